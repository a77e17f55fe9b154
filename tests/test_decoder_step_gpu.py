"""The decoder operators as a W8A8 decoder layer uses them, with the framework's
int8 linears between them:

  RMS norm + int8 -> QKV linear -> rotation and append -> attention over the cache
  -> int8 -> output linear -> residual + RMS norm + int8 -> FFN up (GELU) -> int8
  -> FFN down

Every step is checked on its own inputs: the norm's codes against the oracle's
quantiser on its output, the linears against the oracle's linear block on their
codes, the attention against its 64-bit definition over the cache.  A prompt run
whole, in chunks and token by token leaves the same bits in the cache, and a
captured step that is replayed as the sequences grow gives the eager step's."""
import numpy as np
import pytest
import torch

import oracle
from paritylib import assert_bits_equal, assert_close_fp32, assert_codes_equal, op_as_int
from pagedlib import SPLIT

pytestmark = pytest.mark.gpu
HID, HQ, HKV, D, FFN, PAGE, EPS = 512, 8, 2, 64, 1024, 16, 1e-5


@pytest.fixture(scope="session")
def sq():
    from smoothquant_w8a8_int8_gb300 import binding, build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    binding.load()
    return binding


class Linear:
    def __init__(self, sq, N, K, g):
        W = torch.randn(N, K, generator=g) * 0.05
        self.s = torch.exp(0.3 * torch.randn(K, generator=g)).cuda()
        self.q, self.sw, self.op = sq.pack_weight(W.cuda(), self.s)
        self.bias = (torch.randn(N, generator=g) * 0.02).cuda()


class Layer:
    def __init__(self, sq, seed):
        g = torch.Generator().manual_seed(seed)
        self.sq = sq
        self.qkv = Linear(sq, (HQ + 2 * HKV) * D, HID, g)
        self.out = Linear(sq, HID, HQ * D, g)
        self.up = Linear(sq, FFN, HID, g)
        self.down = Linear(sq, HID, FFN, g)
        self.g1 = (1 + 0.1 * torch.randn(HID, generator=g)).cuda()
        self.g2 = (1 + 0.1 * torch.randn(HID, generator=g)).cuda()
        f = (10000.0 ** (-2 * np.arange(D // 2) / D)).astype(np.float32)
        self.rope = sq.rope_table(torch.from_numpy(f).cuda(), 512)

    def norm(self, h, gain, lin, residual, log):
        q, sx, op, y, _, r = self.sq.rmsnorm_quant(h, gain, EPS, lin.s, residual=residual,
                                                   want_y=True, want_sum=True)
        log.append(("codes", y, lin.s, q, sx, op))
        return op, sx, q, r

    def linear(self, lin, op, sx, q, mode, log):
        y = self.sq.linear_i8(op, sx, lin.op, lin.sw, lin.bias, None, mode)
        log.append(("linear", lin, q, sx, mode, y))
        return y

    def quant(self, x, lin, log):
        q, sx, op = self.sq.quantize_act(x, lin.s)
        log.append(("codes", x, lin.s, q, sx, op))
        return op, sx, q

    def __call__(self, h, cache, starts, lens, max_q, ws, log):
        sq = self.sq
        k, v, table = cache
        op, sx, q, r = self.norm(h, self.g1, self.qkv, None, log)
        qkv = self.linear(self.qkv, op, sx, q, sq.EPI_BIAS, log)
        qs = sq.kv_append(qkv, HQ, k, v, table, starts, lens, rope=self.rope)
        o = sq.paged_attention(qs, k, v, table, starts, lens, max_q=max_q, workspace=ws)
        log.append(("attention", qs, o))
        op, sx, q = self.quant(o, self.out, log)
        a = self.linear(self.out, op, sx, q, sq.EPI_BIAS, log)
        op, sx, q, r = self.norm(a, self.g2, self.up, r, log)
        u = self.linear(self.up, op, sx, q, sq.EPI_BIAS_GELU, log)
        op, sx, q = self.quant(u, self.down, log)
        return self.linear(self.down, op, sx, q, sq.EPI_BIAS, log) + r


def new_cache(sq, B, dtype, pages=64):
    k, v = sq.empty_kv_cache(pages, HKV, PAGE, D, dtype)
    k.fill_(float("nan"))
    v.fill_(float("nan"))
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(1))
    width = pages // B
    return k, v, order[:B * width].view(B, width).int().cuda()


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def check(log):
    for item in log:
        if item[0] == "codes":
            _, y, s, q, sx, op = (x.cpu() if torch.is_tensor(x) else x for x in item)
            qr, sr = oracle.quantize_rows(y.numpy(), s.numpy(), "act")
            assert_codes_equal(q.numpy(), qr)
            assert_codes_equal(op_as_int(op), qr)
            assert_bits_equal(sx.numpy(), sr)
        elif item[0] == "linear":
            _, lin, q, sx, mode, y = item
            acc = oracle.gemm_i32(q.cpu().numpy(), lin.q.cpu().numpy())
            want = oracle.epilogue(acc, sx.cpu().numpy(), lin.sw.cpu().numpy(),
                                   lin.bias.cpu().numpy(), None, mode)
            assert_close_fp32(y.cpu().numpy(), want, "linear")


def attention64(qs, cache, q_lens, kv_lens):
    """(O, bound): the bound of pagedlib.attention_ref with the same terms."""
    k, v, table = (x.cpu() for x in cache)
    Q = qs.double().cpu().view(-1, HQ, D)
    O, bound, row = torch.zeros_like(Q), torch.zeros_like(Q), 0
    for b, (n, length) in enumerate(zip(q_lens, kv_lens)):
        pos = torch.arange(length)
        e = table[b, pos // PAGE].long()
        K, V = k[e, :, pos % PAGE].double(), v[e, :, pos % PAGE].double()
        for i in range(n):
            seen = length - n + i + 1
            for h in range(HQ):
                kk, vv = K[:seen, h * HKV // HQ], V[:seen, h * HKV // HQ]
                s = kk @ Q[row, h] * D ** -0.5
                d = (kk.abs() @ Q[row, h].abs()) * D ** -0.5 * (SPLIT[k.dtype] + 2.0 ** -20) \
                    + 2.0 ** -22 * s.abs()
                O[row, h] = torch.softmax(s, 0) @ vv
                bound[row, h] = vv.abs().max() * (4 * float(d.max()) + 2 * SPLIT[k.dtype]
                                                  + 2.0 ** -20 + 2 * (seen / 16 + 32) * 2.0 ** -23)
            row += 1
    return O.view(row, -1), bound.view(row, -1)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_prompt_whole_and_in_pieces(sq, dtype):
    layer, lens = Layer(sq, 3), [37, 70]
    g = torch.Generator().manual_seed(5)
    hs = [torch.randn(n, HID, generator=g).cuda() for n in lens]
    ws = sq.empty_workspace(sq.paged_attention_workspace_bytes(sum(lens), HQ, HKV, D))
    whole, log = new_cache(sq, 2, dtype), []
    y = layer(torch.cat(hs), whole, ints([0, 37, 107]), ints(lens), 70, ws, log)
    check(log)
    qs, o = log[2][1:]
    ref, bound = attention64(qs, whole, lens, lens)
    assert torch.all((o.double().cpu() - ref).abs() <= bound)
    # in pieces: chunks of unequal length, then single tokens
    pieces, done, outs = new_cache(sq, 2, dtype), [0, 0], [[], []]
    for step in ((30, 61), (5, 7), (1, 1), (1, 0), (0, 1)):
        now = [min(n, lens[b] - done[b]) for b, n in enumerate(step)]
        h = torch.cat([hs[b][done[b]:done[b] + now[b]] for b in range(2)])
        done = [a + b for a, b in zip(done, now)]
        log = []
        z = layer(h, pieces, ints([0, now[0], now[0] + now[1]]), ints(done), max(now), ws, log)
        check(log)
        qs, o = log[2][1:]
        ref, bound = attention64(qs, pieces, now, done)
        assert torch.all((o.double().cpu() - ref).abs() <= bound)
        outs[0].append(z[:now[0]])
        outs[1].append(z[now[0]:])
    assert done == lens
    assert sq.device_status() == sq.SQ_OK
    for a, b in zip(whole[:2], pieces[:2]):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16)), "caches differ"
    assert torch.cat([torch.cat(outs[0]), torch.cat(outs[1])]).shape == y.shape


def test_captured_step_follows_the_sequences(sq):
    B, dtype = 3, torch.bfloat16
    layer = Layer(sq, 7)
    ws = sq.empty_workspace(sq.paged_attention_workspace_bytes(B, HQ, HKV, D))
    eager, graphed = new_cache(sq, B, dtype), new_cache(sq, B, dtype)
    starts, lens = ints([0, 1, 2, 3]), ints([1, 1, 1])
    h = torch.zeros(B, HID, device="cuda")
    step = lambda cache: layer(h, cache, starts, lens, 1, ws, [])  # noqa: E731
    step(eager)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(graphed)
    for n in range(1, 40):
        h.copy_(torch.randn(B, HID, generator=torch.Generator().manual_seed(n)))
        lens.copy_(ints([n, min(n, 20), n // 2]))  # one stops growing, one idles at first
        graph.replay()
        want = step(eager)
        torch.cuda.synchronize()
        assert torch.equal(out, want), f"step {n}"
    assert sq.device_status() == sq.SQ_OK

"""The int8 cache and the gated linear as a W8A8 decoder layer uses them:

  RMS norm + int8 -> QKV linear -> rotation, append to the int8 cache -> attention over
  it -> int8 -> output linear -> residual + RMS norm + int8 -> gated linear -> int8 ->
  down linear

Every step is checked on its own inputs, as in test_decoder_step_gpu.py; a prompt run
whole, in chunks and token by token leaves the same codes and scales in the cache, and a
captured step that is replayed as the sequences grow gives the eager step's bits."""
import pytest
import torch

from pagedlib_i8 import quantise
from test_decoder_step_gpu import (D, FFN, HID, HKV, HQ, PAGE, Layer, check, ints)
from test_gated_gpu import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="session")
def sq():
    from smoothquant_w8a8_int8_gb300 import binding, build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    binding.load()
    return binding


class GatedLayer(Layer):
    def __init__(self, sq, seed, act):
        super().__init__(sq, seed)
        g = torch.Generator().manual_seed(seed + 100)
        gate, up = (torch.randn(FFN, HID, generator=g) * 0.05 for _ in range(2))
        self.act = act
        self.gate_bias = (torch.randn(FFN, generator=g) * 0.02).cuda()
        self.gated_sw, self.gated_op, self.gated_l1 = sq.pack_gated_weight(
            gate.cuda(), up.cuda(), self.up.s, want_l1=True)

    def gated(self, op, sx, q, ws, log):
        y = self.sq.linear_i8_gated(op, sx, self.gated_op, self.gated_sw, FFN, self.act,
                                    bias_gate=self.gate_bias, w_l1=self.gated_l1, workspace=ws)
        log.append(("gated", q, sx, y))
        return y

    def __call__(self, h, cache, starts, lens, max_q, ws, log):
        sq = self.sq
        k, v, ks, vs, table = cache
        op, sx, q, r = self.norm(h, self.g1, self.qkv, None, log)
        qkv = self.linear(self.qkv, op, sx, q, sq.EPI_BIAS, log)
        qs = sq.kv_append(qkv, HQ, k, v, table, starts, lens, rope=self.rope, k_scale=ks,
                          v_scale=vs)
        o = sq.paged_attention(qs, k, v, table, starts, lens, max_q=max_q, workspace=ws[0],
                               k_scale=ks, v_scale=vs)
        log.append(("attention", qkv, qs, o))
        op, sx, q = self.quant(o, self.out, log)
        a = self.linear(self.out, op, sx, q, sq.EPI_BIAS, log)
        op, sx, q, r = self.norm(a, self.g2, self.up, r, log)
        u = self.gated(op, sx, q, ws[1], log)
        op, sx, q = self.quant(u, self.down, log)
        return self.linear(self.down, op, sx, q, sq.EPI_BIAS, log) + r

    def check_gated(self, log):
        for _, q, sx, y in (item for item in log if item[0] == "gated"):
            c = Case.__new__(Case)
            c.M, c.F, c.K, c.x, c.sx = len(q), FFN, HID, q.cpu().float(), sx.cpu()
            c.w, c.sw, c.bias = self.gated_op, self.gated_sw, [self.gate_bias.cpu(), None]
            c.verify(self.sq, self.act, y)


def new_cache(sq, B, pages=64):
    """Codes of every kind and scales that are NaN where no token is."""
    k, v = sq.empty_kv_cache(pages, HKV, PAGE, D, torch.int8)
    ks, vs = sq.empty_kv_scales(pages, HKV, PAGE)
    g = torch.Generator().manual_seed(1)
    for t in (k, v):
        t.copy_(torch.randint(-128, 128, t.shape, generator=g))
    ks.fill_(float("nan"))
    vs.fill_(float("nan"))
    width = pages // B
    table = torch.randperm(pages, generator=g)[:B * width].view(B, width).int().cuda()
    return k, v, ks, vs, table


def workspaces(sq, T):
    return [sq.empty_workspace(sq.paged_attention_workspace_bytes(T, HQ, HKV, D)),
            sq.empty_workspace(max(16, sq.gated_workspace_bytes(T, FFN, HID)))]


def check_attention(log, cache, q_lens, kv_lens):
    """The appended values' codes are the quantiser's, bit by bit, and the output is
    within the bound of pagedlib_i8.attention_ref over the cache as it reads back."""
    qkv, qs, o = next(item for item in log if item[0] == "attention")[1:]
    k, v, ks, vs, table = (x.cpu() for x in cache)
    rows = qkv.cpu().view(-1, HQ + 2 * HKV, D)[:, HQ + HKV:]
    codes, scale = quantise(rows)
    Q, out, row = qs.double().cpu().view(-1, HQ, D), o.double().cpu().view(-1, HQ, D), 0
    for b, (n, length) in enumerate(zip(q_lens, kv_lens)):
        pos = torch.arange(length)
        e = table[b, pos // PAGE].long()
        new = slice(row, row + n)
        assert torch.equal(v[e, :, pos % PAGE][length - n:], codes[new])
        assert torch.equal(vs[e, :, pos % PAGE][length - n:], scale[new])
        wk, wv = ks[e, :, pos % PAGE].double(), vs[e, :, pos % PAGE].double()
        K = k[e, :, pos % PAGE].double() * wk[..., None]
        V = v[e, :, pos % PAGE].double() * wv[..., None]
        for i in range(n):
            seen = length - n + i + 1
            for h in range(HQ):
                hk = h * HKV // HQ
                kk, vv, top = K[:seen, hk], V[:seen, hk], wv[:seen, hk]
                s = kk @ Q[row, h] * D ** -0.5
                d = (kk.abs() @ Q[row, h].abs()) * D ** -0.5 * (2.0 ** -22 + 2.0 ** -20) \
                    + 2.0 ** -22 * s.abs()
                P = torch.softmax(s, 0)
                each = 4 * float(d.max()) + 2.0 ** -21 + 2.0 ** -22 + 2.0 ** -24 \
                    + 2 * (seen / 16 + 32) * 2.0 ** -23
                bound = (P @ vv.abs()) * each + 127 * ((P * top).max() * 2.0 ** -22
                                                       + top.max() * 2.0 ** -100)
                assert torch.all((out[row, h] - P @ vv).abs() <= bound)
            row += 1


@pytest.mark.parametrize("act", [0, 1, 2])
def test_prompt_whole_and_in_pieces(sq, act):
    layer, lens = GatedLayer(sq, 3, act), [37, 70]
    g = torch.Generator().manual_seed(5)
    hs = [torch.randn(n, HID, generator=g).cuda() for n in lens]
    ws = workspaces(sq, sum(lens))
    whole, log = new_cache(sq, 2), []
    y = layer(torch.cat(hs), whole, ints([0, 37, 107]), ints(lens), 70, ws, log)
    check(log)
    layer.check_gated(log)
    check_attention(log, whole, lens, lens)
    # in pieces: chunks of unequal length, then single tokens
    pieces, done, outs = new_cache(sq, 2), [0, 0], [[], []]
    for step in ((30, 61), (5, 7), (1, 1), (1, 0), (0, 1)):
        now = [min(n, lens[b] - done[b]) for b, n in enumerate(step)]
        h = torch.cat([hs[b][done[b]:done[b] + now[b]] for b in range(2)])
        done = [a + b for a, b in zip(done, now)]
        log = []
        z = layer(h, pieces, ints([0, now[0], now[0] + now[1]]), ints(done), max(now), ws, log)
        check(log)
        layer.check_gated(log)
        check_attention(log, pieces, now, done)
        outs[0].append(z[:now[0]])
        outs[1].append(z[now[0]:])
    assert done == lens
    assert sq.device_status() == sq.SQ_OK
    for a, b in zip(whole[:4], pieces[:4]):
        a, b = (x.view(torch.int32) if x.dtype == torch.float32 else x for x in (a, b))
        assert torch.equal(a, b), "caches differ"
    assert torch.cat([torch.cat(outs[0]), torch.cat(outs[1])]).shape == y.shape


def test_captured_step_follows_the_sequences(sq):
    B = 3
    layer, ws = GatedLayer(sq, 7, 0), workspaces(sq, 3)
    eager, graphed = new_cache(sq, B), new_cache(sq, B)
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

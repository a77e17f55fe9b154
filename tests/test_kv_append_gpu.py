"""sq_kv_append and sq_rope_table against their definitions in 64 bits.

Bounds: the table is a rounding of the double functions (half a step plus the
double's own error: 2^-24 (1 + 2^-20) of a value of at most 1).  A rotated
element is x c - y s with c, s off by 2^-24 each, two products and a sum rounded
in fp32 (with or without a fused step): at most 2^-24 (1 + 2 + 1) (|x c| + |y s|),
taken over |x| + |y|.  A cached element adds half a step of its type, relative,
or half the smallest subnormal step of fp16."""
import numpy as np
import pytest
import torch

from pagedlib import HALF_STEP, U32, Batch, rope_ref

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


@pytest.fixture(scope="session")
def sq():
    from smoothquant_w8a8_int8_gb300 import binding, build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    binding.load()
    return binding


def freqs(rot):
    return (10000.0 ** (-2 * np.arange(rot // 2) / max(rot, 1))).astype(np.float32)


def test_rope_table(sq):
    f = freqs(64)
    table = sq.rope_table(torch.from_numpy(f).cuda(), 200000).cpu().numpy().astype(np.float64)
    a = np.arange(200000)[:, None] * f.astype(np.float64)
    tol = U32 * (1 + 2.0 ** -20)
    assert np.max(np.abs(table[..., 0] - np.cos(a))) <= tol
    assert np.max(np.abs(table[..., 1] - np.sin(a))) <= tol
    assert sq.rope_table(torch.from_numpy(f).cuda(), 0).shape == (0, 32, 2)


def run(sq, t, qkv, rot, interleaved, rope_rows=None, in_place=False, stream=None):
    rows = t.table.shape[1] * t.page if rope_rows is None else rope_rows
    rope = sq.rope_table(torch.from_numpy(freqs(rot)).cuda(), rows) if rot else None
    torch.cuda.synchronize()
    q = (qkv[:, :t.Hq * t.D] if in_place
         else torch.full((t.T, t.Hq * t.D), 9.0, device="cuda"))
    got = sq.kv_append(qkv, t.Hq, t.k_d, t.v_d, t.table_d, t.q_start_d, t.kv_len_d, rope=rope,
                       interleaved=interleaved, q_out=q, stream=stream)
    assert got is q
    torch.cuda.synchronize()
    return q.cpu().numpy().astype(np.float64)


def verify(sq, t, rot, interleaved, rope_rows=None, in_place=False, stream=None):
    """Runs the append and checks queries, stored rows, and that nothing else moved."""
    rng = np.random.default_rng(t.T + rot)
    heads = t.Hq + 2 * t.Hkv
    qkv = rng.standard_normal((t.T, heads * t.D)).astype(np.float32)
    before = {n: getattr(t, n + "_d").view(torch.int16).cpu().clone() for n in ("k", "v")}
    dev = torch.from_numpy(qkv).cuda()
    q = run(sq, t, dev, rot, interleaved, rope_rows, in_place, stream)
    if in_place:  # the key and value blocks stay as they were
        assert np.array_equal(dev[:, t.Hq * t.D:].cpu().numpy(), qkv[:, t.Hq * t.D:])
    after = {n: getattr(t, n + "_d").cpu() for n in ("k", "v")}
    rows = t.table.shape[1] * t.page if rope_rows is None else rope_rows
    half, tiny = HALF_STEP[t.dtype], 2.0 ** -25 if t.dtype == FP else 0.0
    written = torch.zeros(t.pages, t.page, dtype=torch.bool)
    first = int(t.q_start[0])
    token = first
    for b in range(t.B):
        n = t.q_lens[b]
        for i in range(n):
            p = t.kv_lens[b] - n + i
            x = qkv[token].reshape(heads, t.D)
            gone = p < 0 or (rot > 0 and p >= rows)
            got_q = q[token].reshape(t.Hq, t.D)
            if gone:
                assert np.all(got_q == 0)
            else:
                want, mag = rope_ref(x[:t.Hq + t.Hkv], p, freqs(rot), rot, interleaved)
                tol = 4 * U32 * mag
                assert np.all(np.abs(got_q - want[:t.Hq]) <= tol[:t.Hq])
                e = int(t.table[b, p // t.page]) if p // t.page < t.table.shape[1] else -1
                if 0 <= e < t.pages:
                    written[e, p % t.page] = True
                    k = after["k"][e, :, p % t.page].double().numpy()
                    v = after["v"][e, :, p % t.page].double().numpy()
                    wk, tk = want[t.Hq:], tol[t.Hq:]
                    assert np.all(np.abs(k - wk) <= tk + half * (np.abs(wk) + tk) + tiny)
                    wv = x[t.Hq + t.Hkv:].astype(np.float64)
                    assert np.all(np.abs(v - wv) <= half * np.abs(wv) + tiny)
            token += 1
    if not in_place:
        assert np.all(q[:first] == 9.0) and np.all(q[token:] == 9.0)
    for n in ("k", "v"):
        same = after[n].view(torch.int16) == before[n]
        assert torch.all(same.all(dim=(1, 3)) | written), f"{n}_cache: other rows written"
    return written


CASES = [
    # q lens, kv lens, Hq, Hkv, D, page, rot, interleaved
    ([1], [1], 1, 1, 64, 16, 64, False),
    ([1, 1, 1], [17, 4000, 64], 8, 2, 128, 16, 128, False),
    ([3, 0, 20], [3, 9, 100], 6, 2, 64, 32, 32, True),
    ([200, 1], [200, 257], 4, 4, 128, 64, 128, True),
    ([7, 5], [7, 300], 7, 1, 64, 256, 8, False),
    ([2, 2], [70, 2], 16, 16, 64, 128, 0, False),
    ([1] * 70, [1 + 3 * i for i in range(70)], 2, 1, 64, 16, 64, False),
    ([1] * 1100, [1 + i % 40 for i in range(1100)], 1, 1, 64, 16, 16, True),
]


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("q,kv,Hq,Hkv,D,page,rot,inter", CASES)
def test_append(sq, q, kv, Hq, Hkv, D, page, rot, inter, dtype):
    t = Batch(q, kv, Hq, Hkv, D, page, dtype, seed=sum(q), front=1, behind=2).cuda()
    assert int(verify(sq, t, rot, inter).sum()) == sum(q)


def test_in_place_and_other_stream(sq):
    t = Batch([5, 1, 30], [6, 200, 90], 8, 2, 128, 32, BF, seed=3).cuda()
    verify(sq, t, 128, False, in_place=True)
    verify(sq, t, 64, True, stream=torch.cuda.Stream())


def test_dropped_tokens(sq):
    """Positions in front of zero, behind the table of angles or of pages, and
    pages outside the cache: nothing is stored, nothing out of range touched."""
    t = Batch([4, 3, 2, 2], [2, 100, 50, 40], 4, 2, 64, 16, BF, seed=5)
    t.table[1, 6] = -1               # positions 96..99 of sequence 1
    t.table[2, 3] = t.pages          # positions 48, 49 of sequence 2
    t.table[3, 2] = 2 ** 31 - 1      # positions 38, 39
    t.cuda()
    assert int(verify(sq, t, 64, False).sum()) == 2  # sequence 0's positions 0 and 1
    assert int(verify(sq, t, 64, False, rope_rows=1).sum()) == 1
    t.kv_len_d[1] = t.kv_lens[1] = 10 ** 6
    verify(sq, t, 64, False, rope_rows=16)


def test_many_pages_beyond_32_bits(sq):
    D, page, Hkv = 128, 256, 8
    pages = (1 << 32) // (Hkv * page * D) + 3
    k, v = sq.empty_kv_cache(pages, Hkv, page, D, BF)
    table = torch.tensor([[pages - 1]], dtype=torch.int32, device="cuda")
    ints = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    qkv = torch.randn(2, (8 + 16) * D, device="cuda")
    sq.kv_append(qkv, 8, k, v, table, ints(0, 2), ints(256))
    want = qkv.view(2, 24, D).bfloat16()
    assert torch.equal(k[-1, :, 254:].transpose(0, 1), want[:, 8:16])
    assert torch.equal(v[-1, :, 254:].transpose(0, 1), want[:, 16:])


def test_graph_follows_the_lengths(sq):
    t = Batch([1, 1], [10, 20], 4, 2, 64, 16, BF, seed=7)
    t.table = torch.arange(8, dtype=torch.int32).view(2, 4) % t.pages
    t.cuda()
    t.k_d, t.v_d = sq.empty_kv_cache(8, 2, 16, 64, BF)
    t.table_d = torch.arange(8, dtype=torch.int32, device="cuda").view(2, 4)
    qkv = torch.randn(2, 8 * 64, device="cuda")
    q = torch.empty(2, 256, device="cuda")
    step = lambda: sq.kv_append(qkv, 4, t.k_d, t.v_d, t.table_d, t.q_start_d,  # noqa: E731
                                t.kv_len_d, q_out=q)
    step()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for n in (1, 33, 64):
        t.kv_len_d.fill_(n)
        t.k_d.zero_()
        g.replay()
        torch.cuda.synchronize()
        want = qkv.view(2, 8, 64)[:, 4:6].bfloat16()
        for b in range(2):
            assert torch.equal(t.k_d[4 * b + (n - 1) // 16, :, (n - 1) % 16], want[b])
        assert int((t.k_d != 0).any(-1).sum()) == 2 * 2

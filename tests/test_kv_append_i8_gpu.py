"""sq_kv_append_i8 against its definition, bit by bit: each step of the rotation and of
the quantiser is one fp32 rounding, so numpy's fp32 steps give the codes, the scales and
the queries themselves."""
import numpy as np
import pytest
import torch

from pagedlib_i8 import BatchI8, quantise

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="session")
def sq():
    from smoothquant_w8a8_int8_gb300 import binding, build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    binding.load()
    return binding


def table_of(sq, rot, rows):
    f = (10000.0 ** (-2 * np.arange(rot // 2) / max(rot, 1))).astype(np.float32)
    return sq.rope_table(torch.from_numpy(f).cuda(), rows)


def rotate(x, angles, interleaved):
    """x [heads, D] in fp32, rotated by (cos, sin) [rot / 2, 2], a rounding a step."""
    out = x.clone()
    n = angles.shape[0]
    i = torch.arange(n)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
    c, s = angles[:, 0], angles[:, 1]
    out[:, a] = x[:, a] * c - x[:, b] * s
    out[:, b] = x[:, a] * s + x[:, b] * c
    return out


def bits(x):
    return x.view(torch.int32) if x.dtype == torch.float32 else x


def verify(sq, t, rot, interleaved, rope_rows=None, in_place=False, stream=None, qkv=None):
    heads = t.Hq + 2 * t.Hkv
    if qkv is None:
        qkv = torch.randn(t.T, heads * t.D, generator=torch.Generator().manual_seed(t.T + rot))
    rows = t.table.shape[1] * t.page if rope_rows is None else rope_rows
    rope = table_of(sq, rot, rows) if rot else None
    names = ("k", "v", "ks", "vs")
    want = {n: getattr(t, n + "_d").cpu().clone() for n in names}
    dev = qkv.cuda()
    q = (dev[:, :t.Hq * t.D] if in_place
         else torch.full((t.T, t.Hq * t.D), 9.0, device="cuda"))
    torch.cuda.synchronize()
    got = sq.kv_append(dev, t.Hq, t.k_d, t.v_d, t.table_d, t.q_start_d, t.kv_len_d, rope=rope,
                       interleaved=interleaved, q_out=q, stream=stream, k_scale=t.ks_d,
                       v_scale=t.vs_d)
    assert got is q
    torch.cuda.synchronize()
    want_q = qkv[:, :t.Hq * t.D].clone() if in_place else torch.full((t.T, t.Hq * t.D), 9.0)
    angles = rope.cpu() if rot else None
    stored, token = 0, int(t.q_start[0])
    for b in range(t.B):
        n = t.q_lens[b]
        for i in range(n):
            p = t.kv_lens[b] - n + i
            x = qkv[token].view(heads, t.D)
            if p < 0 or (rot > 0 and p >= rows):
                want_q[token] = 0
            else:
                y = x[:t.Hq + t.Hkv]
                y = rotate(y, angles[p], interleaved) if rot else y
                want_q[token] = y[:t.Hq].reshape(-1)
                e = int(t.table[b, p // t.page]) if p // t.page < t.table.shape[1] else -1
                if 0 <= e < t.pages:
                    stored += 1
                    r = p % t.page
                    want["k"][e, :, r], want["ks"][e, :, r] = quantise(y[t.Hq:])
                    want["v"][e, :, r], want["vs"][e, :, r] = quantise(x[t.Hq + t.Hkv:])
            token += 1
    assert torch.equal(bits(q.cpu().contiguous()), bits(want_q))
    for n in names:
        got, ref = getattr(t, n + "_d").cpu(), want[n]
        if n in ("ks", "vs"):  # a NaN is a NaN
            assert torch.equal(torch.isnan(got), torch.isnan(ref))
            got, ref = torch.nan_to_num(got), torch.nan_to_num(ref)
        assert torch.equal(bits(got), bits(ref)), n
    if in_place:
        assert torch.equal(dev[:, t.Hq * t.D:].cpu(), qkv[:, t.Hq * t.D:])
    return stored


CASES = [
    # q lens, kv lens, Hq, Hkv, D, page, rot, interleaved
    ([1], [1], 1, 1, 64, 16, 64, False),
    ([1, 1, 1], [17, 1000, 64], 8, 2, 128, 16, 128, False),
    ([3, 0, 20], [3, 9, 100], 6, 2, 64, 32, 32, True),
    ([200, 1], [200, 257], 4, 4, 128, 64, 128, True),
    ([7, 5], [7, 300], 7, 1, 64, 256, 8, False),
    ([2, 2], [70, 2], 16, 16, 64, 128, 0, False),
    ([1] * 70, [1 + 3 * i for i in range(70)], 2, 1, 64, 16, 64, False),
    ([1] * 700, [1 + i % 40 for i in range(700)], 3, 1, 64, 16, 16, True),
    ([340], [345], 5, 5, 128, 16, 64, False),
]


@pytest.mark.parametrize("q,kv,Hq,Hkv,D,page,rot,inter", CASES)
def test_append(sq, q, kv, Hq, Hkv, D, page, rot, inter):
    t = BatchI8(q, kv, Hq, Hkv, D, page, seed=sum(q), front=1, behind=2).cuda()
    assert verify(sq, t, rot, inter) == sum(q)


def test_in_place_and_other_stream(sq):
    t = BatchI8([5, 1, 30], [6, 200, 90], 8, 2, 128, 32, seed=3).cuda()
    verify(sq, t, 128, False, in_place=True)
    verify(sq, t, 64, True, stream=torch.cuda.Stream())


def test_dropped_tokens(sq):
    """Positions in front of zero, behind the table of angles or of pages, and pages
    outside the cache: nothing is stored, nothing out of range touched."""
    t = BatchI8([4, 3, 2, 2], [2, 100, 50, 40], 4, 2, 64, 16, seed=5)
    t.table[1, 6] = -1               # positions 96..99 of sequence 1
    t.table[2, 3] = t.pages          # positions 48, 49 of sequence 2
    t.table[3, 2] = 2 ** 31 - 1      # positions 38, 39
    t.cuda()
    assert verify(sq, t, 64, False) == 2  # sequence 0's positions 0 and 1
    assert verify(sq, t, 64, False, rope_rows=1) == 1
    t.kv_len_d[1] = t.kv_lens[1] = 10 ** 6
    verify(sq, t, 64, False, rope_rows=16)


@pytest.mark.parametrize("D", [64, 128])
def test_rows_of_every_size(sq, D):
    """Zeros, subnormals, the ends of fp32's range, near-ties, and rows that are not
    finite among finite ones."""
    t = BatchI8([12], [30], 4, 2, D, 16, seed=D).cuda()
    g = torch.Generator().manual_seed(1)
    qkv = torch.randn(12, 8, D, generator=g)
    qkv[0] = 0
    qkv[1] *= 1e-41
    qkv[2] *= 2e-38
    qkv[3] *= 1e-33
    qkv[4] = qkv[4] / qkv[4].abs().amax(-1, keepdim=True) * 3.4e38
    qkv[5, 4, 5] = float("nan")
    qkv[5, 6, 7] = float("inf")
    qkv[6, 5, 0] = -float("inf")
    # quotients near half a code: (k + 1/2) scale, and a step on either side
    k = torch.arange(D, dtype=torch.float32) % 120
    scale = torch.rand(8, generator=g) + 0.3
    tie = (k + 0.5) * scale[:, None]
    qkv[7] = tie
    qkv[8] = torch.nextafter(tie, torch.full_like(tie, 1e9))
    qkv[9] = torch.nextafter(tie, torch.zeros_like(tie))
    qkv[7:10, :, 1] = 127 * scale
    verify(sq, t, 0, False, qkv=qkv.view(12, -1))


def test_many_pages_beyond_32_bits(sq):
    D, page, Hkv = 128, 256, 8
    pages = (1 << 32) // (Hkv * page * D) + 3
    k, v = sq.empty_kv_cache(pages, Hkv, page, D, torch.int8)
    ks, vs = sq.empty_kv_scales(pages, Hkv, page)
    table = torch.tensor([[pages - 1]], dtype=torch.int32, device="cuda")
    ints = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    qkv = torch.randn(2, (8 + 16) * D, device="cuda")
    sq.kv_append(qkv, 8, k, v, table, ints(0, 2), ints(256), k_scale=ks, v_scale=vs)
    for cache, scale, at in ((k, ks, 8), (v, vs, 16)):
        codes, s = quantise(qkv.cpu().view(2, 24, D)[:, at:at + 8])
        assert torch.equal(cache[-1, :, 254:].transpose(0, 1).cpu(), codes)
        assert torch.equal(scale[-1, :, 254:].t().cpu(), s)


def test_graph_follows_the_lengths(sq):
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    k, v = sq.empty_kv_cache(8, 2, 16, 64, torch.int8)
    ks, vs = sq.empty_kv_scales(8, 2, 16)
    table, starts, lens = torch.arange(8, dtype=torch.int32, device="cuda").view(2, 4), \
        ints([0, 1, 2]), ints([10, 20])
    qkv = torch.randn(2, 8 * 64, device="cuda")
    q = torch.empty(2, 256, device="cuda")
    step = lambda: sq.kv_append(qkv, 4, k, v, table, starts, lens, q_out=q,  # noqa: E731
                                k_scale=ks, v_scale=vs)
    step()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    codes, scale = quantise(qkv.cpu().view(2, 8, 64)[:, 4:6])
    for n in (1, 33, 64):
        lens.fill_(n)
        k.zero_()
        ks.zero_()
        g.replay()
        torch.cuda.synchronize()
        for b in range(2):
            at = 4 * b + (n - 1) // 16
            assert torch.equal(k[at, :, (n - 1) % 16].cpu(), codes[b])
            assert torch.equal(ks[at, :, (n - 1) % 16].cpu(), scale[b])
        assert int((ks != 0).sum()) == 2 * 2

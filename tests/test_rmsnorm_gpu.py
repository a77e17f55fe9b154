"""sq_rmsnorm_quant: the sum bit for bit, y against the definition in 64 bits,
and the codes, scales and L1 norms bit for bit those of the oracle's quantisers
on the y the kernel stores.

Bound on y, relative: the mean of squares is a sum of non-negative terms in a
tree of at most 32 + 5 + 16 additions behind one product (54 roundings), the
division, the addition of eps; a reciprocal square root halves them and adds its
own, and two products follow: 56 / 2 + 3 = 31 roundings of 2^-24."""
import numpy as np
import pytest
import torch

import oracle
from paritylib import assert_bits_equal, assert_codes_equal, op_as_int, to_dev
from pagedlib import U32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="session")
def sq():
    from smoothquant_w8a8_int8_gb300 import binding, build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    binding.load()
    return binding


def inputs(M, K, seed, spread=1.0):
    rng = np.random.default_rng(seed)
    H = (rng.standard_normal((M, K)) * spread).astype(np.float32)
    H[:, rng.integers(0, K, max(1, K // 100))] *= 20
    R = rng.standard_normal((M, K)).astype(np.float32)
    g = (1 + 0.2 * rng.standard_normal(K)).astype(np.float32)
    s = np.exp(0.5 * rng.standard_normal(K)).astype(np.float32)
    return H, R, g, s


def verify(sq, H, R, g, s, eps, static=0.0, **kw):
    M, K = H.shape
    r = H if R is None else H + R
    Xq, sx, Xop, Y, l1, total = sq.rmsnorm_quant(
        to_dev(H), to_dev(g), eps, to_dev(s), residual=None if R is None else to_dev(R),
        static_scale=static, want_sum=True, want_y=True, want_l1=True, **kw)
    assert np.array_equal(total.cpu().numpy().view(np.uint32), r.view(np.uint32)), "sum"
    y = Y.cpu().numpy()
    r64 = r.astype(np.float64)
    want = r64 / np.sqrt((r64 ** 2).mean(-1, keepdims=True) + np.float32(eps)) * g
    assert np.all(np.abs(y - want) <= 31 * U32 * np.abs(want) * (1 + 1e-6)), "y"
    if static:
        q, scale = oracle.quantize_static(y, s, np.float32(static)), np.float32(static)
        q = q[0] if isinstance(q, tuple) else q
        assert np.all(sx.cpu().numpy() == scale)
    else:
        q, scale = oracle.quantize_rows(y, s, "act")
        assert_bits_equal(sx.cpu().numpy(), scale, "scales")
    assert_codes_equal(Xq.cpu().numpy(), q, "codes")
    assert_codes_equal(op_as_int(Xop), q, "operand")
    assert np.array_equal(l1.cpu().numpy(), np.abs(q.astype(np.int64)).sum(-1))


SHAPES = [(1, 16), (3, 48), (1, 768), (7, 1024), (300, 1040), (2, 4096), (1237, 5136), (5, 8192),
          (33, 4112), (3, 8208), (2, 16384), (700, 2048), (4096, 256)]


@pytest.mark.parametrize("M,K", SHAPES)
@pytest.mark.parametrize("static", [0.0, 0.05])
def test_shapes(sq, M, K, static):
    H, R, g, s = inputs(M, K, M + K)
    verify(sq, H, R, g, s, 1e-5, static)
    verify(sq, H, None, g, s, 1e-6, static)


@pytest.mark.parametrize("K", [1024, 5136])
def test_extreme_smoothing_and_scales(sq, K):
    """Smoothing factors without a usable reciprocal, tiny and huge static
    scales: the codes come from IEEE divisions."""
    H, R, g, s = inputs(9, K, 5)
    s[::7] = 2.0 ** 30
    s[3::11] = 2.0 ** -25
    verify(sq, H, R, g, s, 1e-5)
    verify(sq, H, R, g, s, 1e-5, 0.1)
    H, R, g, s = inputs(9, K, 6)
    verify(sq, H, R, g, s, 1e-5, 2.0 ** -70)
    verify(sq, H, R, g, s, 1e-5, 2.0 ** 70)


def test_zero_rows(sq):
    H, R, g, s = inputs(6, 512, 7)
    H[2], R[2] = 0, 0
    H[4] = -R[4]
    for eps in (1e-5, 0.0):
        out = sq.rmsnorm_quant(to_dev(H), to_dev(g), eps, to_dev(s), residual=to_dev(R),
                               want_y=True)
        Xq, sx, _, Y, _, total = (None if x is None else x.cpu().numpy() for x in
                                  (o.float() if o is not None and o.dtype == torch.bfloat16
                                   else o for o in out))
        assert np.all(Y[[2, 4]] == 0) and np.all(Xq[[2, 4]] == 0) and np.all(sx[[2, 4]] == 1)
        assert np.all(np.isfinite(Y))


@pytest.mark.parametrize("which", ["hidden", "residual"])
def test_sum_in_place(sq, which):
    H, R, g, s = inputs(200, 4096, 8)
    h, r = to_dev(H), to_dev(R)
    base = sq.rmsnorm_quant(h, to_dev(g), 1e-5, to_dev(s), residual=r)
    into = h if which == "hidden" else r
    sx = torch.empty(200, device="cuda")
    op = sq.empty_operand(200, 4096)
    out = sq.rmsnorm_quant(h, to_dev(g), 1e-5, to_dev(s), residual=r,
                           out=(None, sx, op, None, None, into))
    assert out[5] is into and torch.equal(into, base[5])
    assert torch.equal(op, base[2]) and torch.equal(sx, base[1])


def test_stream_and_graph(sq):
    H, R, g, s = inputs(64, 1024, 9)
    h, r, gd, sd = to_dev(H), to_dev(R), to_dev(g), to_dev(s)
    base = sq.rmsnorm_quant(h, gd, 1e-5, sd, residual=r)
    torch.cuda.synchronize()
    side = sq.rmsnorm_quant(h, gd, 1e-5, sd, residual=r, stream=torch.cuda.Stream())
    torch.cuda.synchronize()
    assert torch.equal(side[0], base[0]) and torch.equal(side[5], base[5])
    out = tuple(torch.zeros_like(x) if x is not None else None for x in base)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sq.rmsnorm_quant(h, gd, 1e-5, sd, residual=r, out=out)
    h.copy_(torch.from_numpy(H * 2))
    graph.replay()
    want = sq.rmsnorm_quant(h, gd, 1e-5, sd, residual=r)
    torch.cuda.synchronize()
    for i in (0, 1, 2, 5):
        assert torch.equal(out[i], want[i])


def test_empty(sq):
    out = sq.rmsnorm_quant(torch.empty(0, 64, device="cuda"), torch.ones(64, device="cuda"), 1e-5,
                           torch.ones(64, device="cuda"))
    assert out[0].shape == (0, 64) and out[1].shape == (0,)

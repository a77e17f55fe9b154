"""sq_pack_gated_weight and sq_linear_i8_gated against their definitions in 64 bits.

Bound.  The integer sums are exact.  A projection d = acc (sx sw) + b is rounded three
times in fp32 (acc, sx sw, the fused step): off by at most u (2 |acc sx sw| + |d|), u =
2^-24 (1 + 2^-20 for the products of the small terms).  The activation's slope is at most
1.13, so its input's error counts 1.13 times.  The activation itself:
  SiLU, GELU's tanh form, t / (1 + 2^z): z is rounded at most five times, which moves 2^z
  by a relative 5 u |z| ln 2; 2^x adds 2^-22, 1 + . and the product u each, 1/x 2^-23:
  all of it relative to the result.  2^z beyond fp32's range, or a quotient below it,
  gives zero where the result is below |t| 2^-126.
  GELU: |t| / 2 times erf's error: 1.5e-7 of the formula, and its terms: 2^-22 for the
  exponential, 3 2^-23 for the reciprocal (the polynomial's slope), 2^-21 for six steps of
  a polynomial whose terms stay below 2.
The last product adds u."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
U = 2.0 ** -24 * (1 + 2.0 ** -20)


@pytest.fixture(scope="session")
def sq():
    from smoothquant_w8a8_int8_gb300 import binding, build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    binding.load()
    return binding


def activate(t, act):
    """act(t) in 64 bits and the bound of the kernel's own error."""
    if act == 1:
        y = t * torch.special.erfc(-t / 2 ** 0.5) / 2
        return y, t.abs() / 2 * (1.5e-7 + 2.0 ** -22 + 3 * 2.0 ** -23 + 2.0 ** -21) + U * y.abs()
    z = t if act == 0 else (8 / np.pi) ** 0.5 * (t + 0.044715 * t ** 3)
    y = t * torch.special.expit(z)
    return y, y.abs() * (5 * U * z.abs().clamp(max=200) + 2.0 ** -22 + 2.0 ** -23 + 3 * U) \
        + t.abs() * 2.0 ** -125


class Case:
    def __init__(self, M, F, K, seed=0, bias=(True, True), size=1.0):
        g = torch.Generator().manual_seed(seed)
        rand = lambda *n: torch.randn(*n, generator=g)  # noqa: E731
        self.M, self.F, self.K = M, F, K
        self.x = torch.randint(-127, 128, (M, K), generator=g).float()
        self.sx = (0.5 + torch.rand(M, generator=g)) * 0.02 * size
        self.wg, self.wu, self.s = rand(F, K) * K ** -0.5, rand(F, K) * K ** -0.5, \
            0.5 + torch.rand(K, generator=g)
        self.bias = [rand(F) if b else None for b in bias]

    def packed(self, sq):
        self.sw, self.w, self.l1 = sq.pack_gated_weight(self.wg.cuda(), self.wu.cuda(),
                                                        self.s.cuda(), want_l1=True)
        return self

    def inputs(self):
        return [self.x.bfloat16().cuda(), self.sx.cuda(), self.x.abs().sum(1).int().cuda(),
                *(None if t is None else t.cuda() for t in self.bias)]

    def run(self, sq, act, l1=True, inputs=None, **kw):
        """inputs: kept by the caller where the call is on another stream, which may still
        read them when this returns."""
        x, sx, x_l1, gate, up = inputs or self.inputs()
        return sq.linear_i8_gated(x, sx, self.w, self.sw, self.F, act, gate, up,
                                  x_l1=x_l1 if l1 else None, w_l1=self.l1 if l1 else None, **kw)

    def exact(self, act):
        """(Y, bound) from the packed operand as it is on the GPU."""
        w = self.w.cpu().double().view(-1, 2, 32, self.K)
        sw = self.sw.cpu().double().view(-1, 2, 32)
        side = []
        for i in range(2):
            acc = self.x.double() @ w[:, i].reshape(-1, self.K).t()
            d = (acc * self.sx.double()[:, None] * sw[:, i].reshape(-1))[:, :self.F]
            b = 0 if self.bias[i] is None else self.bias[i].double()
            side.append((d + b, U * (2 * d.abs() + (d + b).abs())))
        (g, dg), (u, du) = side
        y, dy = activate(g, act)
        dy = dy + 1.13 * dg
        return y * u, (y.abs() + dy) * du + dy * u.abs() + U * (y * u).abs() + 2.0 ** -126

    def verify(self, sq, act, got):
        want, bound = self.exact(act)
        over = ((got.double().cpu() - want).abs() - bound)
        assert sq.device_status() == sq.SQ_OK
        assert torch.isfinite(got).all()
        assert float(over.max()) <= 0, f"{float((got.double().cpu() - want).abs().max()):.3e}"


@pytest.mark.parametrize("F,K", [(1, 16), (31, 64), (32, 48), (33, 1040), (200, 512)])
def test_packing(sq, F, K):
    """Each row is sq_pack_weight's, in its place; the filling is zeros with scale 1."""
    c = Case(1, F, K, seed=F).packed(sq)
    rows = sq.gated_rows(F)
    assert rows == -(-F // 32) * 64 and c.w.shape == (rows, K)
    seen = torch.zeros(rows, dtype=torch.bool)
    for i, w in enumerate((c.wg, c.wu)):
        _, sw, op, l1 = sq.pack_weight(w.cuda(), c.s.cuda(), want_l1=True)
        f = torch.arange(F)
        at = f // 32 * 64 + 32 * i + f % 32
        seen[at] = True
        assert torch.equal(c.w[at.cuda()].view(torch.int16), op.view(torch.int16))
        assert torch.equal(c.sw[at.cuda()], sw) and torch.equal(c.l1[at.cuda()], l1)
    rest = (~seen).cuda()
    assert (c.w[rest] == 0).all() and (c.sw[rest] == 1).all() and (c.l1[rest] == 0).all()


def test_packing_rows_of_zeros(sq):
    c = Case(3, 40, 32, seed=1)
    c.wg[5] = 0
    c.packed(sq)
    assert float(c.sw[5]) == 1.0 and int(c.l1[5]) == 0
    c.verify(sq, 0, c.run(sq, 0))


SHAPES = [(1, 1, 16), (1, 96, 64), (2, 33, 1040), (16, 1000, 512), (127, 31, 80), (128, 32, 2080),
          (129, 257, 48), (255, 130, 4112), (256, 128, 64), (257, 515, 1040), (300, 64, 2080),
          (700, 1028, 144), (1030, 40, 32), (7, 300, 2080), (15, 64, 144), (65, 96, 64),
          (20, 12288, 80), (130, 6000, 1056), (3, 14500, 1200)]


@pytest.mark.parametrize("act", [0, 1, 2])
@pytest.mark.parametrize("M,F,K", SHAPES)
def test_gated(sq, M, F, K, act):
    c = Case(M, F, K, seed=M + F + K, bias=(F % 2 == 0, F % 3 != 0)).packed(sq)
    first = c.run(sq, act)
    c.verify(sq, act, first)
    # without the norms: chunks of 1024 added as integers, the same sums
    assert torch.equal(c.run(sq, act, l1=False), first)


@pytest.mark.parametrize("act", [0, 1, 2])
@pytest.mark.parametrize("size", [1e-12, 30.0, 1e18])
def test_range(sq, size, act):
    """Gates far below one, in the tails, and whose square overflows."""
    c = Case(40, 100, 256, seed=5, size=size).packed(sq)
    c.verify(sq, act, c.run(sq, act))


@pytest.mark.parametrize("M,F,K", [(1, 64, 8192), (16, 500, 12288), (128, 1000, 8208),
                                   (130, 33, 8192), (300, 128, 3584), (1, 4000, 12304)])
def test_split_k_is_the_same_bits(sq, M, F, K):
    c = Case(M, F, K, seed=K).packed(sq)
    nbytes = sq.gated_workspace_bytes(M, F, K)
    assert nbytes > 0
    ws = sq.empty_workspace(nbytes)
    want = c.run(sq, 0)
    c.verify(sq, 0, want)
    for _ in range(3):
        assert torch.equal(c.run(sq, 0, workspace=ws), want)


def test_many_tiles(sq):
    """More tiles than fit the GPU at once, a last wave of halves among them."""
    c = Case(2100, 5000, 272, seed=9).packed(sq)
    got = c.run(sq, 0)
    c.verify(sq, 0, got)
    c = Case(200, 21000, 32, seed=10).packed(sq)
    c.verify(sq, 2, c.run(sq, 2))


@pytest.mark.parametrize("K", [1104, 2064])
@pytest.mark.parametrize("rows,columns", [
    ([3], [5]), ([0, 257, 1299], [0, 4999]), (range(0, 1300, 256), range(0, 5000, 400)),
    (range(0, 1300, 512), range(0, 5000, 128)), (range(1300), [17, 2500]), ([], [1, 2]),
    ([700], []), ([300, 301, 1200], range(5000))])
def test_sums_beyond_2_to_the_24(sq, rows, columns, K):
    """A launch whose tiles are summed in one pass where their rows' norms allow it and
    in chunks where they do not: codes of 127 against each other leave fp32's whole
    numbers at K = 1104, so a tile that was summed the wrong way would differ from the
    launch without norms, whose tiles are all chunks."""
    M, F = 1300, 5000
    c = Case(M, F, K, seed=3, bias=(False, True))
    c.wg, c.wu, c.s = c.wg.clamp(-2 / K ** 0.5, 2 / K ** 0.5), c.wu * 0.1, torch.ones(K)
    c.wu[:, 0] = 3.0  # (a row's largest: the others' codes stay small)
    big = 127.0 - (torch.arange(K) % 97 == 0).float()
    c.x = (c.x * 0.5).round()
    c.x[list(rows)] = big
    for w in (c.wg, c.wu):
        w[list(columns)] = torch.flip(big, (0,)) / 127
    c.packed(sq)
    first = c.run(sq, 0)
    assert torch.equal(c.run(sq, 0, l1=False), first)
    limit = 132104  # 127 * limit < 2^24
    assert (c.x.abs().sum(1) > limit).sum() == len(rows)
    if len(columns):
        assert int((c.l1 > limit).sum()) == 2 * len(columns)
    c.verify(sq, 0, first)


def test_rows_are_not_written_beyond_the_output(sq):
    c = Case(130, 101, 64, seed=2).packed(sq)
    whole = torch.full((132 * 101,), 5.0, device="cuda")
    out = whole[104:104 + 130 * 101].view(130, 101)  # (16-byte aligned)
    c.run(sq, 0, out=out)
    assert (whole[:104] == 5).all() and (whole[104 + 130 * 101:] == 5).all()
    c.verify(sq, 0, out)


def test_empty(sq):
    c = Case(4, 8, 32).packed(sq)
    none = torch.empty(0, 32, device="cuda", dtype=torch.bfloat16)
    assert sq.linear_i8_gated(none, torch.empty(0, device="cuda"), c.w, c.sw, 8).shape == (0, 8)
    sw, w = sq.pack_gated_weight(torch.empty(0, 32, device="cuda"),
                                 torch.empty(0, 32, device="cuda"), torch.ones(32, device="cuda"))
    assert w.shape == (0, 32)
    x = c.x.bfloat16().cuda()
    assert sq.linear_i8_gated(x, c.sx.cuda(), w, sw, 0).shape == (4, 0)


def test_streams_and_graph(sq):
    cs = [Case(16, 600, 12288, seed=i).packed(sq) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    ws = [sq.empty_workspace(sq.gated_workspace_bytes(16, 600, 12288)) for _ in cs]
    kept = [c.inputs() for c in cs]
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        got = [c.run(sq, 0, inputs=x, workspace=w, stream=st)
               for c, x, w, st in zip(cs, kept, ws, streams)]
    torch.cuda.synchronize()
    for c, y in zip(cs, got):
        c.verify(sq, 0, y)
    c, out = cs[0], torch.zeros(16, 600, device="cuda")
    x, sx = c.x.bfloat16().cuda(), c.sx.cuda()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sq.linear_i8_gated(x, sx, c.w, c.sw, 600, workspace=ws[0], out=out)
    c.bias = [None, None]
    for size in (1.0, 2.0):
        sx.copy_(c.sx * size)
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        d = Case(16, 600, 12288, seed=0, bias=(False, False))
        d.sx, d.w, d.sw = c.sx * size, c.w, c.sw
        d.verify(sq, 0, out)

"""sq_paged_attention over the range of values: queries whose largest element
ends an octave, rows of very different size side by side, logits far from one.
Lengths, layouts and masks are test_paged_attention_gpu's; the bound is
pagedlib.attention_ref's where no other is derived."""
import pytest
import torch

from pagedlib import SPLIT, Batch, attention_ref
from test_paged_attention_gpu import call, many_behind, poisoned, verify

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16
FEW, MANY = [1, 3], [2, 40]  # tokens of two sequences: 4 heads to a group, so 12 or 160 rows


@pytest.fixture(scope="session")
def sq():
    from smoothquant_w8a8_int8_gb300 import binding, build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    binding.load()
    return binding


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("q", [FEW, MANY])
@pytest.mark.parametrize("top", [2.0 ** -33, 2.0 ** -16, 2.0 ** -8, 1.0, 2.0, 256.0, 2.0 ** 16])
@pytest.mark.parametrize("scale", [0.6931471805599453 / 8, 0.1])
def test_largest_element_at_an_octaves_end(sq, scale, top, q, D, dtype):
    """Every row's largest element is the largest float below `top`, whose
    rounding to fewer bits is `top`, also times the first scale's log2 e; keys that
    make logits of order one."""
    t = Batch(q, [200, 333], 8, 2, D, 32, dtype, seed=D + sum(q))
    rows = t.Q.view(t.T * t.Hq, D)
    rows.mul_(0.3).clamp_(-0.9, 0.9)
    at = torch.arange(rows.shape[0])
    rows[at, at % D] = torch.where(at % 2 == 0, 1.0, -1.0) * (1 - 2.0 ** -24)
    rows.mul_(top)
    t.k = (t.k.float() * (3 / top)).clamp(-65504.0, 65504.0).to(dtype)
    verify(sq, t.cuda(), scale=scale)


def uneven(t, factors):
    """Multiplies the rows (tokens x heads of a group) by `factors` in turn.  Rows of
    2^-13, and keys that make their logits of order one: `factors` of 1 lose their
    bits if a larger row's range is taken for theirs."""
    tok, head = torch.meshgrid(torch.arange(t.T), torch.arange(t.Hq), indexing="ij")
    f = torch.tensor(factors)[(tok * t.G + head % t.G) % len(factors)] * 2.0 ** -13
    t.Q.view(t.T, t.Hq, t.D).mul_(f[..., None])
    t.k = (t.k.float() * 2.0 ** 13).clamp(-65504.0, 65504.0).to(t.dtype)
    return t


@pytest.mark.parametrize("D,dtype", [(64, FP), (128, FP), (64, BF)])
@pytest.mark.parametrize("q,Hq,Hkv", [([1, 3], 8, 2), ([1, 1], 4, 4), ([2, 40], 8, 2),
                                      ([60, 21], 4, 4)])
@pytest.mark.parametrize("factor", [2.0 ** 12, 2.0 ** 20])
def test_rows_of_different_size_side_by_side(sq, factor, q, Hq, Hkv, D, dtype):
    verify(sq, uneven(Batch(q, [150, 333], Hq, Hkv, D, 32, dtype, seed=sum(q)),
                      [1.0, factor, factor, 1.0, 1.0]).cuda())


def beside(sq, t, value):
    """Every third row's queries hold `value` where the keys hold zeros; the others'
    outputs are those of the definition."""
    t.k[..., 7] = 0
    ref, bound = attention_ref(t, t.D ** -0.5)
    rows = t.Q.view(t.T, t.Hq, t.D)
    tok, head = torch.meshgrid(torch.arange(t.T), torch.arange(t.Hq), indexing="ij")
    bad = (tok * t.G + head % t.G) % 3 == 1
    rows[..., 7][bad] = value
    t.cuda()
    got = call(sq, t).double().cpu().view(t.T, t.Hq, t.D)
    assert sq.device_status() == sq.SQ_OK
    ref, bound = ref.view_as(got), bound.view_as(got)
    good = ~bad[..., None] & ~torch.isnan(ref)
    assert good.any() and torch.isfinite(got[good]).all()
    assert float(((got - ref).abs() - bound)[good].max()) <= 0


@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan"), 2.0 ** 40])
@pytest.mark.parametrize("D,dtype", [(64, FP), (128, FP), (64, BF)])
@pytest.mark.parametrize("q,Hq,Hkv", [([1, 3], 8, 2), ([2, 40], 8, 2), ([60, 21], 4, 4)])
def test_a_query_beyond_the_others_stays_in_its_row(sq, q, Hq, Hkv, D, dtype, value):
    beside(sq, Batch(q, [150, 333], Hq, Hkv, D, 32, dtype, seed=sum(q)), value)


@pytest.mark.parametrize("value", [float("inf"), float("nan"), 2.0 ** 40])
@pytest.mark.parametrize("D,dtype", [(64, FP), (128, FP)])
def test_sequences_behind_one_prefix_keep_their_queries(sq, D, dtype, value):
    """The rows of a tile of the prefix's own launch are those of many sequences."""
    kw = dict(Hq=4, D=D, page=64, dtype=dtype, seed=9)
    beside(sq, many_behind(3000, 40, 4, [], **kw), value)
    kw["seed"] = 10
    t = uneven(many_behind(3000, 40, 4, [], **kw), [1.0, 2.0 ** 20, 1.0, 1.0])
    verify(sq, t.cuda())


def sink_batch(q, L, Hq, Hkv, D, dtype, logit, sink, prefix=0, seqs=1):
    """`seqs` sequences of L cached tokens (the first `prefix` shared) and q new
    tokens each.  Position `sink` has the logit `logit` in every row, every other
    position 0; values are of one sign, and the sink's are 0 in the first half of
    the columns."""
    page = 64
    g = torch.Generator().manual_seed(L + q)
    first, pages = prefix // page, -(-L // page)
    own = pages - first
    shared = -(-prefix // page)
    n = shared + seqs * own
    k = torch.zeros(n, Hkv, page, D).to(dtype)
    v = torch.rand(n, Hkv, page, D, generator=g).to(dtype)
    table = torch.full((seqs, pages), -1, dtype=torch.int32)
    for b in range(seqs):
        table[b, first:] = shared + b * own + torch.arange(own)
    where = [(sink // page if sink < prefix else int(table[b, sink // page])) for b in range(seqs)]
    for e in set(where):
        k[e, :, sink % page, 3] = 1.0
        v[e, :, sink % page, :D // 2] = 0.0
    Q = torch.zeros(seqs * q, Hq, D)
    Q[..., 3] = logit
    ints = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    return dict(Q=Q.view(seqs * q, -1).cuda(), k_cache=k.cuda(), v_cache=v.cuda(),
                block_table=table.cuda(), q_start=ints([q * b for b in range(seqs + 1)]),
                kv_len=ints([L] * seqs), max_q=q,
                prefix_pages=torch.arange(shared, dtype=torch.int32).cuda(), prefix_len=prefix)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("q,L,prefix,seqs", [
    (1, 8192, 0, 1), (1, 100000, 0, 1), (4, 3000, 0, 2),     # few rows
    (40, 8192, 0, 1), (40, 50000, 0, 1),                     # many rows
    (1, 9000, 8192, 2), (40, 3000, 2000, 2),                 # the prefix in front
    (1, 40200, 40000, 12), (1, 100200, 100000, 4),           # and in a launch of its own
])
@pytest.mark.parametrize("logit", [16.0, 17.4])
@pytest.mark.parametrize("late", [False, True])
def test_one_key_of_most_weight(sq, q, L, prefix, seqs, D, dtype, logit, late):
    """The others' weights are 2^-23 to 2^-25 of its own, and count together.
    All terms are of one sign, so the error is relative: a weight by 2 d, d =
    2^-22 |logit| (attention_ref's, products exact), by 2^-22 for the exponential
    and by SPLIT; numerator and denominator in L / 16 + 32 steps of 2^-23; and
    2^-37 of the largest weight for each key, half of fp16's smallest step under
    the factor 2^12 that the probabilities carry."""
    Hq, Hkv = 8, 2
    sink = L - q if late else 5
    c = sink_batch(q, L, Hq, Hkv, D, dtype, logit, sink, prefix, seqs)
    got = sq.paged_attention(scale=1.0, **c).double().cpu().view(seqs, q, Hq, D)
    assert sq.device_status() == sq.SQ_OK
    w = torch.ones(L, dtype=torch.float64)
    w[sink] = torch.tensor(logit, dtype=torch.float32).double().exp()
    rel = 2 * (2 * 2.0 ** -22 * logit + 2.0 ** -22 + SPLIT[dtype] + (L / 16 + 32) * 2.0 ** -23)
    table = c["block_table"].cpu().long()
    table[:, :prefix // 64] = torch.arange(prefix // 64)
    pos = torch.arange(L)
    for b in range(seqs):
        pages = table[b, pos // 64]
        pages[pos < prefix] = pos[pos < prefix] // 64
        v = c["v_cache"].cpu()[pages, :, pos % 64].double()      # [L, Hkv, D]
        for i in range(q):
            n = L - q + i + 1
            total = torch.einsum("k,khd->hd", w[:n], v[:n]) / w[:n].sum()
            want = total.repeat_interleave(Hq // Hkv, 0)
            floor = 0.0 if dtype == BF else n * 2.0 ** -37
            assert ((got[b, i] - want).abs() <= want * rel + floor).all()


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("q,prefix", [(FEW, 0), (MANY, 0), (FEW, 150), (MANY, 150),
                                      ([5, 2], 0), ([6], 0)])
@pytest.mark.parametrize("size", [2.0 ** 18, 2.0 ** 22, 2.0 ** 26, 2.0 ** 31, 2.0 ** 40, -2.0 ** 40,
                                  2.0 ** 100])
def test_logits_far_from_one(sq, size, q, prefix, D, dtype):
    """One element of the queries is `size`, the keys' is one of -1, -7/8 ... 7/8:
    logits are whole multiples of size / 64, exact in every format, so a row's
    output is the mean of its values at the largest: within SPLIT, the exponential's
    2^-22, the rounding of log2 e in those weights' common factor (none: they are
    equal) and n / 16 + 32 steps of 2^-23 of the largest value, as attention_ref."""
    kv = [200, 533, 3000][:len(q)] if len(q) > 1 else [3000]   # the last: many pieces
    t = Batch(q, kv, 8, 2, D, 32, dtype, prefix=prefix, seed=sum(q) + D)
    g = torch.Generator().manual_seed(1)
    t.Q.view(t.T, t.Hq, t.D)[:] = 0
    t.Q.view(t.T, t.Hq, t.D)[..., 5] = size
    t.k[:] = 0
    t.k[..., 5] = torch.randint(-8, 8, t.k.shape[:-1], generator=g).to(dtype) / 8
    t.cuda()
    got = call(sq, t, scale=0.125).double().cpu().view(t.T, t.Hq, t.D)
    assert sq.device_status() == sq.SQ_OK
    row = 0
    for b, (n, length) in enumerate(zip(t.q_lens, t.kv_lens)):
        where = [t.row(b, p) for p in range(length)]
        K = torch.stack([t.k[e, :, r, 5] for e, r in where]).double()   # [length, Hkv]
        V = torch.stack([t.v[e, :, r] for e, r in where]).double()
        for i in range(n):
            seen = length - n + i + 1
            x = K[:seen] * (1 if size > 0 else -1)
            top = (x == x.max(0).values).double()
            want = torch.einsum("kh,khd->hd", top, V[:seen]) / top.sum(0)[:, None]
            want = want.repeat_interleave(t.G, 0)
            bound = V[:seen].abs().max() * (2 * SPLIT[dtype] + 2.0 ** -20
                                            + 2 * (seen / 16 + 32) * 2.0 ** -23)
            assert torch.isfinite(got[row]).all()
            assert ((got[row] - want).abs() <= bound).all()
            row += 1


@pytest.mark.parametrize("q", [FEW, MANY])
@pytest.mark.parametrize("dtype,scale,size,keys", [
    (BF, 0.0, 2.0 ** 60, 2.0 ** 50), (FP, 0.0, 2.0 ** 100, 2.0 ** 12),   # equal weights
    (BF, 2.0 ** -110, 2.0 ** 30, 2.0 ** 30), (FP, -2.0 ** -140, 2.0 ** 40, 2.0 ** 10),
    (BF, 2.0 ** 90, 2.0 ** -45, 2.0 ** -45), (BF, -2.0 ** 127, 0.0, 1.0),
    (FP, 2.0 ** 30, 2.0 ** -20, 2.0 ** -12), (FP, 2.0 ** 127, 0.0, 1.0),
    (BF, 2.0 ** -90, 2.0 ** 50, 2.0 ** 38), (FP, 2.0 ** -90, 2.0 ** 80, 2.0 ** 8),
])
def test_scales_of_any_size(sq, dtype, scale, size, keys, q):
    """Queries and keys so that the logits are of order one, or zero."""
    t = Batch(q, [200, 333], 8, 2, 128, 32, dtype, seed=43, spread=size)
    t.k = (t.k.float() * keys).clamp(-2.0 ** 127 if dtype == BF else -65504.0,
                                     2.0 ** 127 if dtype == BF else 65504.0).to(dtype)
    verify(sq, t.cuda(), scale=scale)


@pytest.mark.parametrize("D,dtype", [(64, BF), (128, FP)])
@pytest.mark.parametrize("q,kv,prefix,places", [
    ([1, 3], [900, 700], 0, [(0, 3), (1, 40)]), ([40, 9], [900, 700], 0, [(0, 3), (1, 200)]),
    ([1, 1], [900, 700], 300, [(0, 2), (1, 400)]), ([40, 9], [900, 700], 300, [(0, 2), (1, 400)]),
])
def test_values_that_are_not_finite_and_seen_by_every_row(sq, q, kv, prefix, places, D, dtype):
    """Tiles without a mask: every row that sees them is not finite in their columns."""
    poisoned(sq, Batch(q, kv, 8, 2, D, 32, dtype, prefix=prefix, seed=51), places)

"""sq_paged_attention_i8 where value rows hold nothing but zeros, as the append stores
them: codes of 0 with scale 1, however small the other rows' scales are; and values near
the ends of fp32's range."""
import pytest
import torch

from pagedlib_i8 import BatchI8, attention_ref
from test_paged_attention_i8_gpu import FEW, MANY, call, poisoned, sq  # noqa: F401

pytestmark = pytest.mark.gpu


def token_rows(t, b):
    """(page, row) of every cached token of sequence b."""
    return [at for p in range(t.kv_lens[b]) if (at := t.row(b, p)) is not None]


def verify_rows(sq, t, scale=None, slack=0.0):
    """Against the definition.  A row of zeros adds nothing, so no weight's precision may
    depend on its scale: the bound is attention_ref's with those scales as 0.  A weight
    that is held as two fp16 numbers, the largest below 2^15, is off by 2^-24 at most
    where it is small (each number's half step below fp16's normal range), so by 2^-37 of
    its sequence's largest scale for each key, which its code multiplies by 127 at most.
    (A tile of scales within 2^9 of each other may count rows of zeros among them.)"""
    scale = t.D ** -0.5 if scale is None else scale
    stored = t.vs
    zeros = (t.v == 0).all(-1) & torch.isfinite(stored)
    t.vs = torch.where(zeros, torch.zeros_like(stored), stored)
    ref, bound = attention_ref(t, scale)
    for b in range(t.B):
        if t.kv_lens[b]:
            largest = max(float(t.vs[e, :, r].abs().max()) for e, r in token_rows(t, b))
            near = [float(x) for e, r in token_rows(t, b) for x in stored[e, zeros[e, :, r], r]]
            largest = max([largest] + [x for x in near if x < 2.0 ** 9 * largest])
            bound[t.q_start[b]:t.q_start[b + 1]] += t.kv_lens[b] * 127 * 2.0 ** -37 * largest
    t.vs = stored
    bound = bound + slack
    t.cuda()
    out = torch.full((t.T, t.Hq * t.D), 7.0, device="cuda")
    got = call(sq, t, scale, out=out).double().cpu()
    assert sq.device_status() == sq.SQ_OK
    none = torch.isnan(ref)
    assert (got[none] == 7.0).all()
    over = ((got - ref).abs() - bound)[~none]
    assert torch.isfinite(over).all()
    assert float(over.max()) <= 0, f"{float(over.max()):.3e} over its bound"


def make(q, kv, D, small, lift, zero, prefix=0, seed=0):
    """Value scales `small` times as large; the rows of `zero`'s positions of each sequence
    are zeros, and the key of the first of them stands out by `lift` (log2 of its weight)."""
    t = BatchI8(q, kv, 8, 2, D, 32, seed=seed, prefix=prefix)
    t.vs = t.vs * small
    t.k[:, :, :, 3] = 0
    t.Q.view(t.T, t.Hq, D)[..., 3] = 1.0
    for b in range(t.B):
        for i, p in enumerate(zero):
            if p >= t.kv_lens[b] or (at := t.row(b, p)) is None:
                continue
            e, r = at
            t.v[e, :, r] = 0
            t.vs[e, :, r] = 1.0
            if i == 0:
                t.k[e, :, r] = 0
                t.k[e, :, r, 3] = 127
                t.ks[e, :, r] = lift * 0.6931471805599453 * D ** 0.5 / 127
    return t


@pytest.mark.parametrize("q", [FEW, MANY, [300, 7]])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("small", [1.0, 2.0 ** -13, 2.0 ** -40, 2.0 ** -90])
@pytest.mark.parametrize("lift", [0, 10, 20])
def test_rows_of_zeros(sq, lift, small, D, q):  # noqa: F811
    zero = [5, 0, 37, 64, 65, 66, 129, 200] + list(range(256, 288))
    verify_rows(sq, make(q, [300, 333], D, small, lift, zero, seed=lift + D))


@pytest.mark.parametrize("q", [FEW, MANY])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("zero", [range(0), range(333), range(1, 333), range(0, 333, 2)])
def test_all_or_every_second_row(sq, zero, D, q):  # noqa: F811
    verify_rows(sq, make(q, [300, 333], D, 2.0 ** -30, 0, list(zero), seed=D))


@pytest.mark.parametrize("q", [[1, 2, 1], [1, 70, 20], [1] * 60])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("prefix", [40, 150, 700])
def test_rows_of_zeros_in_a_prefix(sq, prefix, D, q):  # noqa: F811
    kv = [prefix + 30 + n for n in q]
    verify_rows(sq, make(q, kv, D, 2.0 ** -40, 10, [3, 17, prefix - 1, prefix, prefix + 5],
                         prefix=prefix, seed=prefix))


@pytest.mark.parametrize("step", [2.0 ** 7, 2.0 ** 12])
def test_scales_of_rows_of_zeros_that_climb(sq, step):  # noqa: F811
    """Rows of zeros, each of a scale a little above the last one's, in as many steps of a
    long piece of few rows."""
    t = BatchI8([1] * 160, [320] * 160, 8, 8, 64, 32, seed=31)
    t.vs = t.vs * 2.0 ** -60
    for b in range(t.B):
        for i in range(10):
            e, r = t.row(b, 32 * i + (b + i) % 32)
            t.v[e, :, r] = 0
            t.vs[e, :, r] = 2.0 ** -66 * step ** (i + 1)
    verify_rows(sq, t)


@pytest.mark.parametrize("q", [FEW, MANY])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("few", [1, 16])
def test_rows_of_a_few_codes_count(sq, few, D, q):  # noqa: F811
    """Rows with `few` codes that are not zero, in every place of a row in turn."""
    t = BatchI8(q, [300, 333], 8, 2, D, 16, seed=few)
    keep = torch.zeros_like(t.v, dtype=torch.bool)
    for n, (e, r) in enumerate(token_rows(t, 0) + token_rows(t, 1)):
        at = n * few % D
        keep[e, :, r, at:at + few] = True
        t.vs[e, :, r] = 2.0 ** (n % 7)
    t.v = torch.where(keep, t.v | 1, torch.zeros_like(t.v))
    verify_rows(sq, t)


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("q,kv,places", [
    ([3, 2], [40, 17], [(0, 39), (1, 16)]),
    ([40, 30], [40, 300], [(0, 39), (0, 17), (1, 299)]),
])
def test_rows_of_zeros_whose_scale_is_not_finite(sq, q, kv, places, D, value):  # noqa: F811
    """What the append stores for a row that is not finite: the rows that see it are not
    finite, the others do not notice."""
    t = BatchI8(q, kv, 8, 2, D, 32, seed=sum(kv))
    for b, p in places:
        e, r = t.row(b, p)
        t.v[e, :, r] = 0
    poisoned(sq, t, places, "vs", value)


@pytest.mark.parametrize("q", [FEW, MANY, [300, 7]])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("size", [2.0 ** 80, 2.0 ** 100, 2.0 ** 115, 2.0 ** -100])
def test_large_and_small_value_scales(sq, size, D, q):  # noqa: F811
    """Values whose sum over a row's keys is still an fp32 number: 333 of them, each below
    2^3 `size`; and values so small that what a weight may lose, 2^-130, counts."""
    t = BatchI8(q, [300, 333], 8, 2, D, 32, seed=21)
    t.vs = t.vs * size
    verify_rows(sq, t, slack=127 * 333 * 2.0 ** -130 if size < 1 else 0.0)


@pytest.mark.parametrize("q", [FEW, MANY])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("far", [2.0 ** 110, 2.0 ** 60])
def test_one_large_value_row_at_full_weight(sq, far, D, q):  # noqa: F811
    """One key's values far above the others', its weight as theirs."""
    t = BatchI8(q, [140, 333], 8, 2, D, 16, seed=7)
    e, r = t.row(1, 200)
    t.vs[e, :, r] = far
    verify_rows(sq, t)

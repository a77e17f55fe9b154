"""Helpers for the int8 cache's tests: pagedlib's batches with their caches kept as
codes and scales, and the attention's definition in 64 bits with its bound."""
import torch

from pagedlib import Batch


def quantise(x):
    """(codes, scale) of rows in fp32, each step rounded as the operator's."""
    top = x.abs().amax(-1)
    scale = top / torch.full_like(top, 127)
    scale = torch.where(scale == 0, torch.ones_like(scale), scale)
    codes = torch.round(x / scale[..., None]).clamp(-127, 127)
    bad = ~torch.isfinite(top)
    scale[bad] = float("nan")
    codes[bad] = 0
    return codes.to(torch.int8), scale


class BatchI8(Batch):
    """A batch over an int8 cache.  Rows that hold no token have codes of every kind and
    scales that are NaN, infinite or huge."""

    def __init__(self, *args, v_spread=None, **kw):
        args = list(args)
        super().__init__(*args, torch.float32, **kw)
        g = torch.Generator().manual_seed(kw.get("seed", 0) + 1)
        for n in ("k", "v"):
            x = getattr(self, n)
            if n == "v" and v_spread is not None:
                x = x * 2.0 ** ((2 * torch.rand(x.shape[:3] + (1,), generator=g) - 1) * v_spread)
            empty = torch.isnan(x).any(-1)
            codes, scale = quantise(torch.nan_to_num(x))
            noise = torch.randint(-128, 128, codes.shape, generator=g).to(torch.int8)
            codes = torch.where(empty[..., None], noise, codes)
            junk = torch.tensor([float("nan"), float("inf"), -float("inf"), 3e38])
            pick = junk[torch.randint(0, 4, scale.shape, generator=g)]
            setattr(self, n, codes)
            setattr(self, n + "s", torch.where(empty, pick, scale))

    def cuda(self):
        super().cuda()
        self.ks_d, self.vs_d = self.ks.cuda(), self.vs.cuda()
        return self


def attention_ref(t: BatchI8, scale):
    """The definition in 64 bits -> (O [T, Hq * D], bound [T, Hq * D]); rows of no
    sequence are NaN.

    The bound.  A logit is off by at most
      d = |scale| sum |q k| (2^-22 + 2^-20) + 2^-22 |logit|
    (the query's two fp16 numbers; products summed in fp32 in at most a dozen steps of a
    tensor-core instruction, each within 2^-23 of the partial sum; the products with the
    key's scale and with log2 e, and the query's with the scale), so a probability by a
    factor 1 + 2 d (its own and the largest's), to which the exponential adds 2^-22.  A
    weight p v_scale is rounded once (2^-24) and held as two fp16 numbers: 2^-22 of
    itself, or 2^-25 where the row's largest of the step or tile is 2^4 or more: 2^-29 of
    that for each of at most 128 keys.  Numerator and denominator are sums over L keys in
    at most L / 16 + 32 steps (tiles, warps, pieces), each within 2^-23 of the sum of the
    magnitudes so far.  Weights below 2^-100 of the largest count as zero."""
    O = torch.full((t.T, t.Hq, t.D), float("nan"), dtype=torch.float64)
    bound = torch.zeros(t.T, t.Hq, t.D, dtype=torch.float64)
    Q = t.Q.double().view(t.T, t.Hq, t.D)
    row = int(t.q_start[0])
    for b in range(t.B):
        n, length = t.q_lens[b], t.kv_lens[b]
        where = [t.row(b, p) for p in range(length)]
        keys = [p for p in range(length) if where[p] is not None]
        if keys:
            e = torch.tensor([where[p][0] for p in keys])
            r = torch.tensor([where[p][1] for p in keys])
            K = t.k[e, :, r].double() * t.ks[e, :, r].double()[..., None]
            V = t.v[e, :, r].double() * t.vs[e, :, r].double()[..., None]
            vs = t.vs[e, :, r].double().abs()
        at = torch.tensor(keys)
        for i in range(n):
            p = length - n + i
            seen = int((at <= p).sum()) if keys else 0
            if seen == 0:
                O[row] = 0
            else:
                for h in range(t.Hq):
                    q, k, v = Q[row, h], K[:seen, h // t.G], V[:seen, h // t.G]
                    s = scale * (k @ q)
                    d = abs(scale) * (k.abs() @ q.abs()) * (2.0 ** -22 + 2.0 ** -20) \
                        + 2.0 ** -22 * s.abs()
                    P = torch.softmax(s, 0)
                    O[row, h] = P @ v
                    each = 4 * float(d.max()) + 2.0 ** -21 + 2.0 ** -22 + 2.0 ** -24 \
                        + 2 * (seen / 16 + 32) * 2.0 ** -23
                    top = (P * vs[:seen, h // t.G]).max()
                    bound[row, h] = (P @ v.abs()) * each + 127 * (
                        top * 2.0 ** -22 + vs[:seen, h // t.G].max() * 2.0 ** -100)
            row += 1
    return O.view(t.T, -1), bound.view(t.T, -1)

"""Helpers for the decoder operators' tests: random batches over a paged cache,
and their definitions in 64 bits (numpy / torch CPU, no library code)."""
import numpy as np
import torch

U32 = 2.0 ** -24                                            # half a step of fp32
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}  # eps / 2, relative
# what a number loses as a sum of the type's numbers: two roundings in a row for
# fp16; three bf16 numbers hold an fp32 number's 24 bits
SPLIT = {torch.bfloat16: 0.0, torch.float16: 2.0 ** -22}


class Batch:
    """A paged cache and a batch over it, on the CPU.  Rows of the cache that
    hold no token are NaN, table entries behind a sequence's last page are -1,
    and pages stand in random order."""

    def __init__(self, q_lens, kv_lens, Hq, Hkv, D, page, dtype, prefix=0, seed=0, behind=0,
                 front=0, spare=2, spread=1.0):
        rng = np.random.default_rng(seed)
        g = torch.Generator().manual_seed(seed)
        self.q_lens, self.kv_lens = list(q_lens), list(kv_lens)
        self.Hq, self.Hkv, self.D, self.page, self.dtype = Hq, Hkv, D, page, dtype
        self.prefix, self.G, self.B = prefix, Hq // Hkv, len(self.q_lens)
        self.T = front + sum(self.q_lens) + behind
        self.q_start = torch.tensor(front + np.concatenate([[0], np.cumsum(self.q_lens)]),
                                    dtype=torch.int32)
        self.kv_len = torch.tensor(self.kv_lens, dtype=torch.int32)
        first = prefix // page
        shared = -(-prefix // page)
        need = [max(0, -(-n // page) - first) for n in self.kv_lens]
        self.pages = shared + sum(need) + spare
        order = torch.tensor(rng.permutation(self.pages), dtype=torch.int32)
        width = max([1] + [-(-n // page) for n in self.kv_lens]) + 1
        self.table = torch.full((self.B, width), -1, dtype=torch.int32)
        self.prefix_pages = order[:shared].contiguous()
        at = shared
        for b, n in enumerate(need):
            self.table[b, first:first + n] = order[at:at + n]
            at += n
        shape = (self.pages, Hkv, page, D)
        self.k = torch.full(shape, float("nan"), dtype=dtype)
        self.v = torch.full(shape, float("nan"), dtype=dtype)
        rand = lambda *n: torch.randn(*n, generator=g)  # noqa: E731
        for p in range(prefix):
            self._put(self.prefix_pages[p // page], p % page, rand)
        for b, n in enumerate(self.kv_lens):
            for p in range(prefix, n):
                self._put(self.table[b, p // page], p % page, rand)
        self.Q = rand(self.T, Hq * D) * spread

    def _put(self, page, row, rand):
        self.k[int(page), :, row] = rand(self.Hkv, self.D).to(self.dtype)
        self.v[int(page), :, row] = rand(self.Hkv, self.D).to(self.dtype)

    def row(self, b, p):
        """(page, row) of position p of sequence b; None if its page is missing."""
        e = int(self.prefix_pages[p // self.page] if p < self.prefix
                else self.table[b, p // self.page])
        return (e, p % self.page) if 0 <= e < self.pages else None

    def cuda(self):
        for n in ("q_start", "kv_len", "table", "prefix_pages", "k", "v", "Q"):
            setattr(self, n + "_d", getattr(self, n).cuda())
        return self


def attention_ref(t: Batch, scale):
    """The definition in 64 bits -> (O [T, Hq * D], bound [T, Hq * D]); rows of
    no sequence are NaN.

    The bound, per output: a logit is off by at most
      d = |scale| sum |q k| (SPLIT + 2^-20) + 2^-22 |logit|
    (the numbers that stand for q; products summed in fp32 in at most a dozen
    steps of a tensor-core instruction, each within 2^-23 of the partial sum;
    the product with log2 e), so a probability by a factor 1 + 2 d (its own and
    the largest's), to which the exponential adds 2^-22 and its own SPLIT.
    Numerator and denominator are sums over L keys in at most L / 16 + 32 steps
    (tiles, warps, pieces), each within 2^-23 of sum p |v| <= max |v| sum p."""
    O = torch.full((t.T, t.Hq, t.D), float("nan"), dtype=torch.float64)
    bound = torch.zeros(t.T, t.Hq, t.D, dtype=torch.float64)
    Q = t.Q.double().view(t.T, t.Hq, t.D)
    row = int(t.q_start[0])
    for b in range(t.B):
        n, length = t.q_lens[b], t.kv_lens[b]
        where = [t.row(b, p) for p in range(length)]
        keys = [p for p in range(length) if where[p] is not None]
        K = torch.stack([t.k[where[p][0], :, where[p][1]]
                         for p in keys]).double() if keys else None
        V = torch.stack([t.v[where[p][0], :, where[p][1]] for p in keys]).double() if keys else None
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
                    d = abs(scale) * (k.abs() @ q.abs()) * (SPLIT[t.dtype] + 2.0 ** -20) \
                        + 2.0 ** -22 * s.abs()
                    P = torch.softmax(s, 0)
                    O[row, h] = P @ v
                    bound[row, h] = v.abs().max() * (
                        4 * float(d.max()) + 2 * SPLIT[t.dtype] + 2.0 ** -20
                        + 2 * (seen / 16 + 32) * 2.0 ** -23)
            row += 1
    return O.view(t.T, -1), bound.view(t.T, -1)


def rope_ref(x, pos, inv_freq, rot, interleaved):
    """x [heads, D] rotated at position pos, in 64 bits; also the sum of the
    magnitudes of each element's two products."""
    x = np.asarray(x, np.float64)
    out, mag = x.copy(), np.abs(x)
    a = pos * np.asarray(inv_freq, np.float32).astype(np.float64)
    c, s = np.cos(a), np.sin(a)
    i = np.arange(rot // 2)
    ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    out[:, ia] = x[:, ia] * c - x[:, ib] * s
    out[:, ib] = x[:, ia] * s + x[:, ib] * c
    mag[:, ia] = np.abs(x[:, ia]) + np.abs(x[:, ib])
    mag[:, ib] = mag[:, ia]
    return out, mag

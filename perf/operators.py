"""Cases for the operators of a W8A8 decoder layer that stand between its int8
linears: the RMS norm that adds the residual and emits the next linear's int8
operand, the append of rotated keys and values to a paged cache, and the
attention over that cache for a batch whose sequences may share a prefix.

listed() gives the cases, draw() more of the same ranges, prepare() what a
serving loop holds before the call, run() one call (its plain form in torch
operations, or this package's kernels when `own` is set), work() the bytes and
operations a call cannot do without, exact() the same outputs in 64 bits.
"""
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one decode step of 16 sequences: the norm in front of a linear, where
        # latency counts
        {"name": "norm_decode", "op": "norm", "rows": 16, "width": 4096, "scale": 0.0},
        # a prompt chunk of 8192 tokens: bound by memory
        {"name": "norm_prompt", "op": "norm", "rows": 8192, "width": 4096, "scale": 0.0},
        # odd sizes and a calibrated per-tensor scale (Smooth-Static)
        {"name": "norm_static_odd", "op": "norm", "rows": 1237, "width": 5136, "scale": 0.04},
        # one decode step of 64 sequences far into their contexts: a token each
        {"name": "append_decode", "op": "append", "heads": 32, "kv_heads": 8, "dim": 128,
         "type": "bf16", "page": 16, "batch": 64, "q_lo": 1, "q_hi": 1, "kv_lo": 1, "kv_hi": 32768,
         "rot": 128, "pairs": "half", "lens": 1},
        # the chunks of four prompts, about 8000 tokens
        {"name": "append_prompt", "op": "append", "heads": 32, "kv_heads": 8, "dim": 128,
         "type": "bf16", "page": 64, "batch": 4, "q_lo": 1500, "q_hi": 2500, "kv_lo": 2500,
         "kv_hi": 6000, "rot": 128, "pairs": "half", "lens": 2},
        # 16 heads of 64 without sharing, half of each head rotated in
        # neighbouring pairs, ragged chunks
        {"name": "append_partial_fp16", "op": "append", "heads": 16, "kv_heads": 16, "dim": 64,
         "type": "fp16", "page": 32, "batch": 9, "q_lo": 1, "q_hi": 201, "kv_lo": 201,
         "kv_hi": 3001, "rot": 32, "pairs": "neighbours", "lens": 3},
        # one user's next token early in a conversation: latency
        {"name": "attend_one_token", "op": "attend", "heads": 32, "kv_heads": 8, "dim": 128,
         "type": "bf16", "page": 16, "batch": 1, "prefix": 0, "q_lo": 1, "q_hi": 1, "kv_lo": 300,
         "kv_hi": 300, "idle": 0, "lens": 4},
        # one decode step of 64 sequences of every length up to 8192, two of the
        # batch's slots idle (no tokens: rows that nothing is attended by)
        {"name": "attend_decode", "op": "attend", "heads": 32, "kv_heads": 8, "dim": 128,
         "type": "bf16", "page": 16, "batch": 64, "prefix": 0, "q_lo": 1, "q_hi": 1, "kv_lo": 1,
         "kv_hi": 8192, "idle": 2, "lens": 5},
        # one decode step of 128 requests behind one long system prompt
        {"name": "attend_shared_prefix", "op": "attend", "heads": 32, "kv_heads": 8, "dim": 128,
         "type": "bf16", "page": 64, "batch": 128, "prefix": 8192, "q_lo": 1, "q_hi": 1,
         "kv_lo": 1, "kv_hi": 512, "idle": 0, "lens": 6},
        # whole prompts of two requests: bound by the products
        {"name": "attend_prompt", "op": "attend", "heads": 32, "kv_heads": 8, "dim": 128,
         "type": "bf16", "page": 64, "batch": 2, "prefix": 0, "q_lo": 3600, "q_hi": 4096,
         "kv_lo": 4096, "kv_hi": 4500, "idle": 0, "lens": 7},
        # chunks of prompts and single tokens mixed, fp16, 16 heads of 64, behind
        # a prefix that ends inside a page
        {"name": "attend_mixed_fp16", "op": "attend", "heads": 16, "kv_heads": 16, "dim": 64,
         "type": "fp16", "page": 32, "batch": 12, "prefix": 1000, "q_lo": 1, "q_hi": 257,
         "kv_lo": 257, "kv_hi": 2049, "idle": 0, "lens": 8},
        # a few drafted tokens checked at once per request, long contexts
        {"name": "attend_drafts_fp16", "op": "attend", "heads": 24, "kv_heads": 4, "dim": 128,
         "type": "fp16", "page": 128, "batch": 16, "prefix": 0, "q_lo": 2, "q_hi": 5,
         "kv_lo": 4096, "kv_hi": 16384, "idle": 0, "lens": 9},
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["norm", "append", "attend", "attend"])
    if op == "norm":
        width = 16 * _log(rng, 48, 512)
        return {"op": op, "rows": _log(rng, 1, 8192 * 4096 // width), "width": width,
                "scale": rng.choice([0.0, 0.0, 0.03, 0.05])}
    dim = rng.choice([64, 128])
    kv_heads = rng.choice([1, 2, 4, 8]) if dim == 128 else rng.choice([4, 8, 12, 16])
    heads = kv_heads * rng.choice([1, 2, 4, 7, 8] if dim == 128 else [1, 2])
    case = {"op": op, "heads": heads, "kv_heads": kv_heads, "dim": dim,
            "type": rng.choice(["bf16", "fp16"]), "page": rng.choice([16, 32, 64, 128]),
            "lens": rng.randrange(1 << 30)}
    if op == "append":
        chunk = rng.random() < 0.5
        batch = _log(rng, 1, 8) if chunk else _log(rng, 1, 128)
        q_hi = _log(rng, 2, 8192 // batch) if chunk else 1
        return dict(case, batch=batch, q_lo=max(1, q_hi // 2), q_hi=q_hi, kv_lo=q_hi,
                    kv_hi=q_hi + _log(rng, 1, 16000), rot=rng.choice([dim, dim, dim // 2]),
                    pairs=rng.choice(["half", "neighbours"]))
    kind = rng.choice(["decode", "decode", "prefix", "prompt", "mixed"])
    prefix = 0
    if kind == "decode":
        batch, q_hi = _log(rng, 1, 64), rng.choice([1, 1, 1, 4])
        kv_hi = _log(rng, 64, 4000)
    elif kind == "prefix":
        batch, q_hi = _log(rng, 2, 128), rng.choice([1, 1, 2])
        prefix, kv_hi = _log(rng, 128, 8192), _log(rng, 8, 512)
    elif kind == "prompt":
        batch = rng.choice([1, 2, 3])
        q_hi = _log(rng, 128, 6000 // batch)
        kv_hi = q_hi + rng.choice([0, 1, 333])
    else:
        batch, q_hi = _log(rng, 2, 12), _log(rng, 16, 300)
        prefix, kv_hi = rng.choice([0, 77, 1024]), q_hi + _log(rng, 1, 2000)
    return dict(case, batch=batch, prefix=prefix, q_lo=1 if kind == "mixed" else max(1, q_hi // 2),
                q_hi=q_hi, kv_lo=max(q_hi, kv_hi // 4), kv_hi=kv_hi,
                idle=1 if kind == "decode" and batch > 2 and rng.random() < 0.3 else 0)


def _lens(case):
    """(query tokens, cached tokens after the append) of every sequence; the
    cached tokens count the shared prefix.  Idle slots come last: one row of
    queries, nothing cached."""
    r = random.Random(case["lens"])
    q, kv = [], []
    idle = case.get("idle", 0)
    for b in range(case["batch"]):
        q.append(r.randint(case["q_lo"], case["q_hi"]))
        kv.append(case.get("prefix", 0) + max(q[-1], r.randint(case["kv_lo"], case["kv_hi"])))
        if b >= case["batch"] - idle:
            q[-1], kv[-1] = 1, 0
    return q, kv


# ------------------------------------------------------------------ the inputs

def _norm_inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    M, K = case["rows"], case["width"]
    rand = lambda *n: torch.randn(*n, generator=g, device="cuda")  # noqa: E731
    gain = 1 + 0.2 * rand(K)
    hidden = rand(M, K)
    hidden[:, torch.randperm(K, generator=g, device="cuda")[:max(1, K // 100)]] *= 20  # outliers
    smooth = torch.exp(0.5 * rand(K)).clamp(0.2, 8.0)
    return {"case": case, "hidden": hidden, "residual": 2 * rand(M, K), "gain": gain,
            "smooth": smooth, "eps": 1e-5}


def _tables(case, g):
    """Sequence offsets, lengths and the page table, pages in no order."""
    q, kv = _lens(case)
    page = case["page"]
    starts = [0]
    for n in q:
        starts.append(starts[-1] + n)
    prefix = case.get("prefix", 0)
    width = max(1, max(-(-n // page) for n in kv))
    first = prefix // page  # a page that the prefix ends in is each sequence's own
    shared = -(-prefix // page)
    need = [max(0, -(-n // page) - first) for n in kv]
    pages = shared + sum(need)
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(q), width), -1, dtype=torch.int32)
    at = shared
    host = order.cpu()
    for b, n in enumerate(need):
        if n:
            table[b, :first] = host[:first]
            table[b, first:first + n] = host[at:at + n]
        at += n
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    return {"q_start": ints(starts), "kv_len": ints(kv), "table": table.cuda(),
            "prefix_pages": order[:shared].contiguous(), "pages": pages, "tokens": starts[-1],
            "max_q": max(q)}


def _cached_inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    state = {"case": case, **_tables(case, g)}
    hq, hk, d = case["heads"], case["kv_heads"], case["dim"]
    shape = (state["pages"], hk, case["page"], d)
    for name in ("k_cache", "v_cache"):
        state[name] = torch.randn(shape, generator=g, device="cuda", dtype=TYPES[case["type"]])
    if case["op"] == "append":
        # the fused projection's output, and the rotation's table (kept by the model)
        state["qkv"] = torch.randn(state["tokens"], (hq + 2 * hk) * d, generator=g, device="cuda")
        j = torch.arange(case["rot"] // 2, device="cuda", dtype=torch.float64)
        angle = torch.arange(state["table"].shape[1] * case["page"], device="cuda",
                             dtype=torch.float64)[:, None] * 10000.0 ** (-2 * j / case["rot"])
        state["rope"] = torch.stack([angle.cos(), angle.sin()], -1).float().contiguous()
        state["q_out"] = torch.empty(state["tokens"], hq * d, device="cuda")
    else:
        state["q"] = torch.randn(state["tokens"], hq * d, generator=g, device="cuda")
        state["out"] = torch.empty(state["tokens"], hq * d, device="cuda")
    return state


def prepare(case, seed):
    return _norm_inputs(case, seed) if case["op"] == "norm" else _cached_inputs(case, seed)


# ------------------------------------------------------------------ plain forms

def _norm_plain(s):
    total = s["hidden"] + s["residual"]
    y = total * torch.rsqrt(total.square().mean(-1, keepdim=True) + s["eps"]) * s["gain"]
    v = y / s["smooth"]
    fixed = s["case"]["scale"]
    if fixed > 0:
        scale = torch.full((v.shape[0],), fixed, device=v.device)
    else:
        scale = v.abs().amax(-1) / 127
        scale = torch.where(scale == 0, torch.ones_like(scale), scale)
    # int8 codes as the linears' operand holds them: the same whole numbers in bf16
    codes = torch.round(v / scale[:, None]).clamp(-127, 127)
    return {"sum": total, "operand": codes.to(torch.bfloat16), "scale": scale}


def _tokens(s):
    """Each token's sequence, place among its queries and position."""
    q_start, kv_len = s["q_start"].long(), s["kv_len"].long()
    t = torch.arange(s["tokens"], device=q_start.device)
    seq = torch.searchsorted(q_start[1:].contiguous(), t, right=True)
    i = t - q_start[seq]
    return seq, i, kv_len[seq] - (q_start[seq + 1] - q_start[seq]) + i


def _rotate(x, angles, rot, pairs):
    """x [tokens, heads, dim] with its first `rot` elements rotated."""
    cos, sin = angles[:, None, :, 0], angles[:, None, :, 1]
    head, rest = x[..., :rot], x[..., rot:]
    if pairs == "half":
        a, b = head[..., : rot // 2], head[..., rot // 2:]
        return torch.cat([a * cos - b * sin, a * sin + b * cos, rest], -1)
    a, b = head[..., 0::2], head[..., 1::2]
    turned = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    return torch.cat([turned, rest], -1)


def _append_plain(s):
    c = s["case"]
    hq, hk, d = c["heads"], c["kv_heads"], c["dim"]
    seq, _, pos = _tokens(s)
    x = s["qkv"].view(s["tokens"], hq + 2 * hk, d)
    turned = _rotate(x[:, : hq + hk], s["rope"][pos], c["rot"], c["pairs"])
    page = s["table"].long()[seq, pos // c["page"]]
    s["k_cache"][page, :, pos % c["page"]] = turned[:, hq:].to(s["k_cache"].dtype)
    s["v_cache"][page, :, pos % c["page"]] = x[:, hq + hk:].to(s["v_cache"].dtype)
    return {"q": turned[:, :hq].reshape(s["tokens"], hq * d), "k_cache": s["k_cache"],
            "v_cache": s["v_cache"]}


def _attend_plain(s):
    c = s["case"]
    hq, hk, d, page, prefix = c["heads"], c["kv_heads"], c["dim"], c["page"], c["prefix"]
    batch, most, g = c["batch"], s["max_q"], c["heads"] // c["kv_heads"]
    seq, i, pos = _tokens(s)
    # queries padded to [batch, kv head, query x head of the group, dim]
    q = torch.zeros(batch, most, hq, d, device=s["q"].device)
    q[seq, i] = s["q"].view(-1, hq, d)
    q = q.view(batch, most, hk, g, d).transpose(1, 2).reshape(batch, hk, most * g, d)
    at = torch.full((batch, most), -1, dtype=torch.long, device=q.device)
    at[seq, i] = pos
    at = at.repeat_interleave(g, 1)[:, None, :, None]
    # each sequence's own keys and values, then the prefix's, once for all
    first = prefix // page
    own_pages = s["table"][:, first:].long().clamp(min=0)
    gather = lambda cache: cache[own_pages].transpose(1, 2).reshape(  # noqa: E731
        batch, hk, -1, d).float()
    k, v = gather(s["k_cache"]), gather(s["v_cache"])
    key = first * page + torch.arange(k.shape[2], device=q.device)
    logits = torch.matmul(q, k.transpose(-1, -2)) * d ** -0.5
    logits = logits.masked_fill((key > at) | (key < prefix), float("-inf"))
    if prefix:
        once = lambda cache: cache[s["prefix_pages"].long()].transpose(0, 1).reshape(  # noqa: E731
            hk, -1, d)[:, :prefix].float()
        kp, vp = once(s["k_cache"]), once(s["v_cache"])
        all_q = q.transpose(0, 1).reshape(hk, batch * most * g, d)
        front = torch.matmul(all_q, kp.transpose(-1, -2)) * d ** -0.5
        front = front.view(hk, batch, most * g, prefix).transpose(0, 1)
        front = front.masked_fill(torch.arange(prefix, device=q.device) > at, float("-inf"))
        logits = torch.cat([front, logits], -1)
    top = logits.amax(-1, keepdim=True)
    p = torch.exp(logits - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p[..., prefix:], v)
    if prefix:
        part = p[..., :prefix].transpose(0, 1).reshape(hk, batch * most * g, prefix)
        o = o + torch.matmul(part, vp).view(hk, batch, most * g, d).transpose(0, 1)
    o = o / torch.where(total == 0, torch.ones_like(total), total)
    o = o.view(batch, hk, most, g, d).transpose(1, 2).reshape(batch, most, hq * d)
    return {"out": o[seq, i]}


# ------------------------------------------------------------------ the calls

def _norm_own(s):
    from smoothquant_w8a8_int8_gb300 import binding as sq
    _, scale, operand, _, _, total = sq.rmsnorm_quant(
        s["hidden"], s["gain"], s["eps"], s["smooth"], residual=s["residual"],
        static_scale=s["case"]["scale"], want_q=False)
    return {"sum": total, "operand": operand, "scale": scale}


def _append_own(s):
    from smoothquant_w8a8_int8_gb300 import binding as sq
    c = s["case"]
    q = sq.kv_append(s["qkv"], c["heads"], s["k_cache"], s["v_cache"], s["table"], s["q_start"],
                     s["kv_len"], rope=s["rope"], interleaved=c["pairs"] == "neighbours",
                     q_out=s["q_out"])
    return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _attend_own(s):
    from smoothquant_w8a8_int8_gb300 import binding as sq
    c = s["case"]
    if "workspace" not in s:  # kept beside the cache, as a serving loop does
        s["workspace"] = sq.empty_workspace(sq.paged_attention_workspace_bytes(
            s["tokens"], c["heads"], c["kv_heads"], c["dim"], c["prefix"]))
    out = sq.paged_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["q_start"],
                             s["kv_len"], max_q=s["max_q"], prefix_pages=s["prefix_pages"],
                             prefix_len=c["prefix"], workspace=s["workspace"], out=s["out"])
    return {"out": out}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"norm": _norm_own, "append": _append_own, "attend": _attend_own}[op](state)
    return {"norm": _norm_plain, "append": _append_plain, "attend": _attend_plain}[op](state)


def work(case):
    if case["op"] == "norm":
        n = case["rows"] * case["width"]
        # hidden and residual in, sum and operand out, a scale per row, gain and smooth
        return {"bytes": n * (4 + 4 + 4 + 2) + 4 * case["rows"] + 8 * case["width"],
                "flops": 10 * n}
    q, kv = _lens(case)
    hq, hk, d, tokens = case["heads"], case["kv_heads"], case["dim"], sum(q)
    if case["op"] == "append":
        # projections in, queries out in fp32, keys and values out in 16 bits; a
        # row of the rotation's table for each token
        return {"bytes": tokens * (4 * (hq + 2 * hk) * d + 4 * hq * d + 4 * hk * d
                                   + 4 * case["rot"]),
                "flops": 3 * tokens * (hq + hk) * case["rot"]}
    # queries in, outputs out, each sequence's own keys and values, the prefix once
    prefix = case["prefix"]
    own_keys = sum(max(0, n - prefix) for n in kv)
    pairs = sum(sum(max(0, n - m + i + 1) for i in range(m)) for m, n in zip(q, kv))
    return {"bytes": 8 * tokens * hq * d + 4 * hk * d * (own_keys + prefix),
            "flops": 4 * d * hq * pairs}


# ------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        h = s["hidden"].double() + s["residual"].double()
        norm = torch.sqrt((h * h).sum(-1) / h.shape[1] + s["eps"])
        v = h / norm[:, None] * s["gain"].double() / s["smooth"].double()
        if case["scale"] > 0:
            scale = torch.full((h.shape[0],), float(torch.tensor(case["scale"])), device=h.device,
                               dtype=torch.float64)
        else:
            scale = v.abs().max(-1).values / 127
        return {"sum": h, "operand": torch.clamp(torch.round(v / scale[:, None]), -127, 127),
                "scale": scale}
    q_len, kv_len = _lens(case)
    hq, hk, d, page = case["heads"], case["kv_heads"], case["dim"], case["page"]
    table = s["table"].cpu()
    t = 0
    if case["op"] == "append":
        qkv, rope = s["qkv"].double(), s["rope"].double()
        k_cache, v_cache = s["k_cache"].double(), s["v_cache"].double()
        q_out = torch.empty(s["tokens"], hq, d, dtype=torch.float64, device="cuda")
        rot = case["rot"]
        for b, (n, length) in enumerate(zip(q_len, kv_len)):
            pos = torch.arange(length - n, length, device="cuda")
            z = torch.complex(rope[pos, :, 0], rope[pos, :, 1])[:, None]  # [n, 1, rot/2]
            x = qkv[t:t + n].reshape(n, hq + 2 * hk, d).clone()
            r = x[:, : hq + hk, :rot]
            if case["pairs"] == "half":
                w = torch.complex(r[..., : rot // 2].contiguous(),
                                  r[..., rot // 2:].contiguous()) * z
                x[:, : hq + hk, :rot] = torch.cat([w.real, w.imag], -1)
            else:
                w = torch.view_as_complex(r.reshape(n, hq + hk, rot // 2, 2).contiguous()) * z
                x[:, : hq + hk, :rot] = torch.view_as_real(w).reshape(n, hq + hk, rot)
            q_out[t:t + n] = x[:, :hq]
            pages = table[b, pos.cpu() // page].long().cuda()
            k_cache[pages, :, pos % page] = x[:, hq:hq + hk]
            v_cache[pages, :, pos % page] = x[:, hq + hk:]
            t += n
        return {"q": q_out.reshape(s["tokens"], hq * d), "k_cache": k_cache, "v_cache": v_cache}
    out = torch.zeros(s["tokens"], hq, d, dtype=torch.float64, device="cuda")
    g, prefix = hq // hk, case["prefix"]
    front = s["prefix_pages"].cpu()
    for b, (n, length) in enumerate(zip(q_len, kv_len)):
        q = s["q"][t:t + n].double().view(n, hq, d)
        if length > 0:
            # the sequence's pages in order; rows below the prefix's end are the prefix's
            rows = torch.arange(length)
            pages = table[b, rows // page].long()
            pages[rows < prefix] = front[rows[rows < prefix] // page].long()
            pages, at = pages.cuda(), (rows % page).cuda()
            hidden = torch.arange(length, device="cuda")[None, :] > torch.arange(
                length - n, length, device="cuda")[:, None]
            for h in range(hk):
                k = s["k_cache"][pages, h, at].double()
                v = s["v_cache"][pages, h, at].double()
                logits = torch.einsum("ngd,kd->gnk", q[:, h * g:(h + 1) * g], k) / d ** 0.5
                logits.masked_fill_(hidden, float("-inf"))
                out[t:t + n, h * g:(h + 1) * g] = torch.einsum(
                    "gnk,kd->ngd", torch.softmax(logits, -1), v)
        t += n
    return {"out": out.reshape(s["tokens"], hq * d)}

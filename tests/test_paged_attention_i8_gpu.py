"""sq_paged_attention_i8 against its definition in 64 bits: head layouts, page sizes,
lengths of zero, one and many tiles, prefixes that end inside pages and tiles, rows
without a key, anything behind the last token, missing pages, rows of no sequence,
strided queries, streams, graphs and shared workspaces; scales that lie far apart or
are not finite.  The bound is derived in pagedlib_i8.attention_ref."""
import pytest
import torch

from pagedlib_i8 import BatchI8, attention_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="session")
def sq():
    from smoothquant_w8a8_int8_gb300 import binding, build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    binding.load()
    return binding


def call(sq, t, scale=None, **kw):
    kw.setdefault("max_q", max(t.q_lens))
    kw.setdefault("prefix_pages", t.prefix_pages_d if t.prefix else None)
    return sq.paged_attention(kw.pop("Q", t.Q_d), t.k_d, t.v_d, t.table_d, t.q_start_d,
                              t.kv_len_d, prefix_len=t.prefix, scale=scale, k_scale=t.ks_d,
                              v_scale=t.vs_d, **kw)


def verify(sq, t, scale=None, **kw):
    ref, bound = attention_ref(t, t.D ** -0.5 if scale is None else scale)
    out = torch.full((t.T, t.Hq * t.D), 7.0, device="cuda")
    got = call(sq, t, scale, out=out, **kw).double().cpu()
    assert sq.device_status() == sq.SQ_OK
    no_seq = torch.isnan(ref)
    assert torch.all(got[no_seq] == 7.0), "rows of no sequence were written"
    err = (got - ref).abs()[~no_seq]
    over = err - bound[~no_seq]
    assert torch.isfinite(err).all(), "non-finite outputs"
    if over.numel():
        assert float(over.max()) <= 0, f"error {float(err.max()):.3e} over its bound"
    return out


HEADS = [(4, 4), (8, 2), (7, 1), (32, 8), (6, 2), (12, 1), (24, 1), (128, 1)]
LENS = [
    ([1], [1]),
    ([1], [300]),
    ([1, 1, 1], [64, 65, 0]),                    # a slot without tokens
    ([1, 1, 1, 1], [127, 128, 129, 1000]),
    ([0, 3, 1, 0, 2], [5, 3, 17, 0, 130]),       # sequences without queries
    ([4, 2], [2, 70]),                           # rows in front of the first key
    ([33, 1, 70], [33, 400, 200]),               # chunks among single tokens
    ([300], [300]),
    ([5, 257], [1029, 257]),
]


@pytest.mark.parametrize("q,kv", LENS)
@pytest.mark.parametrize("Hq,Hkv", HEADS)
def test_heads_and_lengths(sq, q, kv, Hq, Hkv):
    n = sum(q) + Hq
    t = BatchI8(q, kv, Hq, Hkv, (64, 128)[n % 2], (16, 32, 64, 128, 256)[n % 5], seed=n).cuda()
    verify(sq, t)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_pages(sq, page, D):
    verify(sq, BatchI8([1, 2, 1], [page, page + 1, 3 * page - 1], 8, 2, D, page, seed=page,
                       front=2, behind=3).cuda())
    verify(sq, BatchI8([60, 1], [page + 61, 2 * page], 8, 2, D, page, seed=page + 1, front=1,
                       behind=2).cuda())


@pytest.mark.parametrize("prefix", [1, 16, 40, 100, 128, 200])
@pytest.mark.parametrize("q,kv", [([1, 1, 1], [0, 3, 150]), ([2, 1, 40, 1], [30, 1, 60, 0])])
@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 128), (4, 4, 64), (20, 1, 128)])
def test_shared_prefix(sq, prefix, q, kv, Hq, Hkv, D):
    kv = [prefix + n for n in kv]
    verify(sq, BatchI8(q, kv, Hq, Hkv, D, 16 if prefix % 3 else 64, prefix=prefix, seed=prefix,
                       front=1, behind=1).cuda())


def test_prefix_longer_than_a_sequence(sq):
    """Sequences that end inside the shared prefix see their part of it only."""
    verify(sq, BatchI8([1, 3, 2, 1], [50, 2, 0, 200], 8, 2, 128, 32, prefix=150, seed=3).cuda())


def many_behind(prefix, tiles_per_sm, Hkv, tail, **kw):
    """A batch so large that its shared prefix, read for every sequence, would be more than
    tiles_per_sm key tiles of 128 for each multiprocessor: a launch of its own then."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    n = tiles_per_sm * sms // (Hkv * -(-prefix // 128)) + 1
    q = [1] * n + list(tail)
    kv = [prefix + (i * 7) % 40 for i in range(len(q))]
    kv[1], kv[2] = prefix // 2, 0                     # ends inside the prefix; has no key
    return BatchI8(q, [max(a, b) if b > 1 else a for a, b in zip(kv, q)], kw.pop("Hq"), Hkv,
                   kw.pop("D"), kw.pop("page"), prefix=prefix, front=1, behind=2, **kw)


@pytest.mark.parametrize("prefix,tiles_per_sm,Hkv,tail,kw", [
    (100, 40, 8, [0, 2, 1], dict(Hq=8, D=64, page=16)),
    (128, 40, 8, [], dict(Hq=16, D=128, page=64)),
    (70, 20, 8, [17, 0, 40], dict(Hq=8, D=128, page=32)),
    (60000, 40, 4, [], dict(Hq=4, D=64, page=256)),              # few rows behind a long prefix
])
def test_prefix_in_a_launch_of_its_own(sq, prefix, tiles_per_sm, Hkv, tail, kw):
    t = many_behind(prefix, tiles_per_sm, Hkv, tail, seed=prefix, **kw).cuda()
    verify(sq, t)
    ws = sq.empty_workspace(sq.paged_attention_workspace_bytes(t.T, t.Hq, t.Hkv, t.D, t.prefix))
    first = call(sq, t, workspace=ws)
    out = torch.zeros_like(first)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(sq, t, workspace=ws, out=out)
    for _ in range(3):
        out.zero_()
        g.replay()
        assert torch.equal(out, first)
        assert torch.equal(call(sq, t, workspace=ws), first)
    assert sq.device_status() == sq.SQ_OK


@pytest.mark.parametrize("q,kv,Hq,Hkv,D", [
    ([1], [20011], 4, 1, 64),                    # a thousand pieces of few rows
    ([2, 1], [9000, 12000], 8, 1, 128),
    ([8], [12001], 16, 1, 128),                  # dozens of pieces of many rows
    ([33, 5], [5000, 9000], 8, 2, 64),
])
def test_pieces_joined_by_groups(sq, q, kv, Hq, Hkv, D):
    t = BatchI8(q, kv, Hq, Hkv, D, 64, seed=sum(kv)).cuda()
    ws = sq.empty_workspace(sq.paged_attention_workspace_bytes(t.T, Hq, Hkv, D))
    first = verify(sq, t, workspace=ws)
    for _ in range(5):
        assert torch.equal(call(sq, t, workspace=ws), first)
    assert int(ws[:16384].max()) == 0, "a counter was left behind"


FEW, MANY = [1, 3], [2, 40]  # tokens of two sequences: 4 heads to a group, so 12 or 160 rows


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("q", [FEW, MANY])
@pytest.mark.parametrize("spread", [3, 12, 40])
def test_value_scales_far_apart(sq, spread, q, D):
    """Value rows 2^+-spread in size, keys of every weight among them: small rows of
    much weight count beside large ones of little."""
    t = BatchI8(q, [300, 333], 8, 2, D, 32, seed=spread, v_spread=spread).cuda()
    verify(sq, t)
    verify(sq, t, scale=4.0)


@pytest.mark.parametrize("q", [FEW, MANY])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("far", [2.0 ** 30, 2.0 ** -30, 2.0 ** 100, 0.0])
def test_a_value_row_far_from_the_others(sq, far, D, q):
    """One key's values much larger or smaller than all others, at a weight that makes up
    for it where it is larger."""
    t = BatchI8(q, [140, 333], 8, 2, D, 16, seed=7)
    t.k[:, :, :, 3] = 0
    t.Q.view(t.T, t.Hq, D)[..., 3] = 1.0
    e, r = t.row(1, 200)
    t.vs[e, :, r] = far
    if far > 1:   # 2^-30 of the weight: a logit lower by 30 ln 2, made by one element
        t.k[e, :, r] = 0
        t.k[e, :, r, 3] = -127
        t.ks[e, :, r] = min(torch.log2(torch.tensor(far)).item(), 90) * 0.6931471805599453 \
            * D ** 0.5 / 127
    verify(sq, t.cuda())


def poisoned(sq, t, places, which, value):
    """`places`: (sequence, position) whose scale in every head is `value`.  Rows that
    attend to one are not finite, the others those of the definition."""
    ref, bound = attention_ref(t, t.D ** -0.5)
    hit = torch.zeros(t.T, dtype=torch.bool)
    for b, pos in places:
        page, row = t.row(b, pos)
        getattr(t, which)[page, :, row] = value
        for c in range(t.B) if pos < t.prefix else [b]:
            first = t.kv_lens[c] - t.q_lens[c]
            for i in range(t.q_lens[c]):
                if first + i >= pos:
                    hit[int(t.q_start[c]) + i] = True
    t.cuda()
    out = torch.full((t.T, t.Hq * t.D), 7.0, device="cuda")
    got = call(sq, t, out=out).double().cpu()
    no_seq = torch.isnan(ref).any(-1)
    assert torch.all(got[no_seq] == 7.0)
    assert not torch.isfinite(got[hit]).any(), "a scale that is seen was lost"
    rest = ~hit & ~no_seq
    assert rest.any() and torch.isfinite(got[rest]).all(), "a masked scale was seen"
    assert float(((got - ref).abs() - bound)[rest].max()) <= 0
    assert sq.device_status() == sq.SQ_OK


@pytest.mark.parametrize("which,value", [("ks", float("nan")), ("vs", float("nan")),
                                         ("vs", float("inf"))])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("q,kv,Hq,Hkv,places", [
    ([3, 2], [40, 17], 4, 2, [(0, 39), (1, 16)]),               # few rows: a draft's last token
    ([4, 1], [4, 60], 2, 2, [(0, 2), (1, 59)]),
    ([40, 30], [40, 300], 8, 2, [(0, 39), (0, 17), (1, 299)]),  # chunks
    ([300], [300], 4, 2, [(0, 128), (0, 250), (0, 299)]),
    ([16, 1], [9000, 5], 16, 1, [(0, 8990), (1, 4)]),           # many pieces
])
def test_scales_that_are_not_finite_in_masked_places(sq, q, kv, Hq, Hkv, places, D, which, value):
    poisoned(sq, BatchI8(q, kv, Hq, Hkv, D, 32, seed=sum(kv)), places, which, value)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("q,kv", [([3, 2], [40, 17]), ([40, 30], [40, 300])])
@pytest.mark.parametrize("which,value", [("vs", 3e38), ("vs", 1e-44), ("ks", 3e38)])
def test_extreme_scales_in_masked_places(sq, q, kv, D, which, value):
    """The last position of each sequence, which its last token alone sees."""
    t = BatchI8(q, kv, 8, 2, D, 32, seed=sum(kv))
    ref, bound = attention_ref(t, D ** -0.5)
    for b in range(2):
        page, row = t.row(b, kv[b] - 1)
        getattr(t, which)[page, :, row] = value
    t.cuda()
    got = call(sq, t).double().cpu()
    rest = torch.ones(t.T, dtype=torch.bool)
    rest[t.q_start[1:].long() - 1] = False
    assert float(((got - ref).abs() - bound)[rest].max()) <= 0
    assert sq.device_status() == sq.SQ_OK


@pytest.mark.parametrize("prefix", [40, 130, 300])
@pytest.mark.parametrize("q", [[1, 2, 1], [1, 70, 20]])
@pytest.mark.parametrize("which", ["ks", "vs"])
def test_scales_that_are_not_finite_in_a_prefix(sq, prefix, q, which):
    """Sequences that end inside the prefix do not see its last positions."""
    kv = [prefix // 2, prefix + 80, max(prefix - 1, q[2])]
    for D in (64, 128):
        poisoned(sq, BatchI8(q, kv, 8, 4, D, 16, prefix=prefix, seed=prefix),
                 [(1, prefix - 1), (1, prefix // 2 + 1), (1, prefix + 79)], which, float("nan"))


@pytest.mark.parametrize("q", [FEW, MANY])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("spread,keys", [(2e-5, 2e4), (1e7, 1e-6), (3e-30, 1.0), (0.0, 1.0),
                                         (1e15, 1e-15), (1e-20, 1e20)])
def test_large_and_small_queries(sq, spread, keys, q, D):
    """Queries far from fp16's range, keys that make logits of order one or ten."""
    t = BatchI8(q, [200, 333], 8, 2, D, 32, seed=41, spread=spread)
    t.ks = t.ks * keys
    verify(sq, t.cuda())


@pytest.mark.parametrize("q", [FEW, MANY])
@pytest.mark.parametrize("factor", [2.0 ** 12, 2.0 ** 20])
@pytest.mark.parametrize("D", [64, 128])
def test_rows_of_different_size_side_by_side(sq, factor, q, D):
    t = BatchI8(q, [150, 333], 8, 2, D, 32, seed=sum(q))
    tok, head = torch.meshgrid(torch.arange(t.T), torch.arange(t.Hq), indexing="ij")
    f = torch.tensor([1.0, factor, factor, 1.0, 1.0])[(tok * t.G + head % t.G) % 5] * 2.0 ** -13
    t.Q.view(t.T, t.Hq, t.D).mul_(f[..., None])
    t.ks = t.ks * 2.0 ** 13
    verify(sq, t.cuda())


@pytest.mark.parametrize("q", [FEW, MANY])
@pytest.mark.parametrize("size", [2.0 ** 20, 2.0 ** 26, 2.0 ** 40])
@pytest.mark.parametrize("D", [64, 128])
def test_far_logits(sq, size, q, D):
    """Logits of size and more: one key, which stands out by an eighth of it, has all the
    weight."""
    t = BatchI8(q, [200, 333], 8, 2, D, 32, seed=9)
    t.k[:] = 0
    t.k[..., 5] = 96
    t.ks = torch.where(torch.isfinite(t.ks), torch.full_like(t.ks, 2.0 ** -7), t.ks)
    t.Q[:] = 0
    t.Q.view(t.T, t.Hq, D)[..., 5] = size
    for b in range(2):
        e, r = t.row(b, t.kv_lens[b] - t.q_lens[b])
        t.k[e, :, r, 5] = 108
    t.cuda()
    got = call(sq, t, 1.0).double().cpu()
    row = 0
    for b in range(2):
        e, r = t.row(b, t.kv_lens[b] - t.q_lens[b])
        want = (t.v[e, :, r].double() * t.vs[e, :, r].double()[:, None]).repeat_interleave(4, 0)
        for _ in range(t.q_lens[b]):
            # (a weight's rounding and its two numbers, and the division by the sum)
            err = (got[row].view(t.Hq, D) - want).abs()
            assert float((err - want.abs() * (2.0 ** -21)).max()) <= 0
            row += 1
    assert sq.device_status() == sq.SQ_OK


def test_many_sequences(sq):
    q = [1 + (i % 3 == 0) for i in range(300)]
    kv = [(37 * i) % 200 for i in range(300)]
    verify(sq, BatchI8(q, kv, 4, 2, 64, 16, seed=5).cuda())


@pytest.mark.parametrize("scale", [0.0, -0.1, 1.5])
@pytest.mark.parametrize("q", [[1, 1], [40, 90]])
def test_scales(sq, scale, q):
    """Uniform weights, a negative scale, and peaked weights (logits of +-50)."""
    verify(sq, BatchI8(q, [100, 200], 8, 2, 128, 32, seed=11).cuda(), scale=scale)


@pytest.mark.parametrize("q", [[1, 1], [70, 3]])
def test_missing_pages_are_masked(sq, q):
    t = BatchI8(q, [200, 170], 8, 2, 64, 16, seed=13)
    t.table[0, 3] = -1
    t.table[0, 7] = t.pages
    t.table[1, 0] = 2 ** 31 - 1
    t.table[1, 5] = -2 ** 31
    verify(sq, t.cuda())


@pytest.mark.parametrize("q", [[2, 1], [130, 3]])
def test_all_pages_missing_gives_zeros(sq, q):
    t = BatchI8(q, [200, 170], 8, 2, 128, 16, seed=14)
    t.table[:] = -1
    t.cuda()
    out = call(sq, t)
    assert sq.device_status() == sq.SQ_OK
    assert torch.all(out == 0)


def test_lengths_beyond_the_table_are_clamped(sq):
    t = BatchI8([1, 1], [64, 33], 4, 4, 64, 16, seed=15)
    t.table = t.table[:, :4].contiguous()
    t.cuda()
    want = call(sq, t)
    t.kv_len_d[0] = 2 ** 31 - 1
    got = call(sq, t)
    assert sq.device_status() == sq.SQ_OK
    assert torch.equal(got, want)


def test_strided_queries_and_hint(sq):
    """Queries as a block of columns of a wider matrix; max_q too small or too large only
    chooses another kernel."""
    t = BatchI8([1, 5, 40], [30, 100, 41], 8, 2, 128, 16, seed=17).cuda()
    wide = torch.full((t.T, t.Q.shape[1] + 512), float("nan"), device="cuda")
    wide[:, :t.Q.shape[1]] = t.Q_d
    for max_q in (0, 1, 40, 1 << 20, None):
        verify(sq, t, Q=wide[:, :t.Q.shape[1]], max_q=max_q)


@pytest.mark.parametrize("q", [[1] * 9, [30, 200, 1]])
def test_repeats_are_identical(sq, q):
    t = BatchI8(q, [700 + 13 * i for i in range(len(q))], 8, 2, 128, 32, prefix=300,
                seed=19).cuda()
    ws = sq.empty_workspace(sq.paged_attention_workspace_bytes(t.T, 8, 2, 128, t.prefix))
    first = call(sq, t, workspace=ws)
    for _ in range(5):
        assert torch.equal(call(sq, t, workspace=ws), first)
    other = BatchI8([3, 1], [90, 2000], 8, 2, 128, 16, seed=20).cuda()
    want = call(sq, other)
    assert torch.equal(call(sq, other, workspace=ws), want)   # a smaller call on the same one
    assert torch.equal(call(sq, t, workspace=ws), first)
    assert sq.device_status() == sq.SQ_OK


def test_streams(sq):
    t = BatchI8([1, 1, 60], [200, 900, 64], 8, 2, 128, 32, prefix=100, seed=23).cuda()
    want = call(sq, t)
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(3):  # two streams at once, a workspace each
        got.append(call(sq, t, stream=a))
        with torch.cuda.stream(b):
            got.append(call(sq, t))
    torch.cuda.synchronize()
    assert all(torch.equal(g, want) for g in got)


@pytest.mark.parametrize("q", [[1, 1, 1], [50, 1, 200]])
def test_graphs_share_a_workspace_and_follow_the_lengths(sq, q):
    """Two captured graphs on one workspace, replayed in turn; lengths are read at
    replay."""
    t = BatchI8(q, [300, 240, 500], 8, 2, 128, 16, prefix=64, seed=29).cuda()
    ws = sq.empty_workspace(sq.paged_attention_workspace_bytes(t.T, 8, 2, 128, t.prefix))
    outs = [torch.empty(t.T, t.Q.shape[1], device="cuda") for _ in range(2)]
    call(sq, t, workspace=ws, out=outs[0])
    graphs = []
    for o in outs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(sq, t, workspace=ws, out=o)
        graphs.append(g)
    for lens in ([300, 240, 500], [64, 100, 200], [0, 77, 65]):
        t.kv_len_d.copy_(torch.tensor(lens, dtype=torch.int32))
        want = call(sq, t)
        for g, o in zip(graphs, outs):
            o.fill_(3)
            g.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want) and torch.equal(outs[1], want)
    assert sq.device_status() == sq.SQ_OK


def test_empty_calls(sq):
    t = BatchI8([0, 0], [3, 0], 8, 2, 64, 16, seed=37, behind=4).cuda()
    out = torch.full((t.T, 8 * 64), 5.0, device="cuda")
    call(sq, t, out=out)
    assert torch.all(out == 5.0)
    none = sq.paged_attention(torch.empty(0, 512, device="cuda"), t.k_d, t.v_d, t.table_d,
                              t.q_start_d, t.kv_len_d, k_scale=t.ks_d, v_scale=t.vs_d)
    assert none.shape == (0, 512)


def test_offsets_beyond_32_bits(sq):
    """A cache of more than 2^32 elements: the batch's pages at its far end."""
    D, page, Hkv = 128, 256, 8
    pages = (1 << 32) // (Hkv * page * D) + 40
    t = BatchI8([1, 3], [600, 500], 16, 8, D, page, seed=41)
    u = BatchI8([20, 3], [600, 500], 16, 8, D, page, seed=42)
    for b in (t, u):
        shift = pages - b.pages
        big = [torch.zeros(pages, Hkv, page, D, dtype=torch.int8, device="cuda") for _ in range(2)]
        sc = [torch.zeros(pages, Hkv, page, device="cuda") for _ in range(2)]
        for x, y in zip(big + sc, (b.k, b.v, b.ks, b.vs)):
            x[shift:] = y.cuda()
        b.cuda()
        b.k_d, b.v_d, b.ks_d, b.vs_d = big + sc
        b.table_d = torch.where(b.table_d >= 0, b.table_d + shift, b.table_d).int()
        ref, bound = attention_ref(b, D ** -0.5)
        got = call(sq, b).double().cpu()
        assert float(((got - ref).abs() - bound).max()) <= 0

"""sq_paged_attention against its definition in 64 bits: types, head layouts,
page sizes, lengths of zero, one and many tiles, prefixes that end inside pages
and tiles, rows without a key, pages that end inside a tile with anything behind
the last token, missing pages, rows of no sequence, strided queries, streams,
graphs and shared workspaces.  The bound is derived in pagedlib.attention_ref."""
import pytest
import torch

from pagedlib import Batch, attention_ref

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


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
                              t.kv_len_d, prefix_len=t.prefix, scale=scale, **kw)


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
    D, dtype = (64, 128)[n % 2], (BF, FP)[n // 2 % 2]
    t = Batch(q, kv, Hq, Hkv, D, (16, 32, 64, 128, 256)[n % 5], dtype, seed=n).cuda()
    verify(sq, t)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_pages(sq, page, D, dtype):
    verify(sq, Batch([1, 2, 1], [page, page + 1, 3 * page - 1], 8, 2, D, page, dtype, seed=page,
                     front=2, behind=3).cuda())
    verify(sq, Batch([60, 1], [page + 61, 2 * page], 8, 2, D, page, dtype, seed=page + 1,
                     front=1, behind=2).cuda())


@pytest.mark.parametrize("prefix", [1, 16, 40, 64, 100, 128, 200])
@pytest.mark.parametrize("q,kv", [([1, 1, 1], [0, 3, 150]), ([2, 1, 40, 1], [30, 1, 60, 0])])
@pytest.mark.parametrize("Hq,Hkv,D,dtype", [(8, 2, 128, BF), (4, 4, 64, FP), (20, 1, 128, FP)])
def test_shared_prefix(sq, prefix, q, kv, Hq, Hkv, D, dtype):
    kv = [prefix + n for n in kv]
    verify(sq, Batch(q, kv, Hq, Hkv, D, 16 if prefix % 3 else 64, dtype, prefix=prefix,
                     seed=prefix, front=1, behind=1).cuda())


def test_prefix_longer_than_a_sequence(sq):
    """Sequences that end inside the shared prefix see their part of it only."""
    verify(sq, Batch([1, 3, 2, 1], [50, 2, 0, 200], 8, 2, 128, 32, BF, prefix=150, seed=3).cuda())


@pytest.mark.parametrize("q,kv,Hq,Hkv,D,dtype", [
    ([1], [20011], 4, 1, 64, FP),                # a thousand pieces of few rows
    ([2, 1], [9000, 12000], 8, 1, 128, BF),
    ([8], [12001], 16, 1, 128, BF),              # dozens of pieces of many rows
    ([33, 5], [5000, 9000], 8, 2, 64, FP),
])
def test_pieces_joined_by_groups(sq, q, kv, Hq, Hkv, D, dtype):
    t = Batch(q, kv, Hq, Hkv, D, 64, dtype, seed=sum(kv)).cuda()
    ws = sq.empty_workspace(sq.paged_attention_workspace_bytes(t.T, Hq, Hkv, D))
    first = verify(sq, t, workspace=ws)
    for _ in range(5):
        assert torch.equal(call(sq, t, workspace=ws), first)
    assert int(ws[:16384].max()) == 0, "a counter was left behind"


def many_behind(prefix, tiles_per_sm, Hkv, tail, **kw):
    """A batch of single tokens (and `tail`) so large that its shared prefix,
    read for every sequence, would be more than tiles_per_sm key tiles of 128
    for each multiprocessor: it is attended to in a launch of its own then."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    n = tiles_per_sm * sms // (Hkv * -(-prefix // 128)) + 1
    q = [1] * n + list(tail)
    kv = [prefix + (i * 7) % 40 for i in range(len(q))]
    kv[1], kv[2] = prefix // 2, 0                     # ends inside the prefix; has no key
    return Batch(q, [max(a, b) if b > 1 else a for a, b in zip(kv, q)], kw.pop("Hq"), Hkv,
                 kw.pop("D"), kw.pop("page"), kw.pop("dtype"), prefix=prefix, front=1, behind=2,
                 **kw)


@pytest.mark.parametrize("prefix,tiles_per_sm,Hkv,tail,kw", [
    (100, 40, 8, [0, 2, 1], dict(Hq=8, D=64, page=16, dtype=BF)),
    (128, 40, 8, [], dict(Hq=16, D=128, page=64, dtype=FP)),
    (70, 20, 8, [17, 0, 40], dict(Hq=8, D=128, page=32, dtype=BF)),
    (130, 20, 8, [33, 1], dict(Hq=8, D=64, page=256, dtype=FP)),
    (60000, 40, 4, [], dict(Hq=4, D=64, page=256, dtype=BF)),    # few rows behind a long prefix
    (31000, 40, 2, [1], dict(Hq=2, D=128, page=16, dtype=FP)),
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


@pytest.mark.parametrize("prefix", [1, 127, 128, 129, 300])
@pytest.mark.parametrize("q,kv", [([1, 3, 1], [40, 2, 500]), ([130, 1, 260], [0, 0, 30])])
@pytest.mark.parametrize("D,dtype,page", [(128, BF, 256), (64, FP, 16)])
def test_prefix_in_front_of_own_keys(sq, prefix, q, kv, D, dtype, page):
    """Few sequences, or long ones: the prefix's key tiles stand in front of each
    item's own; the tile in which it ends is read from both page lists."""
    kv = [prefix + max(a, b) for a, b in zip(q, kv)]
    kv[1] = min(kv[1], prefix) // 2 + 1                # ends inside the prefix
    verify(sq, Batch(q, kv, 8, 4, D, page, dtype, prefix=prefix, seed=prefix + D,
                     behind=1).cuda())


def poisoned(sq, t, places):
    """`places`: (sequence, position) whose values are NaN in column 5 and infinite in
    column 38 of every head.  Outputs are the formula's: not finite in those columns
    for the rows that attend to the position, untouched everywhere else."""
    t.cuda()
    ref, bound = attention_ref(t, t.D ** -0.5)
    hit = torch.zeros(t.T, t.Hq, t.D, dtype=torch.bool)
    for b, pos in places:
        page, row = t.row(b, pos)
        t.v_d[page, :, row, 5] = float("nan")
        t.v_d[page, :, row, 38] = float("inf")
        for c in range(t.B) if pos < t.prefix else [b]:
            first = t.kv_lens[c] - t.q_lens[c]
            for i in range(t.q_lens[c]):
                if first + i >= pos:
                    hit[int(t.q_start[c]) + i, :, (5, 38)] = True
    hit = hit.view(t.T, -1)
    out = torch.full((t.T, t.Hq * t.D), 7.0, device="cuda")
    got = call(sq, t, out=out).double().cpu()
    no_seq = torch.isnan(ref)
    assert torch.all(got[no_seq] == 7.0)
    assert not torch.isfinite(got[hit]).any(), "a value that is seen was lost"
    rest = ~hit & ~no_seq
    assert torch.isfinite(got[rest]).all(), "a masked value was seen"
    assert float(((got - ref).abs() - bound)[rest].max()) <= 0
    assert sq.device_status() == sq.SQ_OK


@pytest.mark.parametrize("D,dtype", [(64, BF), (128, FP), (128, BF), (64, FP)])
@pytest.mark.parametrize("q,kv,Hq,Hkv,places", [
    ([3, 2], [40, 17], 4, 2, [(0, 39), (1, 16)]),               # few rows: a draft's last token
    ([4, 1], [4, 60], 2, 2, [(0, 2), (1, 59)]),
    ([40, 30], [40, 300], 8, 2, [(0, 39), (0, 17), (1, 299)]),  # chunks
    ([300], [300], 4, 2, [(0, 128), (0, 250), (0, 299)]),
    ([16, 1], [9000, 5], 16, 1, [(0, 8990), (1, 4)]),           # many pieces
])
def test_values_that_are_not_finite_in_masked_places(sq, q, kv, Hq, Hkv, places, D, dtype):
    poisoned(sq, Batch(q, kv, Hq, Hkv, D, 32, dtype, seed=sum(kv)), places)


@pytest.mark.parametrize("prefix", [40, 130, 300])
@pytest.mark.parametrize("q", [[1, 2, 1], [1, 70, 20]])
def test_values_that_are_not_finite_in_a_prefix(sq, prefix, q):
    """Sequences that end inside the prefix do not see its last positions."""
    kv = [prefix // 2, prefix + 80, max(prefix - 1, q[2])]
    for D, dtype in ((64, FP), (128, BF)):
        poisoned(sq, Batch(q, kv, 8, 4, D, 16, dtype, prefix=prefix, seed=prefix),
                 [(1, prefix - 1), (1, prefix // 2 + 1), (1, prefix + 79)])


@pytest.mark.parametrize("tiles_per_sm,tail", [(40, []), (20, [30])])
def test_values_that_are_not_finite_in_a_prefix_of_its_own(sq, tiles_per_sm, tail):
    t = many_behind(100, tiles_per_sm, 8, tail, Hq=8, D=64, page=32, dtype=BF, seed=3)
    poisoned(sq, t, [(5, 99), (5, 60), (9, t.kv_lens[9] - 1)])


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("q", [[1, 3], [2, 40]])
@pytest.mark.parametrize("spread,keys", [(2e-5, 2e4), (1e7, 1e-6), (3e-30, 1.0), (0.0, 1.0)])
def test_large_and_small_queries(sq, spread, keys, q, dtype):
    """Queries far from the range of the cache's type, keys that make logits of
    order one or ten of them."""
    t = Batch(q, [200, 333], 8, 2, 128, 32, dtype, seed=41, spread=spread)
    # (4.5 deviations of 2e4 pass fp16's largest number, and infinite keys have no logits)
    t.k = (t.k.float() * keys).clamp(-65504.0, 65504.0).to(dtype)
    verify(sq, t.cuda())


def test_many_sequences(sq):
    q = [1 + (i % 3 == 0) for i in range(300)]
    kv = [(37 * i) % 200 for i in range(300)]
    verify(sq, Batch(q, kv, 4, 2, 64, 16, BF, seed=5).cuda())


def test_long_sequence_split_over_the_gpu(sq):
    verify(sq, Batch([1, 1], [9000, 7], 4, 1, 128, 64, BF, seed=6).cuda())
    verify(sq, Batch([20], [5000], 8, 1, 64, 16, FP, seed=7).cuda())


@pytest.mark.parametrize("scale", [0.0, -0.1, 1.5])
@pytest.mark.parametrize("q", [[1, 1], [40, 90]])
def test_scales(sq, scale, q):
    """Uniform weights, a negative scale, and peaked weights (logits of +-50)."""
    verify(sq, Batch(q, [100, 200], 8, 2, 128, 32, FP, seed=11).cuda(), scale=scale)


@pytest.mark.parametrize("q", [[1, 1], [70, 3]])
def test_missing_pages_are_masked(sq, q):
    t = Batch(q, [200, 170], 8, 2, 64, 16, BF, seed=13)
    t.table[0, 3] = -1
    t.table[0, 7] = t.pages
    t.table[1, 0] = 2 ** 31 - 1
    t.table[1, 5] = -2 ** 31
    verify(sq, t.cuda())


@pytest.mark.parametrize("q", [[2, 1], [130, 3]])
def test_all_pages_missing_gives_zeros(sq, q):
    t = Batch(q, [200, 170], 8, 2, 128, 16, BF, seed=14)
    t.table[:] = -1
    t.cuda()
    out = call(sq, t)
    assert sq.device_status() == sq.SQ_OK
    assert torch.all(out == 0)


def test_lengths_beyond_the_table_are_clamped(sq):
    t = Batch([1, 1], [64, 33], 4, 4, 64, 16, BF, seed=15)
    t.table = t.table[:, :4].contiguous()
    t.kv_lens[0] = 64
    t.cuda()
    want = call(sq, t)
    t.kv_len_d[0] = 2 ** 31 - 1
    got = call(sq, t)
    assert sq.device_status() == sq.SQ_OK
    assert torch.equal(got, want)


def test_strided_queries_and_hint(sq):
    """Queries as a block of columns of a wider matrix; max_q too small or too
    large only chooses another kernel."""
    t = Batch([1, 5, 40], [30, 100, 41], 8, 2, 128, 16, BF, seed=17).cuda()
    wide = torch.full((t.T, t.Q.shape[1] + 512), float("nan"), device="cuda")
    wide[:, :t.Q.shape[1]] = t.Q_d
    for max_q in (0, 1, 40, 1 << 20, None):
        verify(sq, t, Q=wide[:, :t.Q.shape[1]], max_q=max_q)


@pytest.mark.parametrize("q", [[1] * 9, [30, 200, 1]])
def test_repeats_are_identical(sq, q):
    """Split rows are joined in a fixed order, and the workspace is reusable as
    it is: call after call gives the same bits."""
    t = Batch(q, [700 + 13 * i for i in range(len(q))], 8, 2, 128, 32, BF, prefix=300,
              seed=19).cuda()
    ws = sq.empty_workspace(sq.paged_attention_workspace_bytes(t.T, 8, 2, 128, t.prefix))
    first = call(sq, t, workspace=ws)
    for _ in range(5):
        assert torch.equal(call(sq, t, workspace=ws), first)
    other = Batch([3, 1], [90, 2000], 8, 2, 128, 16, BF, seed=20).cuda()
    want = call(sq, other)
    assert torch.equal(call(sq, other, workspace=ws), want)   # a smaller call on the same one
    assert torch.equal(call(sq, t, workspace=ws), first)
    assert sq.device_status() == sq.SQ_OK


def test_streams(sq):
    t = Batch([1, 1, 60], [200, 900, 64], 8, 2, 128, 32, FP, prefix=100, seed=23).cuda()
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
    """Two captured graphs on one workspace, replayed in turn; the lengths and
    the table are read at replay."""
    t = Batch(q, [300, 40, 500], 8, 2, 128, 16, BF, prefix=64, seed=29).cuda()
    ws = sq.empty_workspace(sq.paged_attention_workspace_bytes(t.T, 8, 2, 128, t.prefix))
    outs = [torch.empty(t.T, t.Q.shape[1], device="cuda") for _ in range(2)]
    call(sq, t, workspace=ws, out=outs[0])
    graphs = []
    for o in outs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(sq, t, workspace=ws, out=o)
        graphs.append(g)
    for lens in ([300, 40, 500], [64, 400, 200], [0, 600, 65]):
        u = Batch(q, lens, 8, 2, 128, 16, BF, prefix=64, seed=31 + sum(lens), spare=200)
        w = min(t.table.shape[1], u.table.shape[1])
        pages = min(t.pages, u.pages)
        keep = (u.table[:, :w] < pages)
        t.table_d.fill_(-1)
        t.table_d[:, :w] = torch.where(keep, u.table[:, :w], torch.tensor(-1)).cuda().int()
        t.kv_len_d.copy_(u.kv_len)
        t.k_d[:pages] = torch.nan_to_num(u.k[:pages]).cuda()
        t.v_d[:pages] = torch.nan_to_num(u.v[:pages]).cuda()
        want = call(sq, t)
        for g, o in zip(graphs, outs):
            o.fill_(3)
            g.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want) and torch.equal(outs[1], want)
    assert sq.device_status() == sq.SQ_OK


def test_empty_calls(sq):
    t = Batch([0, 0], [3, 0], 8, 2, 64, 16, BF, seed=37, behind=4).cuda()
    out = torch.full((t.T, 8 * 64), 5.0, device="cuda")
    call(sq, t, out=out)
    assert torch.all(out == 5.0)
    none = sq.paged_attention(torch.empty(0, 512, device="cuda"), t.k_d, t.v_d, t.table_d,
                              t.q_start_d, t.kv_len_d)
    assert none.shape == (0, 512)
    empty = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = sq.paged_attention(t.Q_d, t.k_d, t.v_d, t.table_d[:0], empty, t.kv_len_d[:0])
    assert torch.all(out == 0)


def test_offsets_beyond_32_bits(sq):
    """A cache of more than 2^32 elements: the batch's pages at its far end."""
    D, page, Hkv = 128, 256, 8
    pages = (1 << 32) // (Hkv * page * D) + 40
    t = Batch([1, 3], [600, 500], 16, 8, D, page, BF, seed=41)
    big = [torch.zeros(pages, Hkv, page, D, dtype=BF, device="cuda") for _ in range(2)]
    shift = pages - t.pages
    big[0][shift:] = t.k.cuda()
    big[1][shift:] = t.v.cuda()
    t.cuda()
    t.k_d, t.v_d = big
    t.table_d = torch.where(t.table_d >= 0, t.table_d + shift, t.table_d).int()
    ref, bound = attention_ref(t, D ** -0.5)
    got = call(sq, t).double().cpu()
    assert float(((got - ref).abs() - bound).max()) <= 0

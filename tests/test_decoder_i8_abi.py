"""Refusals of the int8 cache's operators at the C boundary and in the binding: each bad
call returns its status before anything touches a GPU."""
import pytest
import torch

from smoothquant_w8a8_int8_gb300 import binding
from smoothquant_w8a8_int8_gb300 import build as sqbuild

OK, INVALID, ALIGN, UNSUP = 0, 1, 2, 3
A = 0x10000       # non-null, 16-byte aligned, never dereferenced
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    sqbuild.build()
    return binding.load()


SHAPE = [
    (dict(T=-1), INVALID), (dict(Hq=0), INVALID), (dict(Hkv=0), INVALID), (dict(Hq=6), INVALID),
    (dict(D=96), UNSUP), (dict(D=0), INVALID), (dict(page_size=48), UNSUP),
    (dict(page_size=8), UNSUP), (dict(page_size=512), UNSUP), (dict(num_pages=-1), INVALID),
    (dict(num_pages=0), INVALID), (dict(B=-1), INVALID), (dict(max_pages=-1), INVALID),
    (dict(T=(1 << 24) + 1), UNSUP), (dict(max_pages=1 << 27), UNSUP),
    (dict(num_pages=1 << 26), UNSUP), (dict(num_pages=1 << 62), UNSUP), (dict(ldq=508), INVALID),
    (dict(ldq=514), ALIGN), (dict(Hq=516, Hkv=4), UNSUP), (dict(q_start=None), INVALID),
    (dict(kv_len=None), INVALID), (dict(table=None), INVALID), (dict(k=None), INVALID),
    (dict(v=None), INVALID), (dict(ks=None), INVALID), (dict(vs=None), INVALID),
    (dict(Q=None), INVALID), (dict(k=A + 8), ALIGN), (dict(v=A + 2), ALIGN),
    (dict(ks=A + 4), ALIGN), (dict(vs=A + 8), ALIGN), (dict(q_start=A + 2), ALIGN),
    (dict(kv_len=A + 1), ALIGN), (dict(table=A + 2), ALIGN), (dict(Q=A + 4), ALIGN),
    (dict(T=0, Q=None, k=None, v=None, ks=None, vs=None, q_start=None), OK),
    (dict(B=0, Q=None, k=None, v=None, ks=None, vs=None, q_start=None, kv_len=None, table=None),
     OK),
]


def fix(a, kw):
    a.update(kw)
    if "ldq" not in kw:
        a["ldq"] = max(0, a["Hq"] * a["D"])
    return a


@pytest.mark.parametrize("kw,want", SHAPE + [
    (dict(rot=-8), INVALID), (dict(rot=72), INVALID), (dict(rot=12), ALIGN),
    (dict(rope=None), INVALID), (dict(rope=A + 8), ALIGN), (dict(positions=-1), INVALID),
    (dict(QKV=None), INVALID), (dict(QKV=A + 4), ALIGN),
])
def test_append(lib, kw, want):
    a = fix(dict(QKV=A, T=4, Hq=8, Hkv=4, D=64, rope=A, positions=100, rot=64, inter=0, q_start=A,
                 kv_len=A, B=2, table=A, max_pages=4, k=A, v=A, ks=A, vs=A, num_pages=8,
                 page_size=16, Q=A, ldq=0), kw)
    assert lib.sq_kv_append_i8(*a.values(), None) == want


@pytest.mark.parametrize("kw,want", SHAPE + [
    (dict(max_q=-1), INVALID), (dict(prefix=-1), INVALID), (dict(prefix=(1 << 30) + 1), UNSUP),
    (dict(prefix=5, pages=None), INVALID), (dict(prefix=5, pages=A + 2), ALIGN),
    (dict(scale=NAN), INVALID), (dict(scale=INF), INVALID), (dict(O=None), INVALID),
    (dict(O=A + 4), ALIGN), (dict(ws=None), INVALID), (dict(ws=A + 8), ALIGN),
])
def test_attention(lib, kw, want):
    a = fix(dict(Q=A, ldq=0, T=4, Hq=8, Hkv=4, D=64, k=A, v=A, ks=A, vs=A, num_pages=8,
                 page_size=16, table=A, max_pages=4, q_start=A, kv_len=A, B=2, max_q=1, pages=None,
                 prefix=0, scale=0.125, O=A, ws=A, ws_bytes=1 << 30), kw)
    assert lib.sq_paged_attention_i8(*a.values(), None) == want


def test_the_16_bit_calls_take_no_int8(lib):
    a = fix(dict(Q=A, ldq=0, T=4, Hq=8, Hkv=4, D=64, k=A, v=A, ctype=2, num_pages=8, page_size=16,
                 table=A, max_pages=4, q_start=A, kv_len=A, B=2, max_q=1, pages=None, prefix=0,
                 scale=0.125, O=A, ws=A, ws_bytes=1 << 30), {})
    assert lib.sq_paged_attention(*a.values(), None) == INVALID


@pytest.mark.parametrize("dtype,scales", [
    (torch.int8, (None, None)), (torch.int8, (0, None)), (torch.bfloat16, (0, 0)),
    (torch.bfloat16, (None, 0)), (torch.int32, (0, 0)), (torch.int8, (0, 0)),
])
def test_binding_refuses(dtype, scales):
    """Scales without an int8 cache, one without the other, other types, CPU tensors."""
    k = torch.zeros(4, 2, 16, 64, dtype=dtype)
    ints = torch.zeros(2, dtype=torch.int32)
    ks, vs = (None if s is None else torch.ones(4, 2, 16) for s in scales)
    with pytest.raises(ValueError):
        binding.kv_append(torch.zeros(1, 8 * 64), 4, k, k, ints.view(1, 2), ints, ints[:1],
                          k_scale=ks, v_scale=vs)
    with pytest.raises(ValueError):
        binding.paged_attention(torch.zeros(1, 256), k, k, ints.view(1, 2), ints, ints[:1],
                                k_scale=ks, v_scale=vs)

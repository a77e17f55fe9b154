"""Refusals of the decoder operators (RMS norm, rotation table, append, paged
attention) at the C boundary and in the binding: each bad call returns its
status before anything touches a GPU."""
import ctypes

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


def rms(lib, **kw):
    a = dict(H=A, residual=A, gamma=A, eps=1e-5, s=A, M=4, K=32, static=0.0, R=A, Y=A, Xq=A, sx=A,
             Xop=A, l1=A)
    a.update(kw)
    return lib.sq_rmsnorm_quant(*a.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(H=None), INVALID), (dict(gamma=None), INVALID), (dict(s=None), INVALID),
    (dict(sx=None), INVALID), (dict(Xq=None, Xop=None), INVALID), (dict(M=-1), INVALID),
    (dict(K=0), INVALID), (dict(K=24), ALIGN), (dict(K=16400), UNSUP),
    (dict(eps=-1e-9), INVALID), (dict(eps=NAN), INVALID), (dict(eps=INF), INVALID),
    (dict(static=-0.1), INVALID), (dict(static=NAN), INVALID), (dict(static=INF), INVALID),
    (dict(H=A + 4), ALIGN), (dict(residual=A + 8), ALIGN), (dict(gamma=A + 4), ALIGN),
    (dict(R=A + 4), ALIGN), (dict(Y=A + 4), ALIGN), (dict(sx=A + 2), ALIGN),
    (dict(l1=A + 1), ALIGN), (dict(Xop=A + 2), ALIGN),
    (dict(M=0, H=None, residual=None, gamma=None, s=None, sx=None, Xq=None, Xop=None), OK),
])
def test_rmsnorm(lib, kw, want):
    assert rms(lib, **kw) == want


@pytest.mark.parametrize("args,want", [
    ((None, 8, 16, A), INVALID), ((A, 8, 16, None), INVALID), ((A, -1, 16, A), INVALID),
    ((A, 8, -8, A), INVALID), ((A, 8, 12, A), ALIGN), ((A + 2, 8, 16, A), ALIGN),
    ((A, 8, 16, A + 8), ALIGN), ((A, 1 << 32, 16, A), UNSUP), ((A, 8, 1032, A), UNSUP),
    ((None, 0, 16, None), OK), ((None, 8, 0, None), OK),
])
def test_rope_table(lib, args, want):
    assert lib.sq_rope_table(*args, None) == want


SHAPE = [
    (dict(T=-1), INVALID), (dict(Hq=0), INVALID), (dict(Hkv=0), INVALID), (dict(Hq=6), INVALID),
    (dict(D=96), UNSUP), (dict(D=0), INVALID), (dict(page_size=48), UNSUP),
    (dict(page_size=8), UNSUP), (dict(page_size=512), UNSUP), (dict(ctype=2), INVALID),
    (dict(ctype=-1), INVALID), (dict(num_pages=-1), INVALID), (dict(num_pages=0), INVALID),
    (dict(B=-1), INVALID), (dict(max_pages=-1), INVALID), (dict(T=(1 << 24) + 1), UNSUP),
    (dict(max_pages=1 << 27), UNSUP), (dict(num_pages=1 << 26), UNSUP),
    (dict(num_pages=1 << 62), UNSUP), (dict(max_pages=1 << 62), UNSUP),
    (dict(ldq=508), INVALID), (dict(ldq=514), ALIGN), (dict(Hq=516, Hkv=4), UNSUP),
    (dict(Hq=8192, Hkv=8192), UNSUP), (dict(q_start=None), INVALID), (dict(kv_len=None), INVALID),
    (dict(table=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID),
    (dict(Q=None), INVALID), (dict(k=A + 8), ALIGN), (dict(v=A + 2), ALIGN),
    (dict(q_start=A + 2), ALIGN), (dict(kv_len=A + 1), ALIGN), (dict(table=A + 2), ALIGN),
    (dict(Q=A + 4), ALIGN),
    (dict(T=0, Q=None, k=None, v=None, q_start=None), OK),
    (dict(B=0, Q=None, k=None, v=None, q_start=None, kv_len=None, table=None), OK),
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
                 kv_len=A, B=2, table=A, max_pages=4, k=A, v=A, ctype=0, num_pages=8,
                 page_size=16, Q=A, ldq=0), kw)
    assert lib.sq_kv_append(*a.values(), None) == want


@pytest.mark.parametrize("kw,want", SHAPE + [
    (dict(max_q=-1), INVALID), (dict(prefix=-1), INVALID), (dict(prefix=(1 << 30) + 1), UNSUP),
    (dict(prefix=5, pages=None), INVALID), (dict(prefix=5, pages=A + 2), ALIGN),
    (dict(scale=NAN), INVALID), (dict(scale=INF), INVALID), (dict(O=None), INVALID),
    (dict(O=A + 4), ALIGN), (dict(ws=None), INVALID), (dict(ws=A + 8), ALIGN),
])
def test_attention(lib, kw, want):
    a = fix(dict(Q=A, ldq=0, T=4, Hq=8, Hkv=4, D=64, k=A, v=A, ctype=0, num_pages=8, page_size=16,
                 table=A, max_pages=4, q_start=A, kv_len=A, B=2, max_q=1, pages=None, prefix=0,
                 scale=0.125, O=A, ws=A, ws_bytes=1 << 30), kw)
    assert lib.sq_paged_attention(*a.values(), None) == want


def test_workspace_bytes(lib):
    n = ctypes.c_size_t(7)
    f = lib.sq_paged_attention_workspace_bytes
    assert f(4, 8, 4, 64, 0, None) == INVALID
    for args, want in (((-1, 8, 4, 64, 0), INVALID), ((4, 8, 3, 64, 0), INVALID),
                       ((4, 8, 4, 80, 0), UNSUP), ((4, 8, 4, 64, -1), INVALID)):
        assert f(*args, ctypes.byref(n)) == want and n.value == 0
    assert f(0, 8, 4, 64, 0, ctypes.byref(n)) == OK and n.value == 0


def test_binding_refuses_cpu_tensors_and_shapes():
    h = torch.zeros(2, 32)
    with pytest.raises(ValueError):
        binding.rmsnorm_quant(h, torch.ones(32), 1e-5, torch.ones(32))
    k = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    ints = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        binding.kv_append(torch.zeros(1, 8 * 64), 4, k, k, ints.view(1, 2), ints, ints[:1])
    with pytest.raises(ValueError):
        binding.paged_attention(torch.zeros(1, 256), k.float(), k.float(), ints.view(1, 2), ints,
                                ints[:1])
    with pytest.raises(ValueError):
        binding.rope_table(torch.zeros(4), 8)

"""Refusals of the gated linear and its packing at the C boundary and in the binding:
each bad call returns its status before anything touches a GPU."""
import ctypes

import pytest
import torch

from smoothquant_w8a8_int8_gb300 import binding
from smoothquant_w8a8_int8_gb300 import build as sqbuild

OK, INVALID, ALIGN, UNSUP = 0, 1, 2, 3
A = 0x10000       # non-null, 16-byte aligned, never dereferenced


@pytest.fixture(scope="module")
def lib():
    sqbuild.build()
    return binding.load()


@pytest.mark.parametrize("F,rows", [(0, 0), (1, 64), (32, 64), (33, 128), (5000, 10048), (-1, 0),
                                    (1 << 24, 1 << 25), ((1 << 24) + 1, 0)])
def test_rows(lib, F, rows):
    assert lib.sq_gated_rows(F) == rows


@pytest.mark.parametrize("kw,want", [
    (dict(Wg=None), INVALID), (dict(Wu=None), INVALID), (dict(s=None), INVALID),
    (dict(sw=None), INVALID), (dict(Wop=None), INVALID), (dict(F=-1), INVALID),
    (dict(K=0), INVALID), (dict(K=24), ALIGN), (dict(F=(1 << 24) + 1), UNSUP),
    (dict(Wg=A + 4), ALIGN), (dict(Wu=A + 8), ALIGN), (dict(s=A + 4), ALIGN),
    (dict(sw=A + 2), ALIGN), (dict(Wop=A + 2), ALIGN), (dict(l1=A + 1), ALIGN),
    (dict(F=0, Wg=None, Wu=None, s=None, sw=None, Wop=None), OK),
])
def test_pack(lib, kw, want):
    a = dict(Wg=A, Wu=A, s=A, F=8, K=32, sw=A, Wop=A, l1=A)
    a.update(kw)
    assert lib.sq_pack_gated_weight(*a.values(), None) == want


@pytest.mark.parametrize("kw,want", [
    (dict(X=None), INVALID), (dict(sx=None), INVALID), (dict(W=None), INVALID),
    (dict(sw=None), INVALID), (dict(Y=None), INVALID), (dict(M=-1), INVALID),
    (dict(F=-1), INVALID), (dict(K=0), INVALID), (dict(act=-1), INVALID), (dict(act=3), INVALID),
    (dict(K=24), ALIGN), (dict(K=133152), UNSUP), (dict(F=(1 << 24) + 1), UNSUP),
    (dict(X=A + 2), ALIGN), (dict(W=A + 8), ALIGN), (dict(Y=A + 4), ALIGN),
    (dict(sx=A + 2), ALIGN), (dict(sw=A + 1), ALIGN), (dict(x_l1=A + 2), ALIGN),
    (dict(w_l1=A + 2), ALIGN), (dict(bg=A + 2), ALIGN), (dict(bu=A + 1), ALIGN),
    (dict(ws=A + 8), ALIGN),
    (dict(M=0, X=None, sx=None, W=None, sw=None, Y=None), OK),
    (dict(F=0, X=None, sx=None, W=None, sw=None, Y=None), OK),
])
def test_gated(lib, kw, want):
    a = dict(X=A, sx=A, x_l1=None, W=A, sw=A, w_l1=None, bg=None, bu=None, M=4, F=8, K=32, act=0,
             Y=A, ws=None, ws_bytes=0)
    a.update(kw)
    assert lib.sq_linear_i8_gated(*a.values(), None) == want


def test_workspace_bytes(lib):
    n = ctypes.c_size_t(7)
    f = lib.sq_gated_workspace_bytes
    assert f(4, 8, 32, None) == INVALID
    for args, want in (((-1, 8, 32), INVALID), ((4, -8, 32), INVALID), ((4, 8, 0), INVALID),
                       ((4, (1 << 24) + 1, 32), UNSUP), ((4, 8, 133152), UNSUP), ((0, 8, 32), OK),
                       ((4, 0, 32), OK)):
        assert f(*args, ctypes.byref(n)) == want and n.value == 0


def test_binding_refuses_cpu_tensors():
    w = torch.zeros(4, 32)
    with pytest.raises(ValueError):
        binding.pack_gated_weight(w, w, torch.ones(32))
    with pytest.raises(ValueError):
        binding.linear_i8_gated(torch.zeros(2, 32, dtype=torch.bfloat16), torch.ones(2),
                                torch.zeros(64, 32, dtype=torch.bfloat16), torch.ones(64), 4)

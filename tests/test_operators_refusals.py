"""Refusals of the codebook operators: every call here is answered before anything is launched."""
import ctypes

import pytest
import torch

import exact_lloyd_means_assign_b200 as km
from exact_lloyd_means_assign_b200 import build as kbuild

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
P = ctypes.c_void_p
F = P(0x10000)          # never dereferenced: validation fails first
f = ctypes.c_float
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    kbuild.build()
    return km._load()


def test_pack4(lib):
    assert lib.km_pack4(None, 4, 10, F, None) == INVALID
    assert lib.km_pack4(F, 4, 10, None, None) == INVALID
    assert lib.km_pack4(F, 0, 10, F, None) == INVALID
    assert lib.km_pack4(F, 4, 0, F, None) == INVALID
    assert lib.km_pack4(F, 4, 1 << 31, F, None) == INVALID
    assert lib.km_pack4(F, 4, 10, P(0x10008), None) == INVALID


def _mv(lib, x=F, dt=1, M=1, packed=F, C=F, R=8, N=64, K=16, scales=None, group=0, y=F):
    return lib.km_matvec4(x, dt, M, packed, C, R, N, K, scales, group, y, None)


def test_matvec4(lib):
    for kw in (dict(x=None), dict(packed=None), dict(C=None), dict(y=None), dict(dt=5), dict(dt=-1), dict(M=0),
               dict(R=0), dict(N=0), dict(K=0), dict(N=1 << 31), dict(M=1 << 31), dict(x=P(0x10001)),
               dict(y=P(0x10001)), dict(packed=P(0x10004)), dict(C=P(0x10002)), dict(scales=P(0x10002), group=32),
               dict(group=32), dict(scales=F), dict(scales=F, group=-32)):
        assert _mv(lib, **kw) == INVALID, kw
    for kw in (dict(K=17), dict(scales=F, group=16), dict(scales=F, group=48)):
        assert _mv(lib, **kw) == UNSUPPORTED, kw


def _lk(lib, C=F, dt=1, ids=F, B=1, N=4, K=4, d=8, Y=F):
    return lib.km_lookup(C, dt, ids, B, N, K, d, f(1), Y, None)


def test_lookup(lib):
    for kw in (dict(C=None), dict(ids=None), dict(Y=None), dict(dt=3), dict(B=0), dict(N=0), dict(K=0), dict(d=0),
               dict(N=1 << 31), dict(K=1 << 31), dict(d=(1 << 20) + 1), dict(C=P(0x10001)), dict(Y=P(0x10001)),
               dict(ids=P(0x10002)), dict(dt=0, C=P(0x10002))):
        assert _lk(lib, **kw) == INVALID, kw


def _lg(lib, dY=F, dt=1, ids=F, B=1, N=4, K=4, d=8, dC=F, ot=0, ws=F, nb=BIG):
    return lib.km_lookup_grad(dY, dt, ids, B, N, K, d, f(1), dC, ot, 0, ws, nb, None)


def test_lookup_grad(lib):
    for kw in (dict(dY=None), dict(ids=None), dict(dC=None), dict(dt=3), dict(ot=3), dict(B=0), dict(N=0), dict(K=0),
               dict(d=0), dict(dY=P(0x10001)), dict(dC=P(0x10002)), dict(ids=P(0x10001)), dict(ws=P(0x10010))):
        assert _lg(lib, **kw) == INVALID, kw
    for kw in (dict(ot=2), dict(dt=0, ot=1), dict(B=1 << 16, N=1 << 15), dict(B=1 << 16, K=1 << 15)):
        assert _lg(lib, **kw) == UNSUPPORTED, kw
    need = lib.km_lookup_grad_workspace_size(1, 4, 4, 8)
    assert need > 0 and need % 256 == 0
    assert _lg(lib, ws=None) == WORKSPACE
    assert _lg(lib, nb=need - 1) == WORKSPACE
    assert lib.km_lookup_grad_workspace_size(1 << 16, 1 << 15, 4, 8) == 0
    assert lib.km_lookup_grad_workspace_size(0, 4, 4, 8) == 0


def _xe(lib, X=F, dt=1, C=F, ids=F, B=1, N=4, K=4, d=8, loss=F, lse=F, ws=F, nb=BIG):
    return lib.km_xent(X, dt, C, ids, B, N, K, d, f(1), loss, lse, ws, nb, None)


def test_xent(lib):
    for kw in (dict(X=None), dict(C=None), dict(ids=None), dict(loss=None, lse=None), dict(dt=4), dict(B=0), dict(N=0),
               dict(K=0), dict(d=0), dict(X=P(0x10001)), dict(C=P(0x10001)), dict(ids=P(0x10001)),
               dict(loss=P(0x10001)), dict(lse=P(0x10002)), dict(ws=P(0x10010)), dict(N=1 << 31)):
        assert _xe(lib, **kw) == INVALID, kw
    assert _xe(lib, B=1 << 16, N=1 << 16) == UNSUPPORTED
    assert _xe(lib, B=1, N=1 << 29, K=1 << 29) == UNSUPPORTED
    need = lib.km_xent_workspace_size(1, 4, 4, 8, 1)
    assert need > 0 and need % 256 == 0
    assert _xe(lib, nb=need - 1) == WORKSPACE and _xe(lib, ws=None) == WORKSPACE
    assert lib.km_xent_workspace_size(1, 4, 4, 8, 7) == 0


def _xg(lib, X=F, dt=1, C=F, ids=F, lse=F, g=F, B=1, N=4, K=4, d=8, dX=F, dC=F, ws=F, nb=BIG):
    return lib.km_xent_grad(X, dt, C, ids, lse, g, B, N, K, d, f(1), dX, dC, ws, nb, None)


def test_xent_grad(lib):
    for kw in (dict(X=None), dict(C=None), dict(ids=None), dict(lse=None), dict(dX=None, dC=None), dict(dt=4),
               dict(B=0), dict(N=0), dict(K=0), dict(d=0), dict(X=P(0x10001)), dict(C=P(0x10001)),
               dict(ids=P(0x10001)), dict(lse=P(0x10002)), dict(g=P(0x10002)), dict(dX=P(0x10001)),
               dict(dC=P(0x10001)), dict(ws=P(0x10010))):
        assert _xg(lib, **kw) == INVALID, kw
    assert _xg(lib, B=1 << 16, N=1 << 16) == UNSUPPORTED
    need = lib.km_xent_grad_workspace_size(1, 4, 4, 8, 1)
    assert need > 0 and need % 256 == 0
    assert _xg(lib, nb=need - 1) == WORKSPACE and _xg(lib, ws=None) == WORKSPACE
    # the scratch is bounded by a piece of the table, not by N x K
    n, k = 1 << 15, 1 << 17
    assert lib.km_xent_grad_workspace_size(1, n, k, 64, 1) < n * k * 2 // 4


def test_binding_refuses_host_tensors_and_wrong_shapes():
    h = torch.float16
    x, packed, C = torch.zeros((1, 64), dtype=h), torch.zeros((4, 32), dtype=torch.uint8), torch.zeros((4, 16))
    for call in (lambda: km.km_matvec4(x, packed, C), lambda: km.km_pack4(torch.zeros((2, 4), dtype=torch.uint8)),
                 lambda: km.km_lookup(torch.zeros((1, 4, 8)), torch.zeros((1, 3), dtype=torch.int32)),
                 lambda: km.km_lookup_grad(torch.zeros((1, 3, 8)), torch.zeros((1, 3), dtype=torch.int32), 4),
                 lambda: km.km_xent(torch.zeros((1, 3, 8)), torch.zeros((1, 4, 8)), torch.zeros((1, 3), dtype=torch.int32)),
                 lambda: km.km_xent_grad(torch.zeros((1, 3, 8)), torch.zeros((1, 4, 8)),
                                         torch.zeros((1, 3), dtype=torch.int32), torch.zeros((1, 3)))):
        with pytest.raises(ValueError):
            call()

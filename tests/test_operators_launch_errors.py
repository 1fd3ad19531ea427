"""Every launch of the codebook operators that fails makes its call fail.

The operators' host code is linked against stand-ins of the CUDA runtime (fake_cudart.c) that launch
nothing and let one numbered call fail; each entry point has to answer KM_ERR_CUDA whichever of its
launches and memsets that is."""
import ctypes
import os
import subprocess

import pytest

from exact_lloyd_means_assign_b200 import build as kbuild

ERR_CUDA = 4
P = ctypes.c_void_p
I64, F32, SZ = ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
A = P(0x100000)         # never dereferenced: nothing is launched
BIG = SZ(1 << 50)
F, H, BF = 0, 1, 2


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    objs = [os.path.join(kbuild.PKG, "_build", u[:-3] + ".o") for u in kbuild.UNITS if u != "km_lib.cu"]
    kbuild.build(force=not all(os.path.exists(o) for o in objs))
    out = str(tmp_path_factory.mktemp("fake") / "libops_fake.so")
    here = os.path.dirname(os.path.abspath(__file__))
    subprocess.run(["gcc", "-w", "-fPIC", "-shared", "-Wl,-Bsymbolic", "-o", out, os.path.join(here, "fake_cudart.c"), *objs,
                    "-lstdc++"], check=True)
    return ctypes.CDLL(out)


def _pack4(lib, R=64, N=128):
    return lib.km_pack4(A, I64(R), I64(N), A, None)


def _matvec4(lib, dt, M, R, N, group=0):
    return lib.km_matvec4(A, dt, I64(M), A, A, I64(R), I64(N), I64(16), A if group else None, I64(group), A, None)


def _lookup(lib, dt, B, N, K, d):
    return lib.km_lookup(A, dt, A, I64(B), I64(N), I64(K), I64(d), F32(1), A, None)


def _lookup_grad(lib, dt, B, N, K, d, acc=0):
    return lib.km_lookup_grad(A, dt, A, I64(B), I64(N), I64(K), I64(d), F32(1), A, F, acc, A, BIG, None)


def _xent(lib, dt, B, N, K, d):
    return lib.km_xent(A, dt, A, A, I64(B), I64(N), I64(K), I64(d), F32(1), A, A, A, BIG, None)


def _xent_grad(lib, dt, B, N, K, d, dX=A, dC=A, scale=1.0):
    return lib.km_xent_grad(A, dt, A, A, A, A, I64(B), I64(N), I64(K), I64(d), F32(scale), dX, dC, A, BIG, None)


CALLS = [
    (_pack4, ()),
    (_matvec4, (F, 1, 64, 128)), (_matvec4, (F, 3, 64, 128)), (_matvec4, (H, 1, 64, 128)), (_matvec4, (BF, 20, 64, 100, 32)),
    (_matvec4, (H, 16, 8192, 4096, 64)), (_matvec4, (BF, 40, 100000, 512)),
    (_lookup, (H, 1, 10, 20, 8)), (_lookup, (F, 2, 100, 20, 3)),
    (_lookup_grad, (H, 1, 100, 20, 8)), (_lookup_grad, (F, 1, 100000, 20, 8)), (_lookup_grad, (BF, 2, 1000000, 5000, 64, 1)),
    (_xent, (F, 1, 100, 200, 8)), (_xent, (H, 2, 100, 200, 12)), (_xent, (BF, 1, 1000, 2000, 256)),
    # one block, blocks that share row tiles, shares of whole row tiles, few table rows, padded rows
    (_xent_grad, (H, 1, 5, 7, 64)), (_xent_grad, (BF, 1, 3000, 1000, 128)), (_xent_grad, (H, 1, 128 * 148, 256, 64)),
    (_xent_grad, (H, 2, 900, 100, 36)), (_xent_grad, (BF, 1, 3000, 1000, 128, None)), (_xent_grad, (BF, 1, 5, 7, 128, A, None)),
    (_xent_grad, (H, 1, 300, 700, 136)), (_xent_grad, (BF, 2, 65536, 5000, 201)), (_xent_grad, (F, 1, 300, 700, 40)),
    (_xent_grad, (H, 1, 300, 700, 200, A, A, 0.0)),
]


@pytest.mark.parametrize("call,args", CALLS)
def test_every_failing_launch_fails_the_call(lib, call, args):
    lib.fake_reset(-1)
    assert call(lib, *args) == 0
    n = ctypes.c_int.in_dll(lib, "fake_calls").value
    assert n >= 1
    for i in range(n):
        lib.fake_reset(i)
        assert call(lib, *args) == ERR_CUDA, f"call {i} of {n} failed unnoticed"
    lib.fake_reset(-1)
    assert call(lib, *args) == 0

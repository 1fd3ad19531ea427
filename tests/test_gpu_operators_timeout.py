"""The bounded waits of the 4-bit products' and the cross entropy's kernels, run out on purpose.

The limit is cut to 20 ms and a test-only switch makes the first block (or SM pair) of each tensor-core
kernel withhold its first stage. The call returns, the error word reports the timeout, and the next
call, which needs the same tensor memory, gives the bits it gave before."""
import time

import pytest
import torch

import exact_lloyd_means_assign_b200 as km

pytestmark = pytest.mark.gpu


def _products(dev, dtype, R, N, M, group):
    g = torch.Generator(device=dev).manual_seed(R)
    codes = torch.randint(0, 16, (R, N), generator=g, device=dev, dtype=torch.uint8)
    C = torch.randn((R, 16), generator=g, device=dev)
    x = torch.randn((M, N), generator=g, device=dev).to(dtype)
    s = torch.rand((R, -(-N // group)), generator=g, device=dev) if group else None
    packed = km.km_pack4(codes)
    return lambda: (km.km_matvec4(x, packed, C, s, group),)


def _xent(dev, dtype, N, K, d, grad):
    g = torch.Generator(device=dev).manual_seed(N)
    X = torch.randn((1, N, d), generator=g, device=dev).to(dtype)
    C = (torch.randn((1, K, d), generator=g, device=dev) * (2 / d ** 0.5)).to(dtype)
    ids = torch.randint(0, K, (1, N), generator=g, device=dev, dtype=torch.int32)
    if not grad:
        return lambda: km.km_xent(X, C, ids)
    _, lse = km.km_xent(X, C, ids)
    return lambda: km.km_xent_grad(X, C, ids, lse)


CASES = [
    ("mma.sync, several stages", lambda dev: _products(dev, torch.float16, 5000, 4096, 1, 0)),
    ("mma.sync, one stage, scales", lambda dev: _products(dev, torch.bfloat16, 40, 100, 20, 32)),
    ("tcgen05, tiles of their own", lambda dev: _products(dev, torch.bfloat16, 40000, 1024, 16, 64)),
    ("tcgen05, a cluster to a tile", lambda dev: _products(dev, torch.float16, 1024, 32768, 30, 0)),
    ("loss", lambda dev: _xent(dev, torch.bfloat16, 3000, 2000, 256, False)),
    ("gradients of long rows", lambda dev: _xent(dev, torch.float16, 3000, 2000, 256, True)),
    ("gradients of short rows", lambda dev: _xent(dev, torch.float16, 3000, 2000, 128, True)),
    ("gradients of short rows, few table rows", lambda dev: _xent(dev, torch.bfloat16, 9000, 100, 40, True)),
]


@pytest.mark.parametrize("name,make", CASES, ids=[c[0] for c in CASES])
def test_a_withheld_stage_times_out_and_the_next_call_is_clean(cuda_device, name, make):
    call = make(cuda_device)
    want = call()
    torch.cuda.synchronize()
    assert km.km_device_error() == 0
    old = km.km_debug_wait_limit(20_000_000)          # 20 ms
    try:
        km.km_debug_inject(3)
        t = time.perf_counter()
        call()
        code = km.km_device_error()                    # synchronises
        elapsed = time.perf_counter() - t
    finally:
        km.km_debug_inject(0)
        km.km_debug_wait_limit(old)
    assert code & 1, "the withheld stage must make a wait run out"
    assert elapsed < 5.0
    again = call()
    torch.cuda.synchronize()
    assert km.km_device_error() == 0
    for a, b in zip(again, want):
        assert torch.equal(a, b)

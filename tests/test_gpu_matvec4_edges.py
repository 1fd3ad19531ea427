"""4-bit products where they can go wrong beside the shapes of test_gpu_matvec4.py."""
import pytest
import torch

import exact_lloyd_means_assign_b200 as km

pytestmark = pytest.mark.gpu


def _fp64(x, codes, C, s=None, group=0):
    W = torch.gather(C.to(x.dtype).double(), 1, codes.long())
    if s is not None:
        W = W * s.double().repeat_interleave(group, 1)[:, :W.shape[1]]
    return x.double() @ W.t()


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("R,N,M", [(16, 1 << 22, 1), (20, 1 << 21, 10), (40, 1 << 21, 20), (128, 1 << 20, 16),
                                   (200, 1 << 20, 30), (5, 1 << 21, 12), (3, (1 << 21) + 5, 30), (7, (1 << 20) + 3, 1)])
def test_long_rows_do_not_drift(cuda_device, dtype, R, N, M):
    # all terms positive. An addition of the tensor cores is off by at most 2^-23 of the running sum and
    # 1024 of them by 1024 2^-23; the fp32 additions behind them (at most 2^22 / 1024 / 16 and a few) have
    # no common direction, nor has the result's rounding: half a step u over sqrt(R M) results, four deviations
    g = torch.Generator(device=cuda_device).manual_seed(R)
    codes = torch.randint(0, 16, (R, N), generator=g, device=cuda_device, dtype=torch.uint8)
    C = (torch.rand((R, 16), generator=g, device=cuda_device) + 0.5) / 64
    x = ((torch.rand((M, N), generator=g, device=cuda_device) + 0.5) * (2.0 ** 16 / N)).to(dtype)
    y = km.km_matvec4(x, km.km_pack4(codes), C)
    torch.cuda.synchronize()
    assert km.km_device_error() == 0
    ref = _fp64(x, codes, C)
    drift = (((y.double() - ref) * ref).sum() / (ref * ref).sum()).item()
    u = torch.finfo(dtype).eps / 2
    assert abs(drift) <= 1024 * 2.0 ** -23 + 4 * u / (R * M) ** 0.5 + 2.0 ** -18


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M", [1, 12, 30])
@pytest.mark.parametrize("group", [32, 64, 128, 96, 384])
def test_an_infinite_last_scale_stays_an_infinity(cuda_device, dtype, M, group):
    # rows that end inside a step: what lies behind their end is no part of the last group
    R, N = 8200, 4136
    g = torch.Generator(device=cuda_device).manual_seed(group)
    codes = torch.randint(0, 16, (R, N), generator=g, device=cuda_device, dtype=torch.uint8)
    C = torch.rand((R, 16), generator=g, device=cuda_device) + 0.5
    x = ((torch.rand((M, N), generator=g, device=cuda_device) + 0.5) / 64).to(dtype)
    s = torch.rand((R, -(-N // group)), generator=g, device=cuda_device) + 0.5
    s[5::7, -1] = float("inf")
    y = km.km_matvec4(x, km.km_pack4(codes), C, s, group)
    torch.cuda.synchronize()
    want = torch.zeros(R, dtype=torch.bool, device=cuda_device)
    want[5::7] = True
    assert (torch.isposinf(y) == want[None]).all() and torch.isfinite(y[:, ~want]).all()

"""Products with 4-bit codebook weights against the fp64 definition.

Tolerance per output, from the arithmetic: the codebook values are rounded to the tokens' type on
both sides, products are exact or rounded in fp32 and summed in fp32. An fp32 sum of N terms taken
as chunks of 16 has a depth of N / 16 + 64 additions at most in every variant, each off by at most
2^-23 of the running magnitude (truncating adders included), so the sum is off by at most
(N / 16 + 64) 2^-23 sum |terms|; the result is rounded once, half a step of its type.
"""
import numpy as np
import pytest
import torch

import exact_lloyd_means_assign_b200 as km
import oracle
from oracle import operators as op

pytestmark = pytest.mark.gpu

DTYPES = [torch.float16, torch.bfloat16, torch.float32]


def _inputs(R, N, M, K, group, dtype, dev, seed=0):
    g = torch.Generator().manual_seed(seed)
    codes = torch.randint(0, K, (R, N), generator=g, dtype=torch.uint8)
    C = torch.randn((R, K), generator=g) * 0.1
    x = torch.randn((M, N), generator=g).to(dtype)
    s = (torch.rand((R, -(-N // group)), generator=g) + 0.1) if group else None
    return codes.to(dev), C.to(dev), x.to(dev), None if s is None else s.to(dev)


def _check(y, x, codes, C, s, group):
    dtype = x.dtype
    Cr = oracle.round_to_dtype(C.cpu(), dtype)
    ref, mag = op.matvec4(oracle.as_f64(x.cpu()), codes.cpu().numpy(), Cr,
                          None if s is None else s.cpu().double().numpy(), group)
    N = x.shape[1]
    tol = torch.finfo(dtype).eps / 2 * np.abs(ref) + (N / 16 + 64) * 2.0 ** -23 * mag
    tol += 2.0 ** -25 if dtype == torch.float16 else 0.0      # half a step of its subnormals
    err = np.abs(y.cpu().double().numpy() - ref)
    assert (err <= tol).all(), f"worst excess {(err - tol).max()} at {np.unravel_index((err - tol).argmax(), err.shape)}"


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("R,N,M,K,group", [
    (1, 1, 1, 1, 0), (1, 1, 1, 16, 32), (3, 7, 2, 4, 0), (16, 32, 1, 16, 32), (17, 33, 9, 16, 32),
    (64, 128, 8, 16, 64), (100, 1999, 3, 8, 0), (65, 1000, 5, 16, 128), (33, 4097, 1, 15, 96),
    (48, 513, 16, 16, 64), (130, 2048, 17, 2, 256), (16, 16384, 1, 16, 32), (7, 20001, 2, 16, 4096),
    (300, 640, 33, 16, 160), (4099, 64, 1, 16, 0), (40, 4096, 70, 16, 128)])
def test_matvec4(cuda_device, dtype, R, N, M, K, group):
    codes, C, x, s = _inputs(R, N, M, K, group, dtype, cuda_device, seed=R + N + M)
    packed = km.km_pack4(codes)
    assert np.array_equal(packed.cpu().numpy(), op.pack4(codes.cpu().numpy()))
    y = km.km_matvec4(x, packed, C, s, group)
    torch.cuda.synchronize()
    _check(y, x, codes, C, s, group)
    assert torch.equal(y, km.km_matvec4(x, packed, C, s, group))


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("R,N,M,K,group", [
    (8192, 4096, 9, 16, 128), (8200, 4104, 16, 16, 64), (4100, 8200, 12, 15, 32), (16500, 2048, 33, 16, 0),
    (2049, 16392, 17, 16, 96), (1024, 32768, 40, 16, 256), (300000, 120, 10, 16, 32), (129, 262144, 9, 4, 4096),
    (33000, 1032, 32, 16, 160)])
def test_more_tokens_on_large_weights(cuda_device, dtype, R, N, M, K, group):
    # the form that decodes into tensor memory: few and many row tiles, reductions shared by a
    # cluster, every class of scale groups, ragged rows, steps and tokens; rows sampled
    codes, C, x, s = _inputs(R, N, M, K, group, dtype, cuda_device, seed=R + N + M)
    packed = km.km_pack4(codes)
    y = km.km_matvec4(x, packed, C, s, group)
    torch.cuda.synchronize()
    assert km.km_device_error() == 0
    g = torch.Generator().manual_seed(1)
    rows = torch.unique(torch.cat([torch.arange(0, min(R, 3)), torch.arange(max(0, R - 130), R),
                                   torch.randint(0, R, (200,), generator=g)])).to(cuda_device)
    _check(y[:, rows], x, codes[rows], C[rows], None if s is None else s[rows], group)
    assert torch.equal(y, km.km_matvec4(x, packed, C, s, group))
    # every token's result is that of the token alone, up to the order of the sums
    one = km.km_matvec4(x[-1:].contiguous(), packed, C, s, group)
    _check(one[:, rows], x[-1:], codes[rows], C[rows], None if s is None else s[rows], group)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_infinities_stay_in_their_row_of_large_weights(cuda_device, dtype):
    R, N, M, group = 8192, 4168, 11, 128
    codes, C, x, s = _inputs(R, N, M, 15, group, dtype, cuda_device, seed=16)
    full = torch.cat([C, torch.full((R, 1), float("inf"), device=cuda_device)], 1).contiguous()   # code 15, unused
    full[7, 0] = float("inf")               # code 0 is also what the padding holds
    codes[7] = torch.where(codes[7] == 0, torch.ones_like(codes[7]), codes[7])
    s[130] = float("nan")
    x[4] = float("nan")
    x[6, 17] = float("inf")
    y = km.km_matvec4(x, km.km_pack4(codes), full, s, group).float()
    torch.cuda.synchronize()
    toks, rows = torch.ones(M, dtype=torch.bool), torch.ones(R, dtype=torch.bool)
    toks[4] = toks[6] = False
    rows[130] = False
    assert torch.isnan(y[4]).all() and torch.isnan(y[:, 130]).all() and not torch.isfinite(y[6]).any()
    assert torch.isfinite(y.cpu()[toks][:, rows]).all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_codes_beyond_the_codebook_stand_for_zero(cuda_device, dtype):
    codes, C, x, _ = _inputs(20, 300, 2, 16, 0, dtype, cuda_device, seed=5)
    C = C[:, :5].contiguous()
    y = km.km_matvec4(x, km.km_pack4(codes), C)
    _check(y, x, codes, C, None, 0)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M", [1, 12])
def test_infinities_stay_in_their_row(cuda_device, dtype, M):
    # an infinite codebook value that no code of the row names, NaN scales of one row, NaN in one
    # token, NaN behind the end of a ragged x: each shows only where the formula has it
    R, N, group = 40, 1000, 128
    codes, C, x, s = _inputs(R, N, M, 15, group, dtype, cuda_device, seed=6)
    full = torch.cat([C, torch.full((R, 1), float("inf"), device=cuda_device)], 1).contiguous()   # code 15
    full[7, 0] = float("inf")
    codes[7] = torch.where(codes[7] == 0, torch.ones_like(codes[7]), codes[7])   # nor row 7's code 0
    s[3] = float("nan")
    if M > 1:
        x[4] = float("nan")
    y = km.km_matvec4(x, km.km_pack4(codes), full, s, group).float()
    torch.cuda.synchronize()
    rows = torch.ones(R, dtype=torch.bool)
    rows[3] = False
    toks = torch.ones(M, dtype=torch.bool)
    if M > 1:
        toks[4] = False
    assert torch.isnan(y[:, 3]).all() and (M == 1 or torch.isnan(y[4]).all())
    good = y.cpu()[toks][:, rows]
    assert torch.isfinite(good).all()
    C2 = full.clone()
    C2[:, 15] = 0
    C2[7, 0] = 0
    s2 = s.clone()
    s2[3] = 0
    x2 = torch.where(torch.isnan(x), torch.zeros_like(x), x)
    _check(torch.where(torch.isnan(y), torch.zeros_like(y), y).to(dtype), x2, codes, C2, s2, group)


def test_unaligned_tokens_and_given_output(cuda_device):
    codes, C, x, s = _inputs(50, 512, 3, 16, 128, torch.bfloat16, cuda_device, seed=7)
    packed = km.km_pack4(codes)
    want = km.km_matvec4(x, packed, C, s, 128)
    buf = torch.empty(x.numel() + 1, dtype=x.dtype, device=cuda_device)
    shifted = buf[1:].view(x.shape)          # contiguous, two bytes off every vector boundary
    shifted.copy_(x)
    out = torch.full((3 * 50 + 2,), 7.0, dtype=x.dtype, device=cuda_device)
    y = km.km_matvec4(shifted, packed, C, s, 128, y=out[1:-1].view(3, 50))
    torch.cuda.synchronize()
    torch.testing.assert_close(y, want, rtol=2.0 ** -7, atol=1e-2)
    _check(y, x, codes, C, s, 128)
    assert out[0] == 7 and out[-1] == 7


def test_encoded_rows_multiply(cuda_device):
    """The whole way: rows fitted and encoded by this library, packed and multiplied."""
    g = torch.Generator().manual_seed(8)
    W = (torch.randn((64, 1024), generator=g) * 0.02).half().to(cuda_device)
    C = km.km_init_grid1d(W[..., None].contiguous(), 16)
    km.km_fit(W[..., None].contiguous(), C, 10)
    codes = km.km_encode1d(W, C)
    x = torch.randn((1, 1024), generator=g).half().to(cuda_device)
    y = km.km_matvec4(x, km.km_pack4(codes), C)
    torch.cuda.synchronize()
    _check(y, x, codes, C.view(64, 16), None, 0)
    # and it is near the product with the weights themselves: 16 values per row carry most of them
    dense = x.float() @ W.float().t()
    assert (y.float() - dense).norm() < 0.2 * dense.norm()


def test_captured_replays_and_other_streams(cuda_device):
    codes, C, x, s = _inputs(200, 2048, 2, 16, 64, torch.float16, cuda_device, seed=9)
    packed = km.km_pack4(codes)
    want = km.km_matvec4(x, packed, C, s, 64)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y1 = km.km_matvec4(x, packed, C, s, 64, stream=side)
    y2 = km.km_matvec4(x, packed, C, s, 64, stream=side.cuda_stream)
    torch.cuda.synchronize()
    assert torch.equal(y1, want) and torch.equal(y2, want)
    xs, ys = x.clone(), torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        km.km_matvec4(xs, packed, C, s, 64, y=ys)
    for k in (1.0, 2.0):
        xs.copy_(x * k)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(ys, km.km_matvec4(x * k, packed, C, s, 64))


def test_offsets_beyond_32_bits(cuda_device):
    # 2^33 codes: the byte offset of the last rows is above 2^32
    R, N = 270336, 32768
    packed = torch.zeros((R, N // 2), dtype=torch.uint8, device=cuda_device)
    packed[-1] = 0x21
    C = torch.zeros((R, 16), device=cuda_device)
    C[:, 0], C[:, 1], C[:, 2] = 1.0, 2.0, 4.0
    x = torch.full((1, N), 2.0 ** -10, dtype=torch.float16, device=cuda_device)
    y = km.km_matvec4(x, packed, C)
    torch.cuda.synchronize()
    assert (y[0, :-1] == 32).all() and y[0, -1] == 96

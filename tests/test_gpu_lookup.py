"""Table lookups (bit-exact) and the table's gradient against the fp64 definition.

The lookup rounds scale * value to fp32 and then to the type: the same two roundings in torch give
the same bits. The gradient sums n_k terms of a row in fp32, each addition off by at most 2^-24 of
the running magnitude, scales (2^-24) and rounds to the output type (half a step), so
|error| <= eps_out / 2 |ref| + (n_k + 2) 2^-24 sum |terms|.
"""
import numpy as np
import pytest
import torch

import exact_lloyd_means_assign_b200 as km
import oracle
from oracle import operators as op

pytestmark = pytest.mark.gpu

DTYPES = [torch.float16, torch.bfloat16, torch.float32]
SHAPES = [(1, 1, 1, 1), (1, 1, 5, 8), (2, 3, 4, 7), (1, 100, 50, 128), (3, 65, 17, 20), (1, 33, 1000, 1024),
          (2, 200, 9, 130), (5, 17, 3, 2), (1, 300, 40, 4096), (40, 5, 6, 16), (1, 64, 2, 1030)]


def _ids(B, N, K, g, kind):
    if kind == "one":
        return torch.full((B, N), K - 1, dtype=torch.int32)
    if kind == "none":
        return torch.full((B, N), -1, dtype=torch.int32)
    ids = torch.randint(0, K, (B, N), generator=g, dtype=torch.int32)
    if kind == "skewed":
        ids = torch.where(torch.rand((B, N), generator=g) < 0.6, torch.zeros_like(ids), ids)
    if kind == "holes":
        r = torch.rand((B, N), generator=g)
        ids[r < 0.2] = -1
        ids[(r >= 0.2) & (r < 0.3)] = K
        ids[(r >= 0.3) & (r < 0.35)] = -2 ** 31
        ids[(r >= 0.35) & (r < 0.4)] = 2 ** 31 - 1
    return ids


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("B,N,K,d", SHAPES)
def test_lookup(cuda_device, dtype, B, N, K, d):
    g = torch.Generator().manual_seed(B * N + K + d)
    C = torch.randn((B, K, d), generator=g).to(dtype).to(cuda_device)
    for kind, scale in (("random", 1.0), ("holes", 11.313708)):
        ids = _ids(B, N, K, g, kind)
        Y = km.km_lookup(C, ids.to(cuda_device), scale)
        torch.cuda.synchronize()
        ok = (ids >= 0) & (ids < K)
        idx = ids.clamp(0, K - 1).long()[..., None].expand(B, N, d)
        ref = torch.gather(C.cpu(), 1, idx).float() * torch.tensor(scale, dtype=torch.float32)
        ref = torch.where(ok[..., None], ref, torch.zeros(())).to(dtype)
        assert torch.equal(Y.cpu(), ref)


def _check_grad(dC, dY, ids, K, scale, prev=None):
    s32 = float(np.float32(scale))
    ref, mag, cnt = op.lookup_grad(oracle.as_f64(dY.cpu()), ids.cpu().numpy(), K, s32)
    if prev is not None:
        ref, mag = ref + oracle.as_f64(prev.cpu()), mag + np.abs(oracle.as_f64(prev.cpu()))
    tol = torch.finfo(dC.dtype).eps / 2 * np.abs(ref) + (cnt[..., None] + 2) * 2.0 ** -24 * mag
    tol += 2.0 ** -25 if dC.dtype == torch.float16 else 0.0
    got = dC.cpu().double().numpy()
    err = np.abs(got - ref)
    assert (err <= tol).all(), f"worst excess {(err - tol).max()}"
    if prev is None:
        assert (got[cnt == 0] == 0).all()
    else:
        assert np.array_equal(got[cnt == 0], oracle.as_f64(prev.cpu())[cnt == 0])


@pytest.mark.parametrize("dtype,out", [(torch.float16, torch.float16), (torch.float16, torch.float32),
                                       (torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32),
                                       (torch.float32, torch.float32)])
@pytest.mark.parametrize("B,N,K,d", SHAPES)
def test_lookup_grad(cuda_device, dtype, out, B, N, K, d):
    g = torch.Generator().manual_seed(B + N * K + d)
    dY = torch.randn((B, N, d), generator=g).to(dtype).to(cuda_device)
    for kind in ("random", "holes", "one", "none", "skewed"):
        ids = _ids(B, N, K, g, kind).to(cuda_device)
        dC = km.km_lookup_grad(dY, ids, K, 1.25, out_dtype=out)
        torch.cuda.synchronize()
        _check_grad(dC, dY, ids, K, 1.25)
        prev = torch.randn((B, K, d), generator=g).to(out).to(cuda_device)
        acc = km.km_lookup_grad(dY, ids, K, 1.25, dC=prev.clone(), accumulate=True)
        torch.cuda.synchronize()
        _check_grad(acc, dY, ids, K, 1.25, prev)


@pytest.mark.parametrize("B,N,K,d", [(1, 5000, 7, 8), (1, 40000, 3, 32), (2, 9000, 70000, 4), (1, 70000, 300000, 1),
                                     (1, 300000, 20, 16), (3, 4096, 1, 64), (1, 4097, 256, 64), (1, 4096, 257, 20),
                                     (1, 65536, 1024, 8), (1, 65537, 1025, 8), (5, 16484, 1200, 8), (3, 30000, 5000, 4),
                                     (100, 1000, 50, 8), (1, 600000, 300, 2), (2, 540000, 3000, 1), (9, 8192, 1024, 16)])
@pytest.mark.parametrize("kind", ["random", "skewed", "holes", "one"])
def test_lookup_grad_large_sorts(cuda_device, B, N, K, d, kind):
    # several sort tiles and passes, runs over many ranges; small integers, so every sum is exact
    g = torch.Generator().manual_seed(N + K)
    ids = _ids(B, N, K, g, kind)
    dY = torch.randint(-8, 9, (B, N, d), generator=g).to(torch.float16)
    dC = km.km_lookup_grad(dY.to(cuda_device), ids.to(cuda_device), K, 0.5)
    again = km.km_lookup_grad(dY.to(cuda_device), ids.to(cuda_device), K, 0.5)
    torch.cuda.synchronize()
    ok = (ids >= 0) & (ids < K)
    rows = torch.where(ok, ids.long() + torch.arange(B)[:, None] * K, B * K).flatten()
    ref = torch.zeros((B * K + 1, d), dtype=torch.float64).index_add_(0, rows, dY.flatten(0, 1).double())
    assert torch.equal(dC.cpu().double(), ref[:-1].view(B, K, d) * 0.5)
    assert torch.equal(dC, again)


def test_lookup_grad_is_deterministic(cuda_device):
    g = torch.Generator().manual_seed(3)
    ids = _ids(1, 50000, 2000, g, "skewed").to(cuda_device)
    dY = torch.randn((1, 50000, 96), generator=g).to(torch.bfloat16).to(cuda_device)
    first = km.km_lookup_grad(dY, ids, 2000, 3.0)
    for _ in range(5):
        assert torch.equal(first, km.km_lookup_grad(dY, ids, 2000, 3.0))


@pytest.mark.parametrize("dtype", DTYPES)
def test_nan_of_ignored_tokens_and_unnamed_rows(cuda_device, dtype):
    g = torch.Generator().manual_seed(4)
    B, N, K, d = 1, 90, 20, 24
    ids = _ids(B, N, K, g, "holes")
    ids[ids == 5] = 6
    bad = (ids < 0) | (ids >= K)
    dY = torch.randn((B, N, d), generator=g).to(dtype)
    dY[bad] = float("nan")
    C = torch.randn((B, K, d), generator=g).to(dtype)
    C[0, 5] = float("inf")
    Y = km.km_lookup(C.to(cuda_device), ids.to(cuda_device), 2.0)
    dC = km.km_lookup_grad(dY.to(cuda_device), ids.to(cuda_device), K, 2.0)
    torch.cuda.synchronize()
    assert torch.isfinite(Y).all() and (Y.cpu()[bad] == 0).all()
    clean = dY.clone()
    clean[bad] = 0
    _check_grad(dC, clean, ids, K, 2.0)


def test_gradient_matches_differences_of_the_lookup(cuda_device):
    # sum(Y * dY) is linear in C: its difference quotient is the gradient, exactly in integers
    g = torch.Generator().manual_seed(5)
    C = torch.randint(-4, 5, (2, 6, 8), generator=g).float().to(cuda_device)
    dY = torch.randint(-4, 5, (2, 30, 8), generator=g).float().to(cuda_device)
    ids = _ids(2, 30, 6, g, "holes").to(cuda_device)
    dC = km.km_lookup_grad(dY, ids, 6, 2.0)
    base = (km.km_lookup(C, ids, 2.0) * dY).sum()
    for b, k, j in ((0, 0, 0), (1, 3, 7), (0, 5, 2), (1, 1, 1)):
        C2 = C.clone()
        C2[b, k, j] += 1
        assert (km.km_lookup(C2, ids, 2.0) * dY).sum() - base == dC[b, k, j]


def test_unaligned_buffers_and_guard_bytes(cuda_device):
    g = torch.Generator().manual_seed(6)
    for dtype in DTYPES:
        C = torch.randn((1, 10, 32), generator=g).to(dtype).to(cuda_device)
        ids = _ids(1, 50, 10, g, "random").to(cuda_device)
        want = km.km_lookup(C, ids, 1.5)
        src = torch.empty(C.numel() + 1, dtype=dtype, device=cuda_device)
        src[1:].copy_(C.flatten())
        dst = torch.full((want.numel() + 2,), 7.0, dtype=dtype, device=cuda_device)
        km.km_lookup(src[1:].view(C.shape), ids, 1.5, Y=dst[1:-1].view(want.shape))
        torch.cuda.synchronize()
        assert torch.equal(dst[1:-1].view(want.shape), want) and dst[0] == 7 and dst[-1] == 7
        gwant = km.km_lookup_grad(want, ids, 10, 1.5, out_dtype=dtype)
        out = torch.full((gwant.numel() + 2,), 7.0, dtype=dtype, device=cuda_device)
        ysrc = torch.empty(want.numel() + 1, dtype=dtype, device=cuda_device)
        ysrc[1:].copy_(want.flatten())
        km.km_lookup_grad(ysrc[1:].view(want.shape), ids, 10, 1.5, dC=out[1:-1].view(gwant.shape))
        torch.cuda.synchronize()
        assert torch.equal(out[1:-1].view(gwant.shape), gwant) and out[0] == 7 and out[-1] == 7


def test_workspace_guard_streams_and_capture(cuda_device):
    g = torch.Generator().manual_seed(7)
    B, N, K, d = 2, 6000, 500, 64
    ids = _ids(B, N, K, g, "skewed").to(cuda_device)
    dY = torch.randn((B, N, d), generator=g).half().to(cuda_device)
    want = km.km_lookup_grad(dY, ids, K, 2.0)
    need = km._load().km_lookup_grad_workspace_size(B, N, K, d)
    ws = torch.full((need + 256,), 0xAB, dtype=torch.uint8, device=cuda_device)
    got = km.km_lookup_grad(dY, ids, K, 2.0, ws=ws[:need])
    torch.cuda.synchronize()
    assert torch.equal(got, want) and (ws[need:] == 0xAB).all()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    s1 = km.km_lookup_grad(dY, ids, K, 2.0, stream=side)
    s2 = km.km_lookup(want.to(torch.float16), ids, 1.0, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(s1, want) and torch.equal(s2, km.km_lookup(want.to(torch.float16), ids, 1.0))
    ids_s, out = ids.clone(), torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        km.km_lookup_grad(dY, ids_s, K, 2.0, dC=out, ws=ws[:need])
    for roll in (0, 1, 77):
        ids_s.copy_(ids.roll(roll, 1))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, km.km_lookup_grad(dY, ids.roll(roll, 1).contiguous(), K, 2.0))


def test_lookup_offsets_beyond_32_bits(cuda_device):
    # 2^32 + values of output, and a table whose last rows lie beyond 2^32 elements
    K, d, N = 1 << 20, 4128, 64
    C = torch.zeros((1, K, d), dtype=torch.float16, device=cuda_device)
    C[0, K - 1] = 3
    ids = torch.full((1, N), K - 1, dtype=torch.int32, device=cuda_device)
    Y = km.km_lookup(C, ids, 2.0)
    torch.cuda.synchronize()
    assert (Y == 6).all()
    dC = km.km_lookup_grad(Y, ids, K, 1.0, dC=C, out_dtype=torch.float16)
    torch.cuda.synchronize()
    assert (dC[0, K - 1] == 6 * N).all() and not dC[0, : K - 1].any()

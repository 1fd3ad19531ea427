"""Cross entropy where it can go wrong beside the shapes of test_gpu_xent.py: rows and labels that
part the lanes of a warp, masked table rows, weights of very different sizes, long reductions.
Tolerances are those of test_gpu_xent.py (the arithmetic stands there) unless a test derives its own.
"""
import pytest
import torch

import exact_lloyd_means_assign_b200 as km
from test_gpu_xent import DTYPES, _check_grad, _check_loss, _inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("N,K,d", [(129, 257, 160), (145, 300, 288), (31, 500, 200), (257 + 17, 131, 136),
                                   (97, 150, 128), (33, 290, 40), (161, 100, 72)])
def test_rows_and_labels_that_part_a_warp(cuda_device, dtype, N, K, d):
    # the last warp's rows end inside it, and every point has a label, so that in each chunk of
    # columns some lanes have work that the others have not
    X, C, ids, g = _inputs(1, N, K, d, dtype, cuda_device, seed=N)
    ids = (torch.arange(N, device=cuda_device, dtype=torch.int32) * 37 % K)[None].contiguous()
    for scale in (1.0, -0.5):
        loss, lse = km.km_xent(X, C, ids, scale)
        dX, dC = km.km_xent_grad(X, C, ids, lse, g, scale)
        torch.cuda.synchronize()
        assert km.km_device_error() == 0
        _check_loss(X, C, ids, scale, loss, lse)
        _check_grad(X, C, ids, g, scale, dX, dC, parts=2 if K <= 128 and d <= 128 and dtype != torch.float32 else 1)


def _fp64(X, C, ids, g, scale=1.0, block=8192):
    """(loss, lse, dX, dC) of one batch in 64 bits on the device."""
    C6, N = C.double(), X.shape[0]
    loss, lse = torch.zeros(N, dtype=torch.float64, device=X.device), torch.zeros(N, dtype=torch.float64, device=X.device)
    rX, rC = torch.zeros(X.shape, dtype=torch.float64, device=X.device), torch.zeros_like(C6)
    for n in range(0, N, block):
        s = slice(n, n + block)
        x = X[s].double()
        z = scale * (x @ C6.t())
        lse[s] = torch.logsumexp(z, 1)
        ok = (ids[s] >= 0) & (ids[s] < C.shape[0])
        rows, t = ok.nonzero()[:, 0], ids[s][ok].long()
        loss[n + rows] = lse[n + rows] - z[rows, t]
        p = torch.exp(z - lse[s, None])
        p[rows, t] -= 1
        w = torch.zeros(x.shape[0], dtype=torch.float64, device=X.device)
        w[rows] = g[s][rows].double() * scale
        p[~ok] = 0
        p *= w[:, None]
        rX[s] = p @ C6
        rC += p.t() @ torch.where(ok[:, None], x, torch.zeros_like(x))
    return loss, lse, rX, rC


def _drift(got, ref):
    """The common relative error of the entries: the slope of got over ref, less one."""
    return (((got.double() - ref) * ref).sum() / (ref * ref).sum()).item()


def _one_signed(N, K, d, dtype, dev, g):
    # positive points against positive rows; labels among the first ten rows, which are zero, so that
    # every gradient beyond them is a sum of terms of one sign
    gen = torch.Generator(device=dev).manual_seed(1)
    X = torch.randn((N, d), generator=gen, device=dev).abs().to(dtype)
    C = (torch.randn((K, d), generator=gen, device=dev).abs() * (0.2 / d ** 0.5)).to(dtype)
    C[:10] = 0
    ids = torch.randint(0, 10, (N,), generator=gen, device=dev, dtype=torch.int32)
    return X, C, ids, torch.full((N,), g, device=dev)


# An addition of the tensor cores is off by at most 2^-23 of the running sum; 1024 of them, the most that
# one accumulator takes, by 1024 2^-23 of a sum of one sign. The rest (exponentials, lse: 2^-18 at these
# logits; roundings of P and of the result, which have no common direction) stays below 2^-16.
MAX_DRIFT = 1024 * 2.0 ** -23 + 2.0 ** -16


@pytest.mark.parametrize("N,K,d,g", [
    (1 << 18, 1 << 14, 128, 1.0),       # dC: 1771 tiles of points to a block
    (1 << 22, 100, 64, 0.25),           # few table rows, P in two parts: 221 tiles of 16 products
    (1 << 14, 1 << 17, 128, 1.0),       # dX: 885 tiles of table rows to a block
])
def test_long_reductions_of_short_rows_do_not_drift(cuda_device, N, K, d, g):
    X, C, ids, gr = _one_signed(N, K, d, torch.float16, cuda_device, g)
    loss, lse = km.km_xent(X[None], C[None], ids[None])
    dX, dC = km.km_xent_grad(X[None], C[None], ids[None], lse, gr[None])
    torch.cuda.synchronize()
    assert km.km_device_error() == 0
    _, _, rX, rC = _fp64(X, C, ids, gr, block=(1 << 27) // K)
    assert abs(_drift(dC[0, 10:], rC[10:])) <= MAX_DRIFT
    assert abs(_drift(dX[0], rX)) <= MAX_DRIFT


@pytest.mark.parametrize("N,K,d,g", [
    (65536, 2048, 1024, 0.25),          # dC: 1024 steps of 64 points
    (1024, 1 << 17, 512, 1.0),          # dX: 2048 steps of 64 table rows
])
def test_long_reductions_of_long_rows_do_not_drift(cuda_device, N, K, d, g):
    X, C, ids, gr = _one_signed(N, K, d, torch.float16, cuda_device, g)
    loss, lse = km.km_xent(X[None], C[None], ids[None])
    dX, dC = km.km_xent_grad(X[None], C[None], ids[None], lse, gr[None])
    torch.cuda.synchronize()
    assert km.km_device_error() == 0
    _, _, rX, rC = _fp64(X, C, ids, gr, block=(1 << 27) // K)
    assert abs(_drift(dC[0, 10:], rC[10:])) <= MAX_DRIFT
    assert abs(_drift(dX[0], rX)) <= MAX_DRIFT


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("low", ["inf", "lowest", "large"])
@pytest.mark.parametrize("d", [40, 64, 136])
@pytest.mark.parametrize("K,dead", [(700, [(0, 200), (500, 700)]), (90, [(0, 64), (80, 90)]), (1500, [(100, 1400)]),
                                    (300, [(0, 1), (64, 128), (256, 300)]), (600, [(0, 256)])])
def test_masked_table_rows(cuda_device, dtype, low, d, K, dead):
    # a column of ones against a column of the table that holds minus infinity, the type's lowest value or
    # another large one where a row is masked: whole chunks and tiles of logits are, and the result is that of the table
    # without those rows
    N = 150
    X, C, _, g = _inputs(1, N, K, d, dtype, cuda_device, seed=K + d)
    g = g.abs() + 1.0 / N
    X[..., -1] = 1
    C[..., -1] = 0
    alive = torch.ones(K, dtype=torch.bool, device=cuda_device)
    for a, b in dead:
        alive[a:b] = False
    sub = C[:, alive].contiguous()
    to_sub = torch.cumsum(alive, 0) - 1
    rows = alive.nonzero()[:, 0]
    ids = rows[torch.arange(N, device=cuda_device) * 7 % len(rows)].to(torch.int32)[None].contiguous()
    ids[0, ::9] = -1
    ids_sub = torch.where(ids >= 0, to_sub[ids.clamp(min=0).long()].to(torch.int32), ids)
    for scale in (1.0, -0.5):
        value = {"inf": -float("inf"), "lowest": torch.finfo(dtype).min, "large": -3e4 if dtype == torch.float16 else -1e30}[low]
        C[:, ~alive, -1] = value if scale > 0 else -value
        loss, lse = km.km_xent(X, C, ids, scale)
        dX, dC = km.km_xent_grad(X, C, ids, lse, g, scale)
        torch.cuda.synchronize()
        assert km.km_device_error() == 0
        _check_loss(X, sub, ids_sub, scale, loss, lse)
        # (with infinities the formula's dX is NaN: 0 times infinity)
        _check_grad(X, sub, ids_sub, g, scale, dX if low != "inf" else None, dC[:, alive].contiguous())
        assert (dC[:, ~alive] == 0).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d", [64, 136])
def test_every_row_masked(cuda_device, dtype, d):
    X, C, ids, _ = _inputs(1, 70, 400, d, dtype, cuda_device, seed=d)
    X[..., -1] = 1
    C[..., -1] = -float("inf")
    loss, lse = km.km_xent(X, C, torch.full_like(ids, -1))
    assert (lse == -float("inf")).all() and (loss == 0).all()
    for low in (torch.finfo(dtype).min, torch.finfo(dtype).min / 2, -3e4):
        C[..., -1] = low
        loss, lse = km.km_xent(X, C, ids)
        # (at 32-bit ranges log K is below the resolution of lse)
        assert torch.isfinite(loss).all()
        assert ((lse.double() - low).abs() <= 2.0 ** -8 * abs(low) + 20).all()


@pytest.mark.parametrize("d,N,K", [(64, 300, 700), (128, 500, 90), (100, 20000, 300)])
@pytest.mark.parametrize("low", [-12, -22, -26])
def test_rows_of_small_weight_beside_large_ones(cuda_device, d, N, K, low):
    # every second point weighs 2^low of the others; its row of dX is what it is alone: two roundings to half a
    # step of the type (P, where sums over the table average it, and the result), and half a step of fp16's subnormals
    dtype = torch.float16
    X, C, ids, _ = _inputs(1, N, K, d, dtype, cuda_device, seed=d)
    g = torch.full((1, N), 2.0 ** 13, device=cuda_device)
    g[0, 1::2] = 2.0 ** (13 + low)
    _, lse = km.km_xent(X, C, ids)
    dX, dC = km.km_xent_grad(X, C, ids, lse, g)
    _, _, rX, rC = _fp64(X[0], C[0], ids[0], g[0])
    small, ref = dX[0, 1::2].double(), rX[1::2]
    rounding = torch.clamp(ref.abs() * 2.0 ** -11, min=2.0 ** -25)
    # (a row's entries of P are off by half a step each, 2^-11 of a probability, with independent signs: in the
    # norm over a row's d values at most 2^-11 |p - label| |C|, the label's entry having no such error)
    assert (small - ref).norm() <= rounding.norm() + 2.0 ** -11 * ref.norm()
    assert ((small - ref).abs() <= 2 * rounding + 2.0 ** -11 * ref.norm(dim=1, keepdim=True) * 4 / d ** 0.5).all()
    # and equal bits whatever the others weigh
    g2 = g.clone()
    g2[0, ::2] = 2.0 ** (13 + low)
    alone, _ = km.km_xent_grad(X, C, ids, lse, g2)
    assert torch.equal(alone[0, 1::2], dX[0, 1::2])


@pytest.mark.parametrize("dtype,d", [(torch.float16, 136), (torch.bfloat16, 200), (torch.float16, 130), (torch.float32, 40),
                                     (torch.float16, 72)])
def test_guards_streams_capture_and_unaligned_rows(cuda_device, dtype, d):
    B, N, K = 2, 300, 700
    X, C, ids, g = _inputs(B, N, K, d, dtype, cuda_device, seed=d)
    loss, lse = km.km_xent(X, C, ids, 0.5)
    dX, dC = km.km_xent_grad(X, C, ids, lse, g, 0.5)

    def off(t):
        # one element off every vector boundary, between guard values
        buf = torch.full((t.numel() + 2,), 7.0, dtype=t.dtype, device=t.device)
        buf[1:-1].copy_(t.flatten())
        return buf, buf[1:-1].view(t.shape)
    for x_off, c_off in ((True, True), (True, False), (False, True)):
        X1, C1 = off(X)[1] if x_off else X, off(C)[1] if c_off else C
        bx, dX1 = off(torch.zeros_like(dX))
        bc, dC1 = off(torch.zeros_like(dC))
        l1, s1 = km.km_xent(X1, C1, ids, 0.5)
        km.km_xent_grad(X1, C1, ids, s1, g, 0.5, dX=dX1, dC=dC1)
        torch.cuda.synchronize()
        _check_loss(X, C, ids, 0.5, l1, s1)
        _check_grad(X, C, ids, g, 0.5, dX1, dC1)
        for b in (bx, bc):
            assert b[0] == 7 and b[-1] == 7
    lib, dt = km._load(), km._dt(dtype)
    n1, n2 = lib.km_xent_workspace_size(B, N, K, d, dt), lib.km_xent_grad_workspace_size(B, N, K, d, dt)
    w1 = torch.full((n1 + 4096,), 0xFF, dtype=torch.uint8, device=cuda_device)
    w2 = torch.full((n2 + 4096,), 0xFF, dtype=torch.uint8, device=cuda_device)
    l2, s2 = km.km_xent(X, C, ids, 0.5, ws=w1[:n1])
    x2, c2 = km.km_xent_grad(X, C, ids, s2, g, 0.5, ws=w2[:n2])
    torch.cuda.synchronize()
    assert torch.equal(l2, loss) and torch.equal(x2, dX) and torch.equal(c2, dC)
    assert (w1[n1:] == 0xFF).all() and (w2[n2:] == 0xFF).all()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    l3, s3 = km.km_xent(X, C, ids, 0.5, stream=side)
    x3, c3 = km.km_xent_grad(X, C, ids, s3, g, 0.5, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(l3, loss) and torch.equal(x3, dX) and torch.equal(c3, dC)
    Xs, lo, ls, gx, gc = X.clone(), torch.empty_like(loss), torch.empty_like(lse), torch.empty_like(dX), torch.empty_like(dC)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        km.km_xent(Xs, C, ids, 0.5, loss=lo, lse=ls, ws=w1[:n1])
        km.km_xent_grad(Xs, C, ids, ls, g, 0.5, dX=gx, dC=gc, ws=w2[:n2])
    for k in (1.0, 0.5):
        Xs.copy_(X * k)
        graph.replay()
        torch.cuda.synchronize()
        rl, rs = km.km_xent(X * k, C, ids, 0.5)
        rx, rc = km.km_xent_grad(X * k, C, ids, rs, g, 0.5)
        assert torch.equal(lo, rl) and torch.equal(gx, rx) and torch.equal(gc, rc)


@pytest.mark.parametrize("dtype,B,N,K,d", [(torch.bfloat16, 2, 32768, 5000, 136), (torch.float16, 3, 20000, 4600, 200),
                                           (torch.float32, 2, 40000, 4000, 24)])
def test_batches_whose_table_comes_in_pieces(cuda_device, dtype, B, N, K, d):
    # more entries of P than are held at a time: several pieces of the table, and dC by batch
    X, C, ids, g = _inputs(B, N, K, d, dtype, cuda_device, seed=N)
    loss, lse = km.km_xent(X, C, ids)
    dX, dC = km.km_xent_grad(X, C, ids, lse, g)
    torch.cuda.synchronize()
    assert km.km_device_error() == 0
    u = torch.finfo(dtype).eps / 2
    for b in range(B):
        rl, rs, rX, rC = _fp64(X[b], C[b], ids[b], g[b])
        assert (lse[b] - rs).abs().max() < 2e-5 and (loss[b] - rl).abs().max() < 4e-5
        # relative norms: half a step of P and of the result at most, plus fp32 sums; fp16 results near its
        # subnormals half a step of those each
        for got, ref in ((dX[b], rX), (dC[b], rC)):
            floor = (2.0 ** -25 * ref.numel() ** 0.5 / ref.norm()).item() if dtype == torch.float16 else 0.0
            assert ((got.double() - ref).norm() / ref.norm()).item() < 2 * u + 2e-5 + floor


def test_small_probabilities_keep_their_bits_in_fp16(cuda_device):
    # table rows that no point has as its label, and points of equal weight: dC of such a row is a sum of
    # probabilities near 2^-22 times that weight alone. Held as they are they would lie among fp16's subnormals
    # (steps of 2^-24: errors of 2^-4 each, 2^-9 and more in a row's sum over 1024 points); times 2^14 they keep all
    # their bits, half a step u = 2^-11 each, and the result is rounded by half a step once more.
    N, K, d, live = 1024, 3000, 64, 20
    for d in (64, 136):
        gen = torch.Generator(device=cuda_device).manual_seed(d)
        X = torch.rand((N, d), generator=gen, device=cuda_device).half() + 0.5
        C = torch.rand((K, d), generator=gen, device=cuda_device).half() * (4 / d)
        X[:, -1] = 1
        C[:, -1] = -8.0
        C[:live, -1] = 4.0                       # the labelled rows take almost all of the softmax
        ids = torch.randint(0, live, (1, N), generator=gen, device=cuda_device, dtype=torch.int32)
        g = torch.full((1, N), 1024.0, device=cuda_device)
        _, lse = km.km_xent(X[None], C[None], ids)
        _, dC = km.km_xent_grad(X[None], C[None], ids, lse, g, want_dX=False)
        torch.cuda.synchronize()
        _, _, _, rC = _fp64(X, C, ids[0], g[0])
        p = rC[live:].abs().max() / (1024 * N)
        assert 2.0 ** -24 < p < 2.0 ** -18, p
        got, ref = dC[0, live:].double(), rC[live:]
        assert ((got - ref).norm() / ref.norm()).item() <= 2 * 2.0 ** -11
        assert ((got - ref).abs() <= 2.0 ** -10 * ref.abs()).all()


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("d", [16384, 16392, 65536, 65541])
def test_logits_of_very_long_rows_do_not_drift(cuda_device, dtype, d):
    # all products positive, one table row: lse is the logit. At most 1024 truncated additions, 2^-23 of the sum
    # each, or d rounded ones, whose errors of 2^-24 have both signs (4 sqrt(d) of them)
    g = torch.Generator(device=cuda_device).manual_seed(d)
    X = (torch.rand((1, 70, d), generator=g, device=cuda_device) + 0.5).to(dtype)
    C = (torch.rand((1, 1, d), generator=g, device=cuda_device) + 0.5).to(dtype)
    ids = torch.zeros((1, 70), dtype=torch.int32, device=cuda_device)
    loss, lse = km.km_xent(X, C, ids, 2.0 ** -10)
    ref = (X[0].double() @ C[0, 0].double()) * 2.0 ** -10
    assert ((lse[0] - ref).abs() <= (1024 * 2.0 ** -23 + 4 * d ** 0.5 * 2.0 ** -24) * ref).all()
    assert (loss.abs() <= 2.0 ** -22 * ref).all()
    C2 = torch.cat([C * 0, C], 1).contiguous()
    loss, lse = km.km_xent(X, C2, ids, 2.0 ** -13)
    dX, dC = km.km_xent_grad(X, C2, ids, lse, None, 2.0 ** -13)
    torch.cuda.synchronize()
    assert km.km_device_error() == 0
    rl, rs, rX, rC = _fp64(X[0], C2[0], ids[0], torch.ones(70, device=cuda_device), 2.0 ** -13)
    u = torch.finfo(dtype).eps / 2
    assert (loss[0] - rl).abs().max() <= 2 * MAX_DRIFT * rs.max() + 2.0 ** -20
    # (P by half a step, with an exponent off by the logit's drift; the result by half a step or fp16's subnormal one)
    for got, ref in ((dX[0], rX), (dC[0], rC)):
        floor = 2.0 ** -25 if dtype == torch.float16 else 0.0
        assert ((got.double() - ref).abs() <= (2.1 * u + 4 * MAX_DRIFT * rs.max()) * ref.abs() + 70 * floor).all()

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
@pytest.mark.parametrize("N,K,d", [(150, 700, 64), (150, 90, 40), (2000, 5000, 128), (150, 700, 136), (9, 20000, 24)])
def test_infinite_table_rows_stay_in_their_column(cuda_device, dtype, N, K, d):
    # dX of a table with infinities is NaN in their column at most; elsewhere it is what finite masks give
    X, C, ids, g = _inputs(1, N, K, d, dtype, cuda_device, seed=N + K)
    X[..., -1] = 1
    C[..., -1] = 0
    dead = torch.arange(K, device=cuda_device) % 3 == 1
    ids = (torch.arange(N, device=cuda_device, dtype=torch.int32) * 3 % (K - 2) // 3 * 3)[None].contiguous()
    ids[0, ::5] = -1
    got = {}
    for low in (-3e4, -float("inf")):
        C[:, dead, -1] = low
        _, lse = km.km_xent(X, C, ids)
        got[low] = km.km_xent_grad(X, C, ids, lse, g)
    (x0, c0), (x1, c1) = got.values()
    assert torch.equal(x0[..., :-1], x1[..., :-1]) and torch.equal(c0, c1)
    assert (x1[0, ::5, :-1] == 0).all()


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


@pytest.mark.parametrize("d,N,K", [(64, 300, 700), (128, 500, 90), (100, 20000, 300), (136, 300, 700), (201, 70, 2100), (512, 4000, 300),
                                   (136, 70000, 2500)])
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
    # and equal bits whatever the others weigh (long rows: as far as 2^24 below the largest)
    g2 = g.clone()
    g2[0, ::2] = 2.0 ** (13 + low)
    alone, _ = km.km_xent_grad(X, C, ids, lse, g2)
    if d <= 128 or low >= -24:
        assert torch.equal(alone[0, 1::2], dX[0, 1::2])
    # dC sums over all of them. An entry of P is off by half a step (and by an exponent's 2^-18), which may fall together
    # over the points; so may 2^-36 of the largest terms, those of a weight of 2^13 (an entry of P holds 14 bits below
    # its row's weight and 10 more, a point of up to 2^3 lies 2^11 below fp16's top)
    tC = torch.zeros_like(rC)
    for n in range(0, N, 8192):
        sl = slice(n, n + 8192)
        p = torch.softmax(X[0, sl].double() @ C[0].double().t(), 1)
        ok = (ids[0, sl] >= 0) & (ids[0, sl] < K)
        p[ok, ids[0, sl][ok].long()] -= 1
        p = p.abs() * torch.where(ok, g[0, sl], torch.zeros_like(g[0, sl]))[:, None]
        p += 2.0 ** (13 - 36 + 11) * ok[:, None]
        tC += p.t() @ X[0, sl].double().abs()
    tC = tC * (2.0 ** -11 + 2.0 ** -18 + (1024 + N / 8192) * 2.0 ** -23) + 2.0 ** -11 * rC.abs() + 2.0 ** -25
    # (results beyond fp16's largest number, 65504, are infinite)
    fits, beyond = rC.abs() + tC < 65504, rC.abs() - tC > 65536
    over = ((dC[0].double() - rC).abs() - tC)[fits]
    assert (over <= 0).all(), (over.max().item(), (over > 0).sum().item())
    assert (dC[0].double()[beyond] == torch.sign(rC[beyond]) * float("inf")).all()


@pytest.mark.parametrize("scale_x", [1.0, 2.0 ** -12, 2.0 ** 9])
@pytest.mark.parametrize("d", [64, 136])
def test_table_rows_of_small_weights_alone(cuda_device, d, scale_x):
    # the labels of the light points are rows that no heavy point has, and whose probabilities under the heavy ones
    # vanish: what these rows of dC hold comes from weights of 2^-12 of the largest
    N, K = 400, 300
    gen = torch.Generator(device=cuda_device).manual_seed(d)
    X = (torch.randn((N, d), generator=gen, device=cuda_device) * scale_x).half()
    C = (torch.randn((K, d), generator=gen, device=cuda_device) * (2 / d ** 0.5)).half()
    light = torch.arange(N, device=cuda_device) % 2 == 1
    X[:, -1] = torch.where(light, -4.0, 4.0) * scale_x
    C[:, -1] = torch.where(torch.arange(K, device=cuda_device) < 150, 6.0, -6.0).half()
    ids = torch.where(light, 150 + torch.arange(N, device=cuda_device) % 150, torch.arange(N, device=cuda_device) % 150).to(torch.int32)
    g = torch.where(light, 1.0 / 4, 1024.0).float() / scale_x
    scale = 1 / scale_x
    _, lse = km.km_xent(X[None], C[None], ids[None], scale)
    dX, dC = km.km_xent_grad(X[None], C[None], ids[None], lse, (g * scale_x)[None], scale)
    torch.cuda.synchronize()
    _, _, rX, rC = _fp64(X, C, ids, g * scale_x, scale)
    # (roundings of P and of the result, half a step each, in the norm of the light rows; fp16's subnormals)
    ref, got = rC[150:], dC[0, 150:].double()
    assert (got - ref).norm() <= 2 * 2.0 ** -11 * ref.norm() + 2.0 ** -25 * ref.numel() ** 0.5
    ref, got = rX[light], dX[0][light].double()
    assert (got - ref).norm() <= 2 * 2.0 ** -11 * ref.norm() + 2.0 ** -25 * ref.numel() ** 0.5


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d,K", [(136, 260), (201, 300), (72, 90)])
def test_points_without_labels_of_other_forms_may_hold_anything(cuda_device, dtype, d, K):
    # long rows, padded ones, and few table rows, with weights that differ by many orders
    X, C, ids, g = _inputs(2, 150, K, d, dtype, cuda_device, seed=d)
    g = g * torch.where(torch.arange(150, device=cuda_device) % 3 == 0, 2.0 ** -9, 1.0)[None]
    bad = (ids < 0) | (ids >= K)
    assert bad.any()
    X[bad] = 0
    _, lse = km.km_xent(X, C, ids)
    dX0, dC0 = km.km_xent_grad(X, C, ids, lse, g)
    for fill in (float("nan"), float("inf"), 6e4):
        X2, g2 = X.clone(), g.clone()
        X2[bad] = fill
        g2[bad] = fill
        loss, lse2 = km.km_xent(X2, C, ids)
        dX, dC = km.km_xent_grad(X2, C, ids, lse2, g2)
        torch.cuda.synchronize()
        assert (loss[bad] == 0).all() and torch.isfinite(loss).all()
        assert torch.equal(dX, dX0) and torch.equal(dC, dC0)


@pytest.mark.parametrize("N,K,d", [((1 << 25) + 3, 3, 64), ((1 << 24) + 5, 40, 136), (5, (1 << 24) + 5, 136), (70000, 70001, 8)])
def test_sizes_beyond_32_bit_offsets(cuda_device, N, K, d):
    # points or a table of more than 2^31 values, more than 2^32 logits; equal rows repeat with a period, so
    # that the results are those of one period, and the last rows show the largest offsets
    dtype, P = torch.bfloat16, 96
    gen = torch.Generator(device=cuda_device).manual_seed(N % 1000)
    x = torch.randn((min(N, P), d), generator=gen, device=cuda_device).to(dtype)
    c = (torch.randn((min(K, P), d), generator=gen, device=cuda_device) * (2 / d ** 0.5)).to(dtype)
    at_x, at_c = torch.arange(N, device=cuda_device) % x.shape[0], torch.arange(K, device=cuda_device) % c.shape[0]
    X, C = x[at_x][None], c[at_c][None]
    ids = (at_x % min(K, c.shape[0])).to(torch.int32)[None]
    g = torch.full((1, N), 1.0 / N, device=cuda_device)
    loss, lse = km.km_xent(X, C, ids)
    dX, dC = km.km_xent_grad(X, C, ids, lse, g)
    torch.cuda.synchronize()
    assert km.km_device_error() == 0
    # one period of points against the table's distinct rows, each as often as it stands there
    times = torch.bincount(at_c, minlength=c.shape[0]).double()
    z = x.double() @ c.double().t()
    rs = torch.logsumexp(z + times.log(), 1)
    t = ids[0, :x.shape[0]].long()
    rl = rs - z.gather(1, t[:, None])[:, 0]
    # (a logit's sum, the exponentials, and at most 320 additions of a tile's and the tiles' sums)
    ez = ((d / 16 + 66) * 2.0 ** -23 * (x.double().abs() @ c.double().abs().t())).max()
    els = ez + 2.0 ** -21 * (z.abs().max() + 2) + 320 * 2.0 ** -24 + 2.0 ** -23 * rs.abs().max()
    assert (lse[0].double() - rs[at_x]).abs().max() <= els
    assert (loss[0].double() - rl[at_x]).abs().max() <= els + ez + 2.0 ** -22 * (rs.abs().max() + z.abs().max())
    p = torch.exp(z - rs[:, None])
    rX = p @ (c.double() * times[:, None]) - c[t].double()
    # (roundings of P and of the result, half a step each, in the norm of a period, first and last)
    u = torch.finfo(dtype).eps / 2
    for sl in (slice(0, x.shape[0]), slice(N - x.shape[0], N)):
        ref = rX[at_x[sl]] / N
        assert (dX[0, sl].double() - ref).norm() <= (2 * u + 2 * els + 2.0 ** -12) * ref.norm()
    # dC of a row: all points' softmax parts, and its label's where it is the first of its kind
    count = torch.bincount(at_x, minlength=x.shape[0]).double()
    soft = (p * count[:, None]).t() @ x.double() / N
    lab = torch.zeros_like(soft).index_add_(0, t, x.double() * count[:, None]) / N
    mag = (p * count[:, None]).t() @ x.double().abs() / N + torch.zeros_like(soft).index_add_(0, t, x.double().abs() * count[:, None]) / N
    for k in {0, min(K, c.shape[0]) - 1, K // 2, K - 1}:
        ref = soft[at_c[k]] - (lab[at_c[k]] if k < c.shape[0] else 0)
        tol = u * ref.abs() + (u + MAX_DRIFT + 2 * els + 2.0 ** -15) * mag[at_c[k]] + 1e-30
        assert ((dC[0, k].double() - ref).abs() <= tol).all()


def test_the_loss_over_very_many_table_rows(cuda_device):
    # 2^24 table rows, alike by the dozen, so that the roundings of the tiles' sums would all point one way. What is
    # left: 20 16-bit products to a logit, an exponential's 2^-21, 64 additions within a tile's half, ten of the joined sums
    N, K, d = 4, (1 << 24) + 5, 16
    gen = torch.Generator(device=cuda_device).manual_seed(3)
    x = torch.randn((N, d), generator=gen, device=cuda_device).half()
    c = (torch.randn((96, d), generator=gen, device=cuda_device) * 0.5).half()
    at = torch.arange(K, device=cuda_device) % 96
    _, lse = km.km_xent(x[None], c[at][None], torch.zeros((1, N), dtype=torch.int32, device=cuda_device))
    z = x.double() @ c.double().t()
    rs = torch.logsumexp(z + torch.bincount(at, minlength=96).double().log(), 1)
    tol = 4 * 2.0 ** -23 * (x.double().abs() @ c.double().abs().t()).max() + 2.0 ** -21 + 80 * 2.0 ** -24 + 2.0 ** -23 * rs.max()
    assert ((lse[0].double() - rs).abs() <= tol).all()

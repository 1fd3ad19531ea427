"""Softmax cross entropy over a table and its gradients against the fp64 definition.

Tolerances, from the arithmetic. A logit is an fp32 sum of d products; in every variant its depth is
at most d / 16 + 64 additions (one more 16-product step for padding), each off by at most 2^-23 of
the running magnitude, so e_z = (d / 16 + 66) 2^-23 scale sum |x c|. An exponential is off by its
argument's rounding, 2^-22 (|z - reference| + 1), and by 2^-21 of itself. A row's sum of
exponentials is positive and at most 256 + tiles additions deep. Hence
  e_lse  = max e_z + 2^-21 (max |z| + 2) + (320 + K / 64) 2^-24,
  e_loss = e_lse + e_z(label).
P carries the relative error e_z + e_lse + 2^-21 (max |z| + 2) on its probability part and is rounded
to its type, half a step u (fp16: P is scaled by f with max |w| f = 2^14, so its absolute floor is half a subnormal step, 2^-25 2^-14 max |w|):
  e_P = |w| (p (e_z + e_lse + ...) + u |p - [label]|) + floor.
The products with C and X then give e_P |C| + depth 2^-23 |P| |C| + half a step of the result.
"""
import numpy as np
import pytest
import torch

import exact_lloyd_means_assign_b200 as km
import oracle
from oracle import operators as op

pytestmark = pytest.mark.gpu

DTYPES = [torch.float16, torch.bfloat16, torch.float32]
SHAPES = [(1, 1, 1, 1), (1, 1, 2, 8), (2, 3, 5, 7), (1, 128, 128, 64), (1, 129, 257, 128), (3, 50, 300, 24),
          (1, 300, 1000, 136), (2, 257, 130, 72), (1, 5, 4099, 33), (1, 1000, 3, 16), (4, 64, 64, 512),
          (1, 200, 520, 1000), (1, 70, 2100, 256), (1, 1, 5000, 64), (1, 2000, 1, 100),
          (2, 384, 640, 128), (3, 129, 385, 65), (1, 40, 1500, 129), (1, 6000, 40, 128), (1, 9, 6000, 72)]


def _inputs(B, N, K, d, dtype, dev, seed, scale_rows=2.0):
    g = torch.Generator().manual_seed(seed)
    X = torch.randn((B, N, d), generator=g).to(dtype)
    C = (torch.randn((B, K, d), generator=g) * (scale_rows / d ** 0.5)).to(dtype)
    ids = torch.randint(0, K, (B, N), generator=g, dtype=torch.int32)
    if N > 4:
        r = torch.rand((B, N), generator=g)
        ids[r < 0.1] = -1
        ids[(r >= 0.1) & (r < 0.15)] = K
        ids[(r >= 0.15) & (r < 0.17)] = 2 ** 31 - 1
    gr = torch.randn((B, N), generator=g) / N
    return X.to(dev), C.to(dev), ids.to(dev), gr.to(dev)


def _errors(X, C, ids, scale):
    X64, C64, i = oracle.as_f64(X.cpu()), oracle.as_f64(C.cpu()), ids.cpu().numpy()
    d, K = X64.shape[2], C64.shape[1]
    loss, lse, z = op.xent(X64, C64, i, scale)
    ez = (d / 16 + 66) * 2.0 ** -23 * abs(scale) * np.einsum("bnd,bkd->bnk", np.abs(X64), np.abs(C64))
    zmax = np.abs(z).max(2)
    eexp = 2.0 ** -21 * (zmax + 2)
    elses = ez.max(2) + eexp + (320 + K / 64) * 2.0 ** -24
    return X64, C64, i, loss, lse, z, ez, eexp, elses


def _check_loss(X, C, ids, scale, loss, lse):
    X64, C64, i, rl, rs, z, ez, eexp, elses = _errors(X, C, ids, scale)
    assert (np.abs(lse.cpu().numpy() - rs) <= elses + 2.0 ** -23 * np.abs(rs)).all()
    got = loss.cpu().numpy()
    assert (np.abs(got - rl) <= elses + ez.max(2) + 2.0 ** -22 * (np.abs(rs) + np.abs(z).max(2))).all()
    bad = (i < 0) | (i >= C64.shape[1])
    assert (got[bad] == 0).all()


def _check_grad(X, C, ids, g, scale, dX, dC, parts=1):
    dtype = X.dtype
    X64, C64, i, rl, rs, z, ez, eexp, elses = _errors(X, C, ids, scale)
    g64 = np.ones(i.shape) if g is None else g.cpu().double().numpy()
    rX, rC, P, p, w = op.xent_grad(X64, C64, i, g64, scale)
    u = torch.finfo(dtype).eps / 2
    aw = np.abs(w)[..., None]
    onehot = np.where(aw > 0, np.abs(P) / np.maximum(aw, 1e-300), 0.0)      # |p - onehot|
    # (two parts: the second is the exact remainder of the first, half a step of it is lost)
    eP = aw * (p * (ez + (elses + eexp + 2.0 ** -23 * np.abs(rs))[..., None]) * 1.01 + (u ** parts + 2.0 ** -22) * onehot)
    if dtype == torch.float16:
        eP += 2.0 ** -39 * np.abs(w).max() * (aw > 0)
    aC, aX, aP = np.abs(C64), np.abs(X64), np.abs(P)
    K, N = C64.shape[1], X64.shape[1]
    tX = np.einsum("bnk,bkd->bnd", eP + (K / 16 + 70) * 2.0 ** -23 * aP, aC) * 1.01 + u * np.abs(rX)
    tC = np.einsum("bnk,bnd->bkd", eP + (N / 16 + 70) * 2.0 ** -23 * aP, np.where(aw > 0, aX, 0)) * 1.01 + u * np.abs(rC)
    if dtype == torch.float16:
        tX, tC = tX + 2.0 ** -25, tC + 2.0 ** -25
    for got, ref, tol in ((dX, rX, tX), (dC, rC, tC)):
        if got is None:
            continue
        err = np.abs(got.cpu().double().numpy() - ref)
        assert (err <= tol).all(), f"worst excess {(err - tol).max()}, {(err > tol).sum()} of {err.size}"
    bad = (i < 0) | (i >= K)
    if dX is not None:
        assert (dX.cpu().double().numpy()[bad] == 0).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("B,N,K,d", SHAPES)
def test_xent_and_gradients(cuda_device, dtype, B, N, K, d):
    X, C, ids, g = _inputs(B, N, K, d, dtype, cuda_device, seed=N + K + d)
    for scale, gr in ((1.0, g), (0.25, None), (-0.5, g), (0.0, g)):
        loss, lse = km.km_xent(X, C, ids, scale)
        dX, dC = km.km_xent_grad(X, C, ids, lse, gr, scale)
        torch.cuda.synchronize()
        assert km.km_device_error() == 0
        _check_loss(X, C, ids, scale, loss, lse)
        _check_grad(X, C, ids, gr, scale, dX, dC)
        again = km.km_xent(X, C, ids, scale)
        aX, aC = km.km_xent_grad(X, C, ids, lse, gr, scale)
        assert torch.equal(again[0], loss) and torch.equal(again[1], lse)
        assert torch.equal(aX, dX) and torch.equal(aC, dC)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("B,N,K,d", [(1, 400, 2, 64), (2, 150, 5, 128), (1, 300, 60, 33), (1, 200, 128, 100)])
def test_few_table_rows_keep_two_parts_of_p(cuda_device, dtype, B, N, K, d):
    X, C, ids, g = _inputs(B, N, K, d, dtype, cuda_device, seed=7 * N + K)
    for scale, gr in ((0.25, None), (-0.5, g)):
        loss, lse = km.km_xent(X, C, ids, scale)
        dX, dC = km.km_xent_grad(X, C, ids, lse, gr, scale)
        _check_grad(X, C, ids, gr, scale, dX, dC, parts=2)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d", [40, 136])
def test_many_pieces_and_split_reductions(cuda_device, dtype, d):
    # a table of several gradient pieces (the scratch holds 2^27 entries of P at a time; rows of up
    # to 128 16-bit values need none) and a reduction over many points; checked through fp64 torch
    # on the device
    B, N, K = 1, 65536, 5000
    X, C, ids, g = _inputs(B, N, K, d, dtype, cuda_device, seed=1)
    loss, lse = km.km_xent(X, C, ids)
    dX, dC = km.km_xent_grad(X, C, ids, lse, g)
    torch.cuda.synchronize()
    X6, C6 = X[0].double(), C[0].double()
    rC, rX = torch.zeros_like(C6), torch.zeros_like(X6)
    for n in range(0, N, 8192):
        sl = slice(n, n + 8192)
        z = X6[sl] @ C6.t()
        ok = (ids[0, sl] >= 0) & (ids[0, sl] < K)
        rs = torch.logsumexp(z, 1)
        assert (lse[0, sl] - rs).abs().max() < 2e-5
        p = torch.exp(z - rs[:, None])
        p[ok, ids[0, sl][ok].long()] -= 1
        p *= torch.where(ok, g[0, sl], torch.zeros_like(g[0, sl]))[:, None]
        rX[sl] = p @ C6
        rC += p.t() @ X6[sl]
    # relative norms: the rounding of P and of the result, half a step each at most, plus fp32 sums;
    # with g near 2^-16 the fp16 results lie among its subnormals, whose half step is 2^-25 for
    # every entry whatever its size, 2^-25 sqrt(entries) in norm
    u = torch.finfo(dtype).eps / 2
    for got, ref in ((dX[0], rX), (dC[0], rC)):
        rel = ((got.double() - ref).norm() / ref.norm()).item()
        floor = (2.0 ** -25 * ref.numel() ** 0.5 / ref.norm()).item() if dtype == torch.float16 else 0.0
        assert rel < 2 * u + 2e-5 + floor, rel


@pytest.mark.parametrize("dtype", DTYPES)
def test_points_without_labels_may_hold_anything(cuda_device, dtype):
    X, C, ids, g = _inputs(2, 150, 260, 64, dtype, cuda_device, seed=2)
    bad = (ids < 0) | (ids >= 260)
    assert bad.any()
    _, lse = km.km_xent(X, C, ids)
    dX0, dC0 = km.km_xent_grad(X, C, ids, lse, g)
    for fill in (float("nan"), float("inf")):
        X2, g2 = X.clone(), g.clone()
        X2[bad] = fill
        g2[bad] = fill
        loss, lse2 = km.km_xent(X2, C, ids)
        dX, dC = km.km_xent_grad(X2, C, ids, lse2, g2)
        torch.cuda.synchronize()
        assert (loss[bad] == 0).all() and torch.isfinite(loss).all()
        assert torch.equal(dX, dX0) and torch.equal(dC, dC0)


@pytest.mark.parametrize("dtype", DTYPES)
def test_no_labels_at_all_and_single_outputs(cuda_device, dtype):
    X, C, ids, g = _inputs(1, 40, 90, 32, dtype, cuda_device, seed=3)
    none = torch.full_like(ids, -1)
    loss, lse = km.km_xent(X, C, none)
    dX, dC = km.km_xent_grad(X, C, none, lse, g)
    torch.cuda.synchronize()
    assert not loss.any() and not dX.any() and not dC.any()
    _, lse = km.km_xent(X, C, ids)
    both = km.km_xent_grad(X, C, ids, lse, g)
    onlyX = km.km_xent_grad(X, C, ids, lse, g, want_dC=False)
    onlyC = km.km_xent_grad(X, C, ids, lse, g, want_dX=False)
    assert onlyX[1] is None and onlyC[0] is None
    assert torch.equal(onlyX[0], both[0]) and torch.equal(onlyC[1], both[1])


def test_large_logits_do_not_overflow(cuda_device):
    X, C, ids, g = _inputs(1, 130, 300, 64, torch.bfloat16, cuda_device, seed=4, scale_rows=200.0)
    loss, lse = km.km_xent(X, C, ids, 4.0)
    dX, dC = km.km_xent_grad(X, C, ids, lse, g, 4.0)
    torch.cuda.synchronize()
    assert torch.isfinite(loss).all() and torch.isfinite(dX).all() and torch.isfinite(dC).all()
    _check_loss(X, C, ids, 4.0, loss, lse)


def test_small_fp16_gradients_keep_their_bits(cuda_device):
    # every probability times every gradient below fp16's smallest number; the loss is scaled at
    # the end only (a large scale_rows-free table, g = 2^-20), results compared before rounding
    # through a table scaled up by 2^12
    X, C, ids, _ = _inputs(1, 200, 4000, 32, torch.float16, cuda_device, seed=5)
    g = torch.full((1, 200), 2.0 ** -8, device=cuda_device)
    _, lse = km.km_xent(X, C, ids)
    dX, _ = km.km_xent_grad(X, C, ids, lse, g)
    X64, C64 = X[0].double(), C[0].double()
    p = torch.softmax(X64 @ C64.t(), 1)
    ok = (ids[0] >= 0) & (ids[0] < 4000)
    p[ok, ids[0][ok].long()] -= 1
    p *= torch.where(ok, 2.0 ** -8, 0.0)[:, None]
    ref = p @ C64
    err = (dX[0].double() - ref).norm() / ref.norm()
    # the result's own rounding (values near 2^-10 and subnormal steps of 2^-24) allows 2^-25 each
    floor = 2.0 ** -25 * ref.numel() ** 0.5 / ref.norm()
    assert err < 2 * 2.0 ** -11 + floor


@pytest.mark.parametrize("dtype", DTYPES)
def test_gradient_matches_differences_of_the_loss(cuda_device, dtype):
    # fp64 differences of the oracle's loss at the rounded inputs, along random directions
    X, C, ids, g = _inputs(1, 60, 100, 40, dtype, cuda_device, seed=6)
    _, lse = km.km_xent(X, C, ids, 0.7)
    dX, dC = km.km_xent_grad(X, C, ids, lse, g, 0.7)
    X64, C64, i, g64 = oracle.as_f64(X.cpu()), oracle.as_f64(C.cpu()), ids.cpu().numpy(), g.cpu().double().numpy()
    rng = np.random.default_rng(0)
    h = 1e-5
    for _ in range(3):
        vX, vC = rng.standard_normal(X64.shape), rng.standard_normal(C64.shape)
        up = (g64 * op.xent(X64 + h * vX, C64 + h * vC, i, 0.7)[0]).sum()
        dn = (g64 * op.xent(X64 - h * vX, C64 - h * vC, i, 0.7)[0]).sum()
        got = (dX.cpu().double().numpy() * vX).sum() + (dC.cpu().double().numpy() * vC).sum()
        # roundings of P and of the results (half a step each), all with independent signs
        u = torch.finfo(dtype).eps / 2
        slack = 4 * u * (np.linalg.norm(oracle.as_f64(dX.cpu())) + np.linalg.norm(oracle.as_f64(dC.cpu())))
        assert abs((up - dn) / (2 * h) - got) < slack + 1e-5


def test_unaligned_rows_guards_streams_and_capture(cuda_device):
    B, N, K, d = 1, 300, 700, 64
    X, C, ids, g = _inputs(B, N, K, d, torch.bfloat16, cuda_device, seed=7)
    loss, lse = km.km_xent(X, C, ids)
    dX, dC = km.km_xent_grad(X, C, ids, lse, g)
    # buffers two bytes off any vector boundary, outputs between guard values
    def off(t):
        buf = torch.full((t.numel() + 2,), 7.0, dtype=t.dtype, device=t.device)
        buf[1:-1].copy_(t.flatten())
        return buf, buf[1:-1].view(t.shape)
    _, X1 = off(X)
    _, C1 = off(C)
    bx, dX1 = off(torch.zeros_like(dX))
    bc, dC1 = off(torch.zeros_like(dC))
    l1, s1 = km.km_xent(X1, C1, ids)
    km.km_xent_grad(X1, C1, ids, s1, g, dX=dX1, dC=dC1)
    torch.cuda.synchronize()
    _check_loss(X, C, ids, 1.0, l1, s1)
    _check_grad(X, C, ids, g, 1.0, dX1, dC1)
    for b in (bx, bc):
        assert b[0] == 7 and b[-1] == 7
    lib = km._load()
    n1 = lib.km_xent_workspace_size(B, N, K, d, 2)
    n2 = lib.km_xent_grad_workspace_size(B, N, K, d, 2)
    w1 = torch.full((n1 + 256,), 0xFF, dtype=torch.uint8, device=cuda_device)
    w2 = torch.full((n2 + 256,), 0xFF, dtype=torch.uint8, device=cuda_device)
    l2, s2 = km.km_xent(X, C, ids, ws=w1[:n1])
    x2, c2 = km.km_xent_grad(X, C, ids, s2, g, ws=w2[:n2])
    torch.cuda.synchronize()
    assert torch.equal(l2, loss) and torch.equal(x2, dX) and torch.equal(c2, dC)
    assert (w1[n1:] == 0xFF).all() and (w2[n2:] == 0xFF).all()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    l3, s3 = km.km_xent(X, C, ids, stream=side)
    x3, c3 = km.km_xent_grad(X, C, ids, s3, g, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(l3, loss) and torch.equal(x3, dX) and torch.equal(c3, dC)
    Xs, lo, ls, gx, gc = X.clone(), torch.empty_like(loss), torch.empty_like(lse), torch.empty_like(dX), torch.empty_like(dC)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        km.km_xent(Xs, C, ids, loss=lo, lse=ls, ws=w1[:n1])
        km.km_xent_grad(Xs, C, ids, ls, g, dX=gx, dC=gc, ws=w2[:n2])
    for k in (1.0, 0.5):
        Xs.copy_(X * k)
        graph.replay()
        torch.cuda.synchronize()
        rl, rs = km.km_xent(X * k, C, ids)
        rx, rc = km.km_xent_grad(X * k, C, ids, rs, g)
        assert torch.equal(lo, rl) and torch.equal(gx, rx) and torch.equal(gc, rc)

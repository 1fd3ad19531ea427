"""The codebook operators together, as a program uses them: points are fitted and labelled, a small
model looks the previous label's row up and predicts the next label over the same table, the table
takes both gradients, and a projection with 4-bit codebook weights reads the result."""
import numpy as np
import pytest
import torch

import exact_lloyd_means_assign_b200 as km
import oracle
from oracle import operators as op

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32])
def test_label_prediction_step(cuda_device, dtype):
    g = torch.Generator().manual_seed(11)
    B, N, K, d = 2, 600, 96, 64
    pts = torch.randn((B, N, d), generator=g).to(dtype).to(cuda_device)
    C32 = pts[:, :K].float().contiguous()
    _, ids, _, _ = km.km_fit(pts, C32, 3, want_ids=True)
    table, _ = km.km_prep(C32, dtype)
    prev, nxt = ids.roll(1, 1).contiguous(), ids.clone()
    prev[:, 0], nxt[:, 0] = -1, -1                      # no predecessor: no input row, no label
    scale = 1 / d ** 0.5
    x = km.km_lookup(table, prev, 1.0)
    loss, lse = km.km_xent(x, table, nxt, scale)
    gr = torch.full((B, N), 1.0 / (B * (N - 1)), device=cuda_device)
    dx, dtab = km.km_xent_grad(x, table, nxt, lse, gr, scale)
    dtab32 = dtab.float()
    km.km_lookup_grad(dx, prev, K, 1.0, dC=dtab32, accumulate=True)
    torch.cuda.synchronize()
    assert km.km_device_error() == 0
    # the same step in fp64 (the activations x are table rows, exact)
    T64, p, n = oracle.as_f64(table.cpu()), prev.cpu().numpy(), nxt.cpu().numpy()
    x64 = op.lookup(T64, p, 1.0)
    rl, _, _ = op.xent(x64, T64, n, scale)
    rX, rC, _, _, _ = op.xent_grad(x64, T64, n, gr.cpu().double().numpy(), scale)
    rT = rC + op.lookup_grad(rX, p, K, 1.0)[0]
    u = torch.finfo(dtype).eps / 2
    assert np.abs(loss.cpu().numpy() - rl).max() < 1e-4
    got = dtab32.cpu().double().numpy()
    # three roundings of half a step (P, dX, dC's rows) in quadrature stay below 2 u in norm; fp16
    # rounds values near its subnormal step 2^-24
    floor = (2.0 ** -25 * (got.size ** 0.5) * 4 / np.linalg.norm(rT)) if dtype == torch.float16 else 0.0
    assert np.linalg.norm(got - rT) < (2 * u + 1e-5 + floor) * np.linalg.norm(rT)
    # and a projection with encoded weights reads the activations
    W = (torch.randn((32, d), generator=g) * 0.05).to(dtype).to(cuda_device)
    cb = km.km_init_grid1d(W[..., None].contiguous(), 16)
    codes = km.km_encode1d(W, cb)
    y = km.km_matvec4(x[0, 1:9].contiguous(), km.km_pack4(codes), cb)
    torch.cuda.synchronize()
    ref, mag = op.matvec4(x64[0, 1:9], codes.cpu().numpy(), oracle.round_to_dtype(cb.cpu().view(32, 16), dtype))
    assert (np.abs(y.cpu().double().numpy() - ref) <= u * np.abs(ref) + 68 * 2.0 ** -23 * mag + 2.0 ** -25).all()

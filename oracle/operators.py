"""fp64 CPU definitions of the codebook operators: products with 4-bit codes, table lookups and
their gradient, softmax cross entropy over a table and its gradient. Plain numpy, one loop per
problem; nothing here is shared with the GPU path."""
from __future__ import annotations

import numpy as np


def pack4(codes):
    """codes [R,N] -> packed [R, 16 * ceil(N / 32)] bytes, even positions in the low halves."""
    R, N = codes.shape
    full = np.zeros((R, 32 * (-(-N // 32))), np.uint8)
    full[:, :N] = codes & 15
    return full[:, 0::2] | (full[:, 1::2] << 4)


def weights4(codes, Cr, scales=None, group=0):
    """The weights [R,N] that codes stand for; Cr [R,K] already rounded, codes >= K are 0."""
    R, N = codes.shape
    table = np.zeros((R, 16))
    table[:, :Cr.shape[1]] = Cr
    W = np.take_along_axis(table, (codes & 15).astype(np.int64), 1)
    if scales is not None:
        W = W * np.repeat(scales, group, axis=1)[:, :N]
    return W


def matvec4(x, codes, Cr, scales=None, group=0):
    """(y [M,R], the sums of the terms' absolute values [M,R])."""
    W = weights4(codes, Cr, scales, group)
    return x @ W.T, np.abs(x) @ np.abs(W).T


def _valid(ids, K):
    return (ids >= 0) & (ids < K)


def lookup(C, ids, scale):
    B, K, d = C.shape
    Y = np.zeros((B, ids.shape[1], d))
    for b in range(B):
        ok = _valid(ids[b], K)
        Y[b, ok] = scale * C[b, ids[b, ok]]
    return Y


def lookup_grad(dY, ids, K, scale):
    """(dC [B,K,d], sums of absolute values [B,K,d], tokens per row [B,K])."""
    B, N, d = dY.shape
    out, mag, cnt = np.zeros((B, K, d)), np.zeros((B, K, d)), np.zeros((B, K), np.int64)
    for b in range(B):
        for n in range(N):
            k = ids[b, n]
            if 0 <= k < K:
                out[b, k] += scale * dY[b, n]
                mag[b, k] += np.abs(scale * dY[b, n])
                cnt[b, k] += 1
    return out, mag, cnt


def xent(X, C, ids, scale):
    """(loss [B,N], lse [B,N], z [B,N,K])."""
    B, N, _ = X.shape
    K = C.shape[1]
    z = scale * np.einsum("bnd,bkd->bnk", X, C)
    m = z.max(2, keepdims=True)
    lse = (m + np.log(np.exp(z - m).sum(2, keepdims=True)))[..., 0]
    loss = np.zeros((B, N))
    for b in range(B):
        for n in range(N):
            if 0 <= ids[b, n] < K:
                loss[b, n] = lse[b, n] - z[b, n, ids[b, n]]
    return loss, lse, z


def xent_grad(X, C, ids, g, scale):
    """(dX, dC, P [B,N,K], p [B,N,K], w [B,N]): P = w (p - onehot), 0 without a label."""
    B, N, _ = X.shape
    K = C.shape[1]
    ok = _valid(ids, K)
    Xc = np.where(ok[..., None], X, 0.0)       # points without a label take no part
    _, lse, z = xent(Xc, C, ids, scale)
    p = np.exp(z - lse[..., None])
    w = np.where(ok, g * scale, 0.0)
    onehot = np.zeros((B, N, K))
    bb, nn = np.nonzero(ok)
    onehot[bb, nn, ids[bb, nn]] = 1.0
    P = w[..., None] * (p - onehot)
    return np.einsum("bnk,bkd->bnd", P, C), np.einsum("bnk,bnd->bkd", P, Xc), P, p, w

"""The fp64 definitions of the codebook operators against brute force and finite differences."""
import numpy as np
import pytest

from oracle import operators as op


def test_pack4_layout():
    codes = np.array([[1, 2, 3], [15, 0, 7]], np.uint8)
    p = op.pack4(codes)
    assert p.shape == (2, 16)
    assert p[0, 0] == 0x21 and p[0, 1] == 0x03 and p[1, 0] == 0x0F and p[1, 1] == 0x07
    assert (p[:, 2:] == 0).all()


@pytest.mark.parametrize("group", [0, 32])
def test_matvec4_is_the_double_sum(group):
    rng = np.random.default_rng(1)
    R, N, M, K = 3, 45, 2, 5
    codes = rng.integers(0, 7, (R, N)).astype(np.uint8)      # 5 and 6 stand for 0
    C, x = rng.standard_normal((R, K)), rng.standard_normal((M, N))
    s = rng.random((R, 2)) if group else None
    y, mag = op.matvec4(x, codes, C, s, group)
    for m in range(M):
        for r in range(R):
            t = [x[m, n] * (C[r, codes[r, n]] if codes[r, n] < K else 0.0) * (s[r, n // group] if group else 1.0)
                 for n in range(N)]
            assert abs(y[m, r] - sum(t)) < 1e-12 and abs(mag[m, r] - sum(map(abs, t))) < 1e-12


def test_lookup_and_its_gradient_are_adjoint():
    rng = np.random.default_rng(2)
    C, dY = rng.standard_normal((2, 6, 3)), rng.standard_normal((2, 9, 3))
    ids = rng.integers(-1, 7, (2, 9))
    Y = op.lookup(C, ids, 1.7)
    dC, _, cnt = op.lookup_grad(dY, ids, 6, 1.7)
    assert abs((Y * dY).sum() - (C * dC).sum()) < 1e-10
    assert cnt.sum() == ((ids >= 0) & (ids < 6)).sum()
    assert (Y[(ids < 0) | (ids >= 6)] == 0).all()


def test_xent_gradient_matches_differences():
    rng = np.random.default_rng(3)
    B, N, K, d, scale = 2, 4, 5, 3, 0.8
    X, C, g = rng.standard_normal((B, N, d)), rng.standard_normal((B, K, d)), rng.standard_normal((B, N))
    ids = rng.integers(0, K, (B, N))
    ids[0, 1], ids[1, 2] = -1, K
    dX, dC, P, p, _ = op.xent_grad(X, C, ids, g, scale)
    np.testing.assert_allclose(p.sum(2), 1.0, rtol=1e-12)
    assert (P[0, 1] == 0).all() and (dX[1, 2] == 0).all()

    def total(X, C):
        return (g * op.xent(X, C, ids, scale)[0]).sum()

    h = 1e-6
    for T, dT, which in ((X, dX, 0), (C, dC, 1)):
        for i in np.ndindex(T.shape):
            a, b = T.copy(), T.copy()
            a[i] += h
            b[i] -= h
            num = (total(a, C) - total(b, C)) if which == 0 else (total(X, a) - total(X, b))
            assert abs(num / (2 * h) - dT[i]) < 1e-7


def test_xent_of_one_row_is_zero():
    X, C = np.ones((1, 2, 3)), np.ones((1, 1, 3))
    loss, lse, _ = op.xent(X, C, np.zeros((1, 2), int), 2.0)
    assert (loss == 0).all() and (lse == 6).all()

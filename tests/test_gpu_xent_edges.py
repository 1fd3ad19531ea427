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

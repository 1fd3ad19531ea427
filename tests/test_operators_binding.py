"""Refusals that the Python binding makes itself, before the library or a device is reached: the check
for a CUDA tensor is taken out, so that host tensors reach the checks behind it."""
import pytest
import torch

import exact_lloyd_means_assign_b200 as km


@pytest.fixture(autouse=True)
def host_tensors(monkeypatch):
    real = km._on_gpu
    monkeypatch.setattr(km, "_on_gpu", lambda t, name: real(t, name) if t is None else t.device)
    monkeypatch.setattr(km, "_launch", lambda *a: pytest.fail("launched"))


X, C = torch.zeros((1, 3, 8)), torch.zeros((1, 4, 8))
IDS, LSE = torch.zeros((1, 3), dtype=torch.int32), torch.zeros((1, 3))
CODES, PACKED, BOOK = torch.zeros((4, 64), dtype=torch.uint8), torch.zeros((4, 32), dtype=torch.uint8), torch.zeros((4, 16))
XH = torch.zeros((1, 64))


@pytest.mark.parametrize("call", [
    lambda: km.km_pack4(None),
    lambda: km.km_matvec4(None, PACKED, BOOK),
    lambda: km.km_matvec4(XH, None, BOOK),
    lambda: km.km_matvec4(XH, PACKED, None),
    lambda: km.km_lookup(None, IDS),
    lambda: km.km_lookup(C, None),
    lambda: km.km_lookup_grad(None, IDS, 4),
    lambda: km.km_lookup_grad(X, None, 4),
    lambda: km.km_xent(None, C, IDS),
    lambda: km.km_xent(X, None, IDS),
    lambda: km.km_xent(X, C, None),
    lambda: km.km_xent_grad(None, C, IDS, LSE),
    lambda: km.km_xent_grad(X, None, IDS, LSE),
    lambda: km.km_xent_grad(X, C, None, LSE),
    lambda: km.km_xent_grad(X, C, IDS, None),
])
def test_a_missing_tensor_is_a_value_error(call):
    with pytest.raises(ValueError):
        call()


def test_optional_tensors_may_be_missing(monkeypatch):
    seen = []
    monkeypatch.setattr(km, "_launch", lambda *a: seen.append(a))
    km.km_xent_grad(X, C, IDS, LSE, None)
    km.km_matvec4(XH, PACKED, BOOK, None)
    assert len(seen) == 2

"""The README's example of codebooks in a model runs as written and its results fit together."""
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example():
    lines = open(os.path.join(ROOT, "README.md")).read().splitlines()
    block = []
    for line in lines[lines.index("## Codebooks in a model") + 1:]:
        if line.startswith("    ") or (block and not line.strip()):
            block.append(line[4:])
        elif block:
            break
    return "\n".join(block)


def test_readme_codebook_example_runs(cuda_device):
    code = _example()
    assert "km.km_matvec4" in code and "km.km_xent_grad" in code
    env = {}
    exec(compile(code, "README.md", "exec"), env)
    torch.cuda.synchronize()
    km = env["km"]
    assert km.km_device_error() == 0
    # the coded weights stand for the weights: 16 values per row, fitted, leave a small error
    dense = env["x"].float() @ env["W"].float().t()
    assert (env["y"].float() - dense).norm() < 0.2 * dense.norm()
    # the gradients of a softmax sum to zero over the table, token by token; so does their sum
    assert torch.isfinite(env["loss"]).all() and torch.isfinite(env["dtable"]).all()
    assert env["dh"].shape == env["h"].shape and env["dtable"].shape == (1, 1024, 128)

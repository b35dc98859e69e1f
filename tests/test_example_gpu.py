"""The example block: generation on the caches gives the whole prompts' outputs, and its backward
pass the derivatives of its forward pass."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def block():
    spec = importlib.util.spec_from_file_location("mamba_block", os.path.join(ROOT, "examples", "mamba_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("bf16", [False, True])
def test_generation_is_the_whole_prompt(block, bf16):
    import torch
    # fp32: the products' order differs between batch sizes; bf16: a rounding of the projections
    # that goes the other way is half a percent of a value, a few of them of the largest
    assert block.serve(dtype=torch.bfloat16 if bf16 else torch.float32) <= (3e-2 if bf16 else 1e-4)


def test_backward_is_the_derivative_of_forward(block):
    # central differences in fp32 forward passes: noise of about 1e-6 |loss terms| / step and a
    # third-order error, both within a percent along the gradient
    for name, (by_backward, by_difference) in block.train().items():
        assert abs(by_backward - by_difference) <= 1e-2 * abs(by_backward), (name, by_backward, by_difference)

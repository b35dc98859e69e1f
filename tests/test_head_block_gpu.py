"""The example block with heads: generation on the caches gives the whole prompts' outputs, and its backward
pass the derivatives of its forward pass (linear attention, its step and gradients, both layer norms, run together)."""
import pytest

from .test_example_gpu import block  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bf16", [False, True])
def test_generation_is_the_whole_prompt(block, bf16):  # noqa: F811
    import torch
    # as the block without heads: fp32, the products' order differs between batch sizes; bf16, a rounding of the
    # projections that goes the other way is half a percent of a value, a few of them of the largest
    got = block.serve(dtype=torch.bfloat16 if bf16 else torch.float32, kind=block.HeadBlock)
    assert got <= (3e-2 if bf16 else 1e-4)


def test_backward_is_the_derivative_of_forward(block):  # noqa: F811
    # central differences in fp32 forward passes: noise of about 1e-6 |loss terms| / step and a
    # third-order error, both within a percent along the gradient
    for name, (by_backward, by_difference) in block.train(kind=block.HeadBlock).items():
        assert abs(by_backward - by_difference) <= 1e-2 * abs(by_backward), (name, by_backward, by_difference)

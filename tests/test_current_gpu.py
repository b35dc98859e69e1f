"""A call on tensors of a GPU that is not the current one runs with theirs current: the default stream's
handle is the same on all of them and stands for the current one's (CPU, with stand-ins)."""
import pytest

from .test_stream_memory import BLOCK, DENSE, calls, gpu  # noqa: F401  (fixture)


@pytest.mark.parametrize("name", BLOCK + DENSE)
@pytest.mark.parametrize("index, device", [(1, 0), (0, 1), (0, 0), (3, 3)])
@pytest.mark.parametrize("given", [None, 7])
def test_runs_on_the_operands_gpu(gpu, name, index, device, given):  # noqa: F811
    g, lib = gpu(0, index, device)
    calls(g.tensor)[name](stream=given)
    assert lib.devices == [index] and g.devices == [device]

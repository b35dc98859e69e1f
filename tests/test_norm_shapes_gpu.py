"""The norms at both sides of every length where a row goes to another number of lanes or pieces, for
every pair of types, forward and gradients: no length without a kernel (bounds as in test_norms_gpu.py)."""
import pytest

from .test_norms_gpu import test_gated_norm as gated_norm
from .test_norms_gpu import test_residual_norm as residual_norm

pytestmark = pytest.mark.gpu

# pieces of 4 elements go over at 32, 64, 128, 256, 512, 1024, 2048, 3072, 4096 and 6144, those of 8 at twice as many
# up to 32768
LENGTHS = [n + e for n in (32, 64, 128, 256, 512, 1024, 2048, 3072, 4096, 6144, 8192, 12288, 16384) for e in (0, 1)]
TYPES = [(False, False), (False, True), (True, False), (True, True)]


@pytest.mark.parametrize("a16, b16", TYPES)
@pytest.mark.parametrize("n", [7, 8, 9, *LENGTHS, 32767, 32768])
def test_every_shape(n, a16, b16):
    gated_norm(3, n, 1, a16, b16, n % 2 == 0)
    residual_norm(2, n, a16, b16, True, True, False)
    residual_norm(2, n, a16, b16, False, n % 2 == 1, False)

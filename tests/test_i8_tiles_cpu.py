"""The shapes of test_gpu_i8_tiles.py reach the kernels that they name, and name
every kernel (host only)."""
import pytest

pytest.importorskip("torch")
import test_gpu_i8_tiles as tiles  # noqa: E402
from test_i8_kernels_cpu import ALL, DENSE_ONLY, kernel  # noqa: E402


@pytest.mark.parametrize("gated,name,shape", [(0, *c) for c in tiles.DENSE + tiles.SLICES]
                         + [(1, *c) for c in tiles.GATED])
def test_the_shapes_that_name_a_kernel_reach_it(gated, name, shape):
    assert kernel(gated, shape) == name


def test_every_kernel_is_named():
    assert {name for name, _ in tiles.DENSE} == ALL - {tiles.FAR}
    assert {name for name, _ in tiles.GATED} == ALL - {tiles.FAR} - DENSE_ONLY

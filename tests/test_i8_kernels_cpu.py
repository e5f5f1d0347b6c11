"""Which kernel a product of matrices in 8 bits takes (sgemm_f32_i8_kernel, host only):
the tests of exact products reach every kernel, dense and gated. A change of the
choice's measured constants that leaves a kernel untested fails here."""
import pytest

pytest.importorskip("torch")
import fp32_gemm_tuning_amd as sg  # noqa: E402
import test_gpu_i8 as products  # noqa: E402

P = 1 << 20   # an address: only its alignment is looked at
DENSE_ONLY = {"rows 32x32", "rows 32x32 through registers"}
FAR = "tile 64x64 of far rows"
ALL = DENSE_ONLY | {FAR, "few 1", "few 2", "few 4", "few 8", "rows 32x64", "rows 32x64 through registers", "rows 64x64",
                    "flat 64x64", "ring 64x128", "flat 64x128", "ring 128x128", "flat 128x128", "tile 128x128",
                    "flat 256x128", "tile 256x256", "flat 256x256", "tile 128x128 of short rows"}


def kernel(gated, shape, layout=(0, 0)):
    M, F, K = shape
    pad, offset = layout
    at, ld = P + offset, max(K + pad, 1)
    return sg.sgemm_f32_i8_kernel(gated, M, F, K, at, ld, at, ld, at, ld)


@pytest.mark.parametrize("gated", [0, 1])
def test_exact_products_reach_every_kernel(gated):
    got = {kernel(gated, s, layout) for s in products.SHAPES for layout in products.LAYOUTS}
    got |= {kernel(gated, s, layout) for s in products.LARGE for layout in products.LAYOUTS[:2]}
    assert got == ALL - {FAR} - (DENSE_ONLY if gated else set())


def test_far_rows_and_what_launches_nothing():
    far = (1 << 31) + 64
    for M in (40, 70):   # test_offsets_past_32_bits
        assert sg.sgemm_f32_i8_kernel(0, M, 3, 300, P, 300, P, far) == FAR
        assert sg.sgemm_f32_i8_kernel(1, M, 3, 300, P, 300, P, far, P, far) == FAR
        assert sg.sgemm_f32_i8_kernel(1, M, 3, 300, P, 300, P, 300, P, far) == FAR
    assert kernel(0, (3, 5, 0)) == kernel(1, (3, 5, 0)) == "zero"
    for shape in ((0, 5, 8), (3, 0, 8), (-1, 5, 8), (3, 5, 131072), (1 << 31, 5, 8), (1 << 30, 1 << 30, 16)):
        assert kernel(0, shape) is None and kernel(1, shape) is None
    assert sg.sgemm_f32_i8_kernel(0, 3, 5, 8, P, 7, P, 8) is None
    assert sg.sgemm_f32_i8_kernel(0, 3, 5, 8, 0, 8, P, 8) is None
    assert sg.sgemm_f32_i8_kernel(1, 3, 5, 8, P, 8, P, 8) is None


def test_what_decides_the_fill():
    # whole 16-byte chunks, in K, the row's distance and the address
    assert kernel(0, (2836, 4253, 144)) == "tile 256x256"
    for bad in (dict(x=P + 8), dict(ldx=152), dict(w=P + 1), dict(ldw=145)):
        v = dict(x=P, ldx=144, w=P, ldw=144) | bad
        assert sg.sgemm_f32_i8_kernel(0, 2836, 4253, 144, *v.values()).startswith("flat")


def test_more_rows_than_a_second_grid_extent_holds():
    # test_more_rows_of_blocks_than_a_second_grid_extent: the rows' kernels put blocks of 32 rows there
    assert kernel(0, (65535 * 32, 16, 10240)).startswith("rows")
    assert not kernel(0, (65535 * 32 + 1, 16, 10240)).startswith("rows")

"""Column-major scales hold what the GEMM copies: G * ld floats, to the end of the last scale's 16-byte line."""
import pytest

from block_scaled_fp8_02_gb300 import _binding as B


@pytest.mark.parametrize("M", [0, 1, 2, 3, 4, 5, 83, 128])
@pytest.mark.parametrize("G", [1, 2, 57])
def test_norm_scales_end_in_the_line_that_the_gemm_copies_last(M, G):
    ld = (M + 3) // 4 * 4
    s = B._col_major_scales(M, G, ld, "cpu")
    assert s.shape == (M, G) and (M == 0 or s.stride() == (1, ld)) and s.storage_offset() == 0
    nbytes = s.untyped_storage().nbytes()
    assert (nbytes + 15) // 16 * 16 == 4 * G * ld

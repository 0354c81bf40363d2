"""Column-major scales own the whole buffer that the GEMM copies: G * ld floats."""
import pytest

from block_scaled_fp8_02_gb300 import _binding as B


@pytest.mark.parametrize("M", [0, 1, 2, 3, 4, 5, 83, 128])
@pytest.mark.parametrize("G", [1, 2, 57])
def test_norm_scales_hold_whole_columns(M, G):
    ld = (M + 3) // 4 * 4
    s = B._col_major_scales(M, G, ld, "cpu")
    assert s.shape == (M, G) and (M == 0 or s.stride() == (1, ld)) and s.storage_offset() == 0
    assert s.untyped_storage().nbytes() >= 4 * G * ld

"""How the 8-bit and grouped products are cut up, before any device work."""
import pytest

import tile_size_selection_amd as tss

# M, N, K whose K is cut into ranges; M N is odd in some, and not a multiple of 4 in others
SPLIT = [(1001, 1001, 4112), (515, 521, 8208), (700, 1003, 2064), (513, 510, 8192), (512, 512, 8192)]


@pytest.mark.parametrize("size", SPLIT)
def test_ranges_partial_sums_start_on_16_byte_borders(size):
    M, N, K = size
    slice_bytes = (M * N + 3) // 4 * 16
    need = tss.gemm_fp8_workspace_size(M, N, K)
    assert need >= 2 * slice_bytes and need % slice_bytes == 0

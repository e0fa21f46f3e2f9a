"""Further refusals of the row operators and the 8-bit and grouped products,
before any device work: calls through the C ABI with addresses that are never
touched, and Python calls with host tensors."""
import pytest

from tile_size_selection_amd import _capi as C
from test_ops_refusals import ALIGN, ARG, DTYPE, GEMM, GROUPED8, _with

SUMS = C.TSS_F32_SUMS


@pytest.mark.parametrize("change,status", [
    (dict(out=C.TSS_E4M3 | SUMS), DTYPE), (dict(out=SUMS), DTYPE), (dict(out=C.TSS_BF16 | 2 * SUMS), DTYPE),
    (dict(out=C.TSS_BF16 | SUMS, A=None), ARG), (dict(out=C.TSS_F16 | SUMS, K=24), ALIGN)])
def test_products_take_fp32_sums_of_their_output_types(change, status):
    assert C.lib().tss_gemm_fp8(*_with(GEMM, **change)) == status
    assert C.lib().tss_gemm_grouped_fp8(*_with(GROUPED8, **change)) == status

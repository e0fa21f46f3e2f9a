"""Further refusals of the row operators and the 8-bit and grouped products,
before any device work: calls through the C ABI with addresses that are never
touched, and Python calls with host tensors."""
import pytest
import torch

import tile_size_selection_amd as tss
from tile_size_selection_amd import _capi as C
from test_ops_refusals import ALIGN, ARG, BACK, DTYPE, GEMM, GROUPED8, NORM, ODD, QUANT, S, F8, _with, z

SUMS = C.TSS_F32_SUMS


@pytest.mark.parametrize("change,status", [
    (dict(out=C.TSS_E4M3 | SUMS), DTYPE), (dict(out=SUMS), DTYPE), (dict(out=C.TSS_BF16 | 2 * SUMS), DTYPE),
    (dict(out=C.TSS_BF16 | SUMS, A=None), ARG), (dict(out=C.TSS_F16 | SUMS, K=24), ALIGN)])
def test_products_take_fp32_sums_of_their_output_types(change, status):
    assert C.lib().tss_gemm_fp8(*_with(GEMM, **change)) == status
    assert C.lib().tss_gemm_grouped_fp8(*_with(GROUPED8, **change)) == status


# a misaligned operand shows that the sizes before it were taken
@pytest.mark.parametrize("change,status", [
    (dict(rows=1 << 22, d=128), ALIGN), (dict(rows=(1 << 23) - 1, d=64), ALIGN), (dict(rows=1 << 23, d=8), ARG)])
def test_norm_takes_many_narrow_rows(change, status):
    assert C.lib().tss_rms_norm(*_with(NORM, x=ODD, **change)) == status
    size = C.lib().tss_rms_norm_backward_workspace_size(change["rows"], change["d"])
    assert size > 0 if status == ALIGN else size == ARG
    assert C.lib().tss_rms_norm_backward(*_with(BACK, dy=ODD, ws_bytes=1 << 30, **change)) == status


@pytest.mark.parametrize("change,status", [
    (dict(rows=1 << 27, d=512), ALIGN), (dict(rows=1 << 28, d=512), ARG), (dict(rows=1 << 27, d=520), ARG),
    (dict(rows=1 << 29, d=128, block_rows=128), ALIGN), (dict(rows=1 << 30, d=128, block_rows=128), ARG)])
def test_quantize_takes_what_a_launch_holds(change, status):
    assert C.lib().tss_quantize_fp8(*_with(QUANT, q=ODD, **change)) == status


@pytest.mark.parametrize("call", [
    lambda h: tss.gemm_fp8(out_dtype="bf16", A=z(4, 128, t=F8), B=z(8, 128, t=F8), sa=z(1, 4, t=S), sb=z(1, 1, t=S), stream=h),
    lambda h: tss.rms_norm(eps=1e-5, x=z(4, 64), weight=z(64), stream=h),
    lambda h: tss.quantize_fp8(gated=False, x=z(4, 64), stream=h),
    lambda h: tss.quantize_fp8("x", stream=h)])
def test_a_stream_wants_tensors_on_a_gpu_in_any_order_of_arguments(call):
    with pytest.raises(ValueError, match="stream"):
        call(1 << 20)


def test_a_stream_of_another_gpu_is_refused(monkeypatch):
    class Stream:
        device = torch.device("cuda:1")

    class Tensor(torch.Tensor):
        device = torch.device("cuda:0")

    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    x, w = z(4, 64).as_subclass(Tensor), z(64).as_subclass(Tensor)
    with pytest.raises(ValueError, match="the stream is of cuda:1, the tensors are on cuda:0"):
        tss.rms_norm(x, w, stream=Stream())


@pytest.mark.parametrize("change,status", [
    (dict(M=65536, N=65536, K=16, C=ODD), ALIGN), (dict(M=(1 << 27) - 1, N=40, K=16, A=ODD), ALIGN),
    (dict(M=1 << 27, N=1, K=16), ARG), (dict(M=1, N=1 << 27, K=16), ARG), (dict(M=(1 << 31) - 1, N=1, K=0), ARG)])
def test_gemm_fp8_takes_operands_below_2_gib_and_what_a_launch_holds(change, status):
    assert C.lib().tss_gemm_fp8(*_with(GEMM, **change)) == status


@pytest.mark.parametrize("change,status", [
    (dict(T=16, E=16, N=(1 << 27) - 8, K=16), ARG), (dict(T=1 << 27, K=16), ARG), (dict(T=1 << 20, N=8192, B=ODD), ALIGN)])
def test_grouped_fp8_takes_what_a_launch_holds(change, status):
    assert C.lib().tss_gemm_grouped_fp8(*_with(GROUPED8, **change)) == status

"""What layer norm, the 8-bit integer products, the sort by expert and its rows
and the gradients' clipping refuse, before any device work: through the C ABI
with addresses that are never touched, and through the Python calls with host
tensors."""
import ctypes

import pytest
import torch

import tile_size_selection_amd as tss
from tile_size_selection_amd import _capi as C

P = 1 << 20       # a 16-byte aligned address
ODD = P + 8       # not 16-byte aligned
OK, ARG, DTYPE, ALIGN, UNSUP = C.TSS_OK, C.TSS_E_ARG, C.TSS_E_DTYPE, C.TSS_E_ALIGN, C.TSS_E_UNSUPPORTED
F16, BF16, F32, E4M3, I8 = C.TSS_F16, C.TSS_BF16, C.TSS_F32, C.TSS_E4M3, C.TSS_I8


def _with(base, **changes):
    return list({**base, **changes}.values())


NORM = dict(rows=4, d=64, dtype=BF16, x=P, residual=P, weight=P, bias=P, eps=1e-5, out_dtype=BF16, y=P, scale=None, h=P,
            mean=P, rstd=P, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(rows=-1), ARG), (dict(d=0), ARG), (dict(rows=1 << 31), ARG), (dict(rows=(1 << 31) - 1, d=512), ARG),
    (dict(d=12), ALIGN), (dict(d=32776), UNSUP), (dict(dtype=9), DTYPE), (dict(dtype=I8), DTYPE),
    (dict(out_dtype=F16), DTYPE), (dict(out_dtype=E4M3), DTYPE), (dict(out_dtype=I8), ARG), (dict(x=None), ARG),
    (dict(weight=None), ARG), (dict(y=None), ARG), (dict(eps=-1.0), ARG), (dict(eps=float("nan")), ARG),
    (dict(x=ODD), ALIGN), (dict(residual=ODD), ALIGN), (dict(weight=ODD), ALIGN), (dict(bias=ODD), ALIGN),
    (dict(y=ODD), ALIGN), (dict(h=ODD), ALIGN), (dict(rows=0, x=None), OK)])
def test_layer_norm_refuses(change, status):
    assert C.lib().tss_layer_norm(*_with(NORM, **change)) == status


BACK = dict(rows=4, d=64, dtype=F32, dy=P, h=P, weight=P, mean=P, rstd=P, dh=None, dx=P, dweight=P, dbias=P, ws=P,
            ws_bytes=1 << 20, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(rows=-1), ARG), (dict(d=20), ALIGN), (dict(d=40000), UNSUP), (dict(dtype=I8), DTYPE), (dict(dy=None), ARG),
    (dict(h=None), ARG), (dict(mean=None), ARG), (dict(rstd=None), ARG), (dict(dx=None), ARG), (dict(dweight=None), ARG),
    (dict(ws=None), ARG), (dict(ws_bytes=63), ARG), (dict(ws=ODD), ALIGN), (dict(dh=ODD), ALIGN), (dict(dx=ODD), ALIGN)])
def test_layer_norm_backward_refuses(change, status):
    assert C.lib().tss_layer_norm_backward(*_with(BACK, **change)) == status


def test_layer_norm_backward_workspace():
    size = C.lib().tss_layer_norm_backward_workspace_size
    assert size(0, 64) == 0 and size(4, 4096) == 4 * 4096 * 8
    assert size(-1, 64) == ARG and size(4, 12) == ALIGN and size(4, 40000) == UNSUP


QUANT = dict(rows=4, d=64, dtype=BF16, x=P, gated=0, q=P, scale=P, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(rows=-1), ARG), (dict(d=0), ARG), (dict(d=4), ALIGN), (dict(d=32776), UNSUP), (dict(dtype=E4M3), DTYPE),
    (dict(x=None), ARG), (dict(q=None), ARG), (dict(scale=None), ARG), (dict(x=ODD), ALIGN), (dict(q=ODD), ALIGN),
    (dict(scale=P + 2), ALIGN), (dict(rows=(1 << 31) - 1, d=4096), ARG)])
def test_quantize_int8_refuses(change, status):
    assert C.lib().tss_quantize_int8(*_with(QUANT, **change)) == status


GEMM = dict(M=4, N=64, K=128, A=P, B=P, sa=P, sb=P, C=P, out=BF16, ws=None, ws_bytes=0, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(M=-1), ARG), (dict(N=-8), ARG), (dict(K=-16), ARG), (dict(K=136), ALIGN), (dict(K=1 << 17), ARG),
    (dict(out=I8), DTYPE), (dict(A=None), ARG), (dict(B=None), ARG), (dict(sa=None), ARG), (dict(sb=None), ARG),
    (dict(C=None), ARG), (dict(A=ODD), ALIGN), (dict(B=ODD), ALIGN), (dict(C=ODD), ALIGN), (dict(sa=P + 2), ALIGN),
    (dict(sb=P + 2), ALIGN), (dict(M=1 << 20, K=2048), ARG), (dict(N=1 << 20, K=2048), ARG), (dict(M=1 << 31), ARG),
    (dict(M=1 << 24, N=1 << 24, K=16), ARG), (dict(M=0), OK), (dict(N=0, A=None), OK)])
def test_gemm_int8_refuses(change, status):
    assert C.lib().tss_gemm_int8(*_with(GEMM, **change)) == status


def test_gemm_int8_wants_its_workspace():
    need = tss.gemm_int8_workspace_size(512, 512, 8192)
    assert need > 0 and need % (512 * 512 * 4) == 0
    big = dict(GEMM, M=512, N=512, K=8192)
    assert C.lib().tss_gemm_int8(*big.values()) == ARG
    assert C.lib().tss_gemm_int8(*_with(big, ws=P, ws_bytes=need - 1)) == ARG
    assert C.lib().tss_gemm_int8(*_with(big, ws=ODD, ws_bytes=need)) == ALIGN
    assert tss.gemm_int8_workspace_size(0, 512, 8192) == 0
    with pytest.raises(tss.TssError):
        tss.gemm_int8_workspace_size(100, 128, 8190)


SORT = dict(tokens=4, top=2, E=8, expert=P, bits=64, sizes=P, row=P, choice=P, ws=None, ws_bytes=0, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(tokens=-1), ARG), (dict(top=0), ARG), (dict(E=0), ARG), (dict(E=4097), ARG), (dict(bits=16), DTYPE),
    (dict(expert=None), ARG), (dict(sizes=None), ARG), (dict(row=None), ARG), (dict(choice=None), ARG),
    (dict(expert=P + 4), ALIGN), (dict(expert=P + 2, bits=32), ALIGN), (dict(sizes=P + 2), ALIGN), (dict(row=P + 1), ALIGN),
    (dict(choice=P + 2), ALIGN), (dict(tokens=1 << 20), ARG), (dict(tokens=1 << 30), ARG),
    (dict(tokens=1 << 20, ws=P, ws_bytes=64), ARG), (dict(tokens=1 << 20, ws=P + 2, ws_bytes=1 << 20), ALIGN)])
def test_sort_refuses(change, status):
    assert C.lib().tss_sort_by_expert(*_with(SORT, **change)) == status


def test_sort_workspace():
    size = C.lib().tss_sort_by_expert_workspace_size
    assert size(0, 2, 8) == 0 and size(64, 8, 256) == 0 and size(1 << 17, 8, 128) > 0
    assert size(-1, 2, 8) == ARG and size(4, 0, 8) == ARG and size(4, 2, 0) == ARG


GATHER = dict(tokens=4, top=2, d=64, dtype=BF16, x=P, row=P, choice=P, rows=P, scale=None, blocks=0, scale_out=None,
              stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(tokens=-1), ARG), (dict(top=0), ARG), (dict(d=0), ARG), (dict(d=12), ALIGN), (dict(dtype=9), DTYPE),
    (dict(x=None), ARG), (dict(row=None), ARG), (dict(rows=None), ARG), (dict(x=ODD), ALIGN), (dict(rows=ODD), ALIGN),
    (dict(blocks=1), ARG), (dict(blocks=1, scale=P, scale_out=P, choice=None), ARG), (dict(blocks=-1), ARG),
    (dict(tokens=1 << 29, d=1024), ARG), (dict(tokens=0, x=None), OK)])
def test_gather_refuses(change, status):
    assert C.lib().tss_gather_rows(*_with(GATHER, **change)) == status


COMBINE = dict(tokens=4, top=2, d=64, dtype=BF16, rows=P, row=P, weight=None, out=BF16, y=P, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(tokens=-1), ARG), (dict(d=12), ALIGN), (dict(dtype=E4M3), DTYPE), (dict(out=F16), DTYPE), (dict(out=I8), DTYPE),
    (dict(rows=None), ARG), (dict(row=None), ARG), (dict(y=None), ARG), (dict(rows=ODD), ALIGN), (dict(y=ODD), ALIGN),
    (dict(tokens=1 << 29, d=1024), ARG)])
def test_combine_refuses(change, status):
    assert C.lib().tss_combine_rows(*_with(COMBINE, **change)) == status


COMBINE_BACK = dict(tokens=4, top=2, d=64, dtype=BF16, dy=P, rows_dtype=BF16, rows=P, row=P, weight=P, drows=P, dweight=P,
                    stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(tokens=-1), ARG), (dict(d=12), ALIGN), (dict(d=32776), UNSUP), (dict(dtype=I8), DTYPE),
    (dict(rows_dtype=F16), DTYPE), (dict(dtype=F32), DTYPE), (dict(dy=None), ARG), (dict(rows=None), ARG),
    (dict(row=None), ARG), (dict(weight=None), ARG), (dict(drows=None), ARG), (dict(dweight=None), ARG),
    (dict(dy=ODD), ALIGN), (dict(rows=ODD), ALIGN), (dict(drows=ODD), ALIGN)])
def test_combine_backward_refuses(change, status):
    assert C.lib().tss_combine_rows_backward(*_with(COMBINE_BACK, **change)) == status


CLIP_NORM = P + (1 << 24)


def clip(at, sizes, types, out=None, max_norm=1.0, norm=CLIP_NORM, ws=P, ws_bytes=1 << 20):
    n = len(at)
    pointers = lambda v: None if v is None else (ctypes.c_void_p * n)(*v)  # noqa: E731
    return C.lib().tss_clip_grad_norm(n, pointers(at), (C.i64 * n)(*sizes), (C.i32 * n)(*types), max_norm, pointers(out),
                                      norm, ws, ws_bytes, None)


Q = P + (1 << 16)


@pytest.mark.parametrize("call,status", [
    (dict(at=[P], sizes=[-1], types=[F32]), ARG), (dict(at=[P], sizes=[1 << 41], types=[F32]), ARG),
    (dict(at=[P], sizes=[8], types=[E4M3]), DTYPE), (dict(at=[None], sizes=[8], types=[F32]), ARG),
    (dict(at=[P], sizes=[8], types=[F32], out=[None]), ARG), (dict(at=[P + 2], sizes=[8], types=[F32]), ALIGN),
    (dict(at=[P + 1], sizes=[8], types=[BF16]), ALIGN), (dict(at=[P], sizes=[8], types=[F32], norm=None), ARG),
    (dict(at=[P], sizes=[8], types=[F32], norm=P + 2), ALIGN), (dict(at=[P], sizes=[1 << 17], types=[F32], ws=None), ARG),
    (dict(at=[P], sizes=[8], types=[F32], ws=P + 4), ALIGN), (dict(at=[P], sizes=[1 << 17], types=[F32], ws_bytes=511), ARG),
    (dict(at=[P], sizes=[8], types=[F32], out=[P], max_norm=-1.0), ARG),
    (dict(at=[P], sizes=[8], types=[F32], out=[P], max_norm=float("nan")), ARG),
    # written twice, in place and not; an output that overlaps an input; one that begins inside another
    (dict(at=[P, P], sizes=[8, 8], types=[F32] * 2, out=[P, P]), ARG),
    (dict(at=[P, P], sizes=[8, 8], types=[F32] * 2, out=[Q, Q]), ARG),
    (dict(at=[P, Q], sizes=[8, 8], types=[F32] * 2, out=[Q, P]), ARG),
    (dict(at=[P], sizes=[8], types=[F32], out=[P + 4]), ARG), (dict(at=[P + 4], sizes=[8], types=[F32], out=[P]), ARG),
    (dict(at=[P, P + 16], sizes=[8, 8], types=[F32] * 2, out=[P, P + 16]), ARG),
    (dict(at=[P, Q], sizes=[8, 8], types=[F32] * 2, out=[P + 64, P + 92]), ARG),
    # the norm's place inside a tensor that is scaled, an output, an input
    (dict(at=[P], sizes=[8], types=[F32], out=[P], norm=P + 28), ARG), (dict(at=[P], sizes=[8], types=[F32], out=[Q], norm=Q), ARG),
    (dict(at=[P], sizes=[8], types=[F32], out=[Q], norm=P + 4), ARG)])
def test_clip_refuses(call, status):
    assert clip(**call) == status


def test_clip_workspace():
    size = lambda *n: C.lib().tss_clip_grad_norm_workspace_size(len(n), (C.i64 * len(n))(*n))  # noqa: E731
    assert size() == 0 and size(0) == 0 and size(-1) == ARG
    # up to 20 units of 2048 elements one workgroup needs none; else 8 bytes a workgroup, 2048 of them at most a table
    assert size(1) == 0 and size(2048 * 20) == 0 and size(2048 * 20 + 1) == 21 * 8 and size(2048 * 12, 1, 0, 2048 * 8) == 21 * 8
    assert size(*[1] * 128) == 128 * 8 and size(*[1] * 129) == 129 * 8 and size(1 << 26) == 2048 * 8


def z(*shape, t=torch.bfloat16):
    return torch.zeros(*shape, dtype=t)


S, I = torch.float32, torch.int32
ORDER = tss.ExpertOrder(z(3, t=I), z(4, 2, t=I), z(8, t=I))
CALLS = {
    "layer norm: host tensors": lambda: tss.layer_norm(z(4, 64), z(64)),
    "layer norm: one dimension": lambda: tss.layer_norm(z(64), z(64)),
    "layer norm: strided rows": lambda: tss.layer_norm(z(4, 128)[:, :64], z(64)),
    "layer norm: weight's length": lambda: tss.layer_norm(z(4, 64), z(32)),
    "layer norm: bias's type": lambda: tss.layer_norm(z(4, 64), z(64), z(64, t=S)),
    "layer norm: output type": lambda: tss.layer_norm(z(4, 64), z(64), out_dtype="e4m3"),
    "layer norm: scale without 8 bits": lambda: tss.layer_norm(z(4, 64), z(64), scale=z(4, t=S)),
    "layer norm: residual_out alone": lambda: tss.layer_norm(z(4, 64), z(64), residual_out=z(4, 64)),
    "layer norm: statistics' length": lambda: tss.layer_norm(z(4, 64), z(64), stats=(z(4, t=S), z(3, t=S))),
    "layer norm backward: mean's type": lambda: tss.layer_norm_backward(z(4, 64), z(4, 64), z(64), z(4), z(4, t=S)),
    "layer norm backward: host tensors": lambda: tss.layer_norm_backward(z(4, 64), z(4, 64), z(64), z(4, t=S), z(4, t=S)),
    "quantize_int8: odd gated row": lambda: tss.quantize_int8(z(4, 65), gated=True),
    "quantize_int8: scale's shape": lambda: tss.quantize_int8(z(4, 256), scale=z(2, 4, t=S)),
    "quantize_int8: host tensors": lambda: tss.quantize_int8(z(4, 64)),
    "gemm_int8: A's type": lambda: tss.gemm_int8(z(4, 64), z(8, 64, t=torch.int8), z(4, t=S), z(8, t=S)),
    "gemm_int8: unsigned": lambda: tss.gemm_int8(z(4, 64, t=torch.uint8), z(8, 64, t=torch.int8), z(4, t=S), z(8, t=S)),
    "gemm_int8: inner sizes": lambda: tss.gemm_int8(z(4, 64, t=torch.int8), z(8, 32, t=torch.int8), z(4, t=S), z(8, t=S)),
    "gemm_int8: sb's length": lambda: tss.gemm_int8(z(4, 64, t=torch.int8), z(8, 64, t=torch.int8), z(4, t=S), z(4, t=S)),
    "gemm_int8: transposed": lambda: tss.gemm_int8(z(4, 64, t=torch.int8), z(64, 64, t=torch.int8).t(), z(4, t=S), z(64, t=S)),
    "gemm_int8: host tensors": lambda: tss.gemm_int8(z(4, 64, t=torch.int8), z(8, 64, t=torch.int8), z(4, t=S), z(8, t=S)),
    "sort: floats": lambda: tss.sort_by_expert(z(4, 2), 3),
    "sort: one dimension": lambda: tss.sort_by_expert(z(4, t=I), 3),
    "sort: no choices": lambda: tss.sort_by_expert(z(4, 0, t=I), 3),
    "sort: strided": lambda: tss.sort_by_expert(z(2, 4, t=I).t(), 3),
    "sort: host tensors": lambda: tss.sort_by_expert(z(4, 2, t=I), 3),
    "gather: other tokens": lambda: tss.gather_rows(z(5, 64), ORDER),
    "gather: scale's length": lambda: tss.gather_rows(z(4, 64), ORDER, z(1, 5, t=S)),
    "gather: scale_out alone": lambda: tss.gather_rows(z(4, 64), ORDER, scale_out=z(1, 8, t=S)),
    "gather: order's type": lambda: tss.gather_rows(z(4, 64), ORDER._replace(row=z(4, 2, t=torch.int64))),
    "gather: choices' length": lambda: tss.gather_rows(z(4, 64), ORDER._replace(choice=z(7, t=I))),
    "gather: host tensors": lambda: tss.gather_rows(z(4, 64), ORDER),
    "combine: rows": lambda: tss.combine_rows(z(4, 64), ORDER),
    "combine: weight's type": lambda: tss.combine_rows(z(8, 64), ORDER, z(4, 2)),
    "combine: out type": lambda: tss.combine_rows(z(8, 64), ORDER, out_dtype="f16"),
    "combine: host tensors": lambda: tss.combine_rows(z(8, 64), ORDER),
    "combine backward: rows' type": lambda: tss.combine_rows_backward(z(4, 64, t=S), z(8, 64), ORDER, z(4, 2, t=S)),
    "combine backward: tokens": lambda: tss.combine_rows_backward(z(3, 64), z(8, 64), ORDER, z(4, 2, t=S)),
    "gather backward: rows": lambda: tss.gather_rows_backward(z(7, 64), ORDER),
    "clip: nothing": lambda: tss.clip_grad_norm([], 1.0),
    "clip: integers": lambda: tss.clip_grad_norm([z(4, t=I)], 1.0),
    "clip: gaps": lambda: tss.clip_grad_norm([z(4, 8)[:, :4]], 1.0),
    "clip: broadcast": lambda: tss.clip_grad_norm([z(1).expand(4)], 1.0),
    "clip: outputs": lambda: tss.clip_grad_norm([z(4)], 1.0, out=[]),
    "clip: output's type": lambda: tss.clip_grad_norm([z(4)], 1.0, out=[z(4, t=S)]),
    "clip: output's order": lambda: tss.clip_grad_norm([z(4, 4)], 1.0, out=[z(4, 4).t()]),
    "clip: host tensors": lambda: tss.clip_grad_norm([z(4)], 1.0),
    "norm: host tensors": lambda: tss.grad_norm([z(4)]),
    "clip: host tensors on a stream": lambda: tss.clip_grad_norm([z(4)], 1.0, stream=0),
}


@pytest.mark.parametrize("call", CALLS.values(), ids=CALLS.keys())
def test_python_calls_refuse(call):
    with pytest.raises(ValueError):
        call()

"""Calls whose outputs or workspace overlap what else they read or write are
refused before any device work (their workgroups run in no order: each such
call would be a race), through the C ABI with addresses that are never touched."""
import ctypes

import pytest

from tile_size_selection_amd import _capi as C

ARG, BF16, F32, I8 = C.TSS_E_ARG, C.TSS_BF16, C.TSS_F32, C.TSS_I8
MIB = 1 << 20


def at(i, off=0):
    """Address `off` bytes into the i-th of many places a MiB long."""
    return (i + 1) * MIB + off


def refused(call, base, change):
    assert set(change) <= set(base)
    return call(*{**base, **change}.values()) == ARG


SORT = dict(tokens=4, top=2, E=8, expert=at(0), bits=64, sizes=at(1), row=at(2), choice=at(3), ws=None, ws_bytes=0, stream=None)
LONG = dict(SORT, tokens=20000, ws=at(4), ws_bytes=MIB)


@pytest.mark.parametrize("base,change", [
    (SORT, dict(row=at(0))), (SORT, dict(row=at(0, 4), bits=32)), (SORT, dict(choice=at(0), bits=32)), (SORT, dict(choice=at(0, 60))),
    (SORT, dict(sizes=at(0, 28), bits=32)), (SORT, dict(row=at(3))), (SORT, dict(choice=at(2, 28))), (SORT, dict(sizes=at(2, 28))),
    (SORT, dict(sizes=at(2, -28))), (SORT, dict(sizes=at(3))), (SORT, dict(row=at(0), choice=at(0), bits=32)),
    (LONG, dict(ws=at(0, 8))), (LONG, dict(ws=at(1))), (LONG, dict(ws=at(2, 159996))), (LONG, dict(ws=at(3, -4)))])
def test_sort(base, change):
    assert refused(C.lib().tss_sort_by_expert, base, change)


GATHER = dict(tokens=4, top=2, d=64, dtype=BF16, x=at(0), row=at(1), choice=at(2), rows=at(3), scale=at(4), blocks=3,
              scale_out=at(5), stream=None)


@pytest.mark.parametrize("change", [
    dict(rows=at(0)), dict(rows=at(0, 496)), dict(rows=at(0, -1008)), dict(rows=at(0), top=1), dict(rows=at(1, 16)),
    dict(rows=at(2, -1008)), dict(rows=at(4, 32)), dict(scale_out=at(4)), dict(scale_out=at(4), top=1), dict(scale_out=at(3, 1020)),
    dict(scale_out=at(0)), dict(scale_out=at(1)), dict(scale_out=at(2, 28)),
    dict(rows=at(0), top=1, choice=None, scale=None, blocks=0, scale_out=None)])
def test_gather(change):
    assert refused(C.lib().tss_gather_rows, GATHER, change)


COMBINE = dict(tokens=4, top=2, d=64, dtype=BF16, rows=at(0), row=at(1), weight=at(2), out=BF16, y=at(3), stream=None)


@pytest.mark.parametrize("change", [
    dict(y=at(0)), dict(y=at(0), top=1), dict(y=at(0, 1008)), dict(y=at(0, -496)), dict(y=at(0, -1008), out=F32), dict(y=at(1)),
    dict(y=at(2, 16)), dict(y=at(0), weight=None)])
def test_combine(change):
    assert refused(C.lib().tss_combine_rows, COMBINE, change)


BACK = dict(tokens=4, top=2, d=64, dtype=BF16, dy=at(0), rows_dtype=BF16, rows=at(1), row=at(2), weight=at(3), drows=at(4),
            dweight=at(5), stream=None)


@pytest.mark.parametrize("change", [
    dict(drows=at(0)), dict(drows=at(0), top=1), dict(drows=at(0, 496)), dict(drows=at(1, 16)), dict(drows=at(1, -16)),
    dict(drows=at(1), rows_dtype=F32), dict(drows=at(2)), dict(drows=at(3, 16)), dict(drows=at(5, -1008)), dict(dweight=at(0)),
    dict(dweight=at(1, 1020)), dict(dweight=at(2)), dict(dweight=at(3, 4)), dict(dweight=at(4, 1020)),
    dict(drows=at(1), dweight=at(1))])
def test_combine_backward(change):
    assert refused(C.lib().tss_combine_rows_backward, BACK, change)


NORM = dict(rows=4, d=64, dtype=BF16, x=at(0), residual=at(1), weight=at(2), bias=at(3), eps=1e-5, out_dtype=BF16, y=at(4),
            scale=None, h=at(5), mean=at(6), rstd=at(7), stream=None)
NORM_I8 = dict(NORM, out_dtype=I8, scale=at(8))


@pytest.mark.parametrize("base,change", [
    (NORM, dict(y=at(0, 128))), (NORM, dict(y=at(0, -128))), (NORM, dict(y=at(1, 496))), (NORM, dict(y=at(2))), (NORM, dict(y=at(3, 112))),
    (NORM, dict(y=at(5))), (NORM, dict(y=at(5, 16))), (NORM, dict(y=at(0), h=at(0))), (NORM, dict(h=at(1, 128))), (NORM, dict(h=at(2))),
    (NORM, dict(mean=at(7))), (NORM, dict(mean=at(0))), (NORM, dict(rstd=at(6, 12))), (NORM, dict(rstd=at(4, 508))), (NORM, dict(mean=at(3))),
    (NORM_I8, dict(y=at(0))), (NORM_I8, dict(y=at(1))), (NORM_I8, dict(y=at(1, 496))), (NORM_I8, dict(scale=at(4, 252))),
    (NORM_I8, dict(scale=at(6))), (NORM_I8, dict(scale=at(0))), (NORM_I8, dict(y=at(5)))])
def test_layer_norm(base, change):
    assert refused(C.lib().tss_layer_norm, base, change)


# 4 rows: one launch; 2000: two, which read dy and h once
NORM_BACK = dict(rows=4, d=64, dtype=BF16, dy=at(0), h=at(1), weight=at(2), mean=at(3), rstd=at(4), dh=at(5), dx=at(6), dweight=at(7),
                 dbias=at(8), ws=at(9), ws_bytes=MIB, stream=None)


@pytest.mark.parametrize("rows", [4, 2000])
@pytest.mark.parametrize("change", [
    dict(dx=at(0, 128)), dict(dx=at(0, -128)), dict(dx=at(1, 128)), dict(dx=at(5, -16)), dict(dx=at(2)), dict(dx=at(3)), dict(dx=at(4, 0)),
    dict(dx=at(7)), dict(dx=at(9)), dict(dweight=at(0)), dict(dweight=at(1, 64)), dict(dweight=at(8)), dict(dbias=at(2)), dict(dbias=at(6)),
    dict(dbias=at(3)), dict(ws=at(0)), dict(ws=at(1, 16)), dict(ws=at(5)), dict(ws=at(6)), dict(ws=at(8)), dict(ws=at(7, -16))])
def test_layer_norm_backward(change, rows):
    assert refused(C.lib().tss_layer_norm_backward, dict(NORM_BACK, rows=rows), change)


QUANT = dict(rows=4, d=64, dtype=BF16, x=at(0), gated=0, q=at(1), scale=at(2), stream=None)


@pytest.mark.parametrize("change", [
    dict(q=at(0)), dict(q=at(0), dtype=F32), dict(q=at(0, 496)), dict(q=at(0, -240)), dict(q=at(0, 512), gated=1), dict(q=at(2, -240)),
    dict(scale=at(0)), dict(scale=at(1, 252)), dict(scale=at(0, 1020), gated=1), dict(scale=at(0, 1020), dtype=F32)])
def test_quantize_int8(change):
    assert refused(C.lib().tss_quantize_int8, QUANT, change)


GEMM = dict(M=4, N=64, K=128, A=at(0), B=at(1), sa=at(2), sb=at(3), C=at(4), out=BF16, ws=None, ws_bytes=0, stream=None)
SPLIT = dict(GEMM, M=256, N=512, K=8192, B=at(8), sa=at(16), sb=at(17), C=at(18), ws=at(24), ws_bytes=1 << 24)


@pytest.mark.parametrize("base,change", [
    (GEMM, dict(C=at(0))), (GEMM, dict(C=at(0, -496))), (GEMM, dict(C=at(0, 496))), (GEMM, dict(C=at(1, 8176))), (GEMM, dict(C=at(2))),
    (GEMM, dict(C=at(3, 240))), (GEMM, dict(C=at(2, -1008), out=F32)),
    (SPLIT, dict(C=at(8))), (SPLIT, dict(ws=at(0))), (SPLIT, dict(ws=at(8, 16))), (SPLIT, dict(ws=at(16))), (SPLIT, dict(ws=at(17))),
    (SPLIT, dict(ws=at(18))), (SPLIT, dict(ws=at(18, -16))), (SPLIT, dict(C=at(24, 16)))])
def test_gemm_int8(base, change):
    assert refused(C.lib().tss_gemm_int8, base, change)


def clip(tensors, out=None, norm=at(30), ws=at(31)):
    """tensors: (address, elements), fp32."""
    n = len(tensors)
    pointers = lambda v: None if v is None else (ctypes.c_void_p * n)(*v)  # noqa: E731
    return C.lib().tss_clip_grad_norm(n, pointers([a for a, _ in tensors]), (C.i64 * n)(*[e for _, e in tensors]), (C.i32 * n)(*[F32] * n),
                                      1.0, pointers(out), norm, ws, MIB, None)


TWO = [(at(0), 200000), (at(1), 100000)]  # 147 sums, 1176 bytes of workspace


@pytest.mark.parametrize("call", [
    dict(norm=at(0, 4)), dict(norm=at(1, 399996)), dict(norm=at(31, 1172)), dict(ws=at(0)), dict(ws=at(1, 399992)), dict(ws=at(1, -1168)),
    dict(ws=at(30)), dict(out=[at(0), at(1)], ws=at(1)), dict(out=[at(2), at(3)], ws=at(3, 8)), dict(out=[at(2), at(3)], ws=at(0)),
    dict(out=[at(2), at(3)], ws=at(30, -1168)), dict(out=[at(2), at(3)], norm=at(31, 8))])
def test_clipping(call):
    assert clip(TWO, **call) == ARG

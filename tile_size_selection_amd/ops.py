"""Row operators (root-mean-square and layer norm, quantisation to 8 bits), the
8-bit and grouped matrix products, and the gradients' norm and clipping: argument checks and marshalling only, as in
api.py; the work is libtss.so's (include/tss.h documents each entry point).

Each call takes stream=, the stream to run on (the current one without it).
Element types are named 'f16', 'bf16', 'f32', 'e4m3', 'e5m2' and 'i8'.  Scales
of 8-bit floating-point tensors are float32, one for each block of 1 or 128
rows x 128 columns, column-block-major: scale[column block][row or row block];
those of 8-bit integers one for each row: scale[row]."""
from __future__ import annotations

import functools
from typing import NamedTuple, Optional, Sequence, Tuple

from . import _capi as C
from .api import _workspace, torch

_DT = {"f16": C.TSS_F16, "bf16": C.TSS_BF16, "f32": C.TSS_F32, "e4m3": C.TSS_E4M3, "e5m2": C.TSS_E5M2,
       "i8": C.TSS_I8}
if torch is not None:
    _TORCH = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32,
              "e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2, "i8": torch.int8}
    _NAME = {v: k for k, v in _TORCH.items()}


def _name(t, what: str, allowed) -> str:
    n = _NAME.get(t.dtype)
    if n not in allowed:
        raise ValueError(f"{what} must be one of {', '.join(allowed)}, not {t.dtype}")
    return n


def _choice(value: str, what: str, allowed) -> str:
    if value not in allowed:
        raise ValueError(f"{what} must be one of {', '.join(allowed)}, not {value!r}")
    return value


def _fits(t, dtype, *shape) -> bool:
    """Whether t is contiguous, of this element type and shape; the first call
    puts the compiled function in its place (it takes a third of the time)."""
    global _fits
    _fits = C.bind().fits
    return _fits(t, dtype, *shape)


def _given(t, what: str, shape, dtype):
    """t, checked: contiguous, of this shape and element type."""
    if not _fits(t, dtype, *shape):
        raise ValueError(f"{what} must be a contiguous {dtype} tensor of shape {tuple(shape)}, not {t.dtype} "
                         f"{tuple(t.shape)}" + ("" if t.is_contiguous() else ", not contiguous"))
    return t


def _out(t, what: str, shape, dtype, device):
    return torch.empty(shape, dtype=dtype, device=device) if t is None else _given(t, what, shape, dtype)


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


# The current stream's handle on a GPU.  torch.cuda.current_stream() makes a
# Stream object for it, which costs 2.7 of the 11.5 us that a call of these
# operators took on the host (a launch itself is 3.3); torch's own code
# generators read the handle this way.
_raw_stream = getattr(getattr(torch, "_C", None), "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _streamed(f):
    """f with stream=None or the stream to run on (a torch stream of the
    tensors' GPU, or a HIP stream's handle).  The stream is made current for
    the call, so that what is allocated in it belongs to that stream too: a
    workspace freed on return is reused behind the launch that uses it."""
    @functools.wraps(f)
    def call(*args, stream=None, **kwargs):
        if stream is None:
            return f(*args, **kwargs)
        device = next((a.device for a in (*args, *kwargs.values()) if isinstance(a, torch.Tensor)), None)
        if device is None or device.type != "cuda":
            raise ValueError(f"stream= needs tensors on a GPU, not on {device}")
        if not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(stream, device=device)
        elif stream.device != device:
            raise ValueError(f"the stream is of {stream.device}, the tensors are on {device}")
        with torch.cuda.stream(stream):
            return f(*args, **kwargs)
    return call


def _call(where: str, fn, tensors, *args):
    """fn(*args, current stream) with the tensors' GPU current; every tensor
    (None aside) must be on it."""
    index = tensors[0].get_device()
    for t in tensors:
        if t is not None and (t.get_device() != index or index < 0):
            raise ValueError("every tensor must be on the same GPU")
    if index == torch.cuda.current_device():
        st = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            st = fn(*args, _raw_stream(index))
    if st != C.TSS_OK:
        C.check(st, where)


_ENTRIES = {}  # the compiled binding's functions that were called, by name


def _entry(name: str):
    f = _ENTRIES.get(name)
    if f is None:
        f = _ENTRIES[name] = getattr(C.bind(), name)
    return f


def _run(name: str, *args):
    """The entry point of this name on args and the current stream, through the
    compiled binding: tensors are given as they are, all on one GPU."""
    st = _entry(name)(*args)
    if st != C.TSS_OK:
        C.check(st, name)


def _size(name: str, *args) -> int:
    """What the entry point of this name, a workspace's size, gives."""
    n = _entry(name)(*args)
    if n < 0:
        C.check(n, name)
    return n


def _blocks(n: int) -> int:
    return (n + 127) // 128


class RmsNorm(NamedTuple):
    y: "torch.Tensor"
    scale: Optional["torch.Tensor"]  # e4m3 output only
    h: Optional["torch.Tensor"]      # x + residual; None without a residual
    rstd: Optional["torch.Tensor"]   # 1 / sqrt(mean(h^2) + eps), where asked for


@_streamed
def rms_norm(x, weight, residual=None, eps: float = 1e-6, out_dtype: Optional[str] = None, out=None, scale=None,
             residual_out=None, rstd=None) -> RmsNorm:
    """h = x + residual (x without one); y = h / sqrt(mean(h^2) + eps) * weight
    over the last dimension of x (rows, d), d a multiple of 8 up to 32768;
    fp32 inside.  out_dtype: x's type (the default) or 'e4m3', with a scale
    for each 128 columns of a row, scale[ceil(d / 128)][rows].  h comes back
    rounded to x's type (residual_out may be residual itself).  rstd: True,
    or a float32 tensor of `rows`, to get the statistics the backward pass
    takes.  out, scale, residual_out: outputs to write into, else allocated."""
    dt = _name(x, "x", ("f16", "bf16", "f32"))
    if x.dim() != 2:
        raise ValueError("x must be (rows, d)")
    rows, d = x.shape
    od = _choice(out_dtype or dt, "out_dtype", (dt, "e4m3"))
    _given(x, "x", (rows, d), x.dtype)
    _given(weight, "weight", (d,), x.dtype)
    out = _out(out, "out", (rows, d), _TORCH[od], x.device)
    if od == "e4m3":
        scale = _out(scale, "scale", (_blocks(d), rows), torch.float32, x.device)
    elif scale is not None:
        raise ValueError("scale is only for out_dtype 'e4m3'")
    if residual is not None:
        _given(residual, "residual", (rows, d), x.dtype)
        residual_out = _out(residual_out, "residual_out", (rows, d), x.dtype, x.device)
    elif residual_out is not None:
        raise ValueError("residual_out needs a residual")
    if rstd is False:
        rstd = None
    elif rstd is not None:
        rstd = _out(None if rstd is True else rstd, "rstd", (rows,), torch.float32, x.device)
    _call("tss_rms_norm", C.lib().tss_rms_norm, (x, weight, out, residual, scale, residual_out, rstd),
          rows, d, _DT[dt], x.data_ptr(), _ptr(residual), weight.data_ptr(), eps, _DT[od], out.data_ptr(), _ptr(scale),
          _ptr(residual_out), _ptr(rstd))
    return RmsNorm(out, scale, residual_out, rstd)


@_streamed
def rms_norm_backward(dy, h, weight, rstd, dh=None, dx=None, dweight=None,
                      workspace=None) -> Tuple["torch.Tensor", "torch.Tensor"]:
    """(dx, dweight) of rms_norm from its h (or x, without a residual) and
    rstd: dx = dh + rstd (dy weight - xhat mean(dy weight xhat)) with xhat =
    h rstd, the gradient of both x and residual (dh: the gradient that arrives
    through h; it may be None), and dweight = sum over rows of dy xhat in
    float32, the same bits on every run.  dx may be dy or dh."""
    dt = _name(dy, "dy", ("f16", "bf16", "f32"))
    if dy.dim() != 2:
        raise ValueError("dy must be (rows, d)")
    rows, d = dy.shape
    _given(dy, "dy", (rows, d), dy.dtype)
    _given(h, "h", (rows, d), dy.dtype)
    _given(weight, "weight", (d,), dy.dtype)
    _given(rstd, "rstd", (rows,), torch.float32)
    if dh is not None:
        _given(dh, "dh", (rows, d), dy.dtype)
    dx = _out(dx, "dx", (rows, d), dy.dtype, dy.device)
    dweight = _out(dweight, "dweight", (d,), torch.float32, dy.device)
    need = C.lib().tss_rms_norm_backward_workspace_size(rows, d)
    if need < 0:
        C.check(int(need), "tss_rms_norm_backward_workspace_size")
    workspace = _workspace(workspace, need, dy.device)
    _call("tss_rms_norm_backward", C.lib().tss_rms_norm_backward,
          (dy, h, weight, rstd, dh, dx, dweight, workspace),
          rows, d, _DT[dt], dy.data_ptr(), h.data_ptr(), weight.data_ptr(), rstd.data_ptr(), _ptr(dh), dx.data_ptr(),
          dweight.data_ptr(), workspace.data_ptr(), workspace.numel() * workspace.element_size())
    return dx, dweight


class LayerNorm(NamedTuple):
    y: "torch.Tensor"
    scale: Optional["torch.Tensor"]  # i8 output only
    h: Optional["torch.Tensor"]      # x + residual; None without a residual
    mean: Optional["torch.Tensor"]   # mean(h) and 1 / sqrt(mean((h - mean)^2) + eps), where asked for
    rstd: Optional["torch.Tensor"]


@_streamed
def layer_norm(x, weight, bias=None, residual=None, eps: float = 1e-5, out_dtype: Optional[str] = None, out=None,
               scale=None, residual_out=None, stats=None) -> LayerNorm:
    """h = x + residual (x without one); y = (h - mean(h)) / sqrt(mean((h -
    mean(h))^2) + eps) * weight + bias (0 without one) over the last dimension
    of x (rows, d), d a multiple of 8 up to 32768; fp32 inside.  out_dtype: x's
    type (the default) or 'i8', with a scale for each row (as quantize_int8
    gives).  h comes back rounded to x's type (residual_out may be residual
    itself).  stats: True, or a pair of float32 tensors of `rows`, to get the
    mean and rstd that the backward pass takes.  out, scale, residual_out:
    outputs to write into, else allocated; out may be x or residual (unless it
    is 'i8', or residual_out is that one), other overlaps are refused."""
    dt = _name(x, "x", ("f16", "bf16", "f32"))
    if x.dim() != 2:
        raise ValueError("x must be (rows, d)")
    rows, d = x.shape
    od = _choice(out_dtype or dt, "out_dtype", (dt, "i8"))
    _given(x, "x", (rows, d), x.dtype)
    _given(weight, "weight", (d,), x.dtype)
    if bias is not None:
        _given(bias, "bias", (d,), x.dtype)
    out = _out(out, "out", (rows, d), _TORCH[od], x.device)
    if od == "i8":
        scale = _out(scale, "scale", (rows,), torch.float32, x.device)
    elif scale is not None:
        raise ValueError("scale is only for out_dtype 'i8'")
    if residual is not None:
        _given(residual, "residual", (rows, d), x.dtype)
        residual_out = _out(residual_out, "residual_out", (rows, d), x.dtype, x.device)
    elif residual_out is not None:
        raise ValueError("residual_out needs a residual")
    mean = rstd = None
    if stats is not None and stats is not False:
        mean, rstd = (None, None) if stats is True else stats
        mean = _out(mean, "mean", (rows,), torch.float32, x.device)
        rstd = _out(rstd, "rstd", (rows,), torch.float32, x.device)
    _run("tss_layer_norm", rows, d, _DT[dt], x, residual, weight, bias, float(eps), _DT[od], out, scale, residual_out, mean,
         rstd)
    return LayerNorm(out, scale, residual_out, mean, rstd)


@_streamed
def layer_norm_backward(dy, h, weight, mean, rstd, dh=None, dx=None, dweight=None, dbias=None, workspace=None):
    """(dx, dweight, dbias) of layer_norm from its h (or x, without a residual),
    mean and rstd: with xhat = (h - mean) rstd and g = dy weight, dx = dh + rstd
    (g - mean(g) - xhat mean(g xhat)), the gradient of both x and residual (dh:
    the gradient that arrives through h; it may be None), dweight = sum over
    rows of dy xhat and dbias = sum over rows of dy in float32, the same bits on
    every run.  dbias False: not computed, None comes back.  dx may be dy, h or
    dh; other overlaps are refused."""
    dt = _name(dy, "dy", ("f16", "bf16", "f32"))
    if dy.dim() != 2:
        raise ValueError("dy must be (rows, d)")
    rows, d = dy.shape
    _given(dy, "dy", (rows, d), dy.dtype)
    _given(h, "h", (rows, d), dy.dtype)
    _given(weight, "weight", (d,), dy.dtype)
    _given(mean, "mean", (rows,), torch.float32)
    _given(rstd, "rstd", (rows,), torch.float32)
    if dh is not None:
        _given(dh, "dh", (rows, d), dy.dtype)
    dx = _out(dx, "dx", (rows, d), dy.dtype, dy.device)
    dweight = _out(dweight, "dweight", (d,), torch.float32, dy.device)
    dbias = None if dbias is False else _out(dbias, "dbias", (d,), torch.float32, dy.device)
    need = _size("tss_layer_norm_backward_workspace_size", rows, d)
    workspace = _workspace(workspace, need, dy.device)
    _run("tss_layer_norm_backward", rows, d, _DT[dt], dy, h, weight, mean, rstd, dh, dx, dweight, dbias, workspace,
         workspace.nbytes)
    return dx, dweight, dbias


@_streamed
def quantize_fp8(x, fp8: str = "e4m3", gated: bool = False, block_rows: int = 1, out=None,
                 scale=None) -> Tuple["torch.Tensor", "torch.Tensor"]:
    """(q, scale) of x (rows, d), or with gated of silu(gate) * up where x is
    (rows, 2 d), gate then up: q in 'e4m3' or 'e5m2' with a float32 scale for
    each block of block_rows (1 or 128) x 128, scale[ceil(d / 128)][rows or
    ceil(rows / 128)].  d a multiple of 8."""
    dt = _name(x, "x", ("f16", "bf16", "f32"))
    _choice(fp8, "fp8", ("e4m3", "e5m2"))
    if block_rows not in (1, 128):
        raise ValueError("block_rows must be 1 or 128")
    if x.dim() != 2 or (gated and x.shape[1] % 2):
        raise ValueError("x must be (rows, d), or (rows, 2 d) with gated")
    rows, d = x.shape
    _given(x, "x", (rows, d), x.dtype)
    if gated:
        d //= 2
    out = _out(out, "out", (rows, d), _TORCH[fp8], x.device)
    scale = _out(scale, "scale", (_blocks(d), rows if block_rows == 1 else _blocks(rows)), torch.float32, x.device)
    _call("tss_quantize_fp8", C.lib().tss_quantize_fp8, (x, out, scale),
          rows, d, _DT[dt], x.data_ptr(), int(gated), _DT[fp8], block_rows, out.data_ptr(), scale.data_ptr())
    return out, scale


@_streamed
def quantize_int8(x, gated: bool = False, out=None, scale=None) -> Tuple["torch.Tensor", "torch.Tensor"]:
    """(q, scale) of x (rows, d), or with gated of silu(gate) * up where x is
    (rows, 2 d), gate then up: q int8 in -127 .. 127 and scale (rows,) float32,
    the row's largest magnitude / 127.  d a multiple of 8 up to 32768.  out and
    scale over x or each other are refused."""
    dt = _name(x, "x", ("f16", "bf16", "f32"))
    if x.dim() != 2 or (gated and x.shape[1] % 2):
        raise ValueError("x must be (rows, d), or (rows, 2 d) with gated")
    rows, d = x.shape
    _given(x, "x", (rows, d), x.dtype)
    if gated:
        d //= 2
    out = _out(out, "out", (rows, d), torch.int8, x.device)
    scale = _out(scale, "scale", (rows,), torch.float32, x.device)
    _run("tss_quantize_int8", rows, d, _DT[dt], x, int(gated), out, scale)
    return out, scale


def _out_type(out_dtype: str, fp32_sums: bool) -> int:
    return _DT[out_dtype] | (C.TSS_F32_SUMS if fp32_sums else 0)


def gemm_fp8_workspace_size(M: int, N: int, K: int) -> int:
    n = C.lib().tss_gemm_fp8_workspace_size(M, N, K)
    if n < 0:
        C.check(int(n), "tss_gemm_fp8_workspace_size")
    return int(n)


@_streamed
def gemm_fp8(A, B, sa, sb, out_dtype: str = "bf16", out=None, workspace=None, fp32_sums: bool = False):
    """C = (A sa) @ (B sb)^T for 8-bit A (M, K), e4m3 or e5m2, and B (N, K),
    e4m3, with sa[ceil(K / 128)][M] and sb[ceil(K / 128)][N or ceil(N / 128)];
    out_dtype 'bf16', 'f16' or 'f32'.  fp32_sums: sums in fp32 throughout, at
    half the rate ('f32' always has them; without it a 16-bit output's blocks
    of 128 are summed in fewer bits, which shows where large products cancel:
    tss_gemm_fp8 in include/tss.h).  K a multiple of 16.  workspace: a device
    tensor of at least gemm_fp8_workspace_size bytes (allocated here when one
    is needed and not given)."""
    adt = _name(A, "A", ("e4m3", "e5m2"))
    _name(B, "B", ("e4m3",))
    if A.dim() != 2 or B.dim() != 2 or A.shape[1] != B.shape[1]:
        raise ValueError(f"shape mismatch {tuple(A.shape)} x {tuple(B.shape)}^T")
    (M, K), N = A.shape, B.shape[0]
    _given(A, "A", (M, K), A.dtype)
    _given(B, "B", (N, K), B.dtype)
    _choice(out_dtype, "out_dtype", ("bf16", "f16", "f32"))
    kb = _blocks(K)
    _given(sa, "sa", (kb, M), torch.float32)
    b_rows = 1 if tuple(sb.shape) == (kb, N) else 128
    _given(sb, "sb", (kb, N if b_rows == 1 else _blocks(N)), torch.float32)
    out = _out(out, "out", (M, N), _TORCH[out_dtype], A.device)
    need = gemm_fp8_workspace_size(M, N, K)
    if need:
        workspace = _workspace(workspace, need, A.device)
    _call("tss_gemm_fp8", C.lib().tss_gemm_fp8, (A, B, sa, sb, out, workspace),
          M, N, K, _DT[adt], A.data_ptr(), B.data_ptr(), sa.data_ptr(), sb.data_ptr(), b_rows, out.data_ptr(),
          _out_type(out_dtype, fp32_sums), _ptr(workspace), 0 if workspace is None else workspace.numel() * workspace.element_size())
    return out


def gemm_int8_workspace_size(M: int, N: int, K: int) -> int:
    return _size("tss_gemm_int8_workspace_size", M, N, K)


@_streamed
def gemm_int8(A, B, sa, sb, out_dtype: str = "bf16", out=None, workspace=None):
    """C = (A sa) @ (B sb)^T for int8 A (M, K) with sa (M,), one scale for each
    token, and int8 B (N, K) with sb (N,), one for each channel; the sums over K
    are exact.  out_dtype 'bf16', 'f16' or 'f32'.  K a multiple of 16 below
    2^17.  workspace: a device tensor of at least gemm_int8_workspace_size bytes
    (allocated here when one is needed and not given).  out and workspace over
    an operand or each other are refused."""
    _name(A, "A", ("i8",))
    _name(B, "B", ("i8",))
    if A.dim() != 2 or B.dim() != 2 or A.shape[1] != B.shape[1]:
        raise ValueError(f"shape mismatch {tuple(A.shape)} x {tuple(B.shape)}^T")
    (M, K), N = A.shape, B.shape[0]
    _given(A, "A", (M, K), A.dtype)
    _given(B, "B", (N, K), B.dtype)
    _choice(out_dtype, "out_dtype", ("bf16", "f16", "f32"))
    _given(sa, "sa", (M,), torch.float32)
    _given(sb, "sb", (N,), torch.float32)
    out = _out(out, "out", (M, N), _TORCH[out_dtype], A.device)
    need = gemm_int8_workspace_size(M, N, K)
    if need:
        workspace = _workspace(workspace, need, A.device)
    _run("tss_gemm_int8", M, N, K, A, B, sa, sb, out, _DT[out_dtype], workspace, 0 if workspace is None else workspace.nbytes)
    return out


def _groups(sizes) -> int:
    if sizes.dim() != 1 or sizes.shape[0] < 1:
        raise ValueError("sizes must hold one int32 per group")
    _given(sizes, "sizes", (sizes.shape[0],), torch.int32)
    return sizes.shape[0]


@_streamed
def gemm_grouped(A, B, sizes, out_dtype: Optional[str] = None, out=None):
    """C[rows of group e] = A[rows of e] @ B[e]: A (T, K) sorted by group, B
    (E, K, N), f16 or bf16; sizes (E,) int32 on the GPU, the rows of each
    group (read on the device, so a captured graph follows them).  Rows past
    their sum come back zero.  out_dtype: A's type (the default) or 'f32'.  K
    and N multiples of 8."""
    dt = _name(A, "A", ("f16", "bf16"))
    if A.dim() != 2 or B.dim() != 3 or A.shape[1] != B.shape[1]:
        raise ValueError(f"shape mismatch {tuple(A.shape)} x {tuple(B.shape)}")
    (T, K), (E, _, N) = A.shape, B.shape
    _given(A, "A", (T, K), A.dtype)
    _given(B, "B", (E, K, N), A.dtype)
    if _groups(sizes) != E:
        raise ValueError("sizes and B disagree on the number of groups")
    od = _choice(out_dtype or dt, "out_dtype", (dt, "f32"))
    out = _out(out, "out", (T, N), _TORCH[od], A.device)
    _call("tss_gemm_grouped", C.lib().tss_gemm_grouped, (A, B, sizes, out),
          T, E, K, N, _DT[dt], A.data_ptr(), B.data_ptr(), sizes.data_ptr(), out.data_ptr(), _DT[od])
    return out


@_streamed
def gemm_grouped_backward(dC, A, B, sizes, dA=None, dB=None, db_dtype: str = "f32", need_dA: bool = True,
                          need_dB: bool = True):
    """(dA, dB) of gemm_grouped: dA[rows of e] = dC[rows of e] @ B[e]^T in A's
    type (rows of no group: zero), dB[e] = A[rows of e]^T @ dC[rows of e] in
    db_dtype ('f32' or A's type; a group without rows: zero).  need_dA or
    need_dB False: that one is not computed and comes back None."""
    dt = _name(A, "A", ("f16", "bf16"))
    if A.dim() != 2 or B.dim() != 3 or dC.dim() != 2 or A.shape[1] != B.shape[1]:
        raise ValueError(f"shape mismatch {tuple(A.shape)} x {tuple(B.shape)}")
    (T, K), (E, _, N) = A.shape, B.shape
    _given(A, "A", (T, K), A.dtype)
    _given(B, "B", (E, K, N), A.dtype)
    _given(dC, "dC", (T, N), A.dtype)
    if _groups(sizes) != E:
        raise ValueError("sizes and B disagree on the number of groups")
    _choice(db_dtype, "db_dtype", ("f32", dt))
    if (dA is not None and not need_dA) or (dB is not None and not need_dB):
        raise ValueError("an output that is not needed must not be given")
    if need_dA:
        dA = _out(dA, "dA", (T, K), A.dtype, A.device)
    if need_dB:
        dB = _out(dB, "dB", (E, K, N), _TORCH[db_dtype], A.device)
    _call("tss_gemm_grouped_backward", C.lib().tss_gemm_grouped_backward, (A, B, dC, sizes, dA, dB),
          T, E, K, N, _DT[dt], dC.data_ptr(), A.data_ptr(), B.data_ptr(), sizes.data_ptr(), _ptr(dA), _ptr(dB),
          _DT[db_dtype])
    return dA, dB


@_streamed
def gemm_grouped_fp8(A, B, sa, sb, sizes, out_dtype: str = "bf16", out=None, fp32_sums: bool = False):
    """C[rows of group e] = (A sa)[rows of e] @ (B[e] sb[e])^T: A (T, K), e4m3
    or e5m2, sorted by group, with sa[ceil(K / 128)][T]; B (E, N, K), e4m3,
    with sb[e][ceil(K / 128)][ceil(N / 128)]; sizes and the rows of no group
    as in gemm_grouped, fp32_sums as in gemm_fp8.  K a multiple of 16, N of 8."""
    adt = _name(A, "A", ("e4m3", "e5m2"))
    _name(B, "B", ("e4m3",))
    if A.dim() != 2 or B.dim() != 3 or A.shape[1] != B.shape[2]:
        raise ValueError(f"shape mismatch {tuple(A.shape)} x {tuple(B.shape)}^T")
    (T, K), (E, N, _) = A.shape, B.shape
    _given(A, "A", (T, K), A.dtype)
    _given(B, "B", (E, N, K), B.dtype)
    _given(sa, "sa", (_blocks(K), T), torch.float32)
    _given(sb, "sb", (E, _blocks(K), _blocks(N)), torch.float32)
    if _groups(sizes) != E:
        raise ValueError("sizes and B disagree on the number of groups")
    _choice(out_dtype, "out_dtype", ("bf16", "f16", "f32"))
    out = _out(out, "out", (T, N), _TORCH[out_dtype], A.device)
    _call("tss_gemm_grouped_fp8", C.lib().tss_gemm_grouped_fp8, (A, B, sa, sb, sizes, out),
          T, E, K, N, _DT[adt], A.data_ptr(), B.data_ptr(), sa.data_ptr(), sb.data_ptr(), sizes.data_ptr(),
          out.data_ptr(), _out_type(out_dtype, fp32_sums))
    return out


_CLIPPED = {_TORCH[n]: _DT[n] for n in ("f16", "bf16", "f32")} if torch is not None else {}


def _refuse_list(grads, out):
    """Says what is wrong with lists of which one tensor cannot be taken."""
    if out is not None and len(out) != len(grads):
        raise ValueError(f"{len(out)} outputs for {len(grads)} gradients")
    for t, o in zip(grads, grads if out is None else out):
        if not (isinstance(t, torch.Tensor) and isinstance(o, torch.Tensor)):
            raise ValueError(f"gradients and outputs must be tensors, not {type(o if isinstance(t, torch.Tensor) else t).__name__}")
        _name(t, "a gradient", ("f16", "bf16", "f32"))
        if o.shape != t.shape or o.dtype != t.dtype or o.stride() != t.stride():
            raise ValueError(f"an output must have its gradient's shape, type and strides, {t.dtype} {tuple(t.shape)} "
                             f"{t.stride()}, not {o.dtype} {tuple(o.shape)} {o.stride()}")
    raise ValueError("gradients must lie in memory without gaps")


def _clip(grads, max_norm: float, out, norm, workspace):
    if out is not None and out is not grads:
        out = list(out)
    if not grads and norm is None:
        raise ValueError("without tensors norm must be given")
    table = C.bind().table(grads, out, _CLIPPED)
    if table is None:
        _refuse_list(grads, out)
    at, sizes, types, to, index = table
    device = grads[0].device if grads else norm.device
    norm = _out(norm, "norm", (), torch.float32, device)
    if grads and norm.get_device() != index:
        raise ValueError("every tensor must be on the same GPU")
    n = len(grads)
    need = _size("tss_clip_grad_norm_workspace_size", n, sizes)
    if need:
        workspace = _workspace(workspace, need, device)
    _run("tss_clip_grad_norm", n, at, sizes, types, float(max_norm), to, norm, workspace,
         0 if workspace is None else workspace.nbytes)
    return norm


def _list_streamed(f):
    """_streamed for calls whose first argument is a sequence of tensors."""
    @functools.wraps(f)
    def call(grads, *args, stream=None, **kwargs):
        grads = list(grads)
        if stream is None:
            return f(grads, *args, **kwargs)
        first = next(iter(grads), kwargs.get("norm"))
        return _streamed(lambda _first: f(grads, *args, **kwargs))(first, stream=stream)
    return call


@_list_streamed
def grad_norm(grads: Sequence["torch.Tensor"], norm=None, workspace=None):
    """The norm over all elements of the tensors (f16, bf16, f32, mixed), a
    float32 scalar on the GPU: squares are added in 64 bits, in a fixed order.
    norm: the scalar to write into (in none of the tensors), else allocated."""
    return _clip(grads, 0.0, None, norm, workspace)


@_list_streamed
def clip_grad_norm(grads: Sequence["torch.Tensor"], max_norm: float, out=None, norm=None, workspace=None):
    """Scales the tensors, in place or into out (a tensor for each, of its
    shape, type and strides), to a norm of at most max_norm: every element times
    min(1, max_norm / (norm + 1e-6)) in float32, rounded once.  Returns grad_norm's
    norm; nothing is read back to the host.  A NaN norm makes every element
    NaN, an infinite one multiplies by 0.  Tensors must lie in memory without
    gaps, and none may be given twice or overlap another that is written, nor
    may norm or workspace lie in one."""
    return _clip(grads, max_norm, grads if out is None else out, norm, workspace)

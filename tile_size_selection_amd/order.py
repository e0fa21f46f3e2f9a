"""Rows sorted by expert and joined again: what stands between a router's
choices and the grouped products.  Argument checks and marshalling only, as in
ops.py; the work is libtss.so's (include/tss.h documents each entry point).

A router gives each of `tokens` tokens `top` choices of an expert.  Their rows,
tokens * top in all, are sorted by expert, a token's in the order of its
choices.  A choice outside 0 .. experts - 1 is dropped: its place is behind the
routed rows, and is written as its complement (~place, a negative number).

An output given to a call may overlap none of its other tensors, apart from
what the call allows: such calls are refused."""
from __future__ import annotations

from typing import NamedTuple, Optional, Tuple

from .api import _workspace, torch
from .ops import _DT, _TORCH, _choice, _given, _name, _out, _run, _size, _streamed

_FLOATS = ("f16", "bf16", "f32")


class ExpertOrder(NamedTuple):
    """sizes (experts,): rows of each expert, what the grouped products take;
    row (tokens, top): each choice's row, the complement of its place where
    dropped; choice (tokens * top,): each row's choice (token * top + j), the
    complement of it behind the routed rows.  All int32."""
    sizes: "torch.Tensor"
    row: "torch.Tensor"
    choice: "torch.Tensor"


def _order(order, tokens: Optional[int] = None) -> Tuple[int, int]:
    """(tokens, top) of an ExpertOrder, checked."""
    shape = order.row.shape
    if len(shape) != 2 or shape[1] < 1:
        raise ValueError("order.row must be (tokens, top)")
    n, top = shape
    if tokens is not None and n != tokens:
        raise ValueError(f"the order is of {n} tokens, not of {tokens}")
    _given(order.row, "order.row", shape, torch.int32)
    _given(order.choice, "order.choice", (n * top,), torch.int32)
    return n, top


@_streamed
def sort_by_expert(expert, experts: int, sizes=None, row=None, choice=None, workspace=None) -> ExpertOrder:
    """ExpertOrder of expert (tokens, top), int32 or int64: the stable order of
    the choices by expert.  experts: 1 to 4096.  sizes, row, choice: outputs to
    write into, else allocated (row may be an int32 expert itself); workspace: a
    device tensor of at least tss_sort_by_expert_workspace_size bytes (allocated
    here when one is needed and not given)."""
    if expert.dim() != 2 or expert.shape[1] < 1 or expert.dtype not in (torch.int32, torch.int64):
        raise ValueError("expert must be (tokens, top) int32 or int64")
    tokens, top = expert.shape
    _given(expert, "expert", (tokens, top), expert.dtype)
    need = _size("tss_sort_by_expert_workspace_size", tokens, top, experts)
    sizes = _out(sizes, "sizes", (experts,), torch.int32, expert.device)
    row = _out(row, "row", (tokens, top), torch.int32, expert.device)
    choice = _out(choice, "choice", (tokens * top,), torch.int32, expert.device)
    if need:
        workspace = _workspace(workspace, need, expert.device)
    _run("tss_sort_by_expert", tokens, top, experts, expert, 64 if expert.dtype == torch.int64 else 32, sizes, row, choice,
         workspace, 0 if workspace is None else workspace.nbytes)
    return ExpertOrder(sizes, row, choice)


@_streamed
def gather_rows(x, order: ExpertOrder, scale=None, out=None, scale_out=None):
    """rows (tokens * top, d) of x (tokens, d) in the order's rows, zero behind
    the routed ones.  x of any type of the library's, d a multiple of 8.  scale
    (.., tokens) float32, such as rms_norm's or quantize_fp8's scales, goes
    along: then (rows, scale (.., tokens * top)) comes back."""
    dt = _name(x, "x", ("f16", "bf16", "f32", "e4m3", "e5m2", "i8"))
    if x.dim() != 2:
        raise ValueError("x must be (tokens, d)")
    tokens, d = x.shape
    _, top = _order(order, tokens)
    _given(x, "x", (tokens, d), x.dtype)
    out = _out(out, "out", (tokens * top, d), x.dtype, x.device)
    blocks = 0
    if scale is not None:
        if scale.dim() < 1 or scale.dim() > 2 or scale.shape[-1] != tokens:
            raise ValueError("scale must be (tokens,) or (blocks, tokens)")
        _given(scale, "scale", tuple(scale.shape), torch.float32)
        blocks = scale.shape[0] if scale.dim() == 2 else 1
        scale_out = _out(scale_out, "scale_out", (*scale.shape[:-1], tokens * top), torch.float32, x.device)
    elif scale_out is not None:
        raise ValueError("scale_out needs scale")
    _run("tss_gather_rows", tokens, top, d, _DT[dt], x, order.row, order.choice, out, scale, blocks, scale_out)
    return out if scale is None else (out, scale_out)


def _combine(rows, order: ExpertOrder, weight, out_dtype: Optional[str], out):
    dt = _name(rows, "rows", _FLOATS)
    tokens, top = _order(order)
    if rows.dim() != 2:
        raise ValueError("rows must be (tokens * top, d)")
    d = rows.shape[1]
    _given(rows, "rows", (tokens * top, d), rows.dtype)
    if weight is not None:
        _given(weight, "weight", (tokens, top), torch.float32)
    od = _choice(out_dtype or dt, "out_dtype", _FLOATS if dt == "f32" else (dt, "f32"))
    out = _out(out, "out", (tokens, d), _TORCH[od], rows.device)
    _run("tss_combine_rows", tokens, top, d, _DT[dt], rows, order.row, weight, _DT[od], out)
    return out


@_streamed
def gather_rows_backward(drows, order: ExpertOrder, out_dtype: Optional[str] = None, out=None):
    """dx (tokens, d) of gather_rows: each token's sum over its rows'
    gradients, in float32 and the order of its choices."""
    return _combine(drows, order, None, out_dtype, out)


@_streamed
def combine_rows(rows, order: ExpertOrder, weight=None, out_dtype: Optional[str] = None, out=None):
    """y (tokens, d): the sum over a token's choices j of weight[t][j] *
    rows[row[t][j]], in float32 and the order of j.  weight (tokens, top)
    float32, or None for 1; dropped choices add nothing, and neither their rows
    nor their weights are read.  rows (tokens * top, d), f16, bf16 or f32;
    out_dtype: rows' type (the default) or 'f32', any of the three for f32 rows."""
    return _combine(rows, order, weight, out_dtype, out)


@_streamed
def combine_rows_backward(dy, rows, order: ExpertOrder, weight, drows=None,
                          dweight=None) -> Tuple["torch.Tensor", "torch.Tensor"]:
    """(drows, dweight) of combine_rows: drows[row[t][j]] = weight[t][j] *
    dy[t] in dy's type (zero behind the routed rows), dweight[t][j] = <dy[t],
    rows[row[t][j]]> in float32 (zero where dropped).  rows: dy's type or f32;
    drows may be rows when the types are the same, dweight may be weight."""
    dt = _name(dy, "dy", _FLOATS)
    rt = _name(rows, "rows", (dt, "f32"))
    if dy.dim() != 2:
        raise ValueError("dy must be (tokens, d)")
    tokens, d = dy.shape
    _, top = _order(order, tokens)
    _given(dy, "dy", (tokens, d), dy.dtype)
    _given(rows, "rows", (tokens * top, d), rows.dtype)
    _given(weight, "weight", (tokens, top), torch.float32)
    drows = _out(drows, "drows", (tokens * top, d), dy.dtype, dy.device)
    dweight = _out(dweight, "dweight", (tokens, top), torch.float32, dy.device)
    _run("tss_combine_rows_backward", tokens, top, d, _DT[dt], dy, _DT[rt], rows, order.row, weight, drows, dweight)
    return drows, dweight

"""An expert layer on the library's operators: the 8-bit forward passes that
serve it, and training steps in bf16 with their gradients.

    python -m tile_size_selection_amd.expert_layer [--tokens N] [--width D] [--hidden F] [--experts E] [--top K]

The layer: h = x + residual; n = rms_norm(h) * w; every token's `top` experts
compute W2[e]^T (silu(n W1[e] gate) * (n W1[e] up)), and their results are
added with the router's weights.  The router's choice is an input here.

forward, backward and forward_fp8 take rows that route() sorted by torch's
operations; forward_sorted, backward_sorted and forward_fp8_sorted sort, gather
and join them by the library's, take a layer norm too, and give the gradient of
the router's weights.  train_step is one of the latter with its gradients
clipped; shared_int8 is an expert that every token passes, in 8-bit integers.
The command runs them on random data and prints how far they are from the same
layer in float32, and how long they take.
"""
from __future__ import annotations

import argparse
from typing import NamedTuple, Optional

from .api import torch
from .ops import (clip_grad_norm, gemm_grouped, gemm_grouped_backward, gemm_grouped_fp8, gemm_int8, layer_norm,
                  layer_norm_backward, quantize_fp8, quantize_int8, rms_norm, rms_norm_backward)
from .order import ExpertOrder, combine_rows, combine_rows_backward, gather_rows, gather_rows_backward, sort_by_expert


class Routing(NamedTuple):
    """Rows sorted by expert: row i of a grouped product is token token[i],
    which gives its result the weight weight[i]; sizes: rows per expert;
    row[t][j]: the row of token t's choice j."""
    token: "torch.Tensor"
    weight: "torch.Tensor"
    sizes: "torch.Tensor"
    row: "torch.Tensor"


def route(expert, weight, experts: int) -> Routing:
    """Routing of expert (tokens, top) integers and weight (tokens, top).  An
    expert outside 0 .. experts - 1 is a dropped choice: its row comes last, is
    in no expert's group and adds nothing."""
    flat = expert.reshape(-1)
    flat = torch.where((flat >= 0) & (flat < experts), flat, experts)
    order = torch.argsort(flat, stable=True)
    row = torch.empty_like(order).scatter_(0, order, torch.arange(order.numel(), device=order.device))
    sizes = (flat[None, :] == torch.arange(experts, device=flat.device)[:, None]).sum(1, dtype=torch.int32)
    return Routing(order // expert.shape[1], weight.reshape(-1)[order], sizes, row.view(expert.shape))


def join(rows, r: Routing):
    """Each token's sum over its choices' rows, in the order of the choices
    (without atomics: the same bits on every run), in float32."""
    return rows.float()[r.row].sum(1)


class Fp8Weights(NamedTuple):
    """W1 (experts, 2 hidden, width) and W2 (experts, width, hidden) in e4m3, scales for 128 x 128 blocks."""
    norm: "torch.Tensor"
    w1: "torch.Tensor"
    s1: "torch.Tensor"
    w2: "torch.Tensor"
    s2: "torch.Tensor"


def quantize_weights(norm, w1, w2) -> Fp8Weights:
    """Fp8Weights of bf16 W1 (experts, width, 2 hidden) and W2 (experts,
    hidden, width), the layout the training step takes."""
    def each(w):
        parts = [quantize_fp8(m.t().contiguous(), block_rows=128) for m in w]
        return torch.stack([q for q, _ in parts]), torch.stack([s for _, s in parts])
    return Fp8Weights(norm, *each(w1), *each(w2))


def forward_fp8(x, residual, w: Fp8Weights, r: Routing):
    """(layer's output, h): bf16 x and residual, 8-bit products."""
    n = rms_norm(x, w.norm, residual, out_dtype="e4m3")
    rows = n.y.view(torch.uint8)[r.token].view(n.y.dtype)
    up = gemm_grouped_fp8(rows, w.w1, n.scale[:, r.token].contiguous(), w.s1, r.sizes)
    act, scale = quantize_fp8(up, gated=True)
    y = gemm_grouped_fp8(act, w.w2, scale, w.s2, r.sizes, out_dtype="f32")
    return join(y * r.weight[:, None], r).to(x.dtype), n.h


class Saved(NamedTuple):
    h: "torch.Tensor"
    rstd: "torch.Tensor"
    rows: "torch.Tensor"
    up: "torch.Tensor"
    act: "torch.Tensor"


def forward(x, residual, norm, w1, w2, r: Routing):
    """(output, h, what backward takes) in x's type; W1 (experts, width, 2
    hidden), W2 (experts, hidden, width)."""
    n = rms_norm(x, norm, residual, rstd=True)
    rows = n.y[r.token]
    up = gemm_grouped(rows, w1, r.sizes)
    gate, lin = up.float().chunk(2, 1)
    act = (torch.nn.functional.silu(gate) * lin).to(x.dtype)
    y = gemm_grouped(act, w2, r.sizes, out_dtype="f32")
    return join(y * r.weight[:, None], r).to(x.dtype), n.h, Saved(n.h, n.rstd, rows, up, act)


def backward(dout, dh, norm, w1, w2, r: Routing, s: Saved):
    """(dx = dresidual, dnorm, dW1, dW2) from the gradients of the output and
    of h; the weights' gradients in float32."""
    dy = (dout.float()[r.token] * r.weight[:, None]).to(dout.dtype)
    dact, dw2 = gemm_grouped_backward(dy, s.act, w2, r.sizes)
    gate, lin = s.up.float().chunk(2, 1)
    sig = torch.sigmoid(gate)
    da = dact.float()
    dup = torch.cat([da * lin * sig * (1 + gate * (1 - sig)), da * gate * sig], 1).to(dout.dtype)
    drows, dw1 = gemm_grouped_backward(dup, s.rows, w1, r.sizes)
    dx, dnorm = rms_norm_backward(join(drows, r).to(dout.dtype), s.h, norm, s.rstd, dh)
    return dx, dnorm, dw1, dw2


def forward_fp8_sorted(x, residual, w: Fp8Weights, expert, weight):
    """forward_fp8 from the router's choices (tokens, top), an expert outside 0
    .. experts - 1 dropped, and their weights (tokens, top) float32."""
    order = sort_by_expert(expert, w.w1.shape[0])
    n = rms_norm(x, w.norm, residual, out_dtype="e4m3")
    rows, scale = gather_rows(n.y, order, n.scale)
    act, scale = quantize_fp8(gemm_grouped_fp8(rows, w.w1, scale, w.s1, order.sizes), gated=True)
    y = gemm_grouped_fp8(act, w.w2, scale, w.s2, order.sizes, out_dtype="f32")
    return combine_rows(y, order, weight, _name_of(x)), n.h


def _name_of(t) -> str:
    return {torch.bfloat16: "bf16", torch.float16: "f16"}[t.dtype]


class Kept(NamedTuple):
    """What backward_sorted takes from forward_sorted."""
    order: ExpertOrder
    h: "torch.Tensor"
    mean: Optional["torch.Tensor"]  # layer norm only
    rstd: "torch.Tensor"
    rows: "torch.Tensor"
    up: "torch.Tensor"
    act: "torch.Tensor"
    y: "torch.Tensor"


def forward_sorted(x, residual, norm, w1, w2, expert, weight, bias=None):
    """(output, h, Kept): forward from the router's choices (tokens, top) and
    their weights (tokens, top) float32.  With a bias the norm is a layer norm."""
    order = sort_by_expert(expert, w1.shape[0])
    if bias is None:
        n, mean = rms_norm(x, norm, residual, rstd=True), None
    else:
        n = layer_norm(x, norm, bias, residual, stats=True)
        mean = n.mean
    rows = gather_rows(n.y, order)
    up = gemm_grouped(rows, w1, order.sizes)
    gate, lin = up.float().chunk(2, 1)
    act = (torch.nn.functional.silu(gate) * lin).to(x.dtype)
    y = gemm_grouped(act, w2, order.sizes)
    return combine_rows(y, order, weight), n.h, Kept(order, n.h, mean, n.rstd, rows, up, act, y)


class Gradients(NamedTuple):
    x: "torch.Tensor"               # and of the residual
    norm: "torch.Tensor"            # the parameters' in float32
    bias: Optional["torch.Tensor"]  # layer norm only
    w1: "torch.Tensor"
    w2: "torch.Tensor"
    weight: "torch.Tensor"


def backward_sorted(dout, dh, norm, w1, w2, weight, k: Kept) -> Gradients:
    """Gradients of forward_sorted from those of its output and of h."""
    dy, dweight = combine_rows_backward(dout, k.y, k.order, weight)
    dact, dw2 = gemm_grouped_backward(dy, k.act, w2, k.order.sizes)
    gate, lin = k.up.float().chunk(2, 1)
    sig = torch.sigmoid(gate)
    da = dact.float()
    dup = torch.cat([da * lin * sig * (1 + gate * (1 - sig)), da * gate * sig], 1).to(dout.dtype)
    drows, dw1 = gemm_grouped_backward(dup, k.rows, w1, k.order.sizes)
    dn, dbias = gather_rows_backward(drows, k.order), None
    if k.mean is None:
        dx, dnorm = rms_norm_backward(dn, k.h, norm, k.rstd, dh)
    else:
        dx, dnorm, dbias = layer_norm_backward(dn, k.h, norm, k.mean, k.rstd, dh)
    return Gradients(dx, dnorm, dbias, dw1, dw2, dweight)


def train_step(x, residual, norm, w1, w2, expert, weight, dout, dh, max_norm: float, bias=None):
    """(output, Gradients, norm): a forward and a backward pass, the parameters'
    gradients (norm, bias, w1, w2) scaled to a norm of at most max_norm."""
    out, _, kept = forward_sorted(x, residual, norm, w1, w2, expert, weight, bias)
    g = backward_sorted(dout, dh, norm, w1, w2, weight, kept)
    total = clip_grad_norm([t for t in (g.norm, g.bias, g.w1, g.w2) if t is not None], max_norm)
    return out, g, total


class Int8Weights(NamedTuple):
    """A layer norm's weight and bias, W1 (2 hidden, width) and W2 (width,
    hidden) in int8 with a scale for each channel (row)."""
    norm: "torch.Tensor"
    bias: "torch.Tensor"
    w1: "torch.Tensor"
    s1: "torch.Tensor"
    w2: "torch.Tensor"
    s2: "torch.Tensor"


def quantize_shared(norm, bias, w1, w2) -> Int8Weights:
    """Int8Weights of W1 (width, 2 hidden) and W2 (hidden, width)."""
    return Int8Weights(norm, bias, *quantize_int8(w1.t().contiguous()), *quantize_int8(w2.t().contiguous()))


def shared_int8(x, residual, w: Int8Weights):
    """(output, h) of an expert that every token passes, behind a layer norm:
    8-bit integers with a scale for each token and channel."""
    n = layer_norm(x, w.norm, w.bias, residual, out_dtype="i8")
    act, scale = quantize_int8(gemm_int8(n.y, w.w1, n.scale, w.s1, _name_of(x)), gated=True)
    return gemm_int8(act, w.w2, scale, w.s2, _name_of(x)), n.h


def reference(x, residual, norm, w1, w2, expert, weight, eps: float = 1e-6, bias=None):
    """(output, h) of the layer in the inputs' type, expert by expert; with a
    bias the norm is a layer norm."""
    h = x + residual
    if bias is None:
        n = h * torch.rsqrt(h.square().mean(1, keepdim=True) + eps) * norm
    else:
        c = h - h.mean(1, keepdim=True)
        n = c * torch.rsqrt(c.square().mean(1, keepdim=True) + eps) * norm + bias
    out = torch.zeros_like(h)
    for e in range(w1.shape[0]):
        gate, lin = (n @ w1[e]).chunk(2, 1)
        y = (torch.nn.functional.silu(gate) * lin) @ w2[e]
        out = out + y * (weight * (expert == e)).sum(1, keepdim=True)
    return out, h


def _timed(f, n: int = 20) -> float:
    """Microseconds of a call among others."""
    for _ in range(3):
        f()
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(n):
        f()
    end.record()
    torch.cuda.synchronize()
    return start.elapsed_time(end) / n * 1e3


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, value in (("tokens", 2048), ("width", 1024), ("hidden", 512), ("experts", 16), ("top", 2)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args()
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    normal = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    bf16 = torch.bfloat16
    x, residual = normal(a.tokens, a.width).to(bf16), normal(a.tokens, a.width).to(bf16)
    norm = (1 + 0.2 * normal(a.width)).to(bf16)
    w1 = (normal(a.experts, a.width, 2 * a.hidden) / a.width ** 0.5).to(bf16)
    w2 = (normal(a.experts, a.hidden, a.width) / a.hidden ** 0.5).to(bf16)
    expert = torch.topk(normal(a.tokens, a.experts), a.top, 1).indices
    weight = torch.softmax(normal(a.tokens, a.top), 1)
    dout, dh = normal(a.tokens, a.width).to(bf16), normal(a.tokens, a.width).to(bf16)
    r = route(expert, weight, a.experts)
    w8 = quantize_weights(norm, w1, w2)

    leaves = [t.float().requires_grad_() for t in (x, norm, w1, w2)]
    out, h = reference(leaves[0], residual.float(), *leaves[1:], expert, weight)
    grads = torch.autograd.grad([out, h], leaves, [dout.float(), dh.float()])
    off = lambda got, want: float((got.float() - want.detach()).norm() / want.detach().norm())  # noqa: E731
    out8, _ = forward_fp8(x, residual, w8, r)
    got, _, saved = forward(x, residual, norm, w1, w2, r)
    back = backward(dout, dh, norm, w1, w2, r, saved)
    print(f"8-bit forward: {off(out8, out):.2e} of the norm from float32, "
          f"{_timed(lambda: forward_fp8(x, residual, w8, r)):.0f} us")
    print(f"bf16 forward:  {off(got, out):.2e}, {_timed(lambda: forward(x, residual, norm, w1, w2, r)):.0f} us")
    print("bf16 backward: " + ", ".join(f"{n} {off(b, w):.2e}" for n, b, w in zip(("dx", "dnorm", "dW1", "dW2"), back, grads))
          + f", {_timed(lambda: backward(dout, dh, norm, w1, w2, r, saved)):.0f} us")

    out8, _ = forward_fp8_sorted(x, residual, w8, expert, weight)
    got, _, kept = forward_sorted(x, residual, norm, w1, w2, expert, weight)
    grad = backward_sorted(dout, dh, norm, w1, w2, weight, kept)
    print(f"rows sorted, gathered and joined by the library: 8-bit forward {off(out8, out):.2e}, "
          f"{_timed(lambda: forward_fp8_sorted(x, residual, w8, expert, weight)):.0f} us; bf16 forward {off(got, out):.2e}, "
          f"{_timed(lambda: forward_sorted(x, residual, norm, w1, w2, expert, weight)):.0f} us; backward "
          + ", ".join(f"{n} {off(b, w):.2e}" for n, b, w in zip(("dx", "dnorm", "dW1", "dW2"), (grad.x, grad.norm, grad.w1, grad.w2), grads))
          + f", {_timed(lambda: backward_sorted(dout, dh, norm, w1, w2, weight, kept)):.0f} us; a step with clipping "
          f"{_timed(lambda: train_step(x, residual, norm, w1, w2, expert, weight, dout, dh, 1.0)):.0f} us")
    bias = (0.2 * normal(a.width)).to(bf16)
    one = torch.zeros(a.tokens, 1, dtype=torch.int64, device="cuda")
    shared, _ = reference(x.float(), residual.float(), norm.float(), w1[:1].float(), w2[:1].float(), one,
                          torch.ones(a.tokens, 1, device="cuda"), 1e-5, bias.float())
    w8i = quantize_shared(norm, bias, w1[0], w2[0])
    got, _ = shared_int8(x, residual, w8i)
    print(f"shared expert in 8-bit integers: {off(got, shared):.2e}, {_timed(lambda: shared_int8(x, residual, w8i)):.0f} us")


if __name__ == "__main__":
    main()

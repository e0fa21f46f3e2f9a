"""The expert layer's passes against the same layer in float64: its 8-bit
forward, its bf16 forward and the gradients of a training step."""
import pytest
import torch

from tile_size_selection_amd import expert_layer as X

pytestmark = pytest.mark.gpu

CUDA = torch.device("cuda:0")


def test_layer_and_its_gradients():
    tokens, width, hidden, experts, top = 150, 272, 144, 6, 2
    g = torch.Generator()
    g.manual_seed(3)
    normal = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    bf16 = torch.bfloat16
    x, residual, dout, dh = (normal(tokens, width).to(bf16) for _ in range(4))
    norm = (1 + 0.2 * normal(width)).to(bf16)
    w1 = (normal(experts, width, 2 * hidden) / width ** 0.5).to(bf16)
    w2 = (normal(experts, hidden, width) / hidden ** 0.5).to(bf16)
    expert = torch.topk(normal(tokens, experts - 1), top, 1).indices  # the last expert gets no rows
    weight = torch.softmax(normal(tokens, top), 1).float()
    leaves = [t.double().requires_grad_() for t in (x, norm, w1, w2)]
    out, h = X.reference(leaves[0], residual.double(), *leaves[1:], expert, weight.double())
    grads = torch.autograd.grad([out, h], leaves, [dout.double(), dh.double()])

    dev = [t.to(CUDA) for t in (x, residual, norm, w1, w2)]
    r = X.route(expert.to(CUDA), weight.to(CUDA), experts)
    assert r.sizes.tolist() == [int((expert == e).sum()) for e in range(experts)]
    off = lambda got, want: float((got.double().cpu() - want.detach()).norm() / want.detach().norm())  # noqa: E731
    got, got_h, saved = X.forward(*dev, r)
    back = X.backward(dout.to(CUDA), dh.to(CUDA), *dev[2:], r, saved)
    # a chain of at most 8 roundings to bf16 (2^-8 each, and of random signs over the norm)
    for what, a, b in zip(("out", "h", "dx", "dnorm", "dW1", "dW2"), (got, got_h, *back), (out, h, *grads)):
        assert off(a, b) <= 8 * 2.0 ** -8, what
    assert (back[2][-1] == 0).all() and (back[3][-1] == 0).all()
    # 8 bits: four roundings to e4m3 (2^-4 each)
    out8, h8 = X.forward_fp8(dev[0], dev[1], X.quantize_weights(*dev[2:]), r)
    assert off(out8, out) <= 4 * 2.0 ** -4 and torch.equal(h8, got_h)

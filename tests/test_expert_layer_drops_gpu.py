"""The expert layer with dropped choices, and the same bits on every run."""
import pytest
import torch

from tile_size_selection_amd import expert_layer as X

pytestmark = pytest.mark.gpu

CUDA = torch.device("cuda:0")


def test_dropped_choices_add_nothing_and_runs_repeat():
    tokens, width, hidden, experts, top = 90, 272, 144, 6, 4
    g = torch.Generator()
    g.manual_seed(5)
    normal = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    bf16 = torch.bfloat16
    x, residual, dout, dh = (normal(tokens, width).to(bf16) for _ in range(4))
    norm = (1 + 0.2 * normal(width)).to(bf16)
    w1 = (normal(experts, width, 2 * hidden) / width ** 0.5).to(bf16)
    w2 = (normal(experts, hidden, width) / hidden ** 0.5).to(bf16)
    expert = torch.topk(normal(tokens, experts), top, 1).indices
    expert[torch.rand(tokens, top, generator=g) < 0.2] = -1
    weight = torch.softmax(normal(tokens, top), 1).float()
    leaves = [t.double().requires_grad_() for t in (x, norm, w1, w2)]
    out, h = X.reference(leaves[0], residual.double(), *leaves[1:], expert, weight.double())
    grads = torch.autograd.grad([out, h], leaves, [dout.double(), dh.double()])
    dev = [t.to(CUDA) for t in (x, residual, norm, w1, w2)]
    r, w8 = X.route(expert.to(CUDA), weight.to(CUDA), experts), X.quantize_weights(*dev[2:])

    def run():
        got, got_h, saved = X.forward(*dev, r)
        return [got, got_h, *X.backward(dout.to(CUDA), dh.to(CUDA), *dev[2:], r, saved), X.forward_fp8(dev[0], dev[1], w8, r)[0]]

    first = run()
    # a chain of at most 8 roundings to bf16 (2^-8 each, and of random signs over the norm); in 8 bits four of 2^-4
    for got, want, bound in zip(first, (out, h, *grads, out), [8 * 2.0 ** -8] * 6 + [4 * 2.0 ** -4]):
        assert float((got.double().cpu() - want.detach()).norm() / want.detach().norm()) <= bound
    for _ in range(10):
        assert all(torch.equal(a, b) for a, b in zip(run(), first))

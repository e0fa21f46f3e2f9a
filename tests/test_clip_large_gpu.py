"""Clipping of 2^28 bytes and more, whose outputs pass the caches by: every
element type with a ragged end, in place and not, off 16-byte borders, and over
several tables of tensors.  Bounds as in the smaller cases' tests."""
import pytest
import torch

import tile_size_selection_amd as tss
import ops_util as U
from test_clip_gpu import CUDA, check, true_norm

pytestmark = pytest.mark.gpu


def tensors(sizes, kinds, seed):
    g = torch.Generator(device=CUDA)
    g.manual_seed(seed)
    return [(0.01 * torch.randn(n, generator=g, device=CUDA)).to(U.TYPES[kinds[i % len(kinds)]]) for i, n in enumerate(sizes)]


CASES = {
    "bf16": ([134217731, 5], ["bf16"]), "f16": ([134217731, 4097], ["f16"]), "f32": ([67108867, 2049], ["f32"]),
    "mixed": ([50000003, 50000001, 50000007, 1, 8191], ["bf16", "f32", "f16"]),
    "two tables": ([700001 + i for i in range(201)], ["bf16", "f32", "f16"]),
    "a few large among many small": ([33 + i for i in range(140)] + [90000001, 9, 10, 45000001], ["f32", "bf16"])}


@pytest.mark.parametrize("ratio", [0.5, 4.0])
@pytest.mark.parametrize("sizes,kinds", CASES.values(), ids=CASES.keys())
def test_clip(sizes, kinds, ratio):
    ts = tensors(sizes, kinds, 1)
    assert sum(t.nbytes for t in ts) >= 2 ** 28
    max_norm = ratio * true_norm(ts)
    before = [t.clone() for t in ts]
    outs = [torch.full_like(t, 7.0) for t in ts]
    norm = tss.clip_grad_norm(ts, max_norm, out=outs)
    check(outs, before, max_norm, norm)
    assert all(torch.equal(t, b) for t, b in zip(ts, before)) and torch.equal(tss.grad_norm(ts), norm)
    assert torch.equal(tss.clip_grad_norm(ts, max_norm), norm)
    assert all(torch.equal(t, o) for t, o in zip(ts, outs))  # in place: the same bits


def test_off_16_byte_borders_and_nothing_beside():
    buf = torch.full((2, 67108900), 7.0, device=CUDA)
    values = tensors([67108867], ["f32"], 2)[0]
    ts, outs = [buf[0, 1:67108868]], [buf[1, 3:67108870]]
    ts[0].copy_(values)
    norm = tss.clip_grad_norm(ts, 1.0, out=outs)
    check(outs, [values], 1.0, norm)
    tss.clip_grad_norm(ts, 1.0)
    assert torch.equal(ts[0], outs[0])
    assert (buf[0, :1] == 7).all() and (buf[0, 67108868:] == 7).all() and (buf[1, :3] == 7).all() and (buf[1, 67108870:] == 7).all()


def test_replays_follow_their_inputs():
    sizes, kinds = CASES["two tables"]
    ts = tensors(sizes, kinds, 3)
    outs = [torch.empty_like(t) for t in ts]
    tss.clip_grad_norm(ts, 0.5, out=outs)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = tss.clip_grad_norm(ts, 0.5, out=outs)
    for seed in (4, 5, 6):
        for t, new in zip(ts, tensors(sizes, kinds, seed)):
            t.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        check(outs, ts, 0.5, norm)
        assert torch.equal(tss.grad_norm(ts), norm)

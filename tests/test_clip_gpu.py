"""The norm over many tensors and clipping, against the definition in 64 bits.

Bounds: the norm's squares are added in 64 bits, so it is off by its rounding
to fp32; the factor is off by its own rounding, the product by one more, and
the output by its type's: half a step + 2^-23."""
import math

import pytest
import torch

import tile_size_selection_amd as tss
import ops_util as U

pytestmark = pytest.mark.gpu

CUDA = torch.device("cuda:0")


def tensors(sizes, seed, kinds=("bf16", "f32", "f16"), spread=0.01):
    g = U.gen(seed)
    return [(spread * U.normal(g, n)).to(U.TYPES[kinds[i % len(kinds)]]).to(CUDA) for i, n in enumerate(sizes)]


def true_norm(ts):
    return math.sqrt(sum(float(t.double().square().sum()) for t in ts))


def check(got, ts, max_norm, norm):
    want = true_norm(ts)
    assert norm.dtype == torch.float32 and norm.shape == ()
    assert abs(float(norm) - want) <= want * 2.0 ** -23
    factor = min(1.0, max_norm / (want + 1e-6))
    for o, t in zip(got, ts):
        half, low = U.half_step({v: k for k, v in U.TYPES.items()}[t.dtype])
        v = t.double() * factor
        assert ((o.double() - v).abs() <= v.abs() * (half + 2.0 ** -23) + low + 2.0 ** -149).all()


SIZES = {
    "one": [1], "small": [5, 1, 300, 4096, 17], "empty ones": [0, 7, 0, 0, 4097, 0], "one workgroup": [2048 * 3 + 1, 5, 2048 * 12, 700, 2047], "a unit more": [2048 * 20, 1], "ragged": [4095, 4096, 4097, 8193, 123457],
    "pieces": [5000003, 1, 2 ** 20], "many": [37 + i for i in range(400)], "a table": [64] * 128, "over a table": [64] * 129,
    "large": [70000001, 33],
    "a small table": [3000] * 5 + [0, 0] + [3001] * 11 + [0], "over it": [3000] * 17}


@pytest.mark.parametrize("ratio", [0.25, 4.0])
@pytest.mark.parametrize("sizes", SIZES.values(), ids=SIZES.keys())
def test_clip(sizes, ratio):
    ts = tensors(sizes, 1)
    max_norm = ratio * true_norm(ts)
    before = [t.clone() for t in ts]
    outs = [torch.full_like(t, 7.0) for t in ts]
    norm = tss.clip_grad_norm(ts, max_norm, out=outs)
    check(outs, before, max_norm, norm)
    assert all(torch.equal(t, b) for t, b in zip(ts, before))
    if ratio > 1:
        assert all(torch.equal(o, b) for o, b in zip(outs, before))
    assert torch.equal(tss.grad_norm(ts), norm)
    given = torch.zeros((), device=CUDA)
    assert tss.clip_grad_norm(iter(ts), max_norm, norm=given) is given and torch.equal(given, norm)
    assert all(torch.equal(t, o) for t, o in zip(ts, outs))  # in place: the same bits


def test_elements_at_any_address():
    buf = torch.randn(3, 70001, generator=U.gen(2)).to(CUDA)
    half = buf.to(torch.bfloat16)
    for i in range(1, 8):
        ts = [buf[0, i:i + 50000], half[1, i:i + 69990], half[2, 2 * i:2 * i + 3], buf[2, i:i]]
        before = [t.clone() for t in ts]
        edges = (buf[0, i - 1].clone(), buf[0, i + 50000].clone(), half[1, i - 1].clone(), half[1, i + 69990].clone())
        norm = tss.clip_grad_norm(ts, 1.0)
        check(ts, before, 1.0, norm)
        assert edges == (buf[0, i - 1], buf[0, i + 50000], half[1, i - 1], half[1, i + 69990])
    out = torch.zeros(50001, device=CUDA)  # from a 16-byte border to off one
    t = torch.randn(50000, generator=U.gen(3)).to(CUDA)
    check([out[1:]], [t], 1.0, tss.clip_grad_norm([t], 1.0, out=[out[1:]]))


def test_orders_in_memory():
    x = torch.randn(4, 6, 5, 7, generator=U.gen(4)).to(CUDA)
    ts = [x.to(memory_format=torch.channels_last), x.permute(3, 1, 0, 2), x[0, 0].t()]
    ts = [t.clone(memory_format=torch.preserve_format) for t in ts]
    before = [t.clone() for t in ts]
    check(ts, before, 2.0, tss.clip_grad_norm(ts, 2.0))


def test_squares_neither_overflow_nor_vanish():
    for scale in (1e30, 1e-30):
        ts = [(scale * torch.randn(10000, generator=U.gen(5)).double()).float().to(CUDA)]
        norm = tss.grad_norm(ts)
        assert abs(float(norm) / true_norm(ts) - 1) <= 2.0 ** -23
    ts = [torch.full((1000,), 3e30, device=CUDA)]
    before = [t.clone() for t in ts]
    check(ts, before, 1.0, tss.clip_grad_norm(ts, 1.0))


def test_norms_that_are_not_finite_or_zero():
    z = torch.zeros(100, device=CUDA)
    assert float(tss.clip_grad_norm([z], 1.0)) == 0 and (z == 0).all()
    assert float(tss.clip_grad_norm([z], 0.0)) == 0 and (z == 0).all()
    a, b = torch.ones(100, device=CUDA), torch.ones(9000, dtype=torch.bfloat16, device=CUDA)
    assert float(tss.clip_grad_norm([a, b], 0.0)) == pytest.approx(math.sqrt(9100)) and (a == 0).all() and (b == 0).all()
    a, b = torch.ones(100, device=CUDA), torch.ones(9000, dtype=torch.bfloat16, device=CUDA)
    assert float(tss.clip_grad_norm([a, b], float("inf"))) == pytest.approx(math.sqrt(9100)) and (a == 1).all()
    a[7] = float("inf")
    assert tss.clip_grad_norm([a, b], 1.0).isinf() and a[7].isnan() and (a[:7] == 0).all() and (b == 0).all()
    a, b = torch.ones(100, device=CUDA), torch.ones(9000, dtype=torch.bfloat16, device=CUDA)
    b[8999] = float("nan")
    assert tss.clip_grad_norm([a, b], 1.0).isnan() and a.isnan().all() and b.isnan().all()


def test_no_tensors():
    norm = torch.full((), 3.0, device=CUDA)
    assert tss.clip_grad_norm([], 1.0, norm=norm) == 0 and tss.grad_norm([], norm=norm) == 0


def test_tensors_given_twice_are_refused():
    t = torch.ones(100, device=CUDA)
    for ts in ([t, t], [t[:60], t[50:]]):
        with pytest.raises(tss.TssError):
            tss.clip_grad_norm(ts, 1.0)
    assert (t == 1).all()
    assert float(tss.grad_norm([t, t])) == pytest.approx(math.sqrt(200))  # a norm reads only
    tss.clip_grad_norm([t[:50], t[50:]], 5.0)
    assert t.allclose(torch.full_like(t, 0.5), rtol=1e-5)


def test_streams_and_a_captured_run():
    ts = tensors([100000, 33, 5000, 70], 6)
    outs = [torch.empty_like(t) for t in ts]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    norm = tss.clip_grad_norm(ts, 0.5, out=outs, stream=stream)
    torch.cuda.current_stream().wait_stream(stream)
    check(outs, ts, 0.5, norm)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = tss.clip_grad_norm(ts, 0.5, out=outs)
    for seed in range(4):
        for t, new in zip(ts, tensors([100000, 33, 5000, 70], 70 + seed)):
            t.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        check(outs, ts, 0.5, held)
        assert torch.equal(tss.grad_norm(ts), held)

"""Root-mean-square norm, its gradients and the 8-bit quantisation against
their definitions in 64 bits.

Bounds: a row's mean of squares is a sum of non-negative fp32 terms over a
fixed tree of at most 8 * 4 + 6 + 16 additions, each off by 2^-24 of the sum,
so y is known to 64 * 2^-24 = 2^-18 of itself before its own rounding; the
gradients to that share of the sum of the magnitudes of their terms."""
import pytest
import torch

import tile_size_selection_amd as tss
import ops_util as U

pytestmark = pytest.mark.gpu

CUDA = torch.device("cuda:0")
REL = 2.0 ** -18
# one row and many; widths of one chunk, one short block, whole blocks, ragged blocks, several chunks a thread
SHAPES = [(1, 8), (1, 4096), (3, 136), (5, 512), (2, 4104), (7, 8200), (3, 16384), (2, 32768), (1030, 264), (1029, 2048),
          (1025, 2056), (1024, 4096)]


def rows_of(shape, dtype, seed, spread=0.7):
    g = U.gen(seed)
    return (U.normal(g, *shape) * torch.exp(spread * U.normal(g, shape[1]))).to(U.TYPES[dtype])


def close(got, want, rel, absolute, what):
    got = got.double().cpu()
    bad = ~((got - want).abs() <= want.abs() * rel + absolute)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {bad.nonzero()[:4].tolist()}"


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("shape", SHAPES)
def test_norm(shape, dtype, residual):
    x = rows_of(shape, dtype, 1)
    r = rows_of(shape, dtype, 2) if residual else None
    w = (1 + 0.2 * U.normal(U.gen(3), shape[1])).to(U.TYPES[dtype])
    y, h, rstd = U.norm_forward(x, r, w, 1e-6)
    dev = lambda t: None if t is None else t.to(CUDA)  # noqa: E731
    half, low = U.half_step(dtype)
    got = tss.rms_norm(dev(x), dev(w), dev(r), rstd=True)
    close(got.y, y, half + REL, low, "y")
    close(got.rstd, rstd, REL, 0, "rstd")
    if residual:
        close(got.h, h, half + 2.0 ** -23, low, "h")
    else:
        assert got.h is None
    assert got.scale is None
    q = tss.rms_norm(dev(x), dev(w), dev(r), out_dtype="e4m3")
    U.check_quantised(q.y, q.scale, y, "e4m3", 1, REL)
    if residual:
        assert torch.equal(q.h, got.h)


def test_norm_in_place_and_on_a_stream():
    x, r = rows_of((37, 1032), "bf16", 4).to(CUDA), rows_of((37, 1032), "bf16", 5).to(CUDA)
    w = torch.ones(1032, dtype=torch.bfloat16, device=CUDA)
    want = tss.rms_norm(x, w, r)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = tss.rms_norm(x, w, r, out=x, residual_out=r, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert got.y is x and got.h is r
    assert torch.equal(x, want.y) and torch.equal(r, want.h)


def test_norm_of_no_rows_zero_rows_and_nan():
    w = torch.ones(136, dtype=torch.float16, device=CUDA)
    none = tss.rms_norm(torch.empty(0, 136, dtype=torch.float16, device=CUDA), w, out_dtype="e4m3")
    assert none.y.shape == (0, 136) and none.scale.shape == (2, 0)
    x = torch.zeros(3, 136, dtype=torch.float16)
    x[1] = 2.0
    x[2, 130] = float("nan")
    got = tss.rms_norm(x.to(CUDA), w, out_dtype="e4m3")
    y = got.y.float().cpu() * U.spread(got.scale.cpu(), 3, 136, 1)
    assert (y[0] == 0).all() and torch.allclose(y[1], torch.ones(136), rtol=2.0 ** -4)
    assert y[2].isnan().all() and got.scale[:, 2].isnan().all()


@pytest.mark.parametrize("with_dh", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("shape", SHAPES)
def test_norm_backward(shape, dtype, with_dh):
    h, dy = rows_of(shape, dtype, 6), rows_of(shape, dtype, 7)
    dh = rows_of(shape, dtype, 8) if with_dh else None
    w = (1 + 0.2 * U.normal(U.gen(9), shape[1])).to(U.TYPES[dtype])
    rstd = U.norm_forward(h, None, w, 1e-6)[2].float()
    dx, dw = U.norm_backward(dy, h, w, rstd, dh)
    dev = lambda t: None if t is None else t.to(CUDA)  # noqa: E731
    got_dx, got_dw = tss.rms_norm_backward(dev(dy), dev(h), dev(w), dev(rstd), dev(dh))
    half, low = U.half_step(dtype)
    xhat, g = (h.double() * rstd.double()[:, None]).abs(), (dy.double() * w.double()).abs()
    terms = rstd.double()[:, None] * (g + xhat * (g * xhat).mean(1, keepdim=True))
    if with_dh:
        terms += dh.double().abs()
    close(got_dx, dx, half, REL * terms + low, "dx")
    # a column's sum: rows / 1024 terms, then 32 + 32 partial sums, on terms known to 2^-22
    close(got_dw, dw, 0, (72 + shape[0] / 1024) * 2.0 ** -24 * (dy.double().abs() * xhat).sum(0) + 1e-40, "dweight")
    again = tss.rms_norm_backward(dev(dy), dev(h), dev(w), dev(rstd), dev(dh))
    assert torch.equal(again[0], got_dx) and torch.equal(again[1], got_dw)


def test_norm_backward_writes_over_its_gradient_and_takes_no_rows():
    h, dy, dh = (rows_of((9, 520), "bf16", s).to(CUDA) for s in (10, 11, 12))
    w = torch.ones(520, dtype=torch.bfloat16, device=CUDA)
    rstd = torch.rand(9, device=CUDA) + 0.5
    want = tss.rms_norm_backward(dy, h, w, rstd, dh)
    for out in (dy, dh):
        keep = out.clone()
        got = tss.rms_norm_backward(dy, h, w, rstd, dh, dx=out)
        assert got[0] is out and torch.equal(out, want[0]) and torch.equal(got[1], want[1])
        out.copy_(keep)
    e = torch.empty(0, 520, dtype=torch.bfloat16, device=CUDA)
    dx, dw = tss.rms_norm_backward(e, e, w, torch.empty(0, device=CUDA), dweight=torch.full((520,), 7.0, device=CUDA))
    assert dx.shape == (0, 520) and (dw == 0).all()


def test_norm_gradient_is_the_slope():
    # the loss sum(dy y) + sum(dh h) along a direction, by central differences of the definition in 64 bits
    x, dy, dh, v = (rows_of((6, 264), "f32", s) for s in (13, 14, 15, 16))
    w = (1 + 0.2 * U.normal(U.gen(17), 264)).float()
    y, h, rstd = U.norm_forward(x, None, w, 1e-6)

    def loss(t):
        a = U.norm_forward(x.double() + t * v.double(), None, w, 1e-6)
        return (a[0] * dy.double()).sum() + (a[1] * dh.double()).sum()

    slope = (loss(1e-5) - loss(-1e-5)) / 2e-5
    dx, _ = tss.rms_norm_backward(dy.to(CUDA), x.to(CUDA), w.to(CUDA), rstd.float().to(CUDA), dh.to(CUDA))
    got = (dx.double().cpu() * v.double()).sum()
    # differences of step 1e-5: off by its square and by 2^-52 / 1e-5 of the loss; dx by 2^-18 of its terms
    size = (dy.double().abs() * y.abs()).sum() + (dh.double() * h).abs().sum()
    assert abs(got - slope) <= (2.0 ** -16) * ((dx.double().cpu() * v.double()).abs().sum() + size)


@pytest.mark.parametrize("fp8", ["e4m3", "e5m2"])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("shape", [(1, 8), (1, 2048), (17, 136), (129, 520), (300, 1032), (256, 128)])
def test_quantize(shape, block_rows, dtype, fp8):
    x = rows_of(shape, dtype, 20)
    q, s = tss.quantize_fp8(x.to(CUDA), fp8, block_rows=block_rows)
    assert q.dtype == U.TYPES[fp8]
    U.check_quantised(q, s, x.double(), fp8, block_rows, 0.0)


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("shape", [(1, 8), (33, 136), (130, 1032)])
def test_quantize_gated(shape, dtype, block_rows):
    rows, d = shape
    g = U.gen(21)
    x = (3 * U.normal(g, rows, 2 * d)).clamp(-12, 12).to(U.TYPES[dtype])
    gate, up = x[:, :d].double(), x[:, d:].double()
    q, s = tss.quantize_fp8(x.to(CUDA), "e4m3", gated=True, block_rows=block_rows)
    # exp of |gate| <= 12 is known to 12 * 1.45 * 2^-23 + 2^-23, the rest to a few 2^-24
    U.check_quantised(q, s, gate * torch.sigmoid(gate) * up, "e4m3", block_rows, 2.0 ** -18)


@pytest.mark.parametrize("fp8", ["e4m3", "e5m2"])
def test_quantize_gated_rounds_as_in_64_bits(fp8):
    # of 4 million values some 30 lie so near a rounding border that fp32 leaves their side open; the result is the
    # definition's for all whose quotient is normal and not within double rounding (2^-24) of a border
    g = U.gen(23)
    x = (2 * U.normal(g, 1024, 2 * 4096)).to(torch.bfloat16)
    gate, up = x[:, :4096].double(), x[:, 4096:].double()
    v = gate * torch.sigmoid(gate) * up
    scale = U.block_amax(v, 1).clamp(min=1e-30) / U.LARGEST[fp8]
    t = v / U.spread(scale, 1024, 4096, 1)
    q, _ = tss.quantize_fp8(x.to(CUDA), fp8, gated=True)
    lowest = {"e4m3": 2.0 ** -6, "e5m2": 2.0 ** -14}[fp8]
    want, low, high = (t.mul(1 + e).float().to(U.TYPES[fp8]).float() for e in (0, -2.0 ** -23, 2.0 ** -23))
    sure = (t.abs() >= lowest) & (low == high)
    assert sure.double().mean() > 0.9
    assert torch.equal(q.float().cpu()[sure], want[sure])


def test_quantize_gated_of_far_gates():
    gate = torch.tensor([[-200.0, -100.0, -88.5, -30.0, 30.0, 100.0, 3e38, 0.0], [float("inf"), 1, 1, 1, 1, 1, 1, 1],
                         [float("-inf"), 1, 1, 1, 1, 1, 1, 1]])
    up = torch.full((3, 8), 1.0)
    up[0, 6] = 1e-36
    v = gate[0].double() * torch.sigmoid(gate[0].double()) * up[0].double()
    q, s = tss.quantize_fp8(torch.cat([gate, up], 1).to(CUDA), gated=True)
    U.check_quantised(q[:1], s[:, :1], v[None], "e4m3", 1, 2.0 ** -18)
    q = q.float().cpu()
    assert s[0, 1].isinf() and q[1, 0].isnan() and (q[1, 1:] == 0).all()
    assert s[0, 2].isnan() and q[2].isnan().all()


def test_quantize_zeros_infinities_and_nan():
    x = torch.ones(4, 256)
    x[0, :128] = 0
    x[1, 3] = float("inf")
    x[2, 200] = float("nan")
    x[3, 128:] = 1e-37
    q, s = tss.quantize_fp8(x.to(CUDA))
    q, s = q.float().cpu(), s.cpu()
    assert (q[0, :128] == 0).all() and s[0, 0] == torch.tensor(1e-30) / 448
    assert s[0, 1].isinf() and q[1, 3].isnan() and (q[1, 4:128] == 0).all()
    assert s[1, 2].isnan() and q[2, 128:].isnan().all() and (q[2, :128] == 448).all()
    assert (q[3, 128:] == 0).all() and (q[3, :128] == 448).all()
    e, t = tss.quantize_fp8(torch.empty(0, 256, device=CUDA), block_rows=128)
    assert e.shape == (0, 256) and t.shape == (2, 0)


@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_keeps_to_its_output(block_rows):
    x = rows_of((131, 392), "bf16", 22).to(CUDA)
    q = torch.full((140, 392), 1.0, device=CUDA).to(torch.float8_e4m3fn)
    s = torch.full((8, 131 if block_rows == 1 else 2), -1.0, device=CUDA)
    tss.quantize_fp8(x, block_rows=block_rows, out=q[:131], scale=s[:4])
    assert (q[131:].float() == 1).all() and (s[4:] == -1).all() and (s[:4] > 0).all()

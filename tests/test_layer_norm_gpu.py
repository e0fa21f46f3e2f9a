"""Layer norm, its gradients and its 8-bit integer output against their
definitions in 64 bits.

Bounds, in 2^-24 of the sum of the terms' magnitudes: a row's sum is a fixed
tree of at most 8 * 4 + 6 + 16 additions, so each of the sums is known to 2^-18
of that.  The first mean's error is taken out by the second sum (to 2^-18 of
itself), so h - mean is off by a rounding of h, of the mean and of the
difference: with R = the row's largest |h|, y is known to |y| 2^-18 + 4 * 2^-24 R
rstd |weight| + 2^-23 |bias| before its own rounding."""
import pytest
import torch

import tile_size_selection_amd as tss
import ops_util as U

pytestmark = pytest.mark.gpu

CUDA = torch.device("cuda:0")
REL = 2.0 ** -18
# one row and many; each number of lanes a row takes, ragged and whole; several waves; several chunks a thread
SHAPES = [(1, 8), (1, 4096), (37, 64), (33, 72), (70, 128), (19, 136), (9, 256), (5, 512), (3, 520), (2, 4104), (7, 8200),
          (3, 16384), (2, 32768), (1030, 264), (1029, 2048), (1025, 2056), (1024, 4096), (1026, 24)]
EPS = 1e-5


def rows_of(shape, dtype, seed, mean=0.5):
    g = U.gen(seed)
    return ((U.normal(g, *shape) + mean * U.normal(g, shape[1])) * torch.exp(0.7 * U.normal(g, shape[1]))).to(U.TYPES[dtype])


def definition(x, residual, weight, bias, eps=EPS):
    """(y, h, mean, rstd) in float64."""
    h = x.double() + (residual.double() if residual is not None else 0)
    mean = h.mean(1)
    c = h - mean[:, None]
    rstd = 1 / torch.sqrt(c.square().mean(1) + eps)
    return c * rstd[:, None] * weight.double() + (bias.double() if bias is not None else 0), h, mean, rstd


def inner(y, h, rstd, weight, bias):
    """The bound above, before y's own rounding."""
    b = bias.double().abs() if bias is not None else 0
    return y.abs() * REL + 4 * 2.0 ** -24 * h.abs().amax(1, keepdim=True) * rstd[:, None] * weight.double().abs() + 2.0 ** -23 * b


def check(got, want, bound, what):
    bad = ~((got.double().cpu() - want).abs() <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {bad.nonzero()[:4].tolist()}"


def params(d, dtype, seed=3):
    g = U.gen(seed)
    return (1 + 0.2 * U.normal(g, d)).to(U.TYPES[dtype]), (0.2 * U.normal(g, d)).to(U.TYPES[dtype])


def dev(t):
    return None if t is None else t.to(CUDA)


@pytest.mark.parametrize("form", ["plain", "residual", "no bias"])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("shape", SHAPES)
def test_norm(shape, dtype, form):
    x = rows_of(shape, dtype, 1)
    r = rows_of(shape, dtype, 2) if form == "residual" else None
    w, b = params(shape[1], dtype)
    b = None if form == "no bias" else b
    y, h, mean, rstd = definition(x, r, w, b)
    half, low = U.half_step(dtype)
    got = tss.layer_norm(dev(x), dev(w), dev(b), dev(r), eps=EPS, stats=True)
    known = inner(y, h, rstd, w, b)
    check(got.y, y, known + (y.abs() + known) * half + low, "y")
    check(got.mean, mean, 2 * 2.0 ** -24 * h.abs().amax(1) + REL * REL * h.abs().mean(1), "mean")
    check(got.rstd, rstd, rstd * REL * 2, "rstd")
    if r is not None:
        check(got.h, h, h.abs() * (half + 2.0 ** -23) + low, "h")
    else:
        assert got.h is None
    assert got.scale is None
    plain = tss.layer_norm(dev(x), dev(w), dev(b), dev(r), eps=EPS)
    assert torch.equal(plain.y, got.y) and plain.mean is None and plain.rstd is None


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("shape", SHAPES)
def test_norm_to_8_bit_integers(shape, dtype):
    x, r = rows_of(shape, dtype, 1), rows_of(shape, dtype, 2)
    w, b = params(shape[1], dtype)
    y, h, _, rstd = definition(x, r, w, b)
    got = tss.layer_norm(dev(x), dev(w), dev(b), dev(r), eps=EPS, out_dtype="i8")
    known = inner(y, h, rstd, w, b)
    scale = y.abs().amax(1) / 127
    check(got.scale, scale, known.amax(1) / 127 + scale * 2.0 ** -23, "scale")
    assert got.y.dtype == torch.int8 and int(got.y.min()) >= -127
    # half a step, what y is known to, and the quotient's rounding
    s = got.scale.double().cpu()[:, None]
    check(got.y.double().cpu() * s, y, s * 0.5 * (1 + 2.0 ** -15) + known + y.abs() * 2.0 ** -23, "values")
    assert (got.y.abs().amax(1) == 127).all()


# rows of several turns of a launch: one wave a row, two, five, nine, and four chunks a thread
TURNS = [(9000, 520), (9001, 1032), (5003, 4104), (4001, 8200), (1103, 16392), (40000, 128)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", TURNS)
def test_rows_taken_in_turn(shape, dtype):
    g = torch.Generator(device=CUDA)
    g.manual_seed(21)
    x, r = ((torch.randn(*shape, generator=g, device=CUDA) + 0.5).to(U.TYPES[dtype]) for _ in range(2))
    w, b = (dev(t) for t in params(shape[1], dtype))
    half, low = U.half_step(dtype)
    for residual in (None, r):
        y, h, mean, rstd = definition(x, residual, w, b)
        known = inner(y, h, rstd, w, b)
        got = tss.layer_norm(x, w, b, residual, eps=EPS, stats=True)
        assert ((got.y.double() - y).abs() <= known + (y.abs() + known) * half + low).all()
        assert ((got.rstd.double() - rstd).abs() <= rstd * REL * 2).all()
        if residual is not None:
            assert ((got.h.double() - h).abs() <= h.abs() * (half + 2.0 ** -23) + low).all()
        q = tss.layer_norm(x, w, b, residual, eps=EPS, out_dtype="i8")
        s = q.scale.double()[:, None]
        assert ((q.y.double() * s - y).abs() <= s * 0.5 * (1 + 2.0 ** -15) + known + y.abs() * 2.0 ** -23).all()
        over = x.clone()
        assert torch.equal(tss.layer_norm(over, w, b, residual, eps=EPS, out=over).y, got.y)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_mean_far_from_zero_costs_no_digits(dtype):
    """Rows of mean 1000 and spread 1 (fp32: 2^-10): what is left is what the elements themselves hold."""
    g = U.gen(4)
    x = (1000 + U.normal(g, 50, 4096) * (1 if dtype == "bf16" else 2.0 ** -10)).to(U.TYPES[dtype])
    x[:, 7] += 16  # bf16 rows are not all alike
    w, b = params(4096, dtype)
    y, h, _, rstd = definition(x, None, w, b)
    got = tss.layer_norm(dev(x), dev(w), dev(b), eps=EPS)
    half, low = U.half_step(dtype)
    known = inner(y, h, rstd, w, b)
    check(got.y, y, known + (y.abs() + known) * half + low, "y")


def test_rows_that_are_constant_or_not_finite_stay_by_themselves():
    x = rows_of((12, 1032), "f32", 5)
    x[1] = 3.0
    x[2] = 0.0
    x[3, 100] = float("nan")
    x[4, 5] = float("inf")
    x[5, 1031] = -float("inf")
    w, b = params(1032, "f32")
    y, h, _, rstd = definition(x, None, w, b)
    for out in (None, "i8"):
        got = tss.layer_norm(dev(x), dev(w), dev(b), eps=EPS, out_dtype=out, stats=True)
        value = got.y.double() if out is None else got.y.double() * got.scale.double()[:, None]
        assert value[3:6].isnan().all()
        rest = [0, 1, 2, 6, 7, 8, 9, 10, 11]
        known = inner(y, h, rstd, w, b)[rest]
        step = 0 if out is None else 0.5 * got.scale.double().cpu()[rest][:, None] * (1 + 2.0 ** -15)
        check(value[rest], y[rest], known + y[rest].abs() * 2.0 ** -23 + step, str(out))
        assert got.rstd[3:6].isnan().all() and got.rstd[1] == got.rstd[2]


def test_outputs_over_inputs_and_beside_others():
    x, r = rows_of((300, 264), "bf16", 6), rows_of((300, 264), "bf16", 7)
    w, b = params(264, "bf16")
    want = tss.layer_norm(dev(x), dev(w), dev(b), dev(r), stats=True)
    dx, dr = dev(x), dev(r)
    got = tss.layer_norm(dx, dev(w), dev(b), dr, out=dx, residual_out=dr)
    assert got.y.data_ptr() == dx.data_ptr() and torch.equal(dx, want.y) and torch.equal(dr, want.h)
    buf = torch.full((302, 264), 7.0, dtype=torch.bfloat16, device=CUDA)
    stats = torch.full((2, 304), 7.0, device=CUDA)
    tss.layer_norm(dev(x), dev(w), dev(b), dev(r), out=buf[1:301], stats=(stats[0, 1:301], stats[1, 1:301]))
    assert torch.equal(buf[1:301], want.y) and (buf[0] == 7).all() and (buf[301] == 7).all()
    assert torch.equal(stats[0, 1:301], want.mean) and torch.equal(stats[1, 1:301], want.rstd)
    assert (stats[:, 0] == 7).all() and (stats[:, 301:] == 7).all()
    assert tss.layer_norm(dev(x)[:0], dev(w)).y.shape == (0, 264)


@pytest.mark.parametrize("with_dh", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("shape", SHAPES + [(9000, 128), (5000, 1024), (3000, 40), (1500, 200), (1024, 72), (1024, 4096), (1025, 4096), (600, 8192), (1300, 520), (2051, 1544), (5000, 264), (187, 11056), (30, 16384), (64, 2056), (65, 504),
                                            (66, 16376),
                                            (40, 2056)])
def test_backward(shape, dtype, with_dh):
    rows, d = shape
    h, dy = rows_of(shape, dtype, 8), rows_of(shape, dtype, 9, mean=0)
    dh = rows_of(shape, dtype, 10) if with_dh else None
    w, _ = params(d, dtype)
    _, _, mean, rstd = definition(h, None, w, None)
    mean, rstd = mean.float(), rstd.float()
    xhat = (h.double() - mean.double()[:, None]) * rstd.double()[:, None]
    g = dy.double() * w.double()
    dx = rstd.double()[:, None] * (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True))
    size = rstd.double()[:, None] * (g.abs() + g.abs().mean(1, keepdim=True) + xhat.abs() * (g * xhat).abs().mean(1, keepdim=True))
    if with_dh:
        dx, size = dx + dh.double(), size + dh.double().abs()
    got = tss.layer_norm_backward(dev(dy), dev(h), dev(w), dev(mean), dev(rstd), dev(dh))
    half, low = U.half_step(dtype)
    check(got[0], dx, dx.abs() * half + size * REL + low, "dx")
    # a column's sum: at most rows / 256 + 1 rows of a lane in turn, then fixed trees of 6 + 4 and 64 + 4 + 16 additions
    # (few rows: rows / 128 + 1 in turn, 4 + 16 additions: fewer up to 9000 rows)
    adds = (rows / 256 + 1 + 10 + 84) * 2.0 ** -24 + 4 * 2.0 ** -24
    check(got[1], (dy.double() * xhat).sum(0), (dy.double() * xhat).abs().sum(0) * adds, "dweight")
    check(got[2], dy.double().sum(0), dy.double().abs().sum(0) * adds, "dbias")
    again = tss.layer_norm_backward(dev(dy), dev(h), dev(w), dev(mean), dev(rstd), dev(dh), dbias=False)
    assert again[2] is None and torch.equal(again[0], got[0]) and torch.equal(again[1], got[1])
    over = dev(dy)
    over = tss.layer_norm_backward(over, dev(h), dev(w), dev(mean), dev(rstd), dev(dh), dx=over)
    assert torch.equal(over[0], got[0])
    check(over[1], (dy.double() * xhat).sum(0), (dy.double() * xhat).abs().sum(0) * adds, "dweight, dx over dy")
    check(over[2], dy.double().sum(0), dy.double().abs().sum(0) * adds, "dbias, dx over dy")
    if with_dh:
        over = dev(dh)
        assert torch.equal(tss.layer_norm_backward(dev(dy), dev(h), dev(w), dev(mean), dev(rstd), over, dx=over)[0], got[0])


def test_gradients_are_differences():
    """Against central differences of the definition in 64 bits."""
    rows, d = 5, 136
    x, dy = U.normal(U.gen(11), rows, d).float(), U.normal(U.gen(12), rows, d).float()
    w, b = params(d, "f32")
    f = tss.layer_norm(dev(x), dev(w), dev(b), stats=True)
    dx, dw, db = tss.layer_norm_backward(dev(dy), dev(x), dev(w), f.mean, f.rstd)
    g = U.gen(13)
    step = 1e-5  # second-order terms 1e-10 of the value, roundings 1e-16 / step = 1e-11
    for at, grad in (("x", dx), ("w", dw), ("b", db)):
        for _ in range(3):
            p = {"x": x.double(), "w": w.double(), "b": b.double()}
            v = U.normal(g, *p[at].shape)

            def value(sign):
                q = {**p, at: p[at] + sign * step * v}
                return float((definition(q["x"], None, q["w"], q["b"])[0] * dy.double()).sum())
            want = (value(1) - value(-1)) / (2 * step)
            size = float((grad.double().cpu() * v).abs().sum())
            assert abs(float((grad.double().cpu() * v).sum()) - want) <= size * REL * 4 + 1e-6, at


def test_no_rows():
    w = torch.ones(64, device=CUDA)
    e = torch.empty(0, 64, device=CUDA)
    dx, dw, db = tss.layer_norm_backward(e, e, w, e[:, 0], e[:, 0], dweight=torch.full((64,), 3.0, device=CUDA))
    assert dx.shape == (0, 64) and (dw == 0).all() and (db == 0).all()


def test_offsets_past_32_bits():
    """2^31 elements and more, in a narrow and a wide form."""
    for rows, d in ((9000011, 256), (1100003, 2048)):
        x = torch.zeros(rows, d, dtype=torch.float16, device=CUDA)
        tail = rows_of((40, d), "f16", 14)
        x[-40:] = dev(tail)
        w, b = params(d, "f16")
        y, h, mean, rstd = definition(tail, None, w, b)
        got = tss.layer_norm(x, dev(w), dev(b), stats=True)
        half, low = U.half_step("f16")
        known = inner(y, h, rstd, w, b)
        check(got.y[-40:], y, known + (y.abs() + known) * half + low, "y")
        assert torch.equal(got.y[0], dev(b)) and torch.equal(got.y[rows // 2], dev(b))
        q = tss.quantize_int8(x)
        assert torch.equal(q[0][-40:], tss.quantize_int8(x[-40:].clone())[0]) and (q[0][-41] == 0).all()
        dy = torch.zeros_like(x)
        dy[-40:] = dev(rows_of((40, d), "f16", 15))
        back = tss.layer_norm_backward(dy, x, dev(w), got.mean, got.rstd)
        small = tss.layer_norm_backward(dy[-40:].clone(), x[-40:].clone(), dev(w), got.mean[-40:].clone(), got.rstd[-40:].clone())
        assert torch.equal(back[0][-40:], small[0]) and (back[0][:-40] == 0).all()
        del x, dy, got, q, back


def test_a_captured_run_follows_its_inputs():
    rows, d = 2000, 264
    x, r, dy = (dev(rows_of((rows, d), "bf16", s)) for s in (16, 17, 18))
    w, b = (dev(t) for t in params(d, "bf16"))

    def run():
        f = tss.layer_norm(x, w, b, r, stats=True)
        q = tss.layer_norm(x, w, b, r, out_dtype="i8")
        return [f.y, f.h, f.mean, f.rstd, q.y, q.scale, *tss.layer_norm_backward(dy, f.h, w, f.mean, f.rstd, r)]

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        run()
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = run()
    for seed in range(4):
        x.copy_(rows_of((rows, d), "bf16", 40 + seed))
        dy.copy_(rows_of((rows, d), "bf16", 50 + seed))
        graph.replay()
        want = run()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(held, want))

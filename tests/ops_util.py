"""Definitions in 64 bits of the row operators and the 8-bit and grouped
products, and the bounds that the tests hold the kernels to."""
import torch

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32,
         "e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
LARGEST = {"e4m3": 448.0, "e5m2": 57344.0}
# half the step of an 8-bit type: relative to a normal value, and absolute below the normal values
HALF_STEP = {"e4m3": (2.0 ** -4, 2.0 ** -10), "e5m2": (2.0 ** -3, 2.0 ** -17)}


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def normal(g, *shape):
    return torch.randn(*shape, generator=g, dtype=torch.float64)


def half_step(dtype):
    """(relative, absolute) rounding error of a 16- or 32-bit type."""
    f = torch.finfo(TYPES[dtype])
    return f.eps / 2, f.tiny * f.eps / 2


def blocks(n):
    return (n + 127) // 128


def block_amax(v, block_rows):
    """Largest |v| of each block_rows x 128 block, [column block][row or row block]."""
    rows, d = v.shape
    p = torch.nn.functional.pad(v.abs(), (0, -d % 128, 0, -rows % block_rows))
    return p.view(p.shape[0] // block_rows, block_rows, blocks(d), 128).amax((1, 3)).t().contiguous()


def spread(scale, rows, d, block_rows):
    """Scales [column block][row block] as one per element, rows x d."""
    return scale.t().repeat_interleave(128, 1)[:, :d].repeat_interleave(block_rows, 0)[:rows]


def check_quantised(q, scale, v, fp8, block_rows, rel):
    """q and scale against the exact values v, themselves known to the kernel
    to `rel` of each: the scale to that and two roundings of 2^-24, q's values
    to half a step of their type besides."""
    want = block_amax(v, block_rows).clamp(min=1e-30) / LARGEST[fp8]
    s = scale.double().cpu()
    assert s.shape == want.shape
    bad = ~((s - want).abs() <= want * (rel + 2.0 ** -23))
    assert not bad.any(), f"scale off at {bad.nonzero()[:4].tolist()}"
    full = spread(s, *v.shape, block_rows)
    got = q.cpu().to(torch.float64) * full
    step, low = HALF_STEP[fp8]
    # the quotient v / scale is known to rel and three roundings; a value that these move across a border is
    # still within half a step of itself after the move
    bound = v.abs() * (step + 2 * rel + 2.0 ** -21) + full * low * (1 + 2.0 ** -10)
    bad = ~((got - v).abs() <= bound)
    assert not bad.any(), f"{int(bad.sum())} values off, first at {bad.nonzero()[:4].tolist()}"


def norm_forward(x, residual, weight, eps):
    """(y, h, rstd) in float64."""
    h = x.double() + (residual.double() if residual is not None else 0)
    r = 1 / torch.sqrt(h.square().mean(1) + eps)
    return h * r[:, None] * weight.double(), h, r


def norm_backward(dy, h, weight, rstd, dh):
    """(dx, dweight) in float64."""
    dy, h, w, r = dy.double(), h.double(), weight.double(), rstd.double()[:, None]
    xhat, g = h * r, dy * w
    dx = r * (g - xhat * (g * xhat).mean(1, keepdim=True))
    return dx + (dh.double() if dh is not None else 0), (dy * xhat).sum(0)


def spans(sizes, T):
    """[(first row, end)] of each group, and the first row of no group."""
    out, at = [], 0
    for n in sizes:
        end = min(at + max(int(n), 0), T)
        out.append((at, end))
        at = end
    return out, at


def values(q, scale, block_rows):
    """The values of 8-bit rows with their scales, float64."""
    return q.to(torch.float64) * spread(scale.double(), *q.shape, block_rows)

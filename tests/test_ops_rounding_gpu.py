"""Gated quantisation with blocks of 1 x 128 rounds as the definition in 64
bits does: over values below the type's smallest normal one, over blocks whose
largest value has a far negative gate, and over far negative gates throughout."""
import pytest
import torch

import tile_size_selection_amd as tss
import ops_util as U

pytestmark = pytest.mark.gpu

CUDA = torch.device("cuda:0")
ROWS, D = 2048, 4096


# exponents of the smallest normal value and of half the smallest one
LOW = {"e4m3": (-6, -10), "e5m2": (-14, -17)}


def inputs(kind, dtype, fp8):
    """(gate, up) on the GPU, in the type that they are given in."""
    g = torch.Generator(device=CUDA)
    g.manual_seed(90)
    normal = lambda: torch.randn(ROWS, D, generator=g, device=CUDA, dtype=torch.float64)  # noqa: E731
    if kind == "small":  # quotients below the smallest normal value
        gate = -4 - 16 * torch.rand(ROWS, D, generator=g, device=CUDA, dtype=torch.float64)
        high, low = LOW[fp8]
        f = 2.0 ** (low + (high - low) * torch.rand(ROWS, D, generator=g, device=CUDA, dtype=torch.float64))
        top = 1000.0 / (1 + torch.exp(torch.tensor(-3.0).double())) * 3  # the block's largest value
        up = f * top.item() / U.LARGEST[fp8] / gate * (1 + torch.exp(-gate))
        gate[:, ::128], up[:, ::128] = 3.0, 1000.0
    elif kind == "top":  # a block's largest value is silu of a gate between -22 and -12
        gate, up = normal(), normal()
        far = -12 - 10 * torch.rand(ROWS, D // 128, generator=g, device=CUDA, dtype=torch.float64)
        gate[:, ::128], up[:, ::128] = far, 20 * torch.exp(-far)
    else:  # gates between -80 and -25
        gate = -25 - 55 * torch.rand(ROWS, D, generator=g, device=CUDA, dtype=torch.float64)
        up = normal() * torch.exp(-gate)
    return gate.to(U.TYPES[dtype]), up.to(U.TYPES[dtype])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("fp8", ["e4m3", "e5m2"])
@pytest.mark.parametrize("kind", ["small", "top", "far"])
def test_quantize_gated_rounds_as_in_64_bits(kind, fp8, dtype):
    gate, up = inputs(kind, dtype, fp8)
    q, s = tss.quantize_fp8(torch.cat([gate, up], 1), fp8, gated=True)
    v = gate.double() / (1 + torch.exp(-gate.double())) * up.double()
    amax = v.view(ROWS, D // 128, 128).abs().amax(2)
    scale = amax.clamp(min=1e-30) / U.LARGEST[fp8]
    # silu is known to 1.22 |gate| + 7 halves of a unit (at most 117 with gates down to -88), the scale to one more
    assert ((s.t().double() - scale).abs() <= scale * 118 * 2.0 ** -24).all()
    t = v / scale.repeat_interleave(128, 1)
    # the result is the definition's for all whose quotient is not within double rounding (2^-24) of a border
    want, low, high = (t.mul(1 + e).float().to(U.TYPES[fp8]).float() for e in (0, -2.0 ** -23, 2.0 ** -23))
    sure = low == high
    assert sure.double().mean() > 0.9
    bad = (q.float() != want) & sure
    assert not bad.any(), f"{int(bad.sum())} differ, first at {bad.nonzero()[:4].tolist()}"


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("fp8", ["e4m3", "e5m2"])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_quantize_rounds_as_fp32_division_does(dtype, fp8, block_rows):
    # scale = amax / largest and q = value / scale in fp32, each rounded as IEEE division is (on the CPU: on the GPU
    # torch multiplies by a constant divisor's reciprocal); many values of a 16-bit type lie exactly on a border
    rows, d = 1500, 4104
    g = U.gen(91)
    x = (U.normal(g, rows, d) * torch.exp(0.7 * U.normal(g, d))).to(U.TYPES[dtype])
    q, s = tss.quantize_fp8(x.to(CUDA), fp8, block_rows=block_rows)
    scale = U.block_amax(x.float(), block_rows).clamp(min=1e-30) / torch.tensor(U.LARGEST[fp8])
    assert torch.equal(s.cpu(), scale)
    want = (x.float() / U.spread(scale, rows, d, block_rows)).to(U.TYPES[fp8])
    assert torch.equal(q.float().cpu(), want.float())

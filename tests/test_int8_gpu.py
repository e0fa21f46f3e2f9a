"""Products of 8-bit integers and their quantisation.

The product's sums are exact, and its scaling has one order, so the oracle
gives the result bit for bit: the sum in 64 bits, rounded to fp32, times sa,
times sb, rounded to the output.  Quantising rounds 127 x / amax, a quotient
known to half a unit of fp32: of 16-bit inputs, x = X 2^-e and amax = A with X,
A of 11 bits, it is a border k + 1/2 or at least 2^-e / 2^12 away from it, far
more than its error of 2^-17-e, so it is the exact quotient's rounding; of fp32
inputs, wherever the border is 2^-17 away."""
import numpy as np
import pytest
import torch

import tile_size_selection_amd as tss
import ops_util as U
from test_int8_plans import WAYS

pytestmark = pytest.mark.gpu

CUDA = torch.device("cuda:0")


def bytes_of(g, *shape):
    return torch.randint(-128, 128, shape, generator=g, dtype=torch.int8)


def scales(g, n):
    return torch.exp(U.normal(g, n)).float()


def product(a, b, sa, sb, out):
    """The definition on the GPU: float64 holds the sums exactly."""
    s = (a.double() @ b.double().t()).float()
    return (s * sa[:, None] * sb).to(U.TYPES[out])


def check(a, b, sa, sb, out, got=None):
    got = tss.gemm_int8(a, b, sa, sb, out) if got is None else got
    want = product(a, b, sa, sb, out)
    bad = got != want
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} differ, first at {bad.nonzero()[:4].tolist()}"


# the sizes that reach every way of running an 8-bit product, and odd ones of every kind
SIZES = sorted(set(WAYS) | {
    (1, 1, 16), (1, 8192, 8192), (3, 17, 48), (16, 256, 512), (17, 256, 512), (33, 1000, 2064), (64, 4104, 1040),
    (129, 130, 128), (1000, 1001, 1024), (255, 4097, 656), (2049, 1100, 4096), (4097, 515, 2048)})


@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_product(M, N, K, out):
    g = U.gen(M * 7 + N * 3 + K)
    a, b = bytes_of(g, M, K).to(CUDA), bytes_of(g, N, K).to(CUDA)
    sa, sb = scales(g, M).to(CUDA), scales(g, N).to(CUDA) * 1e-4
    check(a, b, sa, sb, out)


@pytest.mark.parametrize("M,N,K", [(5, 40, 131056), (600, 300, 131056), (40, 2000, 131056)])
def test_largest_sums(M, N, K):
    """The longest rows at the ends of the range: the sums nearly fill 32 bits."""
    a, b = (torch.full((n, K), -128, dtype=torch.int8, device=CUDA) for n in (M, N))
    a[1::2] = 127
    sa, sb = torch.ones(M, device=CUDA), torch.ones(N, device=CUDA)
    got = tss.gemm_int8(a, b, sa, sb, "f32")
    assert (got[0::2] == float(np.float32(2 ** 14 * K))).all() and (got[1::2] == float(np.float32(-128 * 127 * K))).all()


def test_scales_of_any_size():
    g = U.gen(3)
    a, b = bytes_of(g, 100, 256).to(CUDA), bytes_of(g, 72, 256).to(CUDA)
    sa, sb = scales(g, 100).to(CUDA), scales(g, 72).to(CUDA)
    sa[3], sa[4], sa[5], sb[7], sb[8] = 1e-30, 1e30, float("nan"), 0.0, float("inf")
    got, want = tss.gemm_int8(a, b, sa, sb, "f32"), product(a, b, sa, sb, "f32")
    assert torch.equal(got.nan_to_num(7.0, 8.0, 9.0), want.nan_to_num(7.0, 8.0, 9.0))
    assert torch.equal(got.isnan(), want.isnan()) and got[5].isnan().all()


def test_nothing_beside_the_result_is_written():
    g = U.gen(4)
    for M, N, K in ((5, 23, 64), (70, 131, 4112), (300, 257, 160)):
        a, b, sa, sb = bytes_of(g, M, K).to(CUDA), bytes_of(g, N, K).to(CUDA), scales(g, M).to(CUDA), scales(g, N).to(CUDA)
        for out in ("f32", "bf16"):
            buf = torch.full((M * N + 64,), 7.0, dtype=U.TYPES[out], device=CUDA)
            check(a, b, sa, sb, out, tss.gemm_int8(a, b, sa, sb, out, out=buf[:M * N].view(M, N)))
            assert (buf[M * N:] == 7).all()


def test_empty_sizes():
    e = lambda *s: torch.empty(*s, dtype=torch.int8, device=CUDA)  # noqa: E731
    f = lambda n: torch.ones(n, device=CUDA)  # noqa: E731
    assert tss.gemm_int8(e(0, 64), e(8, 64), f(0), f(8)).shape == (0, 8)
    assert tss.gemm_int8(e(8, 64), e(0, 64), f(8), f(0)).shape == (8, 0)
    for out in ("f32", "bf16"):
        c = torch.full((5, 7), 3.0, dtype=U.TYPES[out], device=CUDA)
        assert (tss.gemm_int8(e(5, 0), e(7, 0), f(5), f(7), out, out=c) == 0).all()


def test_a_given_workspace_and_streams():
    g = U.gen(5)
    M, N, K = 512, 512, 8192
    a, b, sa, sb = bytes_of(g, M, K).to(CUDA), bytes_of(g, N, K).to(CUDA), scales(g, M).to(CUDA), scales(g, N).to(CUDA)
    need = tss.gemm_int8_workspace_size(M, N, K)
    ws = torch.full((need + 64,), 7, dtype=torch.uint8, device=CUDA)
    check(a, b, sa, sb, "bf16", tss.gemm_int8(a, b, sa, sb, workspace=ws[:need]))
    assert (ws[need:] == 7).all()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for _ in range(3):  # two at once, each with a workspace of its own
        for s in streams:
            s.wait_stream(torch.cuda.current_stream())
            outs.append(tss.gemm_int8(a, b, sa, sb, stream=s))
    torch.cuda.synchronize()
    for o in outs:
        check(a, b, sa, sb, "bf16", o)


def check_quantised(x, q, s):
    amax = x.float().abs().amax(1).clamp(min=1e-30)
    assert torch.equal(s.cpu(), amax / 127)
    t = 127 * x.double() / amax.double()[:, None]
    off = q.cpu().double() != torch.round(t)
    if x.dtype == torch.float32:
        off &= ~(((t - torch.floor(t) - 0.5).abs() <= 2.0 ** -17) & ((q.cpu().double() - t).abs() <= 0.5 + 2.0 ** -17))
    assert not off.any(), f"{int(off.sum())} of {off.numel()} off, first at {off.nonzero()[:4].tolist()}"


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,d", [(1, 8), (1, 8192), (37, 64), (19, 136), (9, 256), (5, 520), (2, 4104), (7, 8200), (3, 16384),
                                    (2, 32768), (1030, 264), (1025, 2056), (1026, 24)])
def test_quantisation(rows, d, dtype):
    g = U.gen(6)
    x = (U.normal(g, rows, d) * torch.exp(0.7 * U.normal(g, d))).to(U.TYPES[dtype])
    if rows > 4:
        x[1], x[2, 1:], x[3] = 0, 0, x[3] * 0 + 1e-6
    check_quantised(x, *tss.quantize_int8(x.to(CUDA)))


def test_quantisation_on_rounding_borders():
    """Quotients k + 1/2 and what fp32 holds next to them; halves of 16-bit maxima go to the even number."""
    g = U.gen(7)
    amax = torch.exp(4 * U.normal(g, 4000)).float()
    k = torch.arange(-127, 127).float() + 0.5
    x = torch.cat([amax[:, None], k * (amax[:, None] / 127), torch.zeros(4000, 1)], 1)
    assert x.shape[1] == 256
    check_quantised(x, *tss.quantize_int8(x.to(CUDA)))
    h = torch.cat([amax[:, None], amax[:, None] / 2, -amax[:, None] / 2], 1).repeat(1, 8).to(torch.bfloat16)
    q, s = tss.quantize_int8(h.to(CUDA))
    check_quantised(h, q, s)
    assert (q[:, 1] == 64).all() and (q[:, 2] == -64).all()


def test_rows_that_are_not_finite_stay_by_themselves():
    x = U.normal(U.gen(8), 6, 1032).float()
    x[1, 5], x[2, 6], x[3, 1031] = float("nan"), float("inf"), -float("inf")
    x[1, 9] = torch.tensor(0x7fc12345, dtype=torch.int32).view(torch.float32)  # a NaN with a payload
    q, s = tss.quantize_int8(x.to(CUDA))
    assert s[1].isnan() and s[2].isinf() and s[3].isinf() and s[[0, 4, 5]].isfinite().all()
    assert (q[1:4] == 0).all()
    keep = [0, 4, 5]
    check_quantised(x[keep], q[keep], s[keep])


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,d", [(1, 8), (37, 64), (9, 256), (5, 2056), (1030, 264), (3, 16384), (2, 32768)])
def test_gated_quantisation(rows, d, dtype):
    x = (3 * U.normal(U.gen(9), rows, 2 * d)).to(U.TYPES[dtype])
    x[0, :4] = torch.tensor([-100.0, 100.0, -87.0, 0.0])
    gate, up = x.double()[:, :d], x.double()[:, d:]
    v = gate / (1 + torch.exp(-gate)) * up
    q, s = tss.quantize_int8(x.to(CUDA), gated=True)
    # exp within 1 unit (its argument exact), the sum, quotient and product half a unit each: 2^-21 of v; gates
    # below -87 give less than 2^-120
    scale = v.abs().amax(1).clamp(min=1e-30) / 127
    assert ((s.double().cpu() - scale).abs() <= scale * (2.0 ** -21 + 2.0 ** -23)).all()
    full = s.double().cpu()[:, None]
    assert ((q.double().cpu() * full - v).abs() <= full * 0.5 * (1 + 2.0 ** -15) + v.abs() * 2.0 ** -20 + 2.0 ** -120).all()


def test_captured_products_follow_their_inputs():
    """Two graphs, each with its own split product and its own workspace, replayed in turn with eager calls between."""
    g = U.gen(10)
    M, N, K = 300, 512, 8192
    x = [U.normal(g, M, K).to(torch.bfloat16).to(CUDA) for _ in range(2)]
    b, sb = (t for t in tss.quantize_int8(U.normal(g, N, K).float().to(CUDA)))

    def run(i):
        a, sa = tss.quantize_int8(x[i])
        return [a, sa, tss.gemm_int8(a, b, sa, sb)]

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        run(0)
    torch.cuda.current_stream().wait_stream(stream)
    graphs, held = [torch.cuda.CUDAGraph() for _ in range(2)], []
    for i in range(2):
        with torch.cuda.graph(graphs[i]):
            held.append(run(i))
    for seed in range(4):
        for i in range(2):
            x[i].copy_(U.normal(U.gen(60 + 2 * seed + i), M, K))
            graphs[i].replay()
        want = [run(i) for i in range(2)]
        torch.cuda.synchronize()
        for p, q in zip(held, want):
            assert all(torch.equal(s, t) for s, t in zip(p, q))
            check(p[0], b, p[1], sb, "bf16", p[2])

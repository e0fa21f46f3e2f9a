"""The 8-bit and grouped products against their definitions in 64 bits.

Most inputs are small integers, and most scales powers of two, so that every
fp32 sum is exact whatever the tile, the K split and the order: the result
must equal the definition's, rounded once to the output's type.  The sizes
reach every variant (few rows, the three tiles, K in ranges) and their ragged
edges."""
import pytest
import torch

import tile_size_selection_amd as tss
import ops_util as U

pytestmark = pytest.mark.gpu

CUDA = torch.device("cuda:0")


def ints(g, shape, top, dtype):
    return torch.randint(-top, top + 1, shape, generator=g).to(torch.float32).to(U.TYPES[dtype])


def powers(g, *shape):
    return 2.0 ** torch.randint(-2, 2, shape, generator=g).float()


def equal(got, want, what=""):
    want = want.to(got.dtype)
    bad = got.cpu() != want
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} differ, first at {bad.nonzero()[:4].tolist()}"


def fp8_case(M, N, K, a, b_rows, seed):
    g = U.gen(seed)
    A, B = ints(g, (M, K), 3, a), ints(g, (N, K), 2, "e4m3")
    sa = powers(g, U.blocks(K), M)
    sb = powers(g, U.blocks(K), N if b_rows == 1 else U.blocks(N))
    return A, B, sa, sb


def product(A, B, sa, sb, b_rows):
    a, b = U.values(A, sa, 1).to(CUDA), U.values(B, sb, b_rows).to(CUDA)
    return (a @ b.t().contiguous()).cpu()


FP8_SIZES = [
    (1, 1, 16), (3, 7, 2064), (29, 130, 144), (1, 264, 8192), (3, 136, 144), (16, 16, 128), (17, 24, 112), (31, 1000, 1040),  # few rows
    (33, 3, 16), (77, 129, 2064), (300, 1003, 528), (50, 264, 528), (64, 128, 2064), (100, 1000, 4112), (257, 136, 128),           # 64 x 128, K in ranges
    (2101, 2105, 272), (2100, 2106, 144), (2500, 2200, 128),                                                         # 128 x 128
    (4100, 4104, 400), (4099, 4101, 144), (4096, 4098, 128), (4096, 4096, 128), (8000, 2048, 16),                                       # 256 x 256
]


@pytest.mark.parametrize("b_rows", [128, 1])
@pytest.mark.parametrize("a", ["e4m3", "e5m2"])
@pytest.mark.parametrize("size", FP8_SIZES)
def test_gemm_fp8_is_exact(size, a, b_rows):
    M, N, K = size
    A, B, sa, sb = fp8_case(M, N, K, a, b_rows, M + N + K)
    want = product(A, B, sa, sb, b_rows)
    dev = [t.to(CUDA) for t in (A, B, sa, sb)]
    for out in ("f32", "bf16", "f16"):
        C = torch.full((M + 3, N), float("nan"), dtype=U.TYPES[out], device=CUDA)
        tss.gemm_fp8(*dev, out_dtype=out, out=C[:M])
        equal(C[:M], want, out)
        assert C[M:].isnan().all()


@pytest.mark.parametrize("size", [(5, 264, 4112), (96, 264, 4112), (2100, 2104, 528), (4100, 4104, 528)])
def test_gemm_fp8_of_quantised_values(size):
    M, N, K = size
    g = U.gen(40)
    x = (U.normal(g, M, K) * torch.exp(0.7 * U.normal(g, K))).float().to(CUDA)
    w = (U.normal(g, N, K) / K ** 0.5).float().to(CUDA)
    for b_rows in (1, 128):
        (A, sa), (B, sb) = tss.quantize_fp8(x), tss.quantize_fp8(w, block_rows=b_rows)
        a = U.values(A.cpu(), sa.cpu(), 1).to(CUDA)
        b = U.values(B.cpu(), sb.cpu(), b_rows).to(CUDA).t().contiguous()
        want, size_of = a @ b, a.abs() @ b.abs()
        got = tss.gemm_fp8(A, B, sa, sb, out_dtype="f32").double()
        # at most 128 additions in a block, one a block after it, and the scales' two products, of 2^-24 each
        bound = size_of * (128 + K / 128 + 20) * 2.0 ** -24
        assert ((got - want).abs() <= bound).all()


def test_gemm_fp8_without_products():
    e = torch.empty
    f8, f32 = torch.float8_e4m3fn, torch.float32
    C = tss.gemm_fp8(e(70, 0, dtype=f8, device=CUDA), e(24, 0, dtype=f8, device=CUDA), e(0, 70, dtype=f32, device=CUDA),
                     e(0, 1, dtype=f32, device=CUDA), out=torch.ones(70, 24, dtype=torch.bfloat16, device=CUDA))
    assert (C == 0).all()
    assert tss.gemm_fp8(e(0, 128, dtype=f8, device=CUDA), e(24, 128, dtype=f8, device=CUDA),
                        e(1, 0, dtype=f32, device=CUDA), e(1, 1, dtype=f32, device=CUDA)).shape == (0, 24)


def test_gemm_fp8_nan_stays_in_its_row_and_column():
    A, B, sa, sb = fp8_case(40, 136, 256, "e4m3", 128, 41)
    A[7, 200] = float("nan")
    sa[0, 9] = float("nan")
    B[33, 5] = float("nan")
    C = tss.gemm_fp8(*(t.to(CUDA) for t in (A, B, sa, sb)), out_dtype="f32").isnan().cpu()
    want = torch.zeros(40, 136, dtype=torch.bool)
    want[7] = want[9] = True
    want[:, 33] = True
    assert torch.equal(C, want)


# T and the groups' sizes; sizes may leave rows over, run past T, be zero or negative
GROUPS = [
    (1, [1]), (1, [0, 0, 1]), (5, [0, 2, -4, 0, 3]), (7, [2, 1]), (9, [4, 100, 3]), (20, [0, 0, 0]),
    (64, [2] * 32), (70, [17, 0, 33, 20]), (300, [100, 0, 64, 65, 1]), (150, [1] * 130), (400, [3] * 70 + [0] * 10 + [150]),
    (700, [130, 0, 257, 300]), (1000, [256, 512, 200]), (1300, [700, 0, 513]), (2000, [2000]),
]
WIDTHS = [(16, 8), (144, 264), (272, 136), (400, 520)]
# wide enough for whole rounds of large tiles, and for a last round of whole tiles and of pieces
LARGE = [((2100, [900, 0, 1100]), (144, 5000)), ((2100, [900, 0, 1100]), (144, 8200)), ((1200, [400, 650]), (272, 4104)),
         ((3000, [5, 2990]), (2008 // 16 * 16, 1032))]
CASES = [(g, w) for g in GROUPS for w in WIDTHS] + LARGE
IDS = [f"{g[0]}rows_{len(g[1])}groups_{w[0]}x{w[1]}" for g, w in CASES]


@pytest.mark.parametrize("groups,width", CASES, ids=IDS)
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_grouped_is_exact(groups, width, dtype):
    (T, sizes), (K, N), E = groups, width, len(groups[1])
    g = U.gen(T + K)
    A, B, dC = ints(g, (T, K), 2, dtype), ints(g, (E, K, N), 2, dtype), ints(g, (T, N), 2, dtype)
    at, used = U.spans(sizes, T)
    C, dA = torch.zeros(T, N, dtype=torch.float64), torch.zeros(T, K, dtype=torch.float64)
    dB = torch.zeros(E, K, N, dtype=torch.float64)
    for e, (i, j) in enumerate(at):
        C[i:j] = A[i:j].double() @ B[e].double()
        dA[i:j] = dC[i:j].double() @ B[e].double().t()
        dB[e] = A[i:j].double().t() @ dC[i:j].double()
    A[used:] = float("nan")  # rows of no group are not read
    dC[used:] = float("nan")
    A, B, dC = A.to(CUDA), B.to(CUDA), dC.to(CUDA)
    s = torch.tensor(sizes, dtype=torch.int32, device=CUDA)
    nan = lambda *shape, t: torch.full(shape, float("nan"), dtype=U.TYPES[t], device=CUDA)  # noqa: E731
    for out in (dtype, "f32"):
        got = nan(T + 3, N, t=out)
        tss.gemm_grouped(A, B, s, out_dtype=out, out=got[:T])
        equal(got[:T], C, "C " + out)
        assert got[T:].isnan().all()
        a, b = nan(T + 3, K, t=dtype), nan(E + 1, K, N, t=out)
        tss.gemm_grouped_backward(dC, A, B, s, dA=a[:T], dB=b[:E], db_dtype=out)
        equal(a[:T], dA, "dA")
        equal(b[:E], dB, "dB " + out)
        assert a[T:].isnan().all() and b[E:].isnan().all()
    a, none = tss.gemm_grouped_backward(dC, A, B, s, need_dB=False)
    equal(a, dA, "dA alone")
    assert none is None
    none, b = tss.gemm_grouped_backward(dC, A, B, s, need_dA=False)
    equal(b, dB, "dB alone")
    assert none is None


@pytest.mark.parametrize("groups,width", CASES, ids=IDS)
@pytest.mark.parametrize("a", ["e4m3", "e5m2"])
def test_grouped_fp8_is_exact(groups, width, a):
    (T, sizes), (K, N), E = groups, width, len(groups[1])
    g = U.gen(T + K + 1)
    A, B = ints(g, (T, K), 3, a), ints(g, (E, N, K), 2, "e4m3")
    sa, sb = powers(g, U.blocks(K), T), powers(g, E, U.blocks(K), U.blocks(N))
    at, used = U.spans(sizes, T)
    C = torch.zeros(T, N, dtype=torch.float64)
    for e, (i, j) in enumerate(at):
        C[i:j] = U.values(A[i:j], sa[:, i:j], 1) @ U.values(B[e], sb[e], 128).t()
    A[used:] = float("nan")
    sa[:, used:] = float("nan")
    dev = [t.to(CUDA) for t in (A, B, sa, sb)] + [torch.tensor(sizes, dtype=torch.int32, device=CUDA)]
    for out in ("f32", "bf16", "f16"):
        got = torch.full((T + 3, N), float("nan"), dtype=U.TYPES[out], device=CUDA)
        tss.gemm_grouped_fp8(*dev, out_dtype=out, out=got[:T])
        equal(got[:T], C, out)
        assert got[T:].isnan().all()


def test_grouped_gradients_are_the_slope():
    # sum(dc C) along directions of A and of B, by central differences of the definition in 64 bits (C is linear in each)
    T, sizes, K, N = 90, [40, 0, 45], 64, 72
    g = U.gen(50)
    A, B, dC = (U.normal(g, *s).to(torch.float16) for s in ((T, K), (3, K, N), (T, N)))
    vA, vB = U.normal(g, T, K), U.normal(g, 3, K, N)

    def loss(a, b):
        return sum((dC[i:j].double() * (a[i:j] @ b[e])).sum() for e, (i, j) in enumerate(U.spans(sizes, T)[0]))

    s = torch.tensor(sizes, dtype=torch.int32, device=CUDA)
    dA, dB = tss.gemm_grouped_backward(dC.to(CUDA), A.to(CUDA), B.to(CUDA), s)
    a, b = A.double(), B.double()
    for got, v, slope in ((dA, vA, (loss(a + vA, b) - loss(a - vA, b)) / 2), (dB, vB, (loss(a, b + vB) - loss(a, b - vB)) / 2)):
        terms = (got.double().cpu() * v)
        # dA is rounded to fp16; every sum has at most 128 terms of 2^-24 of magnitudes up to 30 times the result's
        assert abs(terms.sum() - slope) <= (2.0 ** -11 + 2.0 ** -12) * terms.abs().sum()


def test_grouped_replays_follow_the_sizes():
    T, E, K, N = 200, 5, 144, 136
    g = U.gen(60)
    A, B, dC = ints(g, (T, K), 2, "bf16").to(CUDA), ints(g, (E, K, N), 2, "bf16").to(CUDA), ints(g, (T, N), 2, "bf16").to(CUDA)
    A8, B8 = ints(g, (T, K), 2, "e4m3").to(CUDA), ints(g, (E, N, K), 2, "e4m3").to(CUDA)
    sa, sb = powers(g, 2, T).to(CUDA), powers(g, E, 2, 2).to(CUDA)
    x, w = ints(g, (T, K), 2, "bf16").to(CUDA), torch.ones(K, dtype=torch.bfloat16, device=CUDA)
    few, few_s = ints(g, (40, 4096), 2, "e4m3").to(CUDA), powers(g, 32, 40).to(CUDA)
    wide, wide_s = ints(g, (N, 4096), 2, "e4m3").to(CUDA), powers(g, 32, 2).to(CUDA)
    sizes = torch.tensor([50, 0, 20, 70, 40], dtype=torch.int32, device=CUDA)

    def step():
        n = tss.rms_norm(x, w, x, out_dtype="e4m3", rstd=True)
        q = tss.quantize_fp8(x, block_rows=128)
        return [tss.gemm_grouped(A, B, sizes), *tss.gemm_grouped_backward(dC, A, B, sizes),
                tss.gemm_grouped_fp8(A8, B8, sa, sb, sizes), n.y.view(torch.uint8), n.scale, n.h,
                *tss.rms_norm_backward(dC.new_ones(T, K), n.h, w, n.rstd), q[0].view(torch.uint8), q[1],
                tss.gemm_fp8(few, wide, few_s, wide_s)]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = step()
    for new in ([50, 0, 20, 70, 40], [0, 199, 0, 0, 1], [10, 10, 10, 10, 10], [300, 1, 1, 1, 1]):
        sizes.copy_(torch.tensor(new, dtype=torch.int32))
        x.add_(1)
        graph.replay()
        torch.cuda.synchronize()
        for got, want in zip(kept, step()):
            assert torch.equal(got, want), new

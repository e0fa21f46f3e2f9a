"""The 8-bit and grouped products in the ways of running them that depend on
the sizes: small integers and scales that are powers of two, so that every
fp32 sum is exact whatever its order, and the result must equal the
definition's, rounded once to the output's type."""
import pytest
import torch

import tile_size_selection_amd as tss
import ops_util as U
from test_ops_plans import GROUPED, PRODUCTS, SPLIT

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


def check_product(size, a, b_rows, outs=("f32", "bf16", "f16"), **options):
    M, N, K = size
    g = U.gen(M + N + K)
    A, B = ints(g, (M, K), 3, a), ints(g, (N, K), 2, "e4m3")
    sa, sb = powers(g, U.blocks(K), M), powers(g, U.blocks(K), N if b_rows == 1 else U.blocks(N))
    want = (U.values(A, sa, 1).to(CUDA) @ U.values(B, sb, b_rows).to(CUDA).t().contiguous()).cpu()
    dev = [t.to(CUDA) for t in (A, B, sa, sb)]
    need = tss.gemm_fp8_workspace_size(M, N, K)
    for out in outs:
        C = torch.full((M + 3, N), float("nan"), dtype=U.TYPES[out], device=CUDA)
        ws = torch.full((need + 256,), 0x5a, dtype=torch.uint8, device=CUDA)
        tss.gemm_fp8(*dev, out_dtype=out, out=C[:M], workspace=ws[:max(need, 16)], **options)
        equal(C[:M], want, out)
        assert C[M:].isnan().all() and (ws[max(need, 16):] == 0x5a).all()


@pytest.mark.parametrize("b_rows", [128, 1])
@pytest.mark.parametrize("a", ["e4m3", "e5m2"])
@pytest.mark.parametrize("size", SPLIT + [s for s in PRODUCTS if s not in SPLIT])
def test_gemm_fp8_is_exact(size, a, b_rows):
    check_product(size, a, b_rows)


@pytest.mark.parametrize("size", PRODUCTS)
def test_gemm_fp8_with_fp32_sums_is_exact(size):
    check_product(size, "e4m3", 128, ("bf16", "f16", "f32"), fp32_sums=True)


@pytest.mark.parametrize("grouped", [False, True])
@pytest.mark.parametrize("size", [(16, 128, 1024), (900, 1208, 1040), (1700, 1704, 528)])
def test_products_whose_largest_terms_cancel(size, grouped):
    # a pair of outlier columns in every block of 128 whose products cancel, beside values 2^-12 of theirs and less
    M, N, K = size
    g = U.gen(71)
    A, B = U.normal(g, M, K) / 16, U.normal(g, N, K)
    first = torch.arange(0, K, 128)
    A[:, first], A[:, first + 9] = 256.0, 256.0
    B[:, first] = 16.0
    B[:, first + 9] = -16.0
    A, B = A.float().to(U.TYPES["e4m3"]), B.float().to(U.TYPES["e4m3"])
    a, b = A.double().to(CUDA), B.double().t().contiguous().to(CUDA)
    want, terms = a @ b, a.abs() @ b.abs()
    sa, sb = torch.ones(U.blocks(K), M, device=CUDA), torch.ones(U.blocks(K), U.blocks(N), device=CUDA)
    for out in ("bf16", "f16"):
        def call(**sums):
            if grouped:
                sizes = torch.tensor([M], dtype=torch.int32, device=CUDA)
                return tss.gemm_grouped_fp8(A.to(CUDA), B.to(CUDA)[None], sa, sb[None], sizes, out_dtype=out, **sums).double()
            return tss.gemm_fp8(A.to(CUDA), B.to(CUDA), sa, sb, out_dtype=out, **sums).double()
        half, low = U.half_step(out)
        # fp32: an addition for each term of a block, one a block, and a few more at the joins, of 2^-24 each
        bound = terms * (128 + K / 128 + 20) * 2.0 ** -24
        got = call(fp32_sums=True)
        assert ((got - want).abs() <= bound * (1 + half) + want.abs() * half + low).all()
        # the 8-bit instruction: each of a block's products keeps 2^-13 of the block's largest (256 * 16)
        bound = bound + K * 2.0 ** -13 * 4096
        got = call()
        assert ((got - want).abs() <= bound * (1 + half) + want.abs() * half + low).all()


@pytest.mark.parametrize("a", ["e4m3", "e5m2"])
@pytest.mark.parametrize("size", [(300, 24, 256), (1500, 1210, 144), (1001, 1001, 4112), (1700, 1704, 272), (2101, 2105, 272)])
def test_gemm_fp8_takes_every_value(size, a):
    # a row of A holds one value that is not zero, so each element of C is one product, exact in fp32; the values are
    # the type's finite codes, subnormals among them
    M, N, K = size
    g = U.gen(70)
    code = (torch.arange(M) % 256).to(torch.uint8).view(U.TYPES[a])
    code = torch.where(code.float().isfinite(), code.float(), torch.zeros(M))
    A, B = torch.zeros(M, K), ints(g, (N, K), 2, "e4m3")
    k = torch.randint(K, (M,), generator=g)
    A[torch.arange(M), k] = code
    want = code.double()[:, None] * B.double()[:, k].t()
    dev = [t.to(CUDA) for t in (A.to(U.TYPES[a]), B, torch.ones(U.blocks(K), M), torch.ones(U.blocks(K), U.blocks(N)))]
    for out in ("f32", "bf16"):  # (e5m2 passes fp16's largest value)
        equal(tss.gemm_fp8(*dev, out_dtype=out), want, out)


@pytest.mark.parametrize("a", ["e4m3", "e5m2"])
@pytest.mark.parametrize("case", GROUPED)
def test_grouped_fp8_is_exact(case, a):
    T, sizes, K, N = case
    E, g = len(sizes), U.gen(T + K)
    A, B = ints(g, (T, K), 3, a), ints(g, (E, N, K), 2, "e4m3")
    sa, sb = powers(g, U.blocks(K), T), powers(g, E, U.blocks(K), U.blocks(N))
    at, used = U.spans(sizes, T)
    C = torch.zeros(T, N, dtype=torch.float64)
    for e, (i, j) in enumerate(at):
        C[i:j] = (U.values(A[i:j], sa[:, i:j], 1).to(CUDA) @ U.values(B[e], sb[e], 128).to(CUDA).t().contiguous()).cpu()
    A[used:] = float("nan")  # rows of no group are not read
    sa[:, used:] = float("nan")
    dev = [t.to(CUDA) for t in (A, B, sa, sb)] + [torch.tensor(sizes, dtype=torch.int32, device=CUDA)]
    for out in ("f32", "bf16", "f16"):
        got = torch.full((T + 3, N), float("nan"), dtype=U.TYPES[out], device=CUDA)
        for fp32_sums in (False, True):
            tss.gemm_grouped_fp8(*dev, out_dtype=out, out=got[:T].fill_(float("nan")), fp32_sums=fp32_sums)
            equal(got[:T], C, out)
        assert got[T:].isnan().all()


def test_thousands_of_groups():
    T, E, K, N = 3300, 4096, 48, 24
    g = U.gen(80)
    sizes = torch.randint(-1, 3, (E,), generator=g, dtype=torch.int32)
    group = torch.repeat_interleave(torch.arange(E), sizes.clamp(min=0).long())[:T]
    used = group.numel()
    assert 2000 < used < T  # about three quarters of a row a group, and rows of none
    A, B, dC = ints(g, (T, K), 2, "bf16"), ints(g, (E, K, N), 2, "bf16"), ints(g, (T, N), 2, "bf16")
    picked = B.double()[group]
    C, dA, dB = torch.zeros(T, N).double(), torch.zeros(T, K).double(), torch.zeros(E, K, N).double()
    C[:used] = (A[:used].double()[:, :, None] * picked).sum(1)
    dA[:used] = (dC[:used].double()[:, None, :] * picked).sum(2)
    dB.index_add_(0, group, A[:used].double()[:, :, None] * dC[:used].double()[:, None, :])
    dev = [t.to(CUDA) for t in (A, B, dC, sizes)]
    equal(tss.gemm_grouped(dev[0], dev[1], dev[3], out_dtype="f32"), C, "C")
    got = tss.gemm_grouped_backward(dev[2], dev[0], dev[1], dev[3])
    equal(got[0], dA, "dA")
    equal(got[1], dB, "dB")
    f8 = torch.float8_e4m3fn
    ones = lambda *s: torch.ones(*s, device=CUDA)  # noqa: E731
    got = tss.gemm_grouped_fp8(dev[0].to(f8), dev[1].transpose(1, 2).contiguous().to(f8), ones(1, T), ones(E, 1, 1), dev[3],
                               out_dtype="f32")
    equal(got, C, "C of 8 bits")


@pytest.mark.parametrize("handle", [False, True])
def test_calls_by_keyword_on_a_stream(handle):
    g = U.gen(81)
    A, B = ints(g, (40, 256), 3, "e4m3"), ints(g, (24, 256), 2, "e4m3")
    ones = torch.ones(2, 40, device=CUDA), torch.ones(2, 1, device=CUDA)
    a, b = A.to(CUDA), B.to(CUDA)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    C = tss.gemm_fp8(out_dtype="f32", A=a, B=b, sa=ones[0], sb=ones[1], stream=side.cuda_stream if handle else side)
    torch.cuda.current_stream().wait_stream(side)
    equal(C, A.double() @ B.double().t())


@pytest.mark.parametrize("fp32_sums", [False, True])
@pytest.mark.parametrize("size", [(16, 136, 256), (1500, 1210, 272), (1001, 1001, 4112), (1700, 1704, 272), (2101, 2105, 272)])
def test_gemm_fp8_nan_stays_in_its_row_and_column(size, fp32_sums):
    M, N, K = size
    g = U.gen(82)
    A, B = ints(g, (M, K), 3, "e4m3"), ints(g, (N, K), 2, "e4m3")
    sa, sb = powers(g, U.blocks(K), M), powers(g, U.blocks(K), U.blocks(N))
    A[7, K - 1] = float("nan")
    sa[0, 9] = float("nan")
    B[N - 3, 5] = float("nan")
    C = tss.gemm_fp8(*(t.to(CUDA) for t in (A, B, sa, sb)), fp32_sums=fp32_sums)
    want = torch.zeros(M, N, dtype=torch.bool)
    want[7] = want[9] = True
    want[:, N - 3] = True
    assert torch.equal(C.isnan().cpu(), want)


def test_replayed_products_follow_their_inputs():
    # K in ranges with one and two sets of waves, one round of 128 x 128 tiles, and pieces of a last round
    g = U.gen(83)
    cases = []
    for M, N, K in ((513, 510, 8192), (1001, 1001, 4112), (1700, 1704, 272), (2101, 2105, 272)):
        cases.append([t.to(CUDA) for t in (ints(g, (M, K), 3, "e4m3"), ints(g, (N, K), 2, "e4m3"), powers(g, U.blocks(K), M),
                                           powers(g, U.blocks(K), U.blocks(N)))])

    def step():
        return [tss.gemm_fp8(*c, out_dtype=out, fp32_sums=s) for c in cases for out, s in (("f32", False), ("bf16", False), ("bf16", True))]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = step()
    for _ in range(4):
        for c in cases:
            c[2].mul_(2)
        graph.replay()
        torch.cuda.synchronize()
        for got, want in zip(kept, step()):
            assert torch.equal(got, want)

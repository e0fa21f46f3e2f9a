"""The 8-bit and grouped products in the ways of running them that depend on
the sizes: small integers and scales that are powers of two, so that every
fp32 sum is exact whatever its order, and the result must equal the
definition's, rounded once to the output's type."""
import pytest
import torch

import tile_size_selection_amd as tss
import ops_util as U
from test_ops_plans import SPLIT

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
@pytest.mark.parametrize("size", SPLIT)
def test_gemm_fp8_with_k_in_ranges_is_exact(size, a, b_rows):
    check_product(size, a, b_rows)

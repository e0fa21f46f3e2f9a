"""Products of 8-bit integers with few rows, bit for bit: two groups of columns
a workgroup with every kind of ragged edge, and rows of B without number."""
import pytest
import torch

import tile_size_selection_amd as tss
import ops_util as U
from test_int8_gpu import CUDA, bytes_of, check, scales
from test_int8_limits import TWO_GROUPS

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M,N,K", TWO_GROUPS)
def test_two_groups_of_columns(M, N, K, out):
    g = U.gen(M + N + K)
    a, b = bytes_of(g, M, K).to(CUDA), bytes_of(g, N, K).to(CUDA)
    sa, sb = scales(g, M).to(CUDA), scales(g, N).to(CUDA) * 1e-4
    buf = torch.full((M * N + 64,), 7.0, dtype=U.TYPES[out], device=CUDA)
    check(a, b, sa, sb, out, tss.gemm_int8(a, b, sa, sb, out, out=buf[:M * N].view(M, N)))
    assert (buf[M * N:] == 7).all()


@pytest.mark.parametrize("M,N,K,out", [(1, 70000000, 16, "bf16"), (3, 70000001, 16, "f32"), (16, 134217727, 16, "bf16"), (2, 1040000, 2064, "f16")])
def test_as_many_columns_as_memory_takes(M, N, K, out):
    g = torch.Generator(device=CUDA)
    g.manual_seed(N)
    a, b = (torch.randint(-128, 128, (n, K), generator=g, dtype=torch.int8, device=CUDA) for n in (M, N))
    sa, sb = (torch.exp(torch.randn(n, generator=g, device=CUDA)) for n in (M, N))
    got = tss.gemm_int8(a, b, sa, sb, out)
    step = 1 << 24
    for n in range(0, N, step):
        check(a, b[n:n + step], sa, sb[n:n + step], out, got[:, n:n + step])

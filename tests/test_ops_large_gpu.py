"""More rows, columns and elements than a launch with a thread for each holds."""
import pytest
import torch

import tile_size_selection_amd as tss
import ops_util as U

pytestmark = pytest.mark.gpu

CUDA = torch.device("cuda:0")


def test_norm_of_four_million_narrow_rows():
    # a norm over each head: 32768 tokens of 128 heads, and some
    rows, d = (1 << 22) + 5, 128
    g = torch.Generator(device=CUDA)
    g.manual_seed(1)
    x = torch.randn(rows, d, generator=g, device=CUDA, dtype=torch.bfloat16)
    w = (1 + 0.2 * torch.randn(d, generator=g, device=CUDA)).to(torch.bfloat16)
    got = tss.rms_norm(x, w, rstd=True)
    dx, dw = tss.rms_norm_backward(x, x, w, got.rstd)
    for part in (slice(0, 9), slice(rows // 2, rows // 2 + 9), slice(rows - 9, rows)):
        y, h, rstd = U.norm_forward(x[part].cpu(), None, w.cpu(), 1e-6)
        assert ((got.y[part].double().cpu() - y).abs() <= y.abs() * (2.0 ** -8 + 2.0 ** -18)).all()
        r = got.rstd[part].double().cpu()[:, None]
        assert ((r[:, 0] - rstd).abs() <= rstd * 2.0 ** -18).all()
        want, _ = U.norm_backward(x[part].cpu(), x[part].cpu(), w.cpu(), got.rstd[part].cpu(), None)
        size = (h * w.cpu().double()).abs()
        terms = r * (size + (h * r).abs() * (size * (h * r).abs()).mean(1, keepdim=True))
        assert ((dx[part].double().cpu() - want).abs() <= want.abs() * 2.0 ** -8 + 2.0 ** -18 * terms).all()
    # dw = sum of x^2 rstd, terms of one sign: a workgroup (12 a CU) sums 1366 rows, then 200 partial sums at most
    want = (x.double().square() * got.rstd.double()[:, None]).sum(0)
    assert ((dw.double() - want).abs() <= want * (1366 + 200) * 2.0 ** -24).all()


@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_gemm_fp8_of_one_row_and_a_hundred_million_columns(out):
    N, K = 100_000_003, 16
    g = torch.Generator(device=CUDA)
    g.manual_seed(2)
    A = torch.randint(-2, 3, (1, K), generator=g, device=CUDA).float().to(torch.float8_e4m3fn)
    B = torch.randint(-1, 2, (N, K), generator=g, device=CUDA, dtype=torch.int8).to(torch.float8_e4m3fn)
    C = tss.gemm_fp8(A, B, torch.ones(1, 1, device=CUDA), torch.ones(1, U.blocks(N), device=CUDA), out_dtype=out)
    for i in range(0, N, 1 << 23):
        assert torch.equal(C[0, i:i + (1 << 23)].float(), B[i:i + (1 << 23)].float() @ A[0].float())


@pytest.mark.parametrize("shape", [(65600, 65610), (66000, 65536)])
def test_gemm_fp8_of_more_than_2_to_32_elements(shape):
    (M, N), K = shape, 16
    assert M * N > 1 << 32
    g = torch.Generator(device=CUDA)
    g.manual_seed(3)
    A = torch.randint(-2, 3, (M, K), generator=g, device=CUDA, dtype=torch.int8).to(torch.float8_e4m3fn)
    B = torch.randint(-1, 2, (N, K), generator=g, device=CUDA, dtype=torch.int8).to(torch.float8_e4m3fn)
    C = tss.gemm_fp8(A, B, torch.ones(1, M, device=CUDA), torch.ones(1, U.blocks(N), device=CUDA))
    b = B.float().t().contiguous()
    for i in range(0, M, 4100):
        assert torch.equal(C[i:i + 4100].float(), A[i:i + 4100].float() @ b)

"""The operators at the ends of their ranges: tensors of more than 2^31
elements, operands just under 2 GiB, weights that pass 4 GiB over their
groups, no rows and no K, and calls on a stream that is not current."""
import pytest
import torch

import tile_size_selection_amd as tss
import ops_util as U

pytestmark = pytest.mark.gpu

CUDA = torch.device("cuda:0")


def test_rows_past_2_to_31_elements():
    rows, d = 65600, 32768
    x = torch.zeros(rows, d, dtype=torch.bfloat16, device=CUDA)
    g = U.gen(1)
    last = (U.normal(g, 3, d)).to(torch.bfloat16)
    x[-3:] = last.to(CUDA)
    w = torch.ones(d, dtype=torch.bfloat16, device=CUDA)
    n = tss.rms_norm(x, w, out_dtype="e4m3", rstd=True)
    y, h, rstd = U.norm_forward(last, None, w.cpu(), 1e-6)
    U.check_quantised(n.y[-3:], n.scale[:, -3:], y, "e4m3", 1, 2.0 ** -18)
    assert (n.y[:5].view(torch.uint8) == 0).all()
    rs = n.rstd
    del n
    dx, dw = tss.rms_norm_backward(x, x, w, rs)
    want, want_w = U.norm_backward(last, last, w.cpu(), rs[-3:].cpu(), None)
    terms = rs[-3:].double().cpu()[:, None] * (last.double().abs() + y.abs() * (last.double() * y).abs().mean(1, keepdim=True))
    assert ((dx[-3:].double().cpu() - want).abs() <= want.abs() * 2.0 ** -8 + 2.0 ** -18 * terms).all()
    assert ((dw.double().cpu() - want_w).abs() <= 2.0 ** -16 * (last.double() * y).abs().sum(0)).all()
    del dx
    q, s = tss.quantize_fp8(x, block_rows=1)
    U.check_quantised(q[-3:], s[:, -3:], last.double(), "e4m3", 1, 0.0)


def test_gemm_fp8_b_just_under_2_gib():
    M, N, K = 40, 65528, 32752
    assert 2 ** 31 - 2 ** 22 < N * K < 2 ** 31
    g = torch.Generator(device=CUDA)
    g.manual_seed(2)
    A = torch.randint(-1, 2, (M, K), generator=g, device=CUDA, dtype=torch.int8).to(torch.float8_e4m3fn)
    B = torch.empty(N, K, dtype=torch.float8_e4m3fn, device=CUDA)
    for i in range(0, N, 8191):
        B[i:i + 8191] = torch.randint(-1, 2, (min(8191, N - i), K), generator=g, device=CUDA, dtype=torch.int8).to(B.dtype)
    kb = U.blocks(K)
    C = tss.gemm_fp8(A, B, torch.ones(kb, M, device=CUDA), torch.ones(kb, U.blocks(N), device=CUDA), out_dtype="f32")
    for cols in (slice(0, 3), slice(32760, 32770), slice(N - 5, N)):
        assert torch.equal(C[:, cols].double(), A.double() @ B[cols].double().t().contiguous())


def test_grouped_weights_past_4_gib():
    E, K, N = 40, 4096, 16384
    assert E * K * N * 2 > 2 ** 32
    g = U.gen(3)
    A = torch.randint(-2, 3, (7, K), generator=g).to(torch.bfloat16).to(CUDA)
    B = torch.zeros(E, K, N, dtype=torch.bfloat16, device=CUDA)
    B[-1] = torch.randint(-2, 3, (K, N), generator=g).to(torch.bfloat16).to(CUDA)
    sizes = torch.zeros(E, dtype=torch.int32, device=CUDA)
    sizes[-1] = 7
    C = tss.gemm_grouped(A, B, sizes, out_dtype="f32")
    want = A.double() @ B[-1].double()
    assert torch.equal(C.double(), want)
    dA, dB = tss.gemm_grouped_backward(C.to(torch.bfloat16), A, B, sizes)
    assert torch.equal(dB[-1].double(), A.double().t().contiguous() @ C.to(torch.bfloat16).double())
    assert (dB[:-1] == 0).all()
    del dB
    B8 = B.to(torch.float8_e4m3fn).view(E, N, K)
    ones = torch.ones(E, 32, 128, device=CUDA)
    C8 = tss.gemm_grouped_fp8(A.to(torch.float8_e4m3fn), B8, torch.ones(32, 7, device=CUDA), ones, sizes, out_dtype="f32")
    assert torch.equal(C8.double(), A.double() @ B8[-1].double().t().contiguous())


def test_grouped_without_rows_and_without_k():
    bf, f8 = torch.bfloat16, torch.float8_e4m3fn
    new = lambda *s, t=bf: torch.empty(*s, dtype=t, device=CUDA)  # noqa: E731
    sizes = torch.tensor([3, 0], dtype=torch.int32, device=CUDA)
    assert tss.gemm_grouped(new(0, 64), new(2, 64, 24), sizes).shape == (0, 24)
    dA, dB = tss.gemm_grouped_backward(new(0, 24), new(0, 64), new(2, 64, 24), sizes, dB=torch.ones(2, 64, 24, device=CUDA))
    assert dA.shape == (0, 64) and (dB == 0).all()
    ones = torch.ones(5, 24, dtype=bf, device=CUDA)
    assert (tss.gemm_grouped(new(5, 0), new(2, 0, 24), sizes, out=ones) == 0).all()
    dA, dB = tss.gemm_grouped_backward(new(5, 0), torch.ones(5, 64, dtype=bf, device=CUDA), new(2, 64, 0), sizes,
                                       dA=torch.ones(5, 64, dtype=bf, device=CUDA))
    assert (dA == 0).all() and dB.shape == (2, 64, 0)
    ones = torch.ones(5, 24, dtype=bf, device=CUDA)
    e = new(0, 5, t=torch.float32)
    assert (tss.gemm_grouped_fp8(new(5, 0, t=f8), new(2, 24, 0, t=f8), e, new(2, 0, 1, t=torch.float32), sizes,
                                 out=ones) == 0).all()


@pytest.mark.parametrize("handle", [False, True])
def test_calls_on_another_stream_keep_their_workspace(handle):
    # the call's workspace is freed on return; memory taken from the current stream's pool right after must not be it
    g = U.gen(4)
    h, dy = (U.normal(g, 2048, 2048).to(torch.bfloat16).to(CUDA) for _ in range(2))
    w = torch.ones(2048, dtype=torch.bfloat16, device=CUDA)
    rstd = torch.rand(2048, device=CUDA) + 0.5
    want = tss.rms_norm_backward(dy, h, w, rstd)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = tss.rms_norm_backward(dy, h, w, rstd, stream=side.cuda_stream if handle else side)
    trash = [torch.full((1 << 20,), float("nan"), device=CUDA) for _ in range(8)]
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    del trash

"""Outputs over the inputs that a call allows, and beside others without a gap:
the same bits as in places of their own."""
import pytest
import torch

import tile_size_selection_amd as tss
import ops_util as U

pytestmark = pytest.mark.gpu

CUDA = torch.device("cuda:0")


def beside(*sizes, dtype):
    """Tensors of these many elements, each a multiple of 16 bytes, that follow each other in memory."""
    buf = torch.empty(sum(sizes), dtype=dtype, device=CUDA)
    return buf.split(list(sizes))


# one workgroup, several, sums of their own launch, bins that are not kept
@pytest.mark.parametrize("n,experts", [(8, 8), (4000, 100), (40000, 64), (40000, 4096), (5000001, 8)])
def test_sort_over_its_choices(n, experts):
    expert = torch.randint(-1, experts + 1, (n, 1), generator=U.gen(1), dtype=torch.int32).to(CUDA)
    want = tss.sort_by_expert(expert, experts)
    row = expert.clone()
    got = tss.sort_by_expert(row, experts, row=row)
    assert got.row is row and all(torch.equal(a, b) for a, b in zip(got, want))
    packed = torch.empty(2 * n + experts, dtype=torch.int32, device=CUDA)
    sizes, row, choice = packed.split([experts, n, n])
    got = tss.sort_by_expert(expert, experts, sizes=sizes, row=row.view(n, 1), choice=choice)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("tokens,top,d", [(67, 3, 64), (130, 9, 136), (35, 5, 256), (40, 4, 512), (20, 9, 4104), (5, 6, 32768)])
def test_rows_gradients_over_their_inputs(tokens, top, d):
    order = tss.sort_by_expert(torch.randint(-1, 7, (tokens, top), generator=U.gen(2)).to(CUDA), 7)
    g = U.gen(3)
    rows, dy = U.normal(g, tokens * top, d).to(torch.bfloat16).to(CUDA), U.normal(g, tokens, d).to(torch.bfloat16).to(CUDA)
    weight = U.normal(g, tokens, top).float().to(CUDA)
    want = tss.combine_rows_backward(dy, rows, order, weight)
    dweight, drows = weight.clone(), rows.clone()
    got = tss.combine_rows_backward(dy, drows, order, dweight, drows=drows, dweight=dweight)
    assert got[0] is drows and got[1] is dweight and torch.equal(drows, want[0]) and torch.equal(dweight, want[1])


def test_rows_beside_each_other():
    tokens, top, d = 40, 3, 64
    order = tss.sort_by_expert(torch.randint(0, 7, (tokens, top), generator=U.gen(4)).to(CUDA), 7)
    x, rows, y = (t.view(-1, d) for t in beside(tokens * d, tokens * top * d, tokens * d, dtype=torch.float32))
    x.copy_(U.normal(U.gen(5), tokens, d))
    assert torch.equal(tss.gather_rows(x, order, out=rows), tss.gather_rows(x.clone(), order))
    assert torch.equal(tss.combine_rows(rows, order, out=y), tss.combine_rows(rows.clone(), order))


def test_overlaps_are_refused():
    order = tss.sort_by_expert(torch.zeros(8, 1, dtype=torch.int64, device=CUDA), 2)
    x = torch.ones(8, 64, device=CUDA)
    for call in (lambda: tss.gather_rows(x, order, out=x), lambda: tss.combine_rows(x, order, out=x),
                 lambda: tss.sort_by_expert(order.row, 2, choice=order.row.view(-1))):
        with pytest.raises(tss.TssError):
            call()
    assert (x == 1).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,d", [(300, 64), (37, 520), (1300, 2056), (20, 8200), (5, 32768), (2000, 264)])
def test_norms_over_their_inputs(rows, d, dtype):
    g = U.gen(6)
    x, r, dy = (U.normal(g, rows, d).to(U.TYPES[dtype]).to(CUDA) for _ in range(3))
    w, b = ((1 + 0.2 * U.normal(g, d)).to(U.TYPES[dtype]).to(CUDA) for _ in range(2))
    want = tss.layer_norm(x, w, b, r, stats=True)
    over = r.clone()
    assert torch.equal(tss.layer_norm(x, w, b, over, out=over).y, want.y)
    a, c = x.clone(), r.clone()
    got = tss.layer_norm(a, w, b, c, out=c, residual_out=a)  # crosswise
    assert torch.equal(c, want.y) and torch.equal(a, want.h)
    same = tss.layer_norm(x, w, b, x)
    twice = x.clone()
    got = tss.layer_norm(twice, w, b, twice, residual_out=twice)
    assert torch.equal(got.y, same.y) and torch.equal(twice, same.h)
    grads = tss.layer_norm_backward(dy, want.h, w, want.mean, want.rstd, r)
    h = want.h.clone()
    got = tss.layer_norm_backward(dy, h, w, want.mean, want.rstd, r, dx=h)
    assert torch.equal(h, grads[0])
    # few rows are added in another order then: each sum is off by at most rows + 3 roundings of its terms' magnitudes
    xhat = (want.h.double() - want.mean.double()[:, None]) * want.rstd.double()[:, None]
    for p, q, terms in ((got[1], grads[1], dy.double() * xhat), (got[2], grads[2], dy.double())):
        assert ((p.double() - q.double()).abs() <= 2 * (rows + 3) * 2.0 ** -24 * terms.abs().sum(0)).all()


def test_clipping_beside_others():
    """The norm and the workspace right behind and before the tensors."""
    values = U.normal(U.gen(7), 300000).float()
    want = values.to(CUDA)
    norm = tss.clip_grad_norm([want[:200000], want[200000:]], 1.0)
    need = 8 * (98 + 49)
    for first in (0, need // 4):
        buf = torch.zeros(300000 + need // 4 + 4, device=CUDA)
        ts = buf[first:first + 300000]
        ts.copy_(values)
        ws = buf[0:need // 4] if first else buf[300000:300000 + need // 4]
        pair = [ts[:200000], ts[200000:]]
        at = buf[300000 + need // 4]
        assert torch.equal(tss.grad_norm(pair, norm=at, workspace=ws), norm)
        tss.clip_grad_norm(pair, 1.0, norm=at, workspace=ws)
        assert torch.equal(ts, want) and torch.equal(at, norm)
        for call in (dict(norm=ts[5]), dict(norm=at, workspace=ts)):
            with pytest.raises(tss.TssError):
                tss.grad_norm(pair, **call)
        assert torch.equal(ts, want)

"""Choices sorted by expert, their rows gathered and joined, and the gradients,
against their definitions on the CPU: whole numbers and copies exactly, sums in
64 bits.

Bounds: a token's sum over `top` rows in fp32 is off by (top + 1) * 2^-24 of
the sum of its terms' magnitudes before its own rounding; a dot product over d
columns adds 8 * 4 columns of a lane in turn, then a tree of 6 and 16 waves: at
most 8 * 4 + 6 + 16 + 1 roundings, 2^-18 of the sum of the magnitudes."""
import pytest
import torch

import tile_size_selection_amd as tss
import ops_util as U

pytestmark = pytest.mark.gpu

CUDA = torch.device("cuda:0")
TYPES = {**U.TYPES, "i8": torch.int8}


def choices(tokens, top, experts, seed, dropped=0.2, dtype=torch.int64):
    g = U.gen(seed)
    e = torch.randint(0, experts, (tokens, top), generator=g)
    out = torch.rand(tokens, top, generator=g)
    e = torch.where(out < dropped / 2, torch.full_like(e, -1), e)
    return torch.where((out >= dropped / 2) & (out < dropped), e + experts, e).to(dtype)


def defined(expert, experts):
    """(sizes, row, choice) by Python's stable sort."""
    flat = expert.reshape(-1).tolist()
    key = [e if 0 <= e < experts else experts for e in flat]
    order = sorted(range(len(flat)), key=key.__getitem__)
    row = [0] * len(flat)
    for place, i in enumerate(order):
        row[i] = place if key[i] < experts else ~place
    sizes = [0] * (experts + 1)
    for k in key:
        sizes[k] += 1
    choice = [i if key[i] < experts else ~i for i in order]
    return sizes[:experts], torch.tensor(row, dtype=torch.int32).view(expert.shape), torch.tensor(choice, dtype=torch.int32)


def check_sorted(order, expert, experts):
    sizes, row, choice = defined(expert, experts)
    assert order.sizes.tolist() == sizes
    assert torch.equal(order.row.cpu(), row) and torch.equal(order.choice.cpu(), choice)


@pytest.mark.parametrize("dtype", [torch.int64, torch.int32])
@pytest.mark.parametrize("tokens,top,experts", [
    (0, 2, 3), (1, 1, 1), (1, 8, 64), (9, 7, 5), (64, 1, 2), (65, 1, 3), (300, 3, 7), (1024, 8, 256), (1025, 8, 100),
    (4096, 2, 4096), (5000, 6, 160), (33, 5, 4096), (20000, 8, 128), (60000, 5, 999), (100000, 4, 4096), (70001, 3, 1)])
def test_sort(tokens, top, experts, dtype):
    expert = choices(tokens, top, experts, 1, dtype=dtype)
    check_sorted(tss.sort_by_expert(expert.to(CUDA), experts), expert, experts)


@pytest.mark.parametrize("n", [77, 9000])
def test_sort_of_extremes(n):
    """All dropped, all of one expert, and the types' largest and smallest numbers."""
    for expert in (torch.full((n, 1), -1), torch.full((n, 1), 5), torch.zeros(n, 1, dtype=torch.int64), torch.full((n, 1), 6),
                   torch.tensor([2 ** 63 - 1, -2 ** 63, 2 ** 32, -2 ** 32, 2 ** 32 + 5, 5, 0] * n)[:n, None].contiguous(),
                   torch.tensor([2 ** 31 - 1, -2 ** 31, 5], dtype=torch.int32).repeat(n)[:n, None].contiguous()):
        check_sorted(tss.sort_by_expert(expert.to(CUDA), 6), expert, 6)


def test_sort_into_given_tensors_and_on_another_stream():
    expert = choices(4000, 5, 40, 2)
    buf = torch.full((40 + 2 * 20000 + 3,), 7, dtype=torch.int32, device=CUDA)
    sizes, row, choice = buf[1:41], buf[41:20041].view(4000, 5), buf[20042:40042]
    stream = torch.cuda.Stream()
    dev = expert.to(CUDA)
    stream.wait_stream(torch.cuda.current_stream())
    order = tss.sort_by_expert(dev, 40, sizes=sizes, row=row, choice=choice, stream=stream)
    torch.cuda.current_stream().wait_stream(stream)
    assert order.row.data_ptr() == row.data_ptr()
    check_sorted(order, expert, 40)
    assert buf[0] == 7 and buf[20041] == 7 and (buf[40042:] == 7).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32", "e4m3", "e5m2", "i8"])
@pytest.mark.parametrize("tokens,top,d", [(1, 1, 8), (1, 8, 2048), (37, 3, 24), (130, 2, 136), (50, 5, 4104), (700, 8, 512)])
def test_gather(tokens, top, d, dtype):
    expert = choices(tokens, top, 9, 3)
    order = tss.sort_by_expert(expert.to(CUDA), 9)
    bits = torch.randint(-128, 128, (tokens, d * TYPES[dtype].itemsize), generator=U.gen(4), dtype=torch.int8)
    x = bits.view(TYPES[dtype])  # any bits, NaN among them
    scale = U.normal(U.gen(5), 3, tokens).float()
    buf = torch.full((tokens * top * d + 16,), 1, device=CUDA).to(TYPES[dtype])
    rows, got = tss.gather_rows(x.to(CUDA), order, scale.to(CUDA), out=buf[:tokens * top * d].view(-1, d))
    want, want_scale = torch.zeros(tokens * top, bits.shape[1], dtype=torch.int8), torch.zeros(3, tokens * top)
    for r, i in enumerate(order.choice.tolist()):
        if i >= 0:
            want[r], want_scale[:, r] = bits[i // top], scale[:, i // top]
    assert torch.equal(rows.view(torch.int8).cpu(), want) and torch.equal(got.cpu(), want_scale)
    assert (buf[tokens * top * d:].float() == 1).all()
    one = tss.gather_rows(x.to(CUDA), order, scale[0].to(CUDA))[1]
    assert torch.equal(one.cpu(), want_scale[0])
    assert torch.equal(tss.gather_rows(x.to(CUDA), order).view(torch.int8).cpu(), want)


@pytest.mark.parametrize("tokens,top,d", [(9000, 8, 4096), (9001, 8, 4104), (70000, 4, 1024), (40000, 7, 1032)])
def test_gather_of_many_bytes(tokens, top, d):
    order = tss.sort_by_expert(choices(tokens, top, 30, 12).to(CUDA), 30)
    x = torch.randint(-128, 128, (tokens, d), generator=U.gen(13), dtype=torch.int8).to(CUDA)
    rows = tss.gather_rows(x, order)
    kept = order.choice >= 0
    assert torch.equal(rows, x[order.choice.clamp(min=0).long() // top] * kept[:, None])


def of_choices(rows, row):
    return torch.where((row >= 0)[..., None], rows.double()[row.clamp(min=0).long()], 0)


def operands(tokens, top, d, rows_type, seed, experts=7):
    """(order, rows, weight): NaN where nothing may be read."""
    order = tss.sort_by_expert(choices(tokens, top, experts, seed).to(CUDA), experts)
    g = U.gen(seed + 1)
    rows = U.normal(g, tokens * top, d).to(TYPES[rows_type])
    rows[order.choice.cpu() < 0] = float("nan")
    weight = U.normal(g, tokens, top).float()
    return order, rows, torch.where(order.row.cpu() < 0, float("nan"), weight)


PAIRS = [("bf16", "bf16"), ("f16", "f16"), ("f32", "f32"), ("f32", "bf16"), ("f32", "f16"), ("bf16", "f32"), ("f16", "f32")]


@pytest.mark.parametrize("rows_type,out", PAIRS)
@pytest.mark.parametrize("tokens,top,d", [(1, 1, 8), (3, 9, 24), (70, 4, 520), (260, 3, 264), (40, 6, 4104), (5, 17, 2056)])
def test_combine(tokens, top, d, rows_type, out):
    order, rows, weight = operands(tokens, top, d, rows_type, 6)
    row = order.row.cpu()
    half, low = U.half_step(out)
    for w in (weight, None):
        got = tss.combine_rows(rows.to(CUDA), order, None if w is None else w.to(CUDA), out)
        terms = of_choices(rows, row) * (1 if w is None else torch.where(row < 0, 0, w.double())[..., None])
        want, size = terms.sum(1), terms.abs().sum(1)
        assert got.dtype == TYPES[out]
        assert ((got.double().cpu() - want).abs() <= want.abs() * half + size * (top + 1) * 2.0 ** -24 + low).all()
    assert torch.equal(got, tss.gather_rows_backward(rows.to(CUDA), order, out))


@pytest.mark.parametrize("rows_type,dtype", [("bf16", "bf16"), ("f16", "f16"), ("f32", "f32"), ("f32", "bf16"), ("f32", "f16")])
@pytest.mark.parametrize("tokens,top,d", [(1, 1, 8), (67, 3, 64), (130, 2, 136), (35, 5, 256), (40, 4, 512), (20, 9, 4104),
                                          (6, 3, 8200), (5, 5, 16384), (3, 6, 32768)])
def test_combine_backward(tokens, top, d, rows_type, dtype):
    order, rows, weight = operands(tokens, top, d, rows_type, 8)
    dy = U.normal(U.gen(9), tokens, d).to(TYPES[dtype])
    drows, dweight = tss.combine_rows_backward(dy.to(CUDA), rows.to(CUDA), order, weight.to(CUDA))
    row = order.row.cpu()
    place = torch.where(row < 0, ~row, row).long()
    want = torch.zeros(tokens * top, d, dtype=torch.float64)
    want[place.view(-1)] = (torch.where(row < 0, 0, weight.double())[..., None] * dy.double()[:, None]).view(-1, d)
    half, low = U.half_step(dtype)
    assert ((drows.double().cpu() - want).abs() <= want.abs() * (half + 2.0 ** -24) * (1 + half) + 2 * low).all()
    terms = of_choices(rows, row) * dy.double()[:, None]
    assert ((dweight.double().cpu() - terms.sum(2)).abs() <= terms.abs().sum(2) * 2.0 ** -18).all()
    assert (dweight.cpu()[row < 0] == 0).all()
    again = tss.combine_rows_backward(dy.to(CUDA), rows.to(CUDA), order, weight.to(CUDA))
    assert torch.equal(again[0], drows) and torch.equal(again[1], dweight)
    if rows_type == dtype:  # the rows' gradients over the rows
        place = rows.to(CUDA)
        got = tss.combine_rows_backward(dy.to(CUDA), place, order, weight.to(CUDA), drows=place)
        assert torch.equal(got[0], drows) and torch.equal(got[1], dweight)


def test_gradients_are_differences():
    """<dy, combine> is linear in the rows and in the weights apart: a step of
    any size in one gives its gradient's product with the step."""
    tokens, top, d = 30, 3, 264
    order, rows, weight = operands(tokens, top, d, "f32", 10)
    rows, weight = rows.nan_to_num(0.0), weight.nan_to_num(0.0)
    g = U.gen(11)
    dy, vr, vw = U.normal(g, tokens, d), U.normal(g, tokens * top, d), U.normal(g, tokens, top)
    drows, dweight = tss.combine_rows_backward(dy.float().to(CUDA), rows.to(CUDA), order, weight.to(CUDA))

    def value(r, w):
        return float((dy.float().double() * tss.combine_rows(r.float().to(CUDA), order, w.float().to(CUDA)).double().cpu()).sum())
    # terms of size ~3, of which tokens * top * d add at random: roundings of 2^-24 each stay below 1e-5 of the sum's spread
    spread = (tokens * top * d) ** 0.5
    by_rows = value(rows + vr.float(), weight) - value(rows, weight)
    assert abs(by_rows - float((drows.double().cpu() * vr.float().double()).sum())) <= 1e-5 * spread
    by_weight = value(rows, weight + vw.float()) - value(rows, weight)
    assert abs(by_weight - float((dweight.double().cpu() * vw.float().double()).sum())) <= 1e-5 * spread
    dx = tss.gather_rows_backward(drows, order)
    x, vx = U.normal(g, tokens, d).float(), U.normal(g, tokens, d).float()
    moved = tss.gather_rows((x + vx).to(CUDA), order).double().cpu() - tss.gather_rows(x.to(CUDA), order).double().cpu()
    assert abs(float((moved * drows.double().cpu()).sum()) - float((dx.double().cpu() * vx.double()).sum())) <= 1e-5 * spread


def test_indices_past_the_rows_are_not_followed():
    order, rows, weight = operands(20, 4, 264, "bf16", 12)
    rows, weight = rows.nan_to_num(0.0).to(CUDA), weight.nan_to_num(0.0).to(CUDA)
    bad = order.row.clone()
    bad[3, 1], bad[7, 0], bad[9, 2], bad[11, 3] = 80, 2 ** 31 - 1, -81, -2 ** 31
    choice = order.choice.clone()
    choice[5], choice[6], choice[7] = 80, 2 ** 31 - 1, -2 ** 31
    wrong = tss.ExpertOrder(order.sizes, bad, choice)
    zero = torch.where((bad >= 80) | (bad < -80), 0, 1).bool()
    x = U.normal(U.gen(13), 20, 264).to(torch.bfloat16).to(CUDA)
    out = torch.full((80, 264), 5.0, dtype=torch.bfloat16, device=CUDA)
    got, scale = tss.gather_rows(x, wrong, torch.ones(20, device=CUDA), out=out)
    for i, r in enumerate(order.row.view(-1).tolist()):
        want = 5.0 if not zero.view(-1)[i] else x[i // 4] if r >= 0 else 0.0
        assert (got[r if r >= 0 else ~r] == want).all()
    assert (scale[5:8] == 0).all()
    y = tss.combine_rows(rows, wrong, weight)
    kept = torch.where(zero.cpu(), order.row.cpu(), -1)
    terms = of_choices(rows.cpu(), kept) * weight.cpu().double()[..., None]
    assert ((y.double().cpu() - terms.sum(1)).abs() <= terms.abs().sum(1) * (2.0 ** -8 + 5 * 2.0 ** -24)).all()
    drows = torch.full((80, 264), 5.0, dtype=torch.bfloat16, device=CUDA)
    _, dweight = tss.combine_rows_backward(x, rows, wrong, weight, drows=drows)
    assert (dweight[~zero] == 0).all()
    untouched = torch.where(order.row < 0, ~order.row, order.row)[~zero].long()
    assert (drows[untouched] == 5).all()


def test_a_captured_run_follows_its_inputs():
    """Sorted, gathered, joined, and the gradients in one graph: replays on new
    choices, with eager calls between them, give what eager calls give."""
    tokens, top, experts, d = 3000, 4, 50, 264
    g = U.gen(14)
    expert = choices(tokens, top, experts, 15).to(CUDA)
    x, dy = (U.normal(g, tokens, d).to(torch.bfloat16).to(CUDA) for _ in range(2))
    weight = torch.softmax(U.normal(g, tokens, top), 1).float().to(CUDA)

    def run():
        order = tss.sort_by_expert(expert, experts)
        rows = tss.gather_rows(x, order)
        y = tss.combine_rows(rows, order, weight)
        drows, dweight = tss.combine_rows_backward(dy, rows, order, weight)
        return [*order, rows, y, drows, dweight, tss.gather_rows_backward(drows, order)]

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        run()
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = run()
    for seed in range(4):
        expert.copy_(choices(tokens, top, experts, 20 + seed, dropped=0.1 * seed))
        x.copy_(U.normal(U.gen(30 + seed), tokens, d))
        graph.replay()
        want = run()
        torch.cuda.synchronize()
        for a, b in zip(held, want):
            assert torch.equal(a, b)


def test_two_streams_at_once_and_given_workspaces():
    """Sorts on two streams overlap, each with its own workspace; a short one is refused."""
    experts = [choices(20000, 8, 128, 40 + i) for i in range(2)]
    dev = [e.to(CUDA) for e in experts]
    streams = [torch.cuda.Stream() for _ in range(2)]
    spaces = [torch.empty(1 << 20, dtype=torch.uint8, device=CUDA) for _ in range(2)]
    orders = []
    for turn in range(3):
        for i in range(2):
            streams[i].wait_stream(torch.cuda.current_stream())
            orders.append((i, tss.sort_by_expert(dev[i], 128, workspace=spaces[i] if turn else None, stream=streams[i])))
    torch.cuda.synchronize()
    want = [defined(e, 128) for e in experts]
    for i, o in orders:
        assert o.sizes.tolist() == want[i][0] and torch.equal(o.row.cpu(), want[i][1]) and torch.equal(o.choice.cpu(), want[i][2])
    with pytest.raises(ValueError):
        tss.sort_by_expert(dev[0], 128, workspace=torch.empty(64, dtype=torch.uint8, device=CUDA))


def test_rows_past_32_bit_offsets():
    """More than 2^32 bytes and 2^31 elements of rows: the last token's go where the first's do."""
    tokens, top, d = 70001, 4, 8192
    expert = choices(tokens, top, 16, 50)
    order = tss.sort_by_expert(expert.to(CUDA), 16)
    x = torch.zeros(tokens, d, dtype=torch.float16, device=CUDA)
    tail = U.normal(U.gen(51), 50, d).to(torch.float16).to(CUDA)
    x[-50:] = tail
    rows = tss.gather_rows(x, order)
    row = order.row[-50:].long()
    kept = (row >= 0)[..., None]
    assert torch.equal(rows[row.clamp(min=0)] * kept, (tail[:, None] * kept))
    weight = torch.ones(tokens, top, device=CUDA)
    y = tss.combine_rows(rows, order, weight)
    n = kept.sum(1)
    assert torch.equal(y[-50:], (tail.float() * n).half()) and (y[:-50] == 0).all()
    drows, dweight = tss.combine_rows_backward(x, rows, order, weight)
    assert torch.equal(drows, rows)
    want = (tail.double().square().sum(1)[:, None] * kept[..., 0]).cpu()
    assert ((dweight[-50:].double().cpu() - want).abs() <= want * 2.0 ** -18).all() and (dweight[:-50] == 0).all()

"""The expert layer's routing, on the CPU."""
import torch

from tile_size_selection_amd import expert_layer as X


def test_rows_are_sorted_by_expert_and_dropped_choices_come_last():
    expert = torch.tensor([[2, 0], [-1, 1], [0, 3], [1, -1]])  # of 3 experts
    weight = torch.arange(1.0, 9.0).view(4, 2)
    r = X.route(expert, weight, 3)
    assert r.sizes.tolist() == [2, 2, 1] and r.sizes.dtype == torch.int32
    assert r.token.tolist() == [0, 2, 1, 3, 0, 1, 2, 3]
    assert r.weight.tolist() == [2, 5, 4, 7, 1, 3, 6, 8]
    assert (r.token[r.row] == torch.arange(4)[:, None]).all() and torch.equal(r.weight[r.row], weight)
    rows = torch.arange(8.0)[:, None]
    assert torch.equal(X.join(rows, r), rows[r.row].sum(1))


def test_no_tokens():
    r = X.route(torch.empty(0, 2, dtype=torch.int64), torch.empty(0, 2), 3)
    assert r.sizes.tolist() == [0, 0, 0] and r.row.shape == (0, 2)
    assert X.join(torch.empty(0, 5), r).shape == (0, 5)

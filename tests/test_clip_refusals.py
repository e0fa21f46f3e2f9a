"""What the clipping calls refuse of lists that hold other things than tensors."""
import pytest
import torch

import tile_size_selection_amd as tss

T = torch.zeros(4)


@pytest.mark.parametrize("call", [
    lambda: tss.clip_grad_norm([None], 1.0), lambda: tss.grad_norm([None]), lambda: tss.clip_grad_norm([1.0], 1.0),
    lambda: tss.clip_grad_norm([T], 1.0, out=[None]), lambda: tss.clip_grad_norm([None, T], 1.0, out=[T, T]),
    lambda: tss.clip_grad_norm([None], 1.0, norm=T[0])])
def test_what_is_no_tensor(call):
    with pytest.raises(ValueError):
        call()

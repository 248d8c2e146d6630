"""The decode-step operators on the CPU where they can go wrong between the
cases of the other host tests."""
import pytest

import sparse_weight_only_amd as sg

torch = pytest.importorskip("torch")


def ints(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def test_a_mask_table_without_masks_is_refused():
    """An empty tensor's address is null, which the library takes for no masks."""
    for kw in (dict(masks=ints(0, 2)), dict(masks=ints(0, 2), mask_row=ints(2))):
        with pytest.raises(ValueError, match="no mask"):
            sg.adjust_logits(torch.zeros(2, 50), **kw)

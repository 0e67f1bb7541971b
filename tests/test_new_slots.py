"""The slots of new tokens (fp8_layer.new_slots), on the CPU."""
import pytest
import torch

from routed_moe_decode_router_gb300 import fp8_layer


@pytest.mark.parametrize("counts,want", [
    (None, [[14, 15, 16], [-1, -1, -1], [-1, -1, 80]]), ([3, 3, 3], [[14, 15, 16], [-1, -1, -1], [-1, -1, 80]]),
    ([2, 0, 1], [[-1, 15, 16], [-1, -1, -1], [-1, -1, 80]]), ([9, 1, 0], [[14, 15, 16], [-1, -1, -1], [-1, -1, -1]])])
def test_slots(counts, want):
    table = torch.tensor([[0, 1], [2, 3], [5, 4]], dtype=torch.int32)
    lengths = torch.tensor([17, 0, 1], dtype=torch.int32)
    counts = None if counts is None else torch.tensor(counts, dtype=torch.int32)
    assert fp8_layer.new_slots(table, lengths, 3, 16, counts).tolist() == want


@pytest.mark.parametrize("shape", [(3, 1), (1,), (1, 3), (2,), ()])
def test_counts_of_another_shape_are_refused(shape):
    table = torch.zeros(3, 2, dtype=torch.int32)
    lengths = torch.ones(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="counts has shape"):
        fp8_layer.new_slots(table, lengths, 3, 16, torch.ones(shape, dtype=torch.int32))

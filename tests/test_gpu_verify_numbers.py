"""GPU tests of the verification's arithmetic at its borders."""
import math

import pytest
import torch

from routed_moe_decode_router_gb300 import ops

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    yield
    assert ops.device_status() == 0


@pytest.mark.parametrize("p,q,u,kept", [
    (0.25, math.nan, 0.5, True), (0.0, math.nan, 0.0, False),     # NaN counts as 0
    (0.0, -1.0, 0.5, False), (-0.4, -1.0, 0.5, False), (0.25, -math.inf, 0.5, True),
    (0.8, 1.5, 0.75, True), (0.7, 1.5, 0.75, False), (0.8, math.inf, 0.75, True),   # more as 1
    (7.0, 7.0, 0.5, True), (math.inf, math.inf, 0.5, True), (math.nan, 0.0, 0.0, False),
    (0.5, 1.0, 0.5, False), (0.5, 0.5, 1 - 2.0 ** -24, True)])
def test_drafts_of_numbers_that_are_no_probabilities(p, q, u, kept):
    """They count in the acceptance as they do in the draw."""
    target, draft_probs = torch.full((1, 2, 9), 0.125), torch.full((1, 1, 9), 0.125)
    target[0, 0, 4], draft_probs[0, 0, 4] = p, q
    r = ops.verify_draft(torch.tensor([[4]], dtype=torch.int32, device="cuda"), target.cuda(),
                         torch.tensor([[u]], device="cuda"), torch.tensor([0.0], device="cuda"),
                         draft_probs=draft_probs.cuda())
    assert r.accepted.tolist() == [int(kept)]
    assert (r.tokens[0, 0] == 4) == kept

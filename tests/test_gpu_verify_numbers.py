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


def steps(n):
    """A number of steps of 2^-44 as weights that fp32 holds, the largest first."""
    out = []
    while n:
        top = n >> max(0, n.bit_length() - 24) << max(0, n.bit_length() - 24)
        out.append(top * 2.0 ** -44)
        n -= top
    return out


@pytest.mark.parametrize("m", [0xFFFFFF, 0xABCDEF, 0x800001, 0xD00DAD])
@pytest.mark.parametrize("low", [0, 5])
def test_a_number_just_below_a_running_sum(m, low):
    """u times the whole sum is a 2^-24th (or less) of a step below a running sum, less
    than 64 bits of floating point tell apart there: that sum exceeds it."""
    u = m * 2.0 ** -(24 + low)
    one = 1 << (24 + low)
    # the whole sum t near 2^44 with m t = -1 modulo one: k = (m t + 1) / one steps
    t = (1 << 44) - one + (-pow(m, -1, one)) % one
    k, rest = divmod(m * t + 1, one)
    assert rest == 0 and math.floor(u * float(t)) == k and m * t // one == k - 1
    head, tail = steps(k), steps(t - k)
    target = torch.tensor(head + tail, dtype=torch.float64)
    assert torch.equal(target.float().double(), target)
    target = target.float().cuda().view(1, 1, -1)
    none = torch.empty(1, 0, device="cuda")
    r = ops.verify_draft(none.int(), target, none, torch.tensor([u], device="cuda"))
    assert r.tokens.tolist() == [[len(head) - 1]]


@pytest.mark.parametrize("u", [0.0, -0.0, 1e-45, 2.0 ** -126, 2.0 ** -45, 2.0 ** -44, 2.0 ** -43, 1e-9])
def test_small_numbers(u):
    """Ids of one step of 2^-44 each, and one of all the rest."""
    target = torch.full((1, 1, 40), 2.0 ** -44)
    target[0, 0, 39] = 0.75
    total = sum(round(float(x) * 2 ** 44) for x in target[0, 0])
    none = torch.empty(1, 0, device="cuda")
    given = torch.tensor([u], dtype=torch.float32)
    num, den = float(given[0]).as_integer_ratio()
    r = ops.verify_draft(none.int(), target.cuda(), none, given.cuda())
    assert r.tokens.tolist() == [[min(num * total // den, 39)]]

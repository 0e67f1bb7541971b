"""GPU tests of the routed experts' sums over the slots: products that nearly
cancel show in how many bits they are held until they are added."""
import pytest
import torch

from routed_moe_decode_router_gb300 import ops
from tests import ops_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    yield
    assert ops.device_status() == 0


def randn(*shape, seed=0, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(2000 + seed)
    return torch.randn(*shape, generator=g, device="cuda") * std


def stack(*ws):
    qs = [R.weights_fp8(w) for w in ws]
    return torch.stack([q.view(torch.uint8) for q, _ in qs]).view(ops.F8), torch.stack(
        [s for _, s in qs])


# Few pairs; more of them, up to and beyond 2^20 products; many tiles.
@pytest.mark.parametrize("t,hidden,inter", [
    (1, 256, 128), (16, 512, 384), (17, 512, 384), (512, 1024, 128), (513, 1024, 128),
    (700, 2048, 256), (3000, 384, 128)])
def test_slots_that_nearly_cancel(t, hidden, inter):
    """Expert 1 is expert 0 with down scales larger by 2^-5, and its weight is
    the negative: what is left is 2^-5 of a product, so a product rounded to 8
    bits would leave an error of an eighth of it.

    The codes of h are the same in both slots.  So a code of h that falls on
    the other side of a border moves the result by 2^-5 of its own part, and
    the bound is that of one expert with the difference of the scales, plus
    the two products' own fp32 sums."""
    gate, up = randn(inter, hidden, std=0.05), randn(inter, hidden, seed=1, std=0.05)
    gate, gs = stack(gate, gate)
    up, us = stack(up, up)
    down, ds = stack(*[randn(hidden, inter, seed=2, std=0.05)] * 2)
    # scales of 12 bits, so that the larger ones are exact
    ds = (ds.view(torch.int32) & -4096).view(torch.float32)
    ds[1] = ds[0] + ds[0] / 32
    q, s = R.rows_fp8(randn(t, hidden, seed=3))
    ids = torch.tensor([[0, 1]] * t, dtype=torch.int32, device="cuda")
    wts = torch.tensor([[1.0, -1.0]] * t, device="cuda")
    got = ops.experts_fp8(q, s, ids, wts, gate, gs, up, us, down, ds).double()

    one = torch.zeros_like(ids[:, :1])
    want, bound = R.experts(q, s, one, wts[:, :1], gate[:1], gs[:1], up[:1], us[:1], down[:1],
                            ds[:1] - ds[1:])
    g, _ = R.product(q, s, gate[0], gs[0])
    u, _ = R.product(q, s, up[0], us[0])
    h = (g / (1 + torch.exp(-g)) * u).abs()
    sc = h.view(t, -1, 128).amax(2).clamp(min=1e-30) / 448.0
    h = h * (1 + 2.0 ** -4) + R.expand_rows(sc, inter) * 2.0 ** -10     # the code's value, at most
    mag = h @ (R.wide_weights(down[0], ds[0]).abs() + R.wide_weights(down[1], ds[1]).abs()).T
    # each product's sum, and its rounding to fp32 and at the weighted sum
    bound = bound + mag * (R.product_bound(inter) + 2 * R.U) * (1 + R.half_step(torch.bfloat16))
    bad = ~((got - want).abs() <= bound)
    assert not bad.any(), "%d of %d, worst %.3g x its bound" % (
        int(bad.sum()), bad.numel(), float(((got - want).abs() / bound).max()))

"""GPU tests of the FP8 layer's forms: a router in fp32, a shared expert without
a gate."""
import pytest
import torch

from routed_moe_decode_router_gb300 import fp8_layer, ops
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
    g = torch.Generator(device="cuda").manual_seed(4000 + seed)
    return torch.randn(*shape, generator=g, device="cuda") * std


def within(got, want, bound):
    bad = ~((got.double() - want).abs() <= bound)
    assert not bad.any(), "%d of %d, worst %.3g x its bound" % (
        int(bad.sum()), bad.numel(), float(((got.double() - want).abs() / bound).max()))


@pytest.mark.parametrize("rows", [1, 7, 65])
@pytest.mark.parametrize("shared", [0, 384])
def test_router_in_fp32(rows, shared):
    """The logits are those of the unquantised matrix, and decide the experts."""
    lay = fp8_layer.random_layer(512, 16, 256, 4, seed=3, shared_inter=shared, router_fp8=False)
    x, r = randn(rows, 512).to(torch.bfloat16), randn(rows, 512, seed=1).to(torch.bfloat16)
    n = ops.rms_norm(x, lay.norm, residual=r, quantize=True)
    assert lay.router.dtype == torch.float32 and lay.router.shape == (16 + (shared > 0), 512)
    logits = lay.logits(n)
    y, w = n.y.double(), lay.router.double()
    # 512 products and their additions, each one step of fp32 at most
    within(logits, y @ w.T, y.abs() @ w.abs().T * 1024 * R.U)
    out, res = lay.forward(x, r)
    assert torch.equal(res, n.residual)
    ids, wts = ops.route_topk(logits[:, :16], 4)
    assert torch.equal(ids.cpu(), R.route(logits[:, :16], 4)[0])
    add = None
    if shared:
        one = torch.zeros_like(ids[:, :1])
        add = ops.experts_fp8(n.q, n.scales, one, torch.sigmoid(logits[:, 16:]), *lay.shared)
    want, bound = R.experts(n.q, n.scales, ids, wts, *lay.routed, addend=add)
    if shared:      # the gate within 8 steps, so another step of the shared output's bf16
        bound = bound + add.double().abs() * 2 * R.half_step(torch.bfloat16)
    within(out, want, bound)
    # the same experts' weights behind the router in FP8: its logits differ
    eight = fp8_layer.random_layer(512, 16, 256, 4, seed=3, shared_inter=shared)
    assert (eight.logits(n).double() - y @ w.T).abs().max() > 1e-3


@pytest.mark.parametrize("rows", [1, 5, 70])
@pytest.mark.parametrize("router_fp8", [True, False])
def test_shared_expert_without_a_gate(rows, router_fp8):
    lay = fp8_layer.random_layer(512, 16, 256, 4, seed=3, shared_inter=384, shared_gated=False,
                                 router_fp8=router_fp8, scoring="sigmoid", groups=4, group_limit=2,
                                 group_score="top2")
    x = randn(rows, 512).to(torch.bfloat16)
    n = ops.rms_norm(x, lay.norm, quantize=True)
    logits = lay.logits(n)
    assert logits.shape == (rows, 16)
    ids, wts = ops.route_topk(logits, 4, bias=lay.bias, **lay.routing)
    one = torch.zeros_like(ids[:, :1])
    shared, sb = R.experts(n.q, n.scales, one, torch.ones_like(wts[:, :1]), *lay.shared)
    want, bound = R.experts(n.q, n.scales, ids, wts, *lay.routed)
    # the shared output is rounded once more on its way, the sum once
    total = bound + sb + shared.abs() * R.half_step(torch.bfloat16)
    total = total + (want + shared).abs() * R.half_step(torch.bfloat16)
    out, res = lay.forward(x)
    assert res is x
    within(out, want + shared, total)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        again, _ = lay.forward(x)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(again, out)


def test_gate_without_a_shared_expert_is_refused():
    lay = fp8_layer.random_layer(256, 8, 128, 2)
    w = fp8_layer.Fp8Weights
    parts = [w(*lay.routed[i:i + 2]) for i in (0, 2, 4)]
    with pytest.raises(ValueError, match="without shared"):
        fp8_layer.Fp8MoeLayer(lay.norm, randn(8, 256), *parts, 2, shared_gate=randn(256))

"""GPU tests of the norm's e4m3 codes: each is the nearest e4m3 to the normed
value over its scale.  Rows of fp32 return the normed values unrounded, so the
codes can be compared one by one."""
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


def codes(y, scales):
    return (y / scales.repeat_interleave(128, 1)[:, :y.shape[1]]).to(ops.F8).view(torch.uint8)


# Large enough that a quotient 1.5 steps of fp32 off shows, some 10^-5 of them.
@pytest.mark.parametrize("rows,hidden", [(100, 8192), (2048, 4096), (8000, 1000), (4001, 2048),
                                         (1001, 12000)])
def test_codes_are_the_nearest(rows, hidden):
    g = torch.Generator(device="cuda").manual_seed(rows)
    x = torch.randn(rows, hidden, generator=g, device="cuda")
    x = x * torch.exp(torch.randn(hidden, generator=g, device="cuda"))
    w = 1.0 + 0.1 * torch.randn(hidden, generator=g, device="cuda")
    out = ops.rms_norm(x, w, residual=x.flip(0), quantize=True)
    assert torch.equal(out.q.view(torch.uint8), codes(out.y, out.scales))


def test_codes_beside_an_infinity_and_of_the_least_scale():
    w = torch.ones(256, device="cuda")
    w[5] = math.inf
    x = torch.ones(3, 256, device="cuda")
    x[1] = 0.0
    x[1, 200] = 1e-37
    out = ops.rms_norm(x, w, eps=1e-6, quantize=True)
    assert out.scales[0, 0] == math.inf and out.scales[1, 1] == out.scales.new_tensor(1e-30) / 448
    got = out.q.float()
    assert got[0, 5].isnan() and got[0, :5].eq(0).all() and got[0, 6:128].eq(0).all()
    assert got[0, 128:].eq(448).all() and got[1, 5].isnan()     # 0 times infinity
    assert got[1, 128:200].eq(0).all() and got[1, 201:].eq(0).all()
    # 1e-37 / sqrt(eps) over the least scale: 0.0448, between 11 and 12 steps of 2^-8
    assert got[1, 200] == 11 * 2.0 ** -8

"""GPU tests of the attention layer (fp8_layer) for the batches that a server runs:
none, and sequences with fewer new tokens than others."""
import pytest
import torch

from routed_moe_decode_router_gb300 import fp8_layer, ops
from tests.ops_ref import F8

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    yield
    assert ops.device_status() == 0


@pytest.mark.parametrize("residual", [False, True])
def test_no_sequences(residual):
    lay = fp8_layer.random_attention(256, 8, 2, 64, seed=1)
    cache = ops.new_kv_cache(3, 2, 16, 64)
    x = torch.empty(0, 2, 256, dtype=BF, device="cuda")
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    out, res = lay.forward(x, cache, none.view(0, 1), none, residual=x if residual else None)
    assert out.shape == res.shape == (0, 2, 256) and out.dtype == res.dtype == BF

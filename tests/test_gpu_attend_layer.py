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


def test_slots_of_some_of_the_rows():
    table = torch.tensor([[5, 2, -1], [7, 7, 7], [1, 0, 3]], dtype=torch.int32)
    lengths, counts = (torch.tensor(x, dtype=torch.int32) for x in ([20, 2, 49], [1, 4, 3]))
    got = fp8_layer.new_slots(table, lengths, 4, 16, counts)
    assert got.tolist() == [[-1, -1, -1, 35], [-1, -1, 112, 113], [-1, 62, 63, -1]]
    assert fp8_layer.new_slots(table, lengths, 4, 16, counts * 0).tolist() == [[-1] * 4] * 3


@pytest.mark.parametrize("dtype", [F8, BF])
def test_sequences_with_fewer_new_tokens_than_rows(dtype):
    """What the cache holds of the tokens before the new ones stays as it is."""
    heads, kv, dim, hidden, rows, page = 8, 2, 64, 256, 4, 16
    lay = fp8_layer.random_attention(hidden, heads, kv, dim, seed=1)
    g = torch.Generator(device="cuda").manual_seed(5)
    table = torch.arange(12, dtype=torch.int32, device="cuda").view(4, 3)
    cache = ops.new_kv_cache(12, kv, page, dim, dtype)
    old = torch.randn(12 * page, 2, kv, dim, generator=g, device="cuda").to(BF)
    ops.kv_write(cache, old[:, 0], old[:, 1], torch.arange(12 * page, dtype=torch.int32, device="cuda"))
    before = [None if t is None else t.clone() for t in cache]
    lengths = torch.tensor([40, 3, 17, 0], dtype=torch.int32, device="cuda")
    counts = torch.tensor([1, 3, 4, 0], dtype=torch.int32, device="cuda")
    x = torch.randn(4, rows, hidden, generator=g, device="cuda").to(BF)
    out, _ = lay.forward(x, cache, table, lengths, counts=counts)
    n = ops.rms_norm(x.flatten(0, 1), lay.norm, quantize=True)
    qkv = ops.matmul_fp8(n.q, n.scales, *lay.qkv).view(4, rows, -1, dim)
    again = ops.KvCache(*before)
    at = [(b, r) for b in range(4) for r in range(rows - int(counts[b]), rows)]
    slots = torch.tensor([int(table[b, (int(lengths[b]) - rows + r) // page]) * page +
                          (int(lengths[b]) - rows + r) % page for b, r in at], dtype=torch.int32, device="cuda")
    new = torch.stack([qkv[b, r] for b, r in at])
    ops.kv_write(again, new[:, heads:heads + kv].contiguous(), new[:, heads + kv:].contiguous(), slots)
    for a, b in zip(cache, again):
        assert a is b is None or torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    a = ops.attend_paged(qkv[:, :, :heads], again, table, lengths)
    assert torch.equal(out.flatten(0, 1), torch.mm(a.view(4 * rows, -1), lay.out.t()))

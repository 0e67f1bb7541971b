"""GPU tests of the attention over an e4m3 cache whose value scales are at the ends
of what a cache may hold."""
import pytest
import torch

from routed_moe_decode_router_gb300 import ops
from tests import decode_ref as D
from tests.ops_ref import F8, half_step

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    yield
    assert ops.device_status() == 0


def made(lengths, heads, dim, seed=0):
    """(cache in e4m3, table, lengths) of sequences on pages of 16."""
    g = torch.Generator(device="cuda").manual_seed(7000 + seed)
    counts = [-(-n // 16) for n in lengths]
    pages = sum(counts) + 1
    ids = torch.randperm(pages, generator=g, device="cuda").int()
    table = torch.full((len(lengths), max(counts)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(counts):
        table[b, :n] = ids[at:at + n]
        at += n
    (k, ks), (v, vs) = (D.kv_codes(torch.randn(pages, heads, 16, dim, generator=g, device="cuda"))
                        for _ in range(2))
    return ops.KvCache(k, v, ks, vs), table, torch.tensor(lengths, dtype=torch.int32, device="cuda"), g


# sequences that a warp has whole, and ones that many share
LENGTHS = [[300 + i % 40 for i in range(1000)], [700, 3, 1500]]


@pytest.mark.parametrize("lengths", LENGTHS)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("size", [2.0 ** -108, 2.0 ** -120])
def test_values_near_the_least_numbers(lengths, dim, size):
    """Values of 1e-30 and less, which bf16 still holds in full; all tokens weigh alike."""
    cache, table, n, g = made(lengths, 2, dim)
    cache.v_scales.copy_(torch.rand(cache.v_scales.shape, generator=g, device="cuda") * size + size)
    q = (torch.randn(len(lengths), 1, 4, dim, generator=g, device="cuda") * 1e-3).to(BF)
    want, bound = D.attend(q, cache, table, n)
    got = ops.attend_paged(q, cache, table, n).double()
    assert want.abs().mean() > 2.0 ** -120 and ((got - want).abs() <= bound).all()


@pytest.mark.parametrize("lengths", LENGTHS)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_scales_of_either_sign(lengths, dim, dtype):
    """A value is code * scale, whatever the scale's sign."""
    cache, table, n, g = made(lengths, 2, dim, seed=1)
    q = torch.randn(len(lengths), 1, 8, dim, generator=g, device="cuda").to(dtype)
    for s in (cache.k_scales, cache.v_scales):
        s.mul_(torch.where(torch.rand(s.shape, generator=g, device="cuda") < 0.4, -1.0, 1.0))
    want, _ = D.attend(q, cache, table, n)
    # the bound counts magnitudes, and half a step of its own output
    _, bound = D.attend(q, cache._replace(v_scales=cache.v_scales.abs()), table, n)
    got = ops.attend_paged(q, cache, table, n).double()
    assert ((got - want).abs() <= bound + want.abs() * half_step(dtype) * 1.01).all()


@pytest.mark.parametrize("dtype", [BF, HF, torch.float32])
def test_written_rows_with_nan_and_infinities(dtype):
    """A NaN leaves its row's scale to the others; an infinity makes all of its row NaN."""
    cache = ops.new_kv_cache(1, 2, 16, 64)
    x = torch.randn(3, 2, 64, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").to(dtype)
    clean = x.clone()
    x[0, 1, 5], x[1, 0, 63] = float("nan"), -float("inf")
    clean[0, 1, 5] = 0
    # (divided in 64 bits: PyTorch's GPU division by a number is a product with its inverse)
    scales = (clean.double().abs().amax(-1) / 448).float()
    want = (clean.double() / scales.double().unsqueeze(-1)).float().to(F8).float() * scales.unsqueeze(-1)
    want[0, 1, 5], want[1, 0] = float("nan"), float("nan")
    slots = torch.arange(3, dtype=torch.int32, device="cuda")
    ops.kv_write(cache, x, x, slots)
    for got in ops.kv_read(cache, slots, dtype=torch.float32):
        assert torch.equal(got.isnan(), want.isnan())
        assert torch.equal(got.nan_to_num(0.0), want.nan_to_num(0.0))

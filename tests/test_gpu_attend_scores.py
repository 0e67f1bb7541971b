"""GPU tests of the attention with scores so large that their own steps are more than
what the running maximum leaves open."""
import math

import pytest
import torch

from routed_moe_decode_router_gb300 import ops
from tests.ops_ref import F8, half_step

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16
TYPES = [(F8, BF), (F8, HF), (BF, BF), (HF, HF)]


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    yield
    assert ops.device_status() == 0


def scale_of(e):
    """A number of 32 bits that times log2 of Euler's number is 2^e in 32 bits."""
    s = torch.tensor(2.0 ** e / math.log2(math.e), dtype=torch.float32)
    for way in (0.0, math.inf):
        for t in (s, torch.nextafter(s, torch.tensor(way))):
            if float(torch.tensor(float(t) * 1.4426950408889634).float()) == 2.0 ** e:
                return float(t)
    raise AssertionError


# what is added to 2^23 in the scores of 32 tokens after the other
STAIRS = [[0, 1, 2, 3], [3, 2, 1, 0], [1, 2, 0, 3], [0, 8, 16, 18], [1, 9, 2, 3], [0, 0, 1, 1], [5, 4, 6, 7]]


@pytest.mark.parametrize("held,dtype", TYPES)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("e", [-3, 0, 1, 2, 3, 4, 5, 6, 40])
@pytest.mark.parametrize("spread", [False, True])
def test_scores_of_large_steps(held, dtype, dim, e, spread):
    """Scores 2^e (2^23 + m), all of them numbers of 32 bits: a token's weight is 2^(e' m)
    of another's, and a channel of each m says what its tokens have.  With e4m3, value
    scales of many sizes.  spread: one sequence over many warps, or many in one each."""
    heads, page, repeat = 2, 32, 1 if not spread else 60
    many = 1 if spread else 1300
    for stairs in STAIRS if spread or (dim == 64 and e in (0, 3, 4)) else STAIRS[:1]:
        m = torch.tensor(stairs * repeat, device="cuda").repeat_interleave(32)
        n = len(m)
        k = torch.zeros(n // page, heads, page, dim, device="cuda")
        v = torch.zeros_like(k)
        k[..., 0] = 256
        k[..., 1] = m.view(-1, 1, page)
        v.view(-1, heads, page, dim).copy_(torch.nn.functional.one_hot(m, dim).view(-1, 1, page, dim))
        if held == F8:
            g = torch.Generator(device="cuda").manual_seed(n)
            vs = 2.0 ** torch.randint(-9, 10, (n // page, heads, page), generator=g, device="cuda").float()
            cache = ops.KvCache(k.to(F8), v.to(F8), torch.ones_like(vs), vs)
        else:
            vs = torch.ones(n // page, heads, page, device="cuda")
            cache = ops.KvCache(k.to(held), v.to(held))
        table = torch.arange(n // page, dtype=torch.int32, device="cuda").repeat(many, 1)
        q = torch.zeros(many, heads * 4, dim, device="cuda", dtype=dtype)
        q[..., 0], q[..., 1] = 2.0 ** 15, 1
        got = ops.attend_paged(q, cache, table, torch.full((many,), n, dtype=torch.int32, device="cuda"),
                               scale=scale_of(e)).double().view(many, heads, 4, dim)
        w = torch.exp2((m - m.max()).double() * 2.0 ** e)                        # [n]
        vw = vs.transpose(0, 1).reshape(heads, -1).double()                      # [heads, n]
        want = torch.zeros(heads, dim, dtype=torch.float64, device="cuda")
        want.index_add_(1, m, w * vw)
        want = (want / w.sum()).view(1, heads, 1, dim)
        # exact scores: exp2's 2^-22, the weights' two numbers, additions, joins; and where
        # the output's type ends
        off = (got - want).abs()
        rel = half_step(dtype) * 1.01 + (2.0 ** -15 if held == BF else 2.0 ** -20) + (n + 64) * 2.0 ** -23
        tiny = torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2 + 2.0 ** -42 * float(vs.max()) * n
        assert (off <= want * rel + tiny).all(), "%s: %s, not %s" % (
            stairs, got[0, 0, 0, :8].tolist(), want[0, 0, 0, :8].tolist())

"""GPU tests of the attention where a row's largest weight is far above all others,
and those are what its output is made of: the numbers that the weights become for
the second product have to hold them too."""
import math

import pytest
import torch

from routed_moe_decode_router_gb300 import ops
from tests import decode_ref as D
from tests.ops_ref import F8, half_step

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16
TYPES = [(F8, BF), (F8, HF), (HF, HF), (BF, BF)]


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    yield
    assert ops.device_status() == 0


def run(held, dtype, dim, heads, group, lengths, page, nats, every, rows=1, window=0):
    """Keys of nothing but the ones of every `every`th token, whose score is `nats` and
    whose value is in channel 0 alone; the others' values are in every channel, of one
    size each.  Compared with the formula, which is a count of each kind."""
    counts = [-(-n // page) for n in lengths]
    pages = sum(counts)
    place = torch.arange(page * max(counts), device="cuda")
    k = torch.zeros(pages, heads, page, dim, device="cuda")
    v = torch.zeros_like(k)
    small = 2.0 ** (13 + torch.arange(dim, device="cuda") % 3)
    table = torch.full((len(lengths), max(counts)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, c in enumerate(counts):
        table[b, :c] = torch.arange(at, at + c)
        big = (place[:c * page] % every == 0).view(c, 1, page)
        k[at:at + c, ..., 0] = torch.where(big, float(nats), 0.0)
        v[at:at + c] = torch.where(big.unsqueeze(-1), 0.0, small)
        v[at:at + c, ..., 0] = 2.0 ** 15
        at += c
    if held == F8:
        (kc, ks), (vc, vs) = D.kv_codes(k), D.kv_codes(v)
        cache = ops.KvCache(kc, vc, ks, vs)
    else:
        cache = ops.KvCache(k.to(held), v.to(held))
    q = torch.zeros(len(lengths), rows, heads * group, dim, device="cuda", dtype=dtype)
    q[..., 0] = 1
    got = ops.attend_paged(q, cache, table, torch.tensor(lengths, dtype=torch.int32, device="cuda"),
                           scale=1.0, window=window).double()
    kw, vw = D.wide(cache, "k"), D.wide(cache, "v")
    top, kind = float(kw[0, 0, 0]), (vw[0, 0], vw[1, 0])      # of tokens 0 and 1
    w = math.exp(-top)
    for b, n in enumerate(lengths):
        for r in range(rows):
            last = n - rows + r
            lo = max(0, last - window + 1) if window else 0
            bigs = last // every - (lo - 1) // every
            rest = last + 1 - lo - bigs
            want = (kind[0] * bigs + kind[1] * (rest * w)) / (bigs + rest * w)
            # the output's rounding; scores of few roundings of 2^-24 and exp2's 2^-22; a
            # weight as two numbers, 2^-16 (bf16) or 2^-22 of it, f16 2^-44 of the largest;
            # sums, each addition 2^-23, of a warp's share (of four times what 1200 warps
            # have each, and some tiles) and of the shares
            rel = half_step(dtype) * 1.01 + nats * 2.0 ** -21 + 2.0 ** -20 + \
                (2.0 ** -15 if held == BF else 2.0 ** -43 / w) + \
                (min(n, sum(lengths) * heads // 300 + 2048) + 64) * 2.0 ** -23
            off = (got[b, r] - want).abs() / want
            assert (off <= rel).all(), "%d of %d, row %d: %.3g, not %.3g" % (
                int((off > rel).sum()), off.numel(), r, float(off.max()), rel)


@pytest.mark.parametrize("held,dtype", TYPES)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("nats", [14, 16, 17, 18, 22])
@pytest.mark.parametrize("group,lengths,rows,window", [
    (1, [901], 1, 0), (16, [5000, 70], 1, 0), (5, [1200, 65] * 20, 3, 0), (4, [2222], 2, 500)])
def test_weights_far_below_the_largest(held, dtype, dim, nats, group, lengths, rows, window):
    """A token that takes nearly all in every tile or two."""
    run(held, dtype, dim, 2, group, lengths, 48, nats, 40, rows, window)


@pytest.mark.parametrize("held,dtype", TYPES)
@pytest.mark.parametrize("heads,length", [(256, 8192), (16, 131072)])
@pytest.mark.parametrize("nats", [14, 16, 17, 18])
def test_the_first_token_takes_nearly_all(held, dtype, heads, length, nats):
    """One token far above 8191 and 131071 others: half of what is left over is theirs."""
    run(held, dtype, 64, heads, 1, [length], 64, nats, length)

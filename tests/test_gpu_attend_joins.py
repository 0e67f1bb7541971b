"""GPU tests of how the attention's shares of a sequence come together, by outputs
that say what was counted: all tokens weigh alike and a value is one in a channel of
its own stretch of the sequence, so that every channel is a count of its tokens."""
import pytest
import torch

from routed_moe_decode_router_gb300 import ops
from tests.ops_ref import F8, half_step

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16
TYPES = [(F8, BF), (F8, HF), (BF, BF), (HF, HF)]
COUNTERS = 3 * 256      # words at the start of a workspace, which calls leave zero


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    yield
    assert ops.device_status() == 0


class Counted:
    """Sequences of up to longest[b] tokens over a cache whose tokens say where they are:
    a one in channel j // stretch of sequence position j, of every head the same but
    for its sign."""

    def __init__(self, longest, heads, dim, page, held, gone=()):
        self.heads, self.dim, self.page = heads, dim, page
        counts = [-(-n // page) for n in longest]
        pages = sum(counts) + 1
        g = torch.Generator(device="cuda").manual_seed(len(longest))
        ids = torch.randperm(pages, generator=g, device="cuda")
        self.table = torch.full((len(longest), max(counts)), -1, dtype=torch.int32, device="cuda")
        self.stretch = -(-max(longest) // dim)
        k = torch.zeros(pages, heads, page, dim, device="cuda", dtype=torch.float32 if held == F8 else held)
        k[..., 3] = 1            # the same score for all
        v = torch.zeros_like(k)
        sign = torch.where(torch.arange(heads, device="cuda") % 2 == 0, 1.0, -1.0)
        at = 0
        for b, c in enumerate(counts):
            own = ids[at:at + c]
            at += c
            self.table[b, :c] = own.int()
            channel = (torch.arange(c * page, device="cuda") // self.stretch).clamp(max=dim - 1)
            one = torch.nn.functional.one_hot(channel, dim).view(c, 1, page, dim)
            v[own] = (one * sign.view(1, heads, 1, 1)).to(v.dtype)
        for b, p in gone:
            self.table[b, p] = -1
        if held == F8:
            ones = torch.ones(pages, heads, page, device="cuda")
            self.cache = ops.KvCache(k.to(F8), v.to(F8), ones, ones.clone())
        else:
            self.cache = ops.KvCache(k, v)
        self.sign = sign

    def check(self, lengths, rows, group, dtype, window=0, ws=None):
        n = torch.tensor(lengths, dtype=torch.int32, device="cuda")
        g = torch.Generator(device="cuda").manual_seed(3)
        q = torch.randn(len(lengths), rows, group * self.heads, self.dim, generator=g, device="cuda").to(dtype)
        got = ops.attend_paged(q, self.cache, self.table, n, window=window, ws=ws).double()
        pos = torch.arange(self.table.shape[1] * self.page, device="cuda")
        there = (self.table >= 0).repeat_interleave(self.page, 1)             # [B, L]
        channel = (pos // self.stretch).clamp(max=self.dim - 1)
        for r in range(rows):
            last = (n - rows + r).unsqueeze(1)
            see = there & (pos <= last) & (pos < n.unsqueeze(1))
            if window:
                see &= pos > last - window
            count = torch.zeros(len(lengths), self.dim, dtype=torch.float64, device="cuda")
            count.index_add_(1, channel, see.double())
            want = count / count.sum(1, keepdim=True).clamp(min=1)
            want = want[:, None, None] * self.sign.double()[None, :, None, None]
            mine = got[:, r].view(len(lengths), self.heads, group, self.dim)
            # whole numbers times a power of two in every sum (below 2^24 of them): the
            # reciprocal's 2^-23, joins' factors of one (exp2 of 0) and the output's rounding
            off = (mine - want).abs()
            assert (off <= want.abs() * (half_step(dtype) * 1.01 + 2.0 ** -20)).all(), \
                "row %d: worst %.3g of its value" % (r, float((off / want.abs()).nan_to_num().max()))


@pytest.mark.parametrize("held,dtype", TYPES)
@pytest.mark.parametrize("dim,heads,group,rows,page,lengths,window", [
    (64, 1, 8, 1, 64, [70001], 0), (128, 2, 4, 1, 16, [131071], 0), (256, 2, 3, 1, 128, [50021], 0),
    (64, 2, 2, 3, 48, [40000, 9], 0), (128, 1, 16, 4, 64, [9000, 9001, 2], 0),
    (64, 4, 8, 1, 64, [901], 0), (128, 8, 4, 1, 16, [1983, 5, 600], 0), (256, 1, 1, 1, 16, [1500], 0),
    (128, 8, 4, 1, 64, [3000, 77, 0, 5001, 1, 16, 260, 1999] * 4, 0),
    (64, 4, 2, 2, 16, [(37 * i) % 401 for i in range(150)], 0),
    (64, 4, 5, 3, 48, [9001 - 271 * i for i in range(33)], 1024), (128, 1, 1, 1, 32, [30017], 20000),
    (128, 8, 8, 1, 64, [16384 - 500 * i for i in range(32)], 0)])
def test_every_token_counts_once(held, dtype, dim, heads, group, rows, page, lengths, window):
    Counted(lengths, heads, dim, page, held).check(lengths, rows, group, dtype, window)


@pytest.mark.parametrize("held,dtype", TYPES)
def test_pages_that_are_gone_do_not_count(held, dtype):
    gone = [(0, p) for p in range(40, 500)] + [(1, 0), (2, 30)]
    c = Counted([60000, 3000, 2000], 2, 64, 64, held, gone)
    c.check([60000, 3000, 1999], 2, 4, dtype)
    c.check([60000, 3000, 1999], 2, 4, dtype, window=1500)


@pytest.mark.parametrize("held,dtype", TYPES)
@pytest.mark.parametrize("dim,heads,group", [(64, 1, 8), (128, 2, 16), (256, 1, 8)])
def test_a_workspace_from_call_to_call(held, dtype, dim, heads, group):
    """More than 32 sequences, one of them over most thread blocks: its sums are joined
    in groups of blocks and those joined, whose counters are zero again for the next
    call, which has other lengths."""
    longest = [60000] + [100 + i for i in range(39)]
    c = Counted(longest, heads, dim, 64, held)
    ws = ops.AttendWorkspace(len(longest), 1, group * heads, heads, dim)
    for lengths in (longest, [60000] + [1] * 39, [25000] + longest[1:], [0] * 40,
                    [5000] + [0] * 39, longest):
        c.check(lengths, 1, group, dtype, ws=ws)
        assert not ws.buf.view(torch.int32)[:COUNTERS].any()
    # the same workspace with few sequences (a joining kernel), then these again
    few = Counted([20000, 700], heads, dim, 64, held)
    for _ in range(2):
        few.check([20000, 700], 1, group, dtype, ws=ws)
        assert not ws.buf.view(torch.int32)[:COUNTERS].any()
        c.check(longest, 1, group, dtype, ws=ws)
        assert not ws.buf.view(torch.int32)[:COUNTERS].any()


def counts_of_a_page(cache, page, dim):
    """Channel d of the value at place i of every page: 1 where i % dim == d."""
    one = torch.nn.functional.one_hot(torch.arange(page, device="cuda") % dim, dim)
    cache.v.copy_(one.to(cache.v.dtype).expand(cache.v.shape))


@pytest.mark.parametrize("held,dtype", [(F8, BF), (HF, HF)])
@pytest.mark.parametrize("length,window", [
    (1 << 30, 0), ((1 << 30) - 100, 0), (1 << 30, 1000), (1 << 30, (1 << 30) - 7), ((1 << 29) + 33, 1 << 20)])
def test_the_longest_sequences(held, dtype, length, window):
    """2^30 tokens, on pages that come again and again."""
    page, dim = 1024, 64
    cache = ops.new_kv_cache(3, 1, page, dim, held)
    counts_of_a_page(cache, page, dim)
    if held == F8:
        cache.k_scales.fill_(1)
        cache.v_scales.fill_(1)
    table = (torch.arange((1 << 30) // page, device="cuda").int() % 3)[None]
    q = torch.ones(1, 2, 2, dim, dtype=dtype, device="cuda")
    got = ops.attend_paged(q, cache, table, torch.tensor([length], dtype=torch.int32, device="cuda"),
                           window=window).double()
    for r in range(2):
        last = length - 2 + r
        lo = max(0, last - window + 1) if window else 0
        d = torch.arange(dim, device="cuda")

        def below(n):       # tokens of each channel below n: pages are whole rounds of dim
            return n // dim + (d < n % dim).long()
        want = (below(last + 1) - below(lo)).double() / (last + 1 - lo)
        # a warp's share is exact (below 2^24 of them); 1216 shares, and the output
        assert ((got[0, r] - want).abs() <= want * (half_step(dtype) * 1.01 + 1300 * 2.0 ** -24)).all()


def test_the_most_sequences_and_heads():
    """2048 sequences of 1024 heads: two million items of a few tokens, some of none."""
    batch, heads, page, dim = 2048, 1024, 16, 64
    cache = ops.new_kv_cache(3, heads, page, dim, BF)
    counts_of_a_page(cache, page, dim)
    sign = torch.where(torch.arange(heads, device="cuda") % 3 == 0, -1.0, 1.0)
    cache.v.mul_(sign.to(BF)[:, None, None])
    table = torch.randint(0, 3, (batch, 2), device="cuda").int()
    n = torch.arange(batch, device="cuda").int() % 33
    got = ops.attend_paged(torch.ones(batch, heads, dim, dtype=BF, device="cuda"), cache, table, n)
    d = torch.arange(dim, device="cuda")
    count = (d < n[:, None].clamp(max=16)).int() + (d < (n[:, None] - 16)).int()
    want = (count.double() / n[:, None].clamp(min=1)).unsqueeze(1) * sign.double()[:, None]
    assert ((got.double() - want).abs() <= want.abs() * (half_step(BF) * 1.01 + 2.0 ** -20)).all()

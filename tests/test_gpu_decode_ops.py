"""GPU tests of the decoding step's operators against their definitions in 64 bits
(tests/decode_ref.py): the paged cache, attention over it, verification of drafts,
at the sizes, strides and masks where they can go wrong."""
import math

import pytest
import torch

from routed_moe_decode_router_gb300 import ops
from tests import decode_ref as D
from tests.ops_ref import F8

pytestmark = pytest.mark.gpu
BF, HF, FP = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    yield
    assert ops.device_status() == 0


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(9000 + seed)


def randn(*shape, seed=0, std=1.0):
    return torch.randn(*shape, generator=gen(seed), device="cuda") * std


def bits(t):
    return t.contiguous().view(torch.uint8)


def cache_of(pages, heads, page, dim, dtype, seed=0):
    """A cache full of numbers, its keys with larger channels."""
    k = randn(pages, heads, page, dim, seed=seed) * torch.exp(randn(dim, seed=seed + 1, std=0.5))
    v = randn(pages, heads, page, dim, seed=seed + 2)
    if dtype != F8:
        return ops.KvCache(k.to(dtype), v.to(dtype))
    (kc, ks), (vc, vs) = D.kv_codes(k), D.kv_codes(v)
    return ops.KvCache(kc, vc, ks, vs)


# ---------------------------------------------------------------------------
# Cache
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("dtype,held", [(BF, F8), (HF, F8), (FP, F8), (BF, BF), (HF, HF)])
@pytest.mark.parametrize("tokens,heads,page", [(1, 1, 16), (3, 5, 48), (67, 8, 64), (300, 3, 1024)])
def test_cache_written_and_read(dim, dtype, held, tokens, heads, page):
    pages = tokens // page + 3
    cache = cache_of(pages, heads, page, dim, held, seed=7)
    before = [None if t is None else t.clone() for t in cache]
    slots = torch.randperm(pages * page, generator=gen(1), device="cuda")[:tokens].int()
    rows = randn(tokens, 2, heads, dim, seed=2).to(dtype)       # keys and values of one product
    if tokens > 2:
        slots[1] = -1
        slots[2] = pages * page                                 # behind the cache
        rows[0, :, 0] = 0
    ops.kv_write(cache, rows[:, 0], rows[:, 1], slots)
    put = ((slots >= 0) & (slots < pages * page)).nonzero().flatten()
    at = (slots[put] // page).long(), slice(None), (slots[put] % page).long()
    for i, name in enumerate(("k", "v")):
        want, scales = before[i].clone(), before[i + 2]
        if held == F8:
            # the scale to a step, the codes those of the scale that was stored
            ref = rows[put, i].double().abs().amax(-1).clamp(min=1e-30) / 448
            new = getattr(cache, name + "_scales")
            assert ((new[at].double() - ref).abs() <= ref * 2.0 ** -23).all()
            scales = scales.clone()
            scales[at] = new[at]
            assert torch.equal(new, scales)
            codes = (rows[put, i].double() / new[at].double().unsqueeze(-1)).clamp(-448, 448)
            want.view(torch.uint8)[at] = codes.float().to(F8).view(torch.uint8)
        else:
            want[at] = rows[put, i]
        assert torch.equal(bits(getattr(cache, name)), bits(want))
    for out in (BF, HF, FP):
        got = ops.kv_read(cache, slots, dtype=out)
        for i, name in enumerate(("k", "v")):
            want = torch.zeros(tokens, heads, dim, dtype=torch.float64, device="cuda")
            want[put] = D.wide(cache, name)[slots[put].long()]
            if held == F8:      # one rounding of the product to fp32 before
                want = want.float()
            assert torch.equal(got[i], want.to(out))


def test_cache_in_one_tensor_and_beyond_32_bits():
    """Keys, values of a page side by side; byte offsets above 2^32."""
    heads, page, dim, pages = 8, 64, 256, 9000
    both = torch.empty(pages, 2, heads, page, dim, dtype=BF, device="cuda")
    assert both.numel() * 2 > 2 ** 32
    cache = ops.KvCache(both[:, 0], both[:, 1])
    ids = torch.tensor([pages - 1, 0, pages - 3], device="cuda")
    both[ids] = randn(3, 2, heads, page, dim, seed=3).to(BF)
    kept = both[ids].clone()
    slots = (ids[:2] * page + torch.tensor([page - 1, 5], device="cuda")).int()
    k, v = randn(2, heads, dim, seed=4).to(BF), randn(2, heads, dim, seed=5).to(BF)
    ops.kv_write(cache, k, v, slots)
    for i, (p, at) in enumerate(((0, page - 1), (1, 5))):
        kept[p, 0, :, at], kept[p, 1, :, at] = k[i], v[i]
    assert torch.equal(both[ids], kept)
    rk, rv = ops.kv_read(cache, slots)
    assert torch.equal(rk, k) and torch.equal(rv, v)
    q = randn(1, 1, 2 * heads, dim, seed=6).to(BF)
    table = ids.int()[None]
    lengths = torch.tensor([3 * page - 7], dtype=torch.int32, device="cuda")
    small = ops.KvCache(both[ids][:, 0], both[ids][:, 1])
    order = torch.arange(3, dtype=torch.int32, device="cuda")[None]
    want, bound = D.attend(q, small, order, lengths)
    got = ops.attend_paged(q, cache, table, lengths)
    assert ((got.double() - want).abs() <= bound).all()


def test_cache_numbers_at_the_ends_of_their_range():
    cache = ops.new_kv_cache(2, 1, 16, 64)
    x = randn(6, 1, 64, seed=1)
    x[0] *= 1e-38
    x[1] *= 1e37
    x[2, 0, 3] = math.inf
    x[3, 0, 3] = math.nan
    x[4] = 0
    x[5, 0, 0] = -448
    slots = torch.arange(6, dtype=torch.int32, device="cuda")
    ops.kv_write(cache, x, x, slots)
    k, _ = ops.kv_read(cache, slots, dtype=FP)
    ok = [0, 1, 4, 5]
    codes, scales = D.kv_codes(x[ok])
    assert torch.equal(k[ok], codes.float() * scales.unsqueeze(-1))
    assert not k[4].any()
    assert k[2, 0, 3].isnan() and k[3, 0, 3].isnan() and k[3, 0, :3].isfinite().all()


def test_no_tokens_and_no_sequences():
    cache = ops.new_kv_cache(2, 2, 16, 64, dtype=BF)
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    e = torch.empty(0, 2, 64, dtype=BF, device="cuda")
    ops.kv_write(cache, e, e, none)
    k, v = ops.kv_read(cache, none)
    assert k.shape == v.shape == (0, 2, 64)
    out = ops.attend_paged(torch.empty(0, 3, 4, 64, dtype=BF, device="cuda"), cache,
                           torch.empty(0, 1, dtype=torch.int32, device="cuda"), none)
    assert out.shape == (0, 3, 4, 64)
    p = torch.empty(0, 3, 10, device="cuda")
    r = ops.verify_draft(torch.empty(0, 2, dtype=torch.int32, device="cuda"), p,
                         torch.empty(0, 2, device="cuda"), torch.empty(0, device="cuda"))
    assert r.tokens.shape == (0, 3) and r.accepted.shape == (0,)


# ---------------------------------------------------------------------------
# Attention
# ---------------------------------------------------------------------------

def batch_of(lengths, page, seed=0, spare=2):
    """(table, pages): the pages of sequences, in an order of their own."""
    counts = [-(-max(n, 0) // page) for n in lengths]
    pages = sum(counts) + spare
    ids = torch.randperm(pages, generator=gen(seed + 50), device="cuda").int()
    table = torch.full((len(lengths), max(1, max(counts))), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(counts):
        table[b, :n] = ids[at:at + n]
        at += n
    return table, pages


def check(q, cache, table, lengths, ws=None, **kw):
    lengths = torch.as_tensor(lengths, dtype=torch.int32, device="cuda")
    want, bound = D.attend(q, cache, table, lengths, **kw)
    got = ops.attend_paged(q, cache, table, lengths, ws=ws, **kw)
    assert got.dtype == q.dtype and got.shape == q.shape
    bad = ~((got.double() - want).abs() <= bound)
    assert not bad.any(), "%d of %d, worst %.3g x its bound" % (
        int(bad.sum()), bad.numel(), float(((got.double() - want).abs() / bound).nan_to_num().max()))
    return got


TYPES = [(F8, BF), (F8, HF), (BF, BF), (HF, HF)]


@pytest.mark.parametrize("held,dtype", TYPES)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("rows,group,heads,page,lengths,window", [
    (1, 1, 1, 16, [1], 0), (1, 8, 2, 16, [17], 0), (1, 4, 8, 64, [901], 0),
    (1, 3, 2, 48, [5, 0, 16, 333, 1, 48], 0), (1, 7, 1, 32, [1500], 100),
    (4, 8, 2, 64, [64, 3, 700], 0), (3, 5, 2, 48, [129, 1000, 2], 37), (8, 16, 1, 128, [300], 0),
    (2, 1, 3, 16, [31, 32, 33, 1], 1), (64, 1, 2, 16, [40, 100], 16), (5, 3, 1, 16, [15], 3)])
def test_attention_sizes(held, dtype, dim, rows, group, heads, page, lengths, window):
    table, pages = batch_of(lengths, page)
    cache = cache_of(pages, heads, page, dim, held)
    q = randn(len(lengths), rows, group * heads, dim, seed=9).to(dtype)
    got = check(q, cache, table, lengths, window=window)
    again = ops.attend_paged(q, cache, table, torch.tensor(lengths, dtype=torch.int32, device="cuda"),
                             window=window)
    assert torch.equal(got, again)


@pytest.mark.parametrize("held,dtype", TYPES)
@pytest.mark.parametrize("dim,heads,group,rows,lengths", [
    (128, 1, 8, 1, [70001]), (64, 2, 2, 3, [40000, 9]), (256, 1, 1, 1, [30017]),
    (128, 8, 4, 1, [3000, 77, 0, 5001, 1, 16, 260, 1999] * 4),
    (64, 4, 2, 2, [(37 * i) % 401 for i in range(150)])])
def test_attention_long_and_many(held, dtype, dim, heads, group, rows, lengths):
    """Items that many blocks share, and blocks that share many items."""
    table, pages = batch_of(lengths, 64)
    cache = cache_of(pages, heads, 64, dim, held)
    q = randn(len(lengths), rows, group * heads, dim, seed=9).to(dtype)
    ws = ops.AttendWorkspace(len(lengths), rows, group * heads, heads, dim)
    check(q, cache, table, lengths, ws=ws)
    assert not ws.buf[:1024].any()          # ready for the next call


@pytest.mark.parametrize("batch", [32, 33, 1024, 1025, 2048])
def test_attention_of_many_sequences(batch):
    lengths = [(37 * i) % 70 for i in range(batch)]
    lengths[batch // 3] = 3000
    table, pages = batch_of(lengths, 16)
    cache = cache_of(pages, 1, 16, 64, F8)
    q = randn(batch, 1, 3, 64, seed=9).to(BF)
    check(q, cache, table, lengths)


@pytest.mark.parametrize("held,dtype", TYPES)
@pytest.mark.parametrize("batch,page,window", [(1, 48, 0), (2, 16, 30000), (1, 1024, 0), (20, 64, 0)])
def test_long_sequences_with_pages_that_are_gone(held, dtype, batch, page, window):
    """Shares of an item that see nothing, in blocks and in groups of blocks."""
    lengths = [50000 // (1 + b) + 7 for b in range(batch)]
    table, pages = batch_of(lengths, page)
    table[0, 3:table.shape[1] * 2 // 3] = pages + 5
    table[-1, ::3] = -1
    cache = cache_of(pages, 2, page, 64, held)
    q = randn(batch, 3, 4, 64, seed=9).to(dtype)
    check(q, cache, table, lengths, window=window)
    table[:] = -1
    assert not check(q, cache, table, lengths, window=window).any()


@pytest.mark.parametrize("held,dtype", TYPES)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("lengths,heads,group,rows,window", [
    ([1983], 1, 1, 1, 0), ([1100, 30, 0, 2000], 4, 3, 2, 0), ([600] * 3, 8, 4, 1, 0),
    ([4000, 513], 2, 2, 5, 700), ([2100, 2, 1], 1, 16, 2, 0)])
def test_attention_of_few_sequences_spread_over_all_blocks(held, dtype, dim, lengths, heads, group,
                                                           rows, window):
    table, pages = batch_of(lengths, 32)
    cache = cache_of(pages, heads, 32, dim, held)
    q = randn(len(lengths), rows, group * heads, dim, seed=9).to(dtype)
    ws = ops.AttendWorkspace(len(lengths), rows, group * heads, heads, dim)
    got = check(q, cache, table, lengths, ws=ws, window=window)
    table[0, 5:9] = -1
    check(q, cache, table, lengths, ws=ws, window=window)
    lengths = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = ops.attend_paged(q, cache, table, lengths, ws=ws, window=window)
    lengths.sub_(1).clamp_(min=0)
    graph.replay()
    want, bound = D.attend(q, cache, table, lengths, window=window)
    assert ((out.double() - want).abs() <= bound).all() and out.shape == got.shape


def test_infinities_and_nan_that_are_seen():
    """They reach the rows that see them, and those alone.  A weight is two numbers,
    the second of which may be negative or 0, so an infinity may come out as NaN."""
    table, pages = batch_of([100, 100], 16)
    cache = cache_of(pages, 1, 16, 64, BF)
    q = randn(2, 1, 2, 64, seed=9).to(BF)
    lengths = torch.tensor([100, 100], dtype=torch.int32, device="cuda")
    clean = ops.attend_paged(q, cache, table, lengths)
    cache.v[int(table[0, 1]), 0, 3, 5] = math.inf
    got = ops.attend_paged(q, cache, table, lengths)
    assert torch.equal(got[1], clean[1]) and not got[0, 0, :, 5].isfinite().any()
    assert torch.equal(got[0, 0, :, :5], clean[0, 0, :, :5])
    assert torch.equal(got[0, 0, :, 6:], clean[0, 0, :, 6:])
    cache.v[int(table[0, 1]), 0, 3, 5] = 1.0
    clean = ops.attend_paged(q, cache, table, lengths)
    bad = q.clone()
    bad[1, 0, 1, 7] = math.nan
    got = ops.attend_paged(bad, cache, table, lengths)
    assert got[1, 0, 1].isnan().all() and torch.equal(got[1, 0, 0], clean[1, 0, 0])


@pytest.mark.parametrize("held,dtype", TYPES)
@pytest.mark.parametrize("window", [0, 20])
def test_what_a_row_does_not_see_does_not_reach_it(held, dtype, window):
    """NaN and infinities behind the end, before the window, in the tokens after a
    row's own and in pages outside the cache."""
    rows, heads, page, dim, lengths = 4, 2, 16, 128, [40, 2, 0, 64]
    table, pages = batch_of(lengths, page)
    cache = cache_of(pages, heads, page, dim, held)
    q = randn(4, rows, 4, dim, seed=9).to(dtype)
    clean = check(q, cache, table, lengths, window=window)
    used = torch.zeros(pages * page, dtype=torch.bool, device="cuda")
    for b, n in enumerate(lengths):
        for j in range(n):
            if not window or j > n - rows - window:
                used[int(table[b, j // page]) * page + j % page] = True
    for t in cache:
        if t is not None:
            bad = math.nan if t.dtype == F8 else math.inf
            flat = t.transpose(1, 2)
            flat[~used.view(pages, page)] = torch.full_like(flat[~used.view(pages, page)].float(), bad).to(t.dtype)
    assert torch.equal(ops.attend_paged(q, cache, table, torch.tensor(
        lengths, dtype=torch.int32, device="cuda"), window=window), clean)
    # the value (and for e4m3 its scale) of the last token but one of sequence 0
    at = int(table[0, 38 // page]), slice(None), 38 % page
    for poison in ("v", "v_scales", "k"):
        t = getattr(cache, poison)
        if t is None:
            continue
        kept = t[at].clone()
        t[at] = torch.full_like(kept.float(), math.nan if t.dtype == F8 else math.inf).to(t.dtype)
        got = ops.attend_paged(q, cache, table, torch.tensor(lengths, dtype=torch.int32, device="cuda"),
                               window=window)
        assert torch.equal(got[1:], clean[1:]) and torch.equal(got[0, :2], clean[0, :2]), poison
        assert not got[0, 2:].isfinite().any(), poison
        t[at] = kept
    # pages outside the cache
    less = table.clone()
    less[0, 1], less[3, 0] = -1, pages
    check(q, cache, less, lengths, window=window)


@pytest.mark.parametrize("held,dtype", TYPES)
def test_rows_that_see_nothing_are_zero(held, dtype):
    lengths = [3, 0, -5, 20]
    table, pages = batch_of(lengths, 16)
    cache = cache_of(pages, 2, 16, 64, held)
    q = randn(4, 8, 6, 64, seed=9).to(dtype)
    got = check(q, cache, table, lengths)
    assert not got[0, :5].any() and got[0, 5:].any() and not got[1].any() and not got[2].any()
    table[3] = -1
    assert not check(q, cache, table, lengths)[3].any()


@pytest.mark.parametrize("held,dtype", TYPES)
def test_lengths_beyond_the_table_are_the_tables(held, dtype):
    table, pages = batch_of([48, 48], 16)
    cache = cache_of(pages, 1, 16, 64, held)
    q = randn(2, 1, 2, 64, seed=9).to(dtype)
    check(q, cache, table, [49, 2 ** 31 - 1])


@pytest.mark.parametrize("held,dtype", TYPES)
def test_large_scores_and_few_that_count(held, dtype):
    """Scores of +-1000, rising along the sequence: the maximum moves often."""
    n, dim = 700, 128
    table, pages = batch_of([n], 64)
    cache = cache_of(pages, 1, 64, dim, held)
    q = randn(1, 1, 4, dim, seed=9)
    k = torch.empty(n, 1, dim, device="cuda")
    k[:, 0] = q[0, 0, 0] * torch.linspace(-9, 9, n, device="cuda")[:, None]
    k += randn(n, 1, dim, seed=11, std=0.1)
    slots = (table[0].repeat_interleave(64) * 64 + torch.arange(64, device="cuda").repeat(table.shape[1]))[:n].int()
    v = randn(n, 1, dim, seed=12)
    wt = dtype if held != F8 else FP
    ops.kv_write(cache, k.to(wt), v.to(wt), slots)
    check(q.to(dtype), cache, table, [n])
    check(q.to(dtype), cache, table, [n], scale=-0.5)
    check(q.to(dtype), cache, table, [n], scale=0.0)


@pytest.mark.parametrize("dtype", [BF, HF])
def test_scales_of_very_different_size(dtype):
    """Values of 1e-30 to 1e4 beside each other, and tokens without a value."""
    n, dim = 333, 64
    table, pages = batch_of([n], 16)
    cache = cache_of(pages, 2, 16, dim, F8)
    sizes = torch.exp(randn(pages, 2, 16, seed=13, std=4.0)).clamp(max=1e4 if dtype == BF else 100.0)
    cache.v_scales.mul_(sizes)
    cache.v.view(torch.uint8)[::3] = 0
    cache.v_scales[::3] = 1e-30 / 448
    q = randn(1, 2, 8, dim, seed=9).to(dtype)
    check(q, cache, table, [n])
    check((q.float() * 1e-3).to(dtype), cache, table, [n])
    check((q.float() * (1e20 if dtype == BF else 100)).to(dtype), cache, table, [n],
          scale=1e-20 if dtype == BF else 1e-3)


def test_strided_queries_tables_and_outputs():
    lengths = [50, 0, 99]
    table, pages = batch_of(lengths, 16)
    cache = cache_of(pages, 2, 16, 64, F8)
    wide = torch.full((3, 20), 7, dtype=torch.int32, device="cuda")
    wide[:, 3:3 + table.shape[1]] = table
    part = wide[:, 3:3 + table.shape[1]]
    qkv = randn(3, 2, 8 + 4, 64, seed=9).to(BF)           # the rows of one product
    q = qkv[:, :, :8]
    want = ops.attend_paged(q.contiguous(), cache, table, torch.tensor(lengths, dtype=torch.int32, device="cuda"))
    out = torch.full_like(want, 5.0)
    got = ops.attend_paged(q, cache, part, torch.tensor(lengths, dtype=torch.int32, device="cuda"), out=out)
    assert got.data_ptr() == out.data_ptr() and torch.equal(got, want)
    turned = q.transpose(0, 1).contiguous().transpose(0, 1)
    assert torch.equal(ops.attend_paged(turned, cache, part, torch.tensor(lengths, dtype=torch.int32, device="cuda")), want)
    one = ops.attend_paged(q[:, 1], cache, part, torch.tensor(lengths, dtype=torch.int32, device="cuda"))
    assert one.shape == (3, 8, 64) and torch.equal(one, want[:, 1])


def test_workspace_goes_from_shape_to_shape():
    """One workspace, large enough for all, for calls of different shapes in turn."""
    shapes = [(1, 1, 8, 8, 128, [5000]), (1, 4, 16, 2, 64, [900, 3000]), (2, 8, 8, 1, 128, [2000]),
              (3, 1, 4, 4, 256, [700, 800, 900])]
    big = max((ops.AttendWorkspace(64, r, hq, hk, d) for _, r, hq, hk, d, _ in shapes),
              key=lambda w: w.nbytes)
    for _ in range(2):
        for i, (_, r, hq, hk, d, lengths) in enumerate(shapes):
            table, pages = batch_of(lengths, 64)
            cache = cache_of(pages, hk, 64, d, F8, seed=i)
            q = randn(len(lengths), r, hq, d, seed=20 + i).to(BF)
            check(q, cache, table, lengths, ws=big)


def test_attention_captured_and_replayed_with_other_lengths():
    lengths = torch.tensor([3000, 1], dtype=torch.int32, device="cuda")
    table, pages = batch_of([3000, 3000], 64)
    cache = cache_of(pages, 2, 64, 128, F8)
    q = randn(2, 2, 8, 128, seed=9).to(BF)
    ws = ops.AttendWorkspace(2, 2, 8, 2, 128)
    ops.attend_paged(q, cache, table, lengths, ws=ws)
    graphs = []
    for own in (ws, None, ws):                 # two graphs with one workspace, one with its own
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            graphs.append((g, ops.attend_paged(q, cache, table, lengths, ws=own)))
    for new in ([3000, 1], [17, 2999], [0, 0], [1000, 1001]):
        lengths.copy_(torch.tensor(new, dtype=torch.int32))
        want, bound = D.attend(q, cache, table, lengths)
        for g, out in graphs:
            g.replay()
            assert ((out.double() - want).abs() <= bound).all()


def test_calls_on_other_streams_at_once():
    lengths = torch.tensor([2500, 40, 0, 700], dtype=torch.int32, device="cuda")
    table, pages = batch_of([2500, 40, 0, 700], 64)
    cache = cache_of(pages, 4, 64, 128, BF)
    q = randn(4, 1, 16, 128, seed=9).to(BF)
    want = ops.attend_paged(q, cache, table, lengths)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    got = [[] for _ in streams]
    for _ in range(5):
        for s, out in zip(streams, got):
            out.append(ops.attend_paged(q, cache, table, lengths, stream=s))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for out in got for o in out)


def test_attention_refusals():
    cache = cache_of(3, 2, 16, 64, F8)
    q = randn(1, 1, 4, 64).to(BF)
    table = torch.zeros(1, 2, dtype=torch.int32, device="cuda")
    lengths = torch.ones(1, dtype=torch.int32, device="cuda")
    ok = dict(q=q, cache=cache, table=table, lengths=lengths)
    ops.attend_paged(**ok)
    with pytest.raises(ValueError, match="dtype"):
        ops.attend_paged(**{**ok, "q": q.float()})
    with pytest.raises(ValueError, match="elements to a head"):
        ops.attend_paged(**{**ok, "q": randn(1, 1, 2, 128).to(BF)})
    with pytest.raises(ops.N.MoeError, match="q_heads"):
        ops.attend_paged(**{**ok, "q": randn(1, 1, 5, 64).to(BF)})
    with pytest.raises(ValueError, match="dtype"):
        ops.attend_paged(**{**ok, "table": table.long()})
    with pytest.raises(ValueError, match="shape"):
        ops.attend_paged(**{**ok, "lengths": lengths.repeat(2)})
    with pytest.raises(ValueError, match="cpu"):
        ops.attend_paged(**{**ok, "lengths": lengths.cpu()})
    with pytest.raises(ValueError, match="no scales"):
        ops.attend_paged(**{**ok, "cache": ops.KvCache(cache.k.to(BF), cache.v.to(BF), cache.k_scales, cache.v_scales)})
    with pytest.raises(TypeError, match="k_scales"):
        ops.attend_paged(**{**ok, "cache": ops.KvCache(cache.k, cache.v)})
    with pytest.raises(ValueError, match="contiguous in its pages"):
        ops.attend_paged(**{**ok, "cache": cache._replace(k=cache.k.transpose(1, 2).contiguous().transpose(1, 2))})
    with pytest.raises(ops.N.MoeError, match="own type"):
        ops.attend_paged(**{**ok, "cache": ops.KvCache(cache.k.to(HF), cache.v.to(HF))})
    with pytest.raises(ops.N.MoeError, match="two arrays"):
        ops.attend_paged(**{**ok, "cache": cache._replace(v=cache.k)})
    with pytest.raises(ops.N.MoeError, match="window"):
        ops.attend_paged(**ok, window=-1)
    with pytest.raises(ops.N.MoeError, match="scale"):
        ops.attend_paged(**ok, scale=math.nan)
    with pytest.raises(ops.N.MoeError, match="workspace has"):
        ws = ops.AttendWorkspace(1, 1, 4, 2, 64)
        ws.buf = ws.buf[:1024]
        ops.attend_paged(**ok, ws=ws)
    with pytest.raises(ops.N.MoeError, match="out overlaps"):
        ops.attend_paged(**ok, out=q)
    with pytest.raises(ops.N.MoeError, match="aligned"):
        flat = torch.zeros(4 * 64 + 1, dtype=BF, device="cuda")
        ops.attend_paged(**{**ok, "q": flat[1:].view(1, 1, 4, 64)})


# ---------------------------------------------------------------------------
# Verification
# ---------------------------------------------------------------------------

def probs(*shape, seed, std=2.0):
    return torch.softmax(randn(*shape, seed=seed, std=std), -1)


def check_verify(draft, target, accept_u, sample_u, draft_probs=None):
    got = ops.verify_draft(draft, target, accept_u, sample_u, draft_probs=draft_probs)
    tokens, accepted = D.verify(draft, target, accept_u, sample_u, draft_probs)
    assert torch.equal(got.accepted.cpu(), accepted)
    assert torch.equal(got.tokens.cpu(), tokens)
    return got


@pytest.mark.parametrize("certain", [False, True])
@pytest.mark.parametrize("batch,drafts,vocab", [(1, 0, 1), (2, 1, 3), (5, 3, 100), (40, 4, 1000),
                                                (9, 31, 257), (3, 5, 50001), (4, 2, 131072), (2, 1, 1 << 19)])
def test_verify_sizes(certain, batch, drafts, vocab):
    target = probs(batch, drafts + 1, vocab, seed=1)
    q = torch.softmax(torch.log(target[:, :drafts]) + randn(batch, drafts, vocab, seed=2, std=0.5), -1)
    draft = torch.multinomial(q.reshape(-1, vocab), 1, generator=gen(3)).view(batch, drafts).int() \
        if drafts else torch.empty(batch, 0, dtype=torch.int32, device="cuda")
    if certain and drafts:
        draft = torch.where(torch.rand(batch, drafts, generator=gen(6), device="cuda") < 0.5,
                            target[:, :drafts].argmax(-1).int(), draft)
    if batch > 2 and drafts > 1:
        draft[1, drafts // 2] = -1
        draft[2, 0] = vocab
    for seed in range(4):
        accept_u = torch.rand(batch, drafts, generator=gen(10 + seed), device="cuda")
        sample_u = torch.rand(batch, generator=gen(20 + seed), device="cuda")
        check_verify(draft, target, accept_u, sample_u, None if certain else q)


def test_verify_numbers_at_their_ends():
    """sample_u of 0 and just below 1 and outside; rows with nothing, one thing, NaN."""
    vocab = 777
    target = probs(10, 2, vocab, seed=1)
    target[:, :, :5] = 0
    target[:, :, -5:] = 0
    target[1] = 0
    target[2] = 0
    target[2, :, 700] = 1e-6
    target[3, :, 10] = math.nan
    target[3, :, 11] = -0.5
    target[4, :, 12] = math.inf
    target[5] = 1.0
    draft = torch.full((10, 1), 300, dtype=torch.int32, device="cuda")
    draft[6:] = 20
    q = probs(10, 1, vocab, seed=2)
    q[6] = 2.0                  # nowhere less than the target: drawn from the target
    for u in (0.0, 1 - 2.0 ** -24, 1.0, 7.0, -1.0, math.nan, 2.0 ** -140):
        sample_u = torch.full((10,), u, device="cuda")
        for a in (0.0, 1 - 2.0 ** -24, math.nan):
            accept_u = torch.full((10, 1), a, device="cuda")
            for d in (q, None):
                got = check_verify(draft, target, accept_u, sample_u, d)
                assert got.tokens[1, int(got.accepted[1])] == -1


def test_verify_counts_steps_exactly():
    """Equal weights, and a number on the border of two of them: the lower id ends
    where the running sum is the number itself."""
    vocab = 1 << 14
    target = torch.full((vocab // 64, 1, vocab), 2.0 ** -14, device="cuda")
    ids = torch.arange(0, vocab, 64, device="cuda")
    sample_u = ids.float() / vocab
    none = torch.empty(len(ids), 0, device="cuda")
    got = check_verify(none.int(), target, none, sample_u)
    assert torch.equal(got.tokens[:, 0], ids.int())


def test_verify_strided_rows():
    big = torch.zeros(3, 3, 1003, device="cuda")
    big[:, :, 2:1002] = probs(3, 3, 1000, seed=1)
    target = big[:, :, 2:1002]
    q = probs(3, 2, 1000, seed=2)
    draft = target[:, :2].argmax(-1).int()
    u, s = torch.rand(3, 2, generator=gen(4), device="cuda"), torch.rand(3, generator=gen(5), device="cuda")
    check_verify(draft, target, u, s, q)
    got = check_verify(draft, target.contiguous(), u, s, q)
    again = ops.verify_draft(draft, target, u, s, draft_probs=q)
    assert torch.equal(got.tokens, again.tokens)


def test_verify_is_distributed_as_the_target():
    """What comes out first, over many draws: within 5 deviations of the target."""
    vocab, n = 12, 40000
    p, q = probs(vocab, seed=1), probs(vocab, seed=2)
    draft = torch.multinomial(q, n, replacement=True, generator=gen(3)).view(n, 1).int()
    r = ops.verify_draft(draft, p.expand(n, 2, vocab).contiguous(), torch.rand(n, 1, generator=gen(4), device="cuda"),
                         torch.rand(n, generator=gen(5), device="cuda"),
                         draft_probs=q.expand(n, 1, vocab).contiguous())
    seen = torch.bincount(r.tokens[:, 0].long(), minlength=vocab) / n
    assert ((seen - p).abs() <= 5 * torch.sqrt(p * (1 - p) / n) + 1e-4).all()


def test_verify_captured():
    target, q = probs(6, 3, 5000, seed=1), probs(6, 2, 5000, seed=2)
    draft = q.argmax(-1).int()
    u, s = torch.rand(6, 2, generator=gen(4), device="cuda"), torch.rand(6, generator=gen(5), device="cuda")
    ops.verify_draft(draft, target, u, s, draft_probs=q)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = ops.verify_draft(draft, target, u, s, draft_probs=q)
    for seed in range(3):
        u.copy_(torch.rand(6, 2, generator=gen(30 + seed), device="cuda"))
        g.replay()
        tokens, accepted = D.verify(draft, target, u, s, q)
        assert torch.equal(out.tokens.cpu(), tokens) and torch.equal(out.accepted.cpu(), accepted)


def test_verify_refusals():
    t = probs(2, 3, 50, seed=1)
    d, u, s = torch.zeros(2, 2, dtype=torch.int32, device="cuda"), torch.zeros(2, 2, device="cuda"), torch.zeros(2, device="cuda")
    with pytest.raises(ValueError, match="dtype"):
        ops.verify_draft(d, t.half(), u, s)
    with pytest.raises(ValueError, match="shape"):
        ops.verify_draft(d, t[:, :2], u, s)
    with pytest.raises(ValueError, match="shape"):
        ops.verify_draft(d, t, u, s, draft_probs=t)
    with pytest.raises(ValueError, match="contiguous"):
        ops.verify_draft(d, t.transpose(1, 2).contiguous().transpose(1, 2), u, s)
    with pytest.raises(ValueError, match="dtype"):
        ops.verify_draft(d.long(), t, u, s)
    with pytest.raises(ValueError, match="no rows"):
        ops.verify_draft(d, t[:, :0], u, s)


def test_cache_refusals():
    cache = cache_of(3, 2, 16, 64, F8)
    k = randn(4, 2, 64).to(BF)
    slots = torch.arange(4, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="shape"):
        ops.kv_write(cache, k[:, :1], k, slots)
    with pytest.raises(ValueError, match="dtype"):
        ops.kv_write(cache, k, k.float(), slots)
    with pytest.raises(ValueError, match="dtype"):
        ops.kv_write(cache, k, k, slots.long())
    with pytest.raises(ValueError, match="rows of heads"):
        ops.kv_write(cache, k.transpose(1, 2).contiguous().transpose(1, 2), k, slots)
    with pytest.raises(ops.N.MoeError, match="own type"):
        ops.kv_write(ops.KvCache(cache.k.to(HF), cache.v.to(HF)), k, k, slots)
    with pytest.raises(ops.N.MoeError, match="overlaps"):
        both = ops.new_kv_cache(3, 2, 16, 64, dtype=BF)
        ops.kv_write(both, both.k[0].transpose(0, 1)[:4].contiguous(), both.k.view(-1, 2, 64)[:4], slots)
    with pytest.raises(ops.N.MoeError, match="page"):
        ops.kv_read(ops.new_kv_cache(3, 2, 24, 64), slots)
    with pytest.raises(ops.N.MoeError, match="dim"):
        ops.kv_read(ops.new_kv_cache(3, 2, 16, 96), slots)
    with pytest.raises(ValueError, match="dtype"):
        ops.kv_read(cache, slots, dtype=torch.float64)


# ---------------------------------------------------------------------------
# The ends of what calls may ask for
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("held,dtype", [(F8, BF), (HF, HF)])
@pytest.mark.parametrize("heads,group,rows,dim,lengths", [
    (1024, 1, 1, 64, [300, 33]), (1, 256, 1, 64, [1000]), (1, 256, 1, 128, [40, 900]),
    (1, 256, 1, 256, [700, 0, 20]), (3, 4, 64, 128, [63, 600])])
def test_attention_of_most_heads_and_rows(held, dtype, heads, group, rows, dim, lengths):
    table, pages = batch_of(lengths, 16)
    cache = cache_of(pages, heads, 16, dim, held)
    q = randn(len(lengths), rows, group * heads, dim, seed=9).to(dtype)
    check(q, cache, table, lengths)
    check(q, cache, table, lengths, window=50)


def test_two_graphs_share_a_workspace():
    cache = cache_of(300, 2, 16, 128, F8)
    ws = ops.AttendWorkspace(8, 4, 16, 2, 128)
    calls = []
    for rows, lengths in ((1, [2500]), (4, [900, 3, 0, 40, 1000, 7, 64, 65])):
        table, _ = batch_of(lengths, 16, seed=rows)
        q = randn(len(lengths), rows, 16, 128, seed=rows).to(BF)
        n = torch.tensor(lengths, dtype=torch.int32, device="cuda")
        want = check(q, cache, table, lengths)
        ops.attend_paged(q, cache, table, n, ws=ws)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = ops.attend_paged(q, cache, table, n, ws=ws)
        calls.append((graph, out, want, q, table, n))      # a graph reads where they lie
    for _ in range(3):
        for graph, out, want, *_ in calls:
            out.fill_(7)
            graph.replay()
            assert torch.equal(out, want)


def test_verify_counts_the_largest_sums():
    """2^19 weights of 1, by clusters of 256 threads as well as of 512."""
    vocab = 1 << 19
    for batch in (38, 39):
        target = torch.ones(batch, 1, vocab, device="cuda")
        u = torch.rand(batch, generator=gen(3), device="cuda")
        u[0], u[1] = 0.0, 1 - 2.0 ** -24
        none = torch.empty(batch, 0, device="cuda")
        r = ops.verify_draft(none.int(), target, none, u)
        assert torch.equal(r.tokens[:, 0].double(), torch.floor(u.double() * vocab))
        target[:, :, 7::8] = 0         # rows of another sum, and places that none falls to
        r = ops.verify_draft(none.int(), target, none, u)
        at = torch.floor(u.double() * (vocab // 8 * 7))
        assert torch.equal(r.tokens[:, 0].double(), torch.floor(at / 7) + at)


def test_verify_of_the_largest_batch():
    batch, vocab = 65535, 5
    want = torch.randint(0, vocab, (batch, 2), generator=gen(1), device="cuda")
    target = torch.nn.functional.one_hot(want, vocab).float()
    draft = torch.randint(0, vocab, (batch, 1), generator=gen(2), device="cuda").int()
    u = torch.rand(batch, 1, generator=gen(3), device="cuda")
    r = ops.verify_draft(draft, target, u, u[:, 0].contiguous())
    good = draft[:, 0] == want[:, 0]
    assert torch.equal(r.accepted, good.int())
    assert torch.equal(r.tokens[:, 0], want[:, 0].int())
    assert torch.equal(r.tokens[:, 1], torch.where(good, want[:, 1], -1).int())

"""GPU tests of a decoding step made of the operators together: the attention of a
layer over a paged cache (fp8_layer), the MoE layer behind it, and the verification
of the tokens that were drafted for it."""
import pytest
import torch

from routed_moe_decode_router_gb300 import fp8_layer, ops
from tests import decode_ref as D
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


def randn(*shape, seed=0, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(5000 + seed)
    return torch.randn(*shape, generator=g, device="cuda") * std


def cache_for(lengths, rows, page, heads, dim, dtype):
    """A cache with the sequences' tokens but the last `rows`, and their tables."""
    counts = [-(-n // page) for n in lengths]
    pages = sum(counts) + 1
    ids = torch.randperm(pages, device="cuda").int()
    table = torch.full((len(lengths), max(counts) + 1), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(counts):
        table[b, :n] = ids[at:at + n]
        at += n
    cache = ops.new_kv_cache(pages, heads, page, dim, dtype)
    for b, n in enumerate(lengths):
        if n > rows:
            slots = fp8_layer.new_slots(table[b:b + 1], torch.tensor([n - rows], device="cuda"),
                                        n - rows, page).flatten()
            k, v = (randn(n - rows, heads, dim, seed=10 * b + i).to(BF) for i in range(2))
            ops.kv_write(cache, k, v, slots)
    return cache, table, torch.tensor(lengths, dtype=torch.int32, device="cuda")


def test_new_slots():
    table = torch.tensor([[5, 2, -1], [7, 7, 7], [1, 0, 3]], dtype=torch.int32)
    lengths = torch.tensor([20, 2, 49], dtype=torch.int32)
    got = fp8_layer.new_slots(table, lengths, 4, 16)
    assert got.tolist() == [[32, 33, 34, 35], [-1, -1, 112, 113], [61, 62, 63, -1]]
    assert fp8_layer.new_slots(table, torch.tensor([34, 0, 0]), 3, 16).tolist() == [[47, -1, -1], [-1] * 3, [-1] * 3]


@pytest.mark.parametrize("dtype", [F8, BF])
@pytest.mark.parametrize("rows,window", [(1, 0), (4, 0), (3, 25)])
def test_attention_layer(dtype, rows, window):
    heads, kv, dim, hidden, page = 8, 2, 64, 256, 16
    lay = fp8_layer.random_attention(hidden, heads, kv, dim, seed=1, window=window)
    cache, table, lengths = cache_for([40, 3, 77, 1], rows, page, kv, dim, dtype)
    x, r = randn(4, rows, hidden, seed=90).to(BF), randn(4, rows, hidden, seed=91).to(BF)
    before = [None if t is None else t.clone() for t in cache]
    out, res = lay.forward(x, cache, table, lengths, residual=r, ws=lay.workspace(4, rows))
    # the same product, its keys and values in their slots and nothing else touched
    n = ops.rms_norm(x.flatten(0, 1), lay.norm, residual=r.flatten(0, 1), quantize=True)
    qkv = ops.matmul_fp8(n.q, n.scales, *lay.qkv).view(4 * rows, -1, dim)
    again = ops.KvCache(*before)
    slots = fp8_layer.new_slots(table, lengths, rows, page).flatten()
    ops.kv_write(again, qkv[:, heads:heads + kv].contiguous(), qkv[:, heads + kv:].contiguous(), slots)
    for a, b in zip(cache, again):
        assert a is b is None or torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    want, bound = D.attend(qkv[:, :heads].unflatten(0, (4, rows)), cache, table, lengths, window=window)
    a = ops.attend_paged(qkv[:, :heads].unflatten(0, (4, rows)), cache, table, lengths, window=window)
    assert ((a.double() - want).abs() <= bound).all()
    assert torch.equal(out.flatten(0, 1), torch.mm(a.view(4 * rows, -1), lay.out.t()))
    assert torch.equal(res.flatten(0, 1), n.residual)


def test_rotation_is_asked_for_with_the_positions():
    seen = []

    def rotate(q, k, pos):
        seen.append(pos.tolist())
        return -q, -k
    lay = fp8_layer.random_attention(256, 4, 2, 64, seed=1, rotate=rotate)
    plain = fp8_layer.random_attention(256, 4, 2, 64, seed=1)
    x = randn(2, 2, 256, seed=3).to(BF)
    outs = []
    for layer in (lay, plain):       # both turned: the scores stay, with nothing else in the cache
        cache, table, lengths = cache_for([2, 1], 2, 16, 2, 64, BF)
        outs.append(layer.forward(x, cache, table, lengths)[0])
    assert seen == [[0, 1, 0, 0]]
    assert torch.equal(*outs)


def test_wrong_heads_are_refused():
    w = fp8_layer.quantize_weights(randn(6 * 64, 128))
    with pytest.raises(ValueError, match="heads"):
        fp8_layer.Fp8AttentionLayer(randn(128).to(BF), w, randn(128, 5 * 64).to(BF), 4, 1)


@pytest.mark.parametrize("captured", [False, True])
def test_speculative_step(captured):
    """Three sequences with drafted tokens, one of them with fewer, through attention
    and experts to the target's probabilities, and the drafts that stay."""
    drafts, vocab, hidden = 3, 777, 256
    rows = drafts + 1
    attention = fp8_layer.random_attention(hidden, 8, 2, 64, seed=1)
    experts = fp8_layer.random_layer(hidden, 16, 128, 4, seed=2)
    embed, head = randn(vocab, hidden, seed=4).to(BF), randn(vocab, hidden, seed=5, std=0.2).to(BF)
    cache, table, lengths = cache_for([30, 17, 70], rows, 16, 2, 64, F8)
    ws = attention.workspace(3, rows)
    q = torch.softmax(randn(3, drafts, vocab, seed=6, std=2.0), -1)
    first = torch.tensor([[1], [2], [3]], device="cuda")
    draft = torch.multinomial(q.flatten(0, 1), 1).view(3, drafts).int()
    draft[1, 2] = -1
    u, s = torch.rand(3, drafts, device="cuda"), torch.rand(3, device="cuda")

    def step():
        x = embed[torch.cat([first, draft.clamp(min=0).long()], 1)]
        a, res = attention.forward(x, cache, table, lengths, ws=ws)
        y, res = experts.forward(a.flatten(0, 1), res.flatten(0, 1).contiguous())
        logits = (y + res).float() @ head.t().float()
        probs = torch.softmax(logits, -1).view(3, rows, vocab)
        return probs, ops.verify_draft(draft, probs, u, s, draft_probs=q)
    probs, got = step()
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            probs, got = step()
        u.uniform_()
        graph.replay()
    tokens, accepted = D.verify(draft, probs, u, s, q)
    assert torch.equal(got.tokens.cpu(), tokens) and torch.equal(got.accepted.cpu(), accepted)
    # the next step goes on from what stayed
    after = lengths - rows + 1 + got.accepted
    assert (after >= lengths - rows + 1).all() and (after <= lengths).all()

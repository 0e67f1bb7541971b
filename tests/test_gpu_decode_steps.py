"""GPU tests of decoding steps one after the other: what a verify step leaves in the
cache, and the steps that go on from it."""
import math

import pytest
import torch

from routed_moe_decode_router_gb300 import fp8_layer, ops
from tests import decode_ref as D
from tests.ops_ref import F8

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
HEADS, KV, DIM, HIDDEN, PAGE, VOCAB, DRAFTS = 8, 2, 64, 256, 16, 777, 3
ROWS = DRAFTS + 1


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    yield
    assert ops.device_status() == 0


class Model:
    """One layer, an embedding and a head; sequences of `before` tokens in its cache."""

    def __init__(self, before, dtype):
        self.g = torch.Generator(device="cuda").manual_seed(77)
        self.attention = fp8_layer.random_attention(HIDDEN, HEADS, KV, DIM, seed=1)
        self.experts = fp8_layer.random_layer(HIDDEN, 16, 128, 4, seed=2)
        self.embed = self.randn(VOCAB, HIDDEN).to(BF)
        self.head = (self.randn(VOCAB, HIDDEN) * 0.2)
        self.batch, self.width = len(before), 8
        pages = self.batch * self.width
        self.table = torch.randperm(pages, generator=self.g, device="cuda").view(self.batch, -1).int()
        self.cache = ops.new_kv_cache(pages, KV, PAGE, DIM, dtype)
        self.ws = self.attention.workspace(self.batch, ROWS)
        for b, n in enumerate(before):
            slots = self.slots(b, range(n))
            k, v = self.randn(n, KV, DIM).to(BF), self.randn(n, KV, DIM).to(BF)
            ops.kv_write(self.cache, k, v, slots)

    def randn(self, *shape):
        return torch.randn(*shape, generator=self.g, device="cuda")

    def slots(self, b, positions):
        return torch.tensor([int(self.table[b, j // PAGE]) * PAGE + j % PAGE for j in positions],
                            dtype=torch.int32, device="cuda")

    def probs(self, tokens, cache, lengths):
        """The target's probabilities after each of the tokens [B, R]."""
        a, res = self.attention.forward(self.embed[tokens.clamp(min=0).long()], cache, self.table,
                                        lengths, ws=self.ws)
        y, res = self.experts.forward(a.flatten(0, 1), res.flatten(0, 1).contiguous())
        return torch.softmax((y + res).float() @ self.head.t(), -1).unflatten(0, (self.batch, -1))


def drafts_for(m, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    q = torch.softmax(torch.randn(m.batch, DRAFTS, VOCAB, generator=g, device="cuda") * 2, -1)
    draft = torch.multinomial(q.flatten(0, 1), 1, generator=g).view(m.batch, DRAFTS).int()
    return q, draft, torch.rand(m.batch, DRAFTS, generator=g, device="cuda") * 0.05, \
        torch.rand(m.batch, generator=g, device="cuda")


@pytest.mark.parametrize("dtype", [F8, BF])
def test_a_step_goes_on_from_the_tokens_that_stayed(dtype):
    """Two verify steps; the second sees the same as over a cache that holds the tokens
    that stayed and, everywhere else, NaN.  Each is replayed from a graph as well."""
    before = [30, 17, 70, 0]
    m = Model(before, dtype)
    first = torch.tensor([[1], [2], [3], [4]], dtype=torch.int32, device="cuda")
    n = torch.tensor(before, dtype=torch.int32, device="cuda")
    for step in range(2):
        q, draft, u, s = drafts_for(m, step)
        draft[1, 2] = -1
        tokens, lengths = torch.cat([first, draft], 1), n + ROWS
        kept = [None if t is None else t.clone() for t in m.cache]

        def run():
            probs = m.probs(tokens, m.cache, lengths)
            return probs, ops.verify_draft(draft, probs, u, s, draft_probs=q)
        probs, got = run()
        after = [None if t is None else t.clone() for t in m.cache]
        want = D.verify(draft, probs, u, s, q)
        assert torch.equal(got.tokens.cpu(), want[0]) and torch.equal(got.accepted.cpu(), want[1])
        for t, old in zip(m.cache, kept):
            if t is not None:
                t.copy_(old)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            again = run()
        graph.replay()
        assert torch.equal(again[0], probs) and torch.equal(again[1].tokens, got.tokens)
        for t, new in zip(m.cache, after):
            assert t is None or torch.equal(t.view(torch.uint8), new.view(torch.uint8))
        # the same over the tokens before and nothing else that is a number
        clean = ops.KvCache(*(None if t is None else torch.full_like(t.float(), math.nan).to(t.dtype)
                              for t in m.cache))
        for b in range(m.batch):
            held = m.slots(b, range(int(n[b]))).long()
            at = held // PAGE, slice(None), held % PAGE
            for t, src in zip(clean, kept):
                if t is not None:
                    flat = t.view(torch.uint8) if t.dtype == F8 else t
                    flat[at] = (src.view(torch.uint8) if t.dtype == F8 else src)[at]
        assert torch.equal(m.probs(tokens, clean, lengths), probs)
        assert probs.isfinite().all()
        first = got.tokens.gather(1, got.accepted[:, None].long())
        n = n + 1 + got.accepted
    assert 0 < int(n.sum()) - sum(before) - 2 * m.batch < 2 * m.batch * DRAFTS   # some stayed, some not


@pytest.mark.parametrize("dtype", [F8, BF])
def test_rows_of_a_verify_step_are_steps_of_one_token(dtype):
    """Each row's attention is that of a step which ends with its token."""
    before = [30, 17, 70, 0]
    m = Model(before, dtype)
    lengths = torch.tensor(before, dtype=torch.int32, device="cuda") + ROWS
    m.probs(torch.arange(m.batch * ROWS, device="cuda").view(m.batch, ROWS), m.cache, lengths)
    q = m.randn(m.batch, ROWS, HEADS, DIM).to(BF)
    together = ops.attend_paged(q, m.cache, m.table, lengths)
    for r in range(ROWS):
        n = lengths - ROWS + 1 + r
        want, bound = D.attend(q[:, r:r + 1], m.cache, m.table, n)
        one = ops.attend_paged(q[:, r], m.cache, m.table, n)
        assert ((one.double() - want[:, 0]).abs() <= bound[:, 0]).all()
        assert ((together[:, r].double() - want[:, 0]).abs() <= bound[:, 0]).all()


@pytest.mark.parametrize("dtype", [F8, BF])
@pytest.mark.parametrize("batch,length,window", [(1, 40, 0), (4, 300, 0), (3, 1000, 0), (40, 700, 0), (2, 5000, 90)])
def test_each_call_sees_what_the_one_before_it_wrote(dtype, batch, length, window):
    """Calls that start while the one before still runs: the same slots written, read
    and attended to in turn, with other values each time, from one graph."""
    g = torch.Generator(device="cuda").manual_seed(9)
    steps, heads = 12, 4
    width = length // PAGE + 1
    cache = ops.new_kv_cache(batch * width, heads, PAGE, 128, dtype)
    table = torch.randperm(batch * width, generator=g, device="cuda").view(batch, width).int()
    lengths = torch.full((batch,), length, dtype=torch.int32, device="cuda")
    every = fp8_layer.new_slots(table, lengths, length, PAGE).flatten()
    last = fp8_layer.new_slots(table, lengths, 2, PAGE).flatten()
    q = torch.randn(batch, 2, 8, 128, generator=g, device="cuda").to(BF)
    rows = [torch.randn(2, len(s), heads, 128, generator=g, device="cuda").to(BF)
            for s in (every, last) * steps]
    ws = ops.AttendWorkspace(batch, 2, 8, heads, 128)

    def run(wait):
        out = []
        for i in range(steps):
            for j, slots in enumerate((every, last)):
                ops.kv_write(cache, *rows[2 * i + j], slots)
                wait()
                for call in (lambda: ops.attend_paged(q, cache, table, lengths, window=window, ws=ws),
                             lambda: torch.stack(ops.kv_read(cache, last))):
                    out.append(call())
                    wait()
        return out
    want = run(torch.cuda.synchronize)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run(lambda: None)
    for _ in range(5):
        for t in got:
            t.fill_(7)
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(got, want))

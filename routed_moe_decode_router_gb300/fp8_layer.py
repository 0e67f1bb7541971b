"""A routed MoE layer with FP8 weights, for any number of token rows, and the
attention before it: the operators of ops.py as one step of a model, from the
previous layer's output to this layer's.

    norm (+ residual)  ->  queries, keys, values  ->  cache  ->  attention
                       ->  output product
    norm (+ residual)  ->  router logits  ->  experts of each row
                       ->  shared expert  ->  routed experts, added to it

``python -m routed_moe_decode_router_gb300.fp8_layer`` runs a layer of the
decode workload's shape with random weights over one, 64 and 4096 rows, and both
halves of it over one new token of 1 and 64 sequences and four of 16.
"""
from __future__ import annotations

from typing import NamedTuple, Optional

import torch

from . import ops

_E4M3_MAX = 448.0


class Fp8Weights(NamedTuple):
    codes: torch.Tensor     # float8_e4m3fn [..., N, K]
    scales: torch.Tensor    # float32 [..., ceil(N / 128), ceil(K / 128)]


def quantize_weights(w: torch.Tensor) -> Fp8Weights:
    """w [..., N, K] as e4m3 codes with one scale per block of 128 x 128 (a
    load-time step, in plain PyTorch)."""
    n, k = w.shape[-2:]
    nb, kb = -(-n // 128), -(-k // 128)
    pad = torch.nn.functional.pad(w.float(), (0, kb * 128 - k, 0, nb * 128 - n))
    blocks = pad.unflatten(-1, (kb, 128)).unflatten(-3, (nb, 128))   # [..., nb, 128, kb, 128]
    scales = blocks.abs().amax((-3, -1)).clamp(min=1e-30) / _E4M3_MAX
    codes = (blocks / scales[..., :, None, :, None]).clamp(-_E4M3_MAX, _E4M3_MAX)
    codes = codes.flatten(-2).flatten(-3, -2)[..., :n, :k].to(ops.F8).contiguous()
    return Fp8Weights(codes, scales.contiguous())


class Fp8MoeLayer:
    """The layer's weights on a CUDA device, and its forward call.

    norm [H] (bf16); router [E, H] and, with a gated shared expert, its gate
    vector [H], which become one matrix (the gate as its last row); gate, up
    [E, I, H] and down [E, H, I]; shared: the same three matrices
    [1, Is, H] / [1, H, Is] or None, its output added as it is without a gate
    vector.  The routing arguments are those of ops.route_topk.

    router_fp8: the router's matrix as FP8 weights, the logits from the FP8
    rows that the experts read, in one of the package's products; which of two
    experts with near logits is taken then depends on the rounding to e4m3.
    False, for a router trained in bf16 or fp32: its matrix in fp32, the logits
    an fp32 matrix product with the normed rows in bf16."""

    def __init__(self, norm: torch.Tensor, router: torch.Tensor, gate: Fp8Weights,
                 up: Fp8Weights, down: Fp8Weights, top_k: int, *,
                 shared: Optional[tuple] = None, shared_gate: Optional[torch.Tensor] = None,
                 router_fp8: bool = True, eps: float = 1e-6,
                 bias: Optional[torch.Tensor] = None, **routing):
        if shared is None and shared_gate is not None:
            raise ValueError("shared_gate is given without shared")
        self.norm, self.eps, self.top_k = norm, eps, top_k
        self.experts = router.shape[0]
        if shared_gate is not None:
            router = torch.cat([router, shared_gate[None].to(router.dtype)])
        self.router = quantize_weights(router) if router_fp8 else router.float()
        self.router_fp8 = router_fp8
        self.routed = (*gate, *up, *down)
        self.shared = None if shared is None else tuple(t for w in shared for t in w)
        self.shared_gated = shared_gate is not None
        self.bias, self.routing = bias, routing

    def logits(self, n: ops.NormOut) -> torch.Tensor:
        """[T, E] (and the shared gate's column) in fp32 of the normed rows."""
        if self.router_fp8:
            return ops.matmul_fp8(n.q, n.scales, *self.router, out_dtype=torch.float32)
        return torch.mm(n.y.float(), self.router.t())

    def forward(self, x: torch.Tensor, residual: Optional[torch.Tensor] = None):
        """(out, residual) [T, H] bf16 of x and the running residual: out is
        what the next layer's norm adds to the returned residual."""
        n = ops.rms_norm(x, self.norm, eps=self.eps, residual=residual, quantize=True,
                         keep=not self.router_fp8)
        logits = self.logits(n)
        ids, wts = ops.route_topk(logits[:, :self.experts], self.top_k, bias=self.bias,
                                  **self.routing)
        out = None
        if self.shared is not None:
            # the shared expert is one expert that every row chooses, its
            # weight 1 or the sigmoid of the gate row's logit
            if self.shared_gated:
                one, gate = ops.route_topk(logits[:, self.experts:], 1, scoring="sigmoid",
                                           norm_topk_prob=False)
            else:
                one, gate = torch.zeros_like(ids[:, :1]), torch.ones_like(wts[:, :1])
            out = ops.experts_fp8(n.q, n.scales, one, gate, *self.shared)
        out = ops.experts_fp8(n.q, n.scales, ids, wts, *self.routed, addend=out, out=out)
        return out, x if residual is None else n.residual


def new_slots(table: torch.Tensor, lengths: torch.Tensor, rows: int, page: int,
              counts: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The slots [B, rows] (int32) of the last `rows` tokens of sequences whose
    pages are table [B, W] and whose lengths, these tokens among them, are lengths
    [B]; -1 for positions before the first token or behind the table, for page
    numbers that no cache has, and with counts [B] for all but the last counts[b]
    tokens."""
    pos = lengths[:, None] - rows + torch.arange(rows, device=table.device)
    at = torch.div(pos, page, rounding_mode="floor")
    ids = table.gather(1, at.clamp(0, table.shape[1] - 1).long()).long()
    slots = ids * page + pos % page
    there = (pos >= 0) & (at < table.shape[1]) & (ids >= 0) & (slots < 1 << 31)
    if counts is not None:
        if counts.shape != lengths.shape:
            raise ValueError("counts has shape %s, expected %s" % (tuple(counts.shape), tuple(lengths.shape)))
        there &= pos >= (lengths - counts)[:, None]
    return torch.where(there, slots, -1).to(torch.int32)


class Fp8AttentionLayer:
    """The attention of a layer over a paged cache, and its forward call.

    norm [H] (bf16); qkv: FP8 weights [(heads + 2 kv_heads) dim, H], queries, keys
    and values in this order; out [H, heads dim] (bf16; its product is PyTorch's).
    rotate: (q, k, positions) -> (q, k), the position embedding of queries
    [T, heads, dim] and keys [T, kv_heads, dim], or None.  window and scale as in
    ops.attend_paged."""

    def __init__(self, norm: torch.Tensor, qkv: Fp8Weights, out: torch.Tensor, heads: int,
                 kv_heads: int, *, eps: float = 1e-6, rotate=None, window: int = 0,
                 scale: Optional[float] = None):
        dim, rest = divmod(qkv.codes.shape[0], heads + 2 * kv_heads)
        if rest or out.shape[1] != heads * dim:
            raise ValueError("qkv has %d rows and out %d columns, which are not those of %d and %d "
                             "heads" % (qkv.codes.shape[0], out.shape[1], heads, kv_heads))
        self.norm, self.qkv, self.out = norm, qkv, out
        self.heads, self.kv_heads, self.dim = heads, kv_heads, dim
        self.eps, self.rotate, self.window, self.scale = eps, rotate, window, scale

    def workspace(self, batch: int, rows: int) -> ops.AttendWorkspace:
        return ops.AttendWorkspace(batch, rows, self.heads, self.kv_heads, self.dim)

    def forward(self, x: torch.Tensor, cache: ops.KvCache, table: torch.Tensor,
                lengths: torch.Tensor, residual: Optional[torch.Tensor] = None,
                ws: Optional[ops.AttendWorkspace] = None, counts: Optional[torch.Tensor] = None):
        """(out, residual) [B, R, H] bf16 of the last R tokens x of B sequences:
        their keys and values are written to the cache, and they see what it then
        holds.  table [B, W] and lengths [B] (the new tokens among them) as in
        ops.attend_paged.  counts [B]: how many of its R rows a sequence's new tokens
        are, the last ones; without it all are, and overwrite what the cache has at
        their positions.  The other rows are not written, and what comes out for
        them is of no token.  Lengths are within the table: tokens behind it are not
        written, and their rows see what the last of it do."""
        b, r, h = x.shape
        flat = None if residual is None else residual.reshape(b * r, h)
        n = ops.rms_norm(x.reshape(b * r, h), self.norm, eps=self.eps, residual=flat,
                         quantize=True, keep=False)
        rows = ops.matmul_fp8(n.q, n.scales, *self.qkv).unflatten(1, (-1, self.dim))
        q, k, v = rows.split([self.heads, self.kv_heads, self.kv_heads], dim=1)
        if self.rotate is not None:
            pos = lengths[:, None] - r + torch.arange(r, device=x.device)
            q, k = self.rotate(q, k, pos.clamp(min=0).flatten())
        slots = new_slots(table, lengths, r, cache.k.shape[2], counts)
        ops.kv_write(cache, k, v, slots.flatten())
        a = ops.attend_paged(q.unflatten(0, (b, r)), cache, table, lengths, scale=self.scale,
                             window=self.window, ws=ws)
        out = torch.mm(a.view(b * r, self.heads * self.dim), self.out.t()).view(b, r, h)
        return out, x if residual is None else n.residual.view(b, r, h)


def random_attention(hidden: int, heads: int, kv_heads: int, dim: int, seed: int = 0,
                     device="cuda", **kw) -> Fp8AttentionLayer:
    """An attention layer with weights N(0, 0.02)."""
    g = torch.Generator(device=device).manual_seed(seed)

    def normal(*shape, std=0.02):
        return torch.randn(*shape, generator=g, device=device) * std

    return Fp8AttentionLayer((1 + normal(hidden)).to(torch.bfloat16),
                             quantize_weights(normal((heads + 2 * kv_heads) * dim, hidden)),
                             normal(hidden, heads * dim).to(torch.bfloat16), heads, kv_heads, **kw)


def random_layer(hidden: int, experts: int, inter: int, top_k: int, seed: int = 0,
                 device="cuda", shared_inter: int = 0, shared_gated: bool = True,
                 router_fp8: bool = True, **routing) -> Fp8MoeLayer:
    """A layer with weights N(0, 0.02), as the package's synthetic layers."""
    g = torch.Generator(device=device).manual_seed(seed)

    def normal(*shape, std=0.02):
        return torch.randn(*shape, generator=g, device=device) * std

    def stack(e, n, k):
        return quantize_weights(normal(e, n, k))

    shared = gate = None
    if shared_inter:
        shared = (stack(1, shared_inter, hidden), stack(1, shared_inter, hidden),
                  stack(1, hidden, shared_inter))
        gate = normal(hidden) if shared_gated else None
    bias = None
    if routing.get("scoring") == "sigmoid":
        bias = torch.rand(experts, generator=g, device=device) * 0.2 - 0.1
    return Fp8MoeLayer((1 + normal(hidden)).to(torch.bfloat16), normal(experts, hidden),
                       stack(experts, inter, hidden), stack(experts, inter, hidden),
                       stack(experts, hidden, inter), top_k, shared=shared, shared_gate=gate,
                       router_fp8=router_fp8, bias=bias, **routing)


def _timed(run):
    """(outputs, microseconds) of a call, replayed from a CUDA graph."""
    run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    for _ in range(3):
        graph.replay()
    start.record()
    for _ in range(20):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    return out, start.elapsed_time(end) / 20 * 1e3


def main():
    layer = random_layer(2048, 128, 768, 8, shared_inter=768)
    for rows in (1, 64, 4096):
        x = torch.randn(rows, 2048, device="cuda").to(torch.bfloat16)
        r = torch.randn(rows, 2048, device="cuda").to(torch.bfloat16)
        (out, _), us = _timed(lambda: layer.forward(x, r))
        if ops.device_status() != 0 or not torch.isfinite(out).all():
            raise RuntimeError("the layer of %d rows did not finish" % rows)
        print("%5d rows: %8.1f us per layer, %10.0f rows/s" % (rows, us, rows / us * 1e6))
    attention = random_attention(2048, 32, 4, 128)
    length, page = 4096, 64
    for batch, rows in ((1, 1), (64, 1), (16, 4)):
        cache = ops.new_kv_cache(batch * length // page, 4, page, 128)
        table = torch.randperm(batch * length // page, device="cuda").view(batch, -1).int()
        lengths = torch.full((batch,), length, dtype=torch.int32, device="cuda")
        x = torch.randn(batch, rows, 2048, device="cuda").to(torch.bfloat16)
        r = torch.randn(batch, rows, 2048, device="cuda").to(torch.bfloat16)
        ws = attention.workspace(batch, rows)

        def step():
            a, res = attention.forward(x, cache, table, lengths, residual=r, ws=ws)
            return layer.forward(a.flatten(0, 1), res.flatten(0, 1))
        (out, _), us = _timed(step)
        if ops.device_status() != 0 or not torch.isfinite(out).all():
            raise RuntimeError("the layer of %d sequences did not finish" % batch)
        print("%5d sequences of %d, %d new tokens each: %8.1f us per layer with its attention"
              % (batch, length, rows, us))


if __name__ == "__main__":
    main()

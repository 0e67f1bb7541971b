"""PyTorch-facing calls of the FP8 layer operators (include/moe_ops.h): norm
with an FP8 output, grouped expert routing, the block-scaled FP8 product and
the routed experts, for any number of token rows; and of a decoding step's
others: the paged cache of keys and values, attention over it, and the
verification of drafted tokens.

Like layer.py it only marshals: tensors are checked by their attributes
before any pointer reaches the library, every step runs in the CUDA library
on the given (or current) stream, and every call can be captured into a CUDA
graph (after a first call outside of one, which looks up what the library
keeps per device).  Outputs made by a call belong to the stream it runs on.
The checks and the output tensors are made in the extension
csrc/ops_binding.cpp.  FP8 rows are float8_e4m3fn [T, K] with float32 scales
[T, ceil(K / 128)]; FP8 weights float8_e4m3fn [N, K] with float32 scales
[ceil(N / 128), ceil(K / 128)] (experts: one more leading dimension).
"""
from __future__ import annotations

import importlib.machinery
import importlib.util
import os
from typing import NamedTuple, Optional

import torch

from . import build as _build
from . import native as N

F8 = torch.float8_e4m3fn
_DTYPES = {torch.bfloat16: N.MOEOP_BF16, torch.float16: N.MOEOP_FP16,
           torch.float32: N.MOEOP_FP32}
_SCORING = {"softmax": N.MOE_SCORING_SOFTMAX, "sigmoid": N.MOE_SCORING_SIGMOID}
_GROUP_SCORE = {"max": N.MOEOP_GROUP_MAX, "top2": N.MOEOP_GROUP_TOP2}


class NormOut(NamedTuple):
    y: Optional[torch.Tensor]          # normed rows, x's type
    residual: Optional[torch.Tensor]   # x + residual, x's type
    q: Optional[torch.Tensor]          # e4m3 codes of the normed rows
    scales: Optional[torch.Tensor]     # one per row and 128 inputs


_ext = None


def _load():
    """The built extension (raises if it was never built, like native.lib())."""
    global _ext
    if _ext is None:
        N.lib()
        if not os.path.exists(_build.BINDING):
            raise RuntimeError("extension %s is missing: build it first "
                               "(python -c 'import __graft_entry__ as g; g.build()')"
                               % _build.BINDING)
        if _build.built_for() != _build.target():
            raise RuntimeError("extension %s was built for %s, this is %s: build it again"
                               % (_build.BINDING, _build.built_for() or "another PyTorch",
                                  _build.target()))
        loader = importlib.machinery.ExtensionFileLoader("_moe_ops", _build.BINDING)
        mod = importlib.util.module_from_spec(
            importlib.util.spec_from_loader("_moe_ops", loader))
        loader.exec_module(mod)
        mod.set_error_class(N.MoeError)
        _ext = mod
    return _ext


def rms_norm(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6,
             residual: Optional[torch.Tensor] = None, quantize: bool = False,
             keep: bool = True, residual_out: Optional[torch.Tensor] = None,
             stream=None) -> NormOut:
    """Root-mean-square norm of x [T, H] (bf16, fp16 or fp32; rows may be
    strided), with the residual added first if there is one, and the sum
    returned.  quantize: also as FP8 rows; keep=False: only as FP8 rows.
    residual_out: where the sum goes (x or residual itself for in place)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return rms_norm(x, weight, eps, residual, quantize, keep, residual_out)
    return NormOut(*(_ext or _load()).rms_norm(x, weight, eps, residual, bool(quantize),
                                               bool(keep), residual_out))


def route_topk(logits: torch.Tensor, top_k: int, scoring: str = "softmax",
               bias: Optional[torch.Tensor] = None, groups: int = 1, group_limit: int = 1,
               group_score: str = "max", norm_topk_prob: bool = True,
               routed_scaling_factor: float = 1.0, stream=None):
    """(ids [T, top_k] int32, wts [T, top_k] float32) of logits [T, E] (fp32,
    bf16 or fp16; rows may be strided), in descending order of the selection
    key.  scoring: "softmax" or "sigmoid"; bias [E] float32 is added for the
    selection only; group_score: "max" or "top2".  Experts whose logit or bias
    is -inf or NaN are not taken: id -1, weight 0 where none is left.  A bias
    of +inf puts its expert first."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return route_topk(logits, top_k, scoring, bias, groups, group_limit, group_score,
                              norm_topk_prob, routed_scaling_factor)
    try:
        scoring_code, score_code = _SCORING[scoring], _GROUP_SCORE[group_score]
    except KeyError:
        raise ValueError("scoring must be 'softmax' or 'sigmoid' and group_score 'max' or 'top2', "
                         "not %r and %r" % (scoring, group_score)) from None
    return (_ext or _load()).route_topk(
        logits, top_k, scoring_code, bias, groups, group_limit, score_code,
        bool(norm_topk_prob), routed_scaling_factor)


def matmul_fp8(a: torch.Tensor, a_scales: torch.Tensor, b: torch.Tensor, b_scales: torch.Tensor,
               out_dtype: torch.dtype = torch.bfloat16, out: Optional[torch.Tensor] = None,
               stream=None) -> torch.Tensor:
    """a [M, K] (FP8 rows) times the transpose of b [N, K] (FP8 weights):
    [M, N] in out_dtype (bf16, fp16 or fp32).  K and the row strides of a and
    b are multiples of 16."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return matmul_fp8(a, a_scales, b, b_scales, out_dtype, out)
    code = _DTYPES.get(out_dtype if out is None else out.dtype)
    if code is None:
        raise ValueError("out_dtype is %s, expected bfloat16, float16 or float32" % out_dtype)
    return (_ext or _load()).matmul_fp8(a, a_scales, b, b_scales, code, out)


class ExpertsWorkspace:
    """Caller-owned scratch of experts_fp8 for calls of up to `rows` rows.
    Calls that overlap on the GPU need one each."""

    def __init__(self, rows: int, top_k: int, hidden: int, inter: int, experts: int,
                 device="cuda"):
        self.nbytes = N.moeop_experts_workspace_size(
            N.ExpertsConfig(hidden, inter, experts, top_k), rows)
        self.buf = torch.empty(self.nbytes, dtype=torch.uint8, device=device)

    @property
    def ptr(self) -> int:
        return self.buf.data_ptr()


def experts_fp8(q: torch.Tensor, scales: torch.Tensor, ids: torch.Tensor, wts: torch.Tensor,
                gate: torch.Tensor, gate_scales: torch.Tensor, up: torch.Tensor,
                up_scales: torch.Tensor, down: torch.Tensor, down_scales: torch.Tensor,
                ws: Optional[ExpertsWorkspace] = None, addend: Optional[torch.Tensor] = None,
                out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The routed experts (SwiGLU) of FP8 rows q [T, H]: bf16 [T, H], the
    weighted sum over each row's experts in slot order (+ addend).  gate, up
    [E, I, H] and down [E, H, I] are FP8 weights, ids / wts [T, k] as
    route_topk gives them (ids outside [0, E) contribute nothing).  Without
    `ws` the scratch comes from PyTorch's allocator for the call."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return experts_fp8(q, scales, ids, wts, gate, gate_scales, up, up_scales, down,
                               down_scales, ws, addend, out)
    return (_ext or _load()).experts_fp8(
        q, scales, ids, wts, gate, gate_scales, up, up_scales, down, down_scales,
        None if ws is None else ws.buf, addend, out)


class KvCache(NamedTuple):
    """A paged cache of keys and values: k, v [pages, heads, page, dim] of bf16,
    fp16 or e4m3, with e4m3 one float32 scale per head and place,
    [pages, heads, page].  Contiguous but for the stride of the pages, so that
    keys and values may lie in one tensor.  page: a multiple of 16 up to 1024;
    dim: 64, 128 or 256.  A slot is a place in it: page number * page + place."""
    k: torch.Tensor
    v: torch.Tensor
    k_scales: Optional[torch.Tensor] = None
    v_scales: Optional[torch.Tensor] = None


def new_kv_cache(pages: int, heads: int, page: int, dim: int, dtype: torch.dtype = F8,
                 device="cuda") -> KvCache:
    """An empty cache (zeros) in e4m3, bf16 or fp16."""
    k, v = (torch.zeros(pages, heads, page, dim, dtype=dtype, device=device) for _ in range(2))
    if dtype != F8:
        return KvCache(k, v)
    return KvCache(k, v, *(torch.zeros(pages, heads, page, device=device) for _ in range(2)))


def kv_write(cache: KvCache, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor,
             stream=None) -> None:
    """Write the keys and values [T, heads, dim] of T tokens to their slots
    (int32 [T]; one outside the cache, as -1, is passed over).  An e4m3 cache
    takes bf16, fp16 or fp32 and quantises: scale = max(amax of the dim, 1e-30) /
    448 (a NaN leaves it to the others; an infinity makes its row NaN); a cache of
    16 bits takes its own type.  Tokens may be strided.  The slots
    of a call are distinct: a slot given twice holds nothing defined."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return kv_write(cache, k, v, slots)
    return (_ext or _load()).kv_write(*cache, k, v, slots)


def kv_read(cache: KvCache, slots: torch.Tensor, dtype: torch.dtype = torch.bfloat16,
            stream=None):
    """(k, v) [T, heads, dim] in dtype (bf16, fp16 or fp32) of the slots (int32
    [T]; one outside the cache gives zeros)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return kv_read(cache, slots, dtype)
    code = _DTYPES.get(dtype)
    if code is None:
        raise ValueError("dtype is %s, expected bfloat16, float16 or float32" % dtype)
    return (_ext or _load()).kv_read(*cache, slots, code)


class AttendWorkspace:
    """Caller-owned scratch of attend_paged for calls of these rows, heads and
    dim and up to `batch` sequences (initialised here, on the current stream).
    Calls that overlap on the GPU need one each."""

    def __init__(self, batch: int, rows: int, q_heads: int, heads: int, dim: int,
                 device="cuda"):
        self.nbytes = N.moeop_attend_workspace_size(batch, rows, q_heads, heads, dim)
        self.buf = torch.zeros(self.nbytes, dtype=torch.uint8, device=device)

    @property
    def ptr(self) -> int:
        return self.buf.data_ptr()


def attend_paged(q: torch.Tensor, cache: KvCache, table: torch.Tensor, lengths: torch.Tensor,
                 scale: Optional[float] = None, window: int = 0,
                 ws: Optional[AttendWorkspace] = None, out: Optional[torch.Tensor] = None,
                 stream=None) -> torch.Tensor:
    """Attention of the last R tokens of each sequence over its cached tokens,
    their own among them (write them first).

    q [B, R, q_heads, dim] (or [B, q_heads, dim], R = 1) in bf16 or fp16, the
    cache's own type where that is one of 16 bits; B and R may be strided.  table
    [B, W] int32: the pages of each sequence in order; lengths [B] int32: its
    tokens.  Row r is at position length - R + r and sees the positions up to its
    own, with a window the last `window` of them.  A page number outside the cache
    (as -1) takes its tokens out; a row that sees nothing is zero, so a free place
    of a batch has length 0, and a sequence with fewer new tokens has them in its
    last rows.  scale: 1 / sqrt(dim) if not given.  Returns q's shape and type."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return attend_paged(q, cache, table, lengths, scale, window, ws, out)
    return (_ext or _load()).attend_paged(*cache, q, table, lengths, scale, window,
                                          None if ws is None else ws.buf, out)


class VerifyOut(NamedTuple):
    tokens: torch.Tensor     # int32 [B, K + 1]: the drafts that stay, one more token, then -1
    accepted: torch.Tensor   # int32 [B]: how many drafts stay


def verify_draft(draft: torch.Tensor, target_probs: torch.Tensor, accept_u: torch.Tensor,
                 sample_u: torch.Tensor, draft_probs: Optional[torch.Tensor] = None,
                 stream=None) -> VerifyOut:
    """Which of the K drafted tokens [B, K] (int32; a negative one ends a
    sequence's drafts) stay, and the token after them, so that what comes out is
    distributed as the target.  target_probs [B, K + 1, V], draft_probs [B, K, V]
    float32 (none: the drafts are certain); accept_u [B, K] and sample_u [B]:
    uniform float32 numbers in [0, 1).  Draft i stays while accept_u * draft_probs <
    target_probs at it; the next token is drawn from max(target - draft, 0) where a
    draft is refused, else from the target, as the lowest id whose running sum
    exceeds sample_u times the whole (-1 where no probability is positive)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return verify_draft(draft, target_probs, accept_u, sample_u, draft_probs)
    return VerifyOut(*(_ext or _load()).verify_draft(draft, target_probs, accept_u, sample_u,
                                                     draft_probs))


def device_status(stream=None) -> int:
    """Synchronise and read (then clear) the operators' device status word."""
    s = stream if stream is not None else torch.cuda.current_stream()
    return N.moeop_read_device_status(s.cuda_stream)

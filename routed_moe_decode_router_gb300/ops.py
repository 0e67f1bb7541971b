"""PyTorch-facing calls of the FP8 layer operators (include/moe_ops.h): norm
with an FP8 output, grouped expert routing, the block-scaled FP8 product and
the routed experts, for any number of token rows.

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


def device_status(stream=None) -> int:
    """Synchronise and read (then clear) the operators' device status word."""
    s = stream if stream is not None else torch.cuda.current_stream()
    return N.moeop_read_device_status(s.cuda_stream)

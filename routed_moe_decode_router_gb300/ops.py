"""PyTorch-facing calls of the FP8 layer operators (include/moe_ops.h): norm
with an FP8 output, grouped expert routing, the block-scaled FP8 product and
the routed experts, for any number of token rows.

Like layer.py it only marshals: tensors are checked by their attributes
before any pointer reaches the library, every step runs in the CUDA library
on the given (or current) stream, and every call can be captured into a CUDA
graph.  FP8 rows are float8_e4m3fn [T, K] with float32 scales
[T, ceil(K / 128)]; FP8 weights float8_e4m3fn [N, K] with float32 scales
[ceil(N / 128), ceil(K / 128)] (experts: one more leading dimension).
"""
from __future__ import annotations

from typing import NamedTuple, Optional

import torch

from . import native as N

F8 = torch.float8_e4m3fn
_DTYPES = {torch.bfloat16: N.MOEOP_BF16, torch.float16: N.MOEOP_FP16,
           torch.float32: N.MOEOP_FP32}


class NormOut(NamedTuple):
    y: Optional[torch.Tensor]          # normed rows, x's type
    residual: Optional[torch.Tensor]   # x + residual, x's type
    q: Optional[torch.Tensor]          # e4m3 codes of the normed rows
    scales: Optional[torch.Tensor]     # one per row and 128 inputs


def _blocks(n: int) -> int:
    return -(-n // N.MOEOP_BLOCK)


def _stream(stream) -> int:
    return (stream if stream is not None else torch.cuda.current_stream()).cuda_stream


def _need(t, name: str, dtype, shape, device, rows_only: bool = False):
    """Refuse a tensor the kernels would misread.  rows_only: a row stride is
    taken, so only the last dimension has to be contiguous."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.dtype != dtype:
        raise ValueError("%s has dtype %s, expected %s" % (name, t.dtype, dtype))
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    if not t.is_contiguous() and not (rows_only and t.dim() == 2 and t.stride(1) == 1):
        raise ValueError("%s must be contiguous%s" % (name, " in its rows" if rows_only else ""))
    if t.device != device:
        raise ValueError("%s is on %s, expected %s" % (name, t.device, device))


def _cuda(t, name: str, dims: int) -> torch.device:
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.dim() != dims:
        raise ValueError("%s has %d dimensions, expected %d" % (name, t.dim(), dims))
    if t.device.type != "cuda":
        raise ValueError("%s is on %s; it must be in CUDA device memory" % (name, t.device))
    if t.device.index != torch.cuda.current_device():
        raise ValueError("%s is on %s, which is not the current device" % (name, t.device))
    return t.device


def _row_stride(t: torch.Tensor) -> int:
    # the stride of a single row means nothing and may be anything
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def _ptr(t: Optional[torch.Tensor]) -> int:
    return 0 if t is None else t.data_ptr()


def rms_norm(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6,
             residual: Optional[torch.Tensor] = None, quantize: bool = False,
             keep: bool = True, residual_out: Optional[torch.Tensor] = None,
             stream=None) -> NormOut:
    """Root-mean-square norm of x [T, H] (bf16, fp16 or fp32; rows may be
    strided), with the residual added first if there is one, and the sum
    returned.  quantize: also as FP8 rows; keep=False: only as FP8 rows.
    residual_out: where the sum goes (x or residual itself for in place)."""
    dev = _cuda(x, "x", 2)
    if x.dtype not in _DTYPES:
        raise ValueError("x has dtype %s, expected bfloat16, float16 or float32" % x.dtype)
    rows, hidden = x.shape
    _need(x, "x", x.dtype, (rows, hidden), dev, rows_only=True)
    _need(weight, "weight", x.dtype, (hidden,), dev)
    if residual is not None:
        _need(residual, "residual", x.dtype, (rows, hidden), dev, rows_only=True)
        if residual_out is None:
            residual_out = torch.empty((rows, hidden), dtype=x.dtype, device=dev)
    elif residual_out is not None:
        raise ValueError("residual_out is given without residual")
    if residual_out is not None:
        _need(residual_out, "residual_out", x.dtype, (rows, hidden), dev)
    if not keep and not quantize:
        raise ValueError("keep=False without quantize leaves no output")
    y = torch.empty((rows, hidden), dtype=x.dtype, device=dev) if keep else None
    q = torch.empty((rows, hidden), dtype=F8, device=dev) if quantize else None
    scales = torch.empty((rows, _blocks(hidden)), dtype=torch.float32,
                         device=dev) if quantize else None
    if rows:
        N.moeop_rms_norm(x.data_ptr(), _row_stride(x), _ptr(residual),
                         0 if residual is None else _row_stride(residual), weight.data_ptr(),
                         rows, hidden, _DTYPES[x.dtype], eps, _ptr(y), _ptr(residual_out),
                         _ptr(q), _ptr(scales), _stream(stream))
    return NormOut(y, residual_out, q, scales)


def route_topk(logits: torch.Tensor, top_k: int, scoring: str = "softmax",
               bias: Optional[torch.Tensor] = None, groups: int = 1, group_limit: int = 1,
               group_score: str = "max", norm_topk_prob: bool = True,
               routed_scaling_factor: float = 1.0, stream=None):
    """(ids [T, top_k] int32, wts [T, top_k] float32) of logits [T, E] (fp32,
    bf16 or fp16; rows may be strided), in descending order of the selection
    key.  scoring: "softmax" or "sigmoid"; bias [E] float32 is added for the
    selection only; group_score: "max" or "top2".  Experts whose logit is
    -inf or NaN are not taken: id -1, weight 0 where none is left."""
    dev = _cuda(logits, "logits", 2)
    if logits.dtype not in _DTYPES:
        raise ValueError("logits has dtype %s, expected float32, bfloat16 or float16"
                         % logits.dtype)
    rows, experts = logits.shape
    _need(logits, "logits", logits.dtype, (rows, experts), dev, rows_only=True)
    if bias is not None:
        _need(bias, "bias", torch.float32, (experts,), dev)
    if scoring not in ("softmax", "sigmoid"):
        raise ValueError("scoring must be 'softmax' or 'sigmoid', not %r" % (scoring,))
    if group_score not in ("max", "top2"):
        raise ValueError("group_score must be 'max' or 'top2', not %r" % (group_score,))
    cfg = N.RouteConfig(
        num_experts=experts, top_k=top_k,
        scoring=N.MOE_SCORING_SIGMOID if scoring == "sigmoid" else N.MOE_SCORING_SOFTMAX,
        groups=groups, group_limit=group_limit,
        group_score=N.MOEOP_GROUP_TOP2 if group_score == "top2" else N.MOEOP_GROUP_MAX,
        norm_topk_prob=int(bool(norm_topk_prob)), routed_scaling_factor=routed_scaling_factor,
        dtype=_DTYPES[logits.dtype])
    if top_k < 0:
        raise ValueError("top_k=%d must not be negative" % top_k)
    ids = torch.empty((rows, top_k), dtype=torch.int32, device=dev)
    wts = torch.empty((rows, top_k), dtype=torch.float32, device=dev)
    N.moeop_route_topk(cfg, _ptr(logits), _row_stride(logits), _ptr(bias), rows, _ptr(ids),
                       _ptr(wts), _stream(stream))
    return ids, wts


def matmul_fp8(a: torch.Tensor, a_scales: torch.Tensor, b: torch.Tensor, b_scales: torch.Tensor,
               out_dtype: torch.dtype = torch.bfloat16, out: Optional[torch.Tensor] = None,
               stream=None) -> torch.Tensor:
    """a [M, K] (FP8 rows) times the transpose of b [N, K] (FP8 weights):
    [M, N] in out_dtype (bf16, fp16 or fp32).  K and the row strides of a and
    b are multiples of 16."""
    dev = _cuda(a, "a", 2)
    _cuda(b, "b", 2)
    m, k = a.shape
    n = b.shape[0]
    _need(a, "a", F8, (m, k), dev, rows_only=True)
    _need(b, "b", F8, (n, k), dev, rows_only=True)
    _need(a_scales, "a_scales", torch.float32, (m, _blocks(k)), dev)
    _need(b_scales, "b_scales", torch.float32, (_blocks(n), _blocks(k)), dev)
    if out is not None:
        out_dtype = out.dtype
    if out_dtype not in _DTYPES:
        raise ValueError("out_dtype is %s, expected bfloat16, float16 or float32" % out_dtype)
    if out is None:
        out = torch.empty((m, n), dtype=out_dtype, device=dev)
    _need(out, "out", out_dtype, (m, n), dev)
    N.moeop_matmul_fp8(_ptr(a), _row_stride(a), _ptr(a_scales), _ptr(b), _row_stride(b),
                       _ptr(b_scales), m, n, k, _ptr(out), _DTYPES[out_dtype], _stream(stream))
    return out


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
    `ws` the scratch comes from PyTorch's allocator for the call, which then
    has to run on the current stream."""
    dev = _cuda(q, "q", 2)
    _cuda(gate, "gate", 3)
    _cuda(ids, "ids", 2)
    t, h = q.shape
    e, inter = gate.shape[:2]
    k = ids.shape[1]
    _need(q, "q", F8, (t, h), dev)
    _need(scales, "scales", torch.float32, (t, _blocks(h)), dev)
    _need(ids, "ids", torch.int32, (t, k), dev)
    _need(wts, "wts", torch.float32, (t, k), dev)
    hb, ib = _blocks(h), _blocks(inter)
    for name, w, sc, shape, sshape in (
            ("gate", gate, gate_scales, (e, inter, h), (e, ib, hb)),
            ("up", up, up_scales, (e, inter, h), (e, ib, hb)),
            ("down", down, down_scales, (e, h, inter), (e, hb, ib))):
        _need(w, name, F8, shape, dev)
        _need(sc, name + "_scales", torch.float32, sshape, dev)
    if addend is not None:
        _need(addend, "addend", torch.bfloat16, (t, h), dev)
    if out is None:
        out = torch.empty((t, h), dtype=torch.bfloat16, device=dev)
    _need(out, "out", torch.bfloat16, (t, h), dev)
    if ws is None:
        if stream is not None and stream != torch.cuda.current_stream():
            raise ValueError("a call on another stream than the current one needs a workspace")
        ws = ExpertsWorkspace(t, k, h, inter, e, device=dev)
    elif ws.buf.device != dev:
        raise ValueError("the workspace is on %s, expected %s" % (ws.buf.device, dev))
    N.moeop_experts_fp8(
        N.ExpertsConfig(h, inter, e, k),
        N.ExpertsWeights(_ptr(gate), _ptr(up), _ptr(down), _ptr(gate_scales), _ptr(up_scales),
                         _ptr(down_scales)),
        _ptr(q), _ptr(scales), _ptr(ids), _ptr(wts), _ptr(addend), _ptr(out), t, ws.ptr,
        ws.nbytes, _stream(stream))
    return out


def device_status(stream=None) -> int:
    """Synchronise and read (then clear) the operators' device status word."""
    return N.moeop_read_device_status(_stream(stream))

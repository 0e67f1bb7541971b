// moeop_api.cu -- host side of the ABI declared in include/moe_ops.h: every
// check, before the first launch.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "moeop.cuh"

using namespace moe;
using namespace moe::op;

namespace {

moe_status fail(moe_status s, const char *fmt, ...) {
    char msg[400];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(msg, sizeof msg, fmt, ap);
    va_end(ap);
    return set_error(s, msg);
}
moe_status ok() {
    set_error(MOE_OK, "");
    return MOE_OK;
}
moe_status launched(cudaError_t e, const char *what) {
    return e == cudaSuccess ? ok() : fail(MOE_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool overlap(const void *a, size_t na, const void *b, size_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return a && b && na && nb && x < y + nb && y < x + na;
}
// Bytes from the first to the last element of `rows` strided rows.
size_t span(int64_t rows, int64_t stride, int64_t cols, size_t size) {
    return rows < 1 ? 0 : ((size_t)(rows - 1) * stride + cols) * size;
}
// NULL or misaligned.
bool bad(const void *p, size_t a) { return !p || !aligned(p, a); }

size_t type_size(int dtype) { return dtype == MOEOP_FP32 ? 4 : 2; }

moe_status check_dtype(int dtype, const char *what) {
    if (dtype < MOEOP_BF16 || dtype > MOEOP_FP32)
        return fail(MOE_ERR_INVALID_ARG, "%s=%d: must be bf16 (0), fp16 (1) or fp32 (2)", what,
                    dtype);
    return MOE_OK;
}

moe_status check_experts(const moeop_experts_config *c, int rows) {
    if (!c) return fail(MOE_ERR_INVALID_ARG, "cfg is NULL");
    if (c->hidden < 128 || c->hidden > 32768 || c->hidden % 128)
        return fail(MOE_ERR_INVALID_ARG, "hidden=%d: must be a multiple of 128 in [128, 32768]",
                    c->hidden);
    if (c->inter < 128 || c->inter > 32768 || c->inter % 128)
        return fail(MOE_ERR_INVALID_ARG, "inter=%d: must be a multiple of 128 in [128, 32768]",
                    c->inter);
    if (c->num_experts < 1 || c->num_experts > MOEOP_MAX_EXPERTS)
        return fail(MOE_ERR_INVALID_ARG, "num_experts=%d: must be in [1, %d]", c->num_experts,
                    MOEOP_MAX_EXPERTS);
    if (c->top_k < 1 || c->top_k > MOEOP_MAX_TOPK)
        return fail(MOE_ERR_INVALID_ARG, "top_k=%d: must be in [1, %d]", c->top_k, MOEOP_MAX_TOPK);
    if (rows < 0 || (int64_t)rows * c->top_k > (1 << 26))
        return fail(MOE_ERR_INVALID_ARG, "rows=%d: rows * top_k must be in [0, 2^26]", rows);
    return MOE_OK;
}

}  // namespace

extern "C" {

moe_status moeop_rms_norm(const void *x, int64_t x_stride, const void *residual,
                          int64_t residual_stride, const void *weight, int rows, int hidden,
                          int dtype, float eps, void *y, void *residual_out, uint8_t *q,
                          float *scales, void *stream) {
    moe_status s;
    if ((s = check_dtype(dtype, "dtype")) != MOE_OK) return s;
    if (rows < 0 || rows > (1 << 30))
        return fail(MOE_ERR_INVALID_ARG, "rows=%d: must be in [0, 2^30]", rows);
    if (hidden < 1 || hidden > MOEOP_MAX_NORM_HIDDEN)
        return fail(MOE_ERR_INVALID_ARG, "hidden=%d: must be in [1, %d]", hidden,
                    MOEOP_MAX_NORM_HIDDEN);
    if (!(eps >= 0.f) || !std::isfinite(eps))
        return fail(MOE_ERR_INVALID_ARG, "eps=%g: must be finite and not negative", (double)eps);
    if (!y && !q) return fail(MOE_ERR_INVALID_ARG, "one of y and q is required");
    if (!q != !scales) return fail(MOE_ERR_INVALID_ARG, "q and scales come together");
    if (rows == 0) return ok();
    const size_t es = type_size(dtype);
    if (bad(x, es) || bad(weight, es) || !aligned(residual, es) || !aligned(y, es) ||
        !aligned(residual_out, es) || !aligned(scales, 4))
        return fail(MOE_ERR_INVALID_ARG, "a pointer is NULL or not aligned to its type");
    if (x_stride < hidden || (residual && residual_stride < hidden))
        return fail(MOE_ERR_INVALID_ARG, "a row stride is less than hidden=%d", hidden);
    const size_t nx = span(rows, x_stride, hidden, es);
    const size_t nr = span(rows, residual_stride, hidden, es);
    const size_t n = (size_t)rows * hidden, ns = (size_t)rows * ((hidden + 127) / 128) * 4;
    const struct { const void *p; size_t n; } outs[4] = {
        {y, n * es}, {residual_out, n * es}, {q, n}, {scales, ns}};
    for (int i = 0; i < 4; ++i) {
        // the sum may be written over the rows it was read from
        const bool over_x = i == 1 && residual_out == x && x_stride == hidden;
        const bool over_r = i == 1 && residual_out == residual && residual_stride == hidden;
        if ((!over_x && overlap(outs[i].p, outs[i].n, x, nx)) ||
            (!over_r && overlap(outs[i].p, outs[i].n, residual, nr)) ||
            overlap(outs[i].p, outs[i].n, weight, hidden * es))
            return fail(MOE_ERR_INVALID_ARG, "an output overlaps an input");
        for (int j = 0; j < i; ++j)
            if (overlap(outs[i].p, outs[i].n, outs[j].p, outs[j].n))
                return fail(MOE_ERR_INVALID_ARG, "two outputs overlap");
    }
    NormParams p{x, residual, weight, x_stride, residual ? residual_stride : 0, rows, hidden, dtype,
                 eps, y, residual_out, q, scales};
    const bool vec = hidden % 8 == 0 && (x_stride * (int64_t)es) % 16 == 0 &&
                     (p.residual_stride * (int64_t)es) % 16 == 0 && aligned(x, 16) &&
                     aligned(residual, 16) && aligned(weight, 16) && aligned(y, 16) &&
                     aligned(residual_out, 16) && aligned(q, 8);
    return launched(launch_rms_norm(p, vec, static_cast<cudaStream_t>(stream)), "norm launch");
}

moe_status moeop_route_topk(const moeop_route_config *cfg, const void *logits,
                            int64_t logits_stride, const float *bias, int rows, int32_t *ids,
                            float *wts, void *stream) {
    if (!cfg) return fail(MOE_ERR_INVALID_ARG, "cfg is NULL");
    const moeop_route_config &c = *cfg;
    moe_status s;
    if ((s = check_dtype(c.dtype, "dtype")) != MOE_OK) return s;
    if (c.num_experts < 1 || c.num_experts > MOEOP_MAX_EXPERTS)
        return fail(MOE_ERR_INVALID_ARG, "num_experts=%d: must be in [1, %d]", c.num_experts,
                    MOEOP_MAX_EXPERTS);
    if (c.groups < 1 || c.groups > MOEOP_MAX_GROUPS || c.num_experts % c.groups)
        return fail(MOE_ERR_INVALID_ARG, "groups=%d: must be in [1, %d] and divide num_experts=%d",
                    c.groups, MOEOP_MAX_GROUPS, c.num_experts);
    if (c.group_limit < 1 || c.group_limit > c.groups)
        return fail(MOE_ERR_INVALID_ARG, "group_limit=%d: must be in [1, groups=%d]",
                    c.group_limit, c.groups);
    const int open = c.group_limit * (c.num_experts / c.groups);
    if (c.top_k < 1 || c.top_k > MOEOP_MAX_TOPK || c.top_k > open)
        return fail(MOE_ERR_INVALID_ARG,
                    "top_k=%d: must be in [1, min(%d, the %d experts of group_limit groups)]",
                    c.top_k, MOEOP_MAX_TOPK, open);
    if (c.scoring != MOE_SCORING_SOFTMAX && c.scoring != MOE_SCORING_SIGMOID)
        return fail(MOE_ERR_INVALID_ARG, "scoring=%d: must be softmax (0) or sigmoid (1)",
                    c.scoring);
    if (c.group_score != MOEOP_GROUP_MAX && c.group_score != MOEOP_GROUP_TOP2)
        return fail(MOE_ERR_INVALID_ARG, "group_score=%d: must be max (0) or top2 (1)",
                    c.group_score);
    if (c.norm_topk_prob & ~1) return fail(MOE_ERR_INVALID_ARG, "norm_topk_prob must be 0 or 1");
    if (!std::isfinite(c.routed_scaling_factor))
        return fail(MOE_ERR_INVALID_ARG, "routed_scaling_factor is not finite");
    if (rows < 0 || rows > (1 << 30))
        return fail(MOE_ERR_INVALID_ARG, "rows=%d: must be in [0, 2^30]", rows);
    if (rows == 0) return ok();
    if (bad(logits, type_size(c.dtype)) || !aligned(bias, 4) || bad(ids, 4) || bad(wts, 4))
        return fail(MOE_ERR_INVALID_ARG, "a pointer is NULL or not aligned to its type");
    if (logits_stride < c.num_experts)
        return fail(MOE_ERR_INVALID_ARG, "the row stride is less than num_experts=%d",
                    c.num_experts);
    const size_t nl = span(rows, logits_stride, c.num_experts, type_size(c.dtype));
    const size_t n = (size_t)rows * c.top_k * 4, nb = (size_t)c.num_experts * 4;
    if (overlap(ids, n, logits, nl) || overlap(wts, n, logits, nl) || overlap(ids, n, wts, n) ||
        overlap(ids, n, bias, nb) || overlap(wts, n, bias, nb))
        return fail(MOE_ERR_INVALID_ARG, "the outputs overlap each other or an input");
    const RouteParams p{c, logits, logits_stride, bias, rows, ids, wts};
    return launched(launch_route_topk(p, static_cast<cudaStream_t>(stream)), "route launch");
}

moe_status moeop_matmul_fp8(const uint8_t *a, int64_t a_stride, const float *a_scales,
                            const uint8_t *b, int64_t b_stride, const float *b_scales, int m,
                            int n, int k, void *out, int out_dtype, void *stream) {
    moe_status s;
    if ((s = check_dtype(out_dtype, "out_dtype")) != MOE_OK) return s;
    if (m < 0) return fail(MOE_ERR_INVALID_ARG, "m=%d: must not be negative", m);
    if (n < 1 || n > (1 << 24)) return fail(MOE_ERR_INVALID_ARG, "n=%d: must be in [1, 2^24]", n);
    if (k < 16 || k > (1 << 24) || k % 16)
        return fail(MOE_ERR_INVALID_ARG, "k=%d: must be a multiple of 16 in [16, 2^24]", k);
    if (((int64_t)m + 127) / 128 * ((n + 127) / 128) > 0x3FFFFFFF)
        return fail(MOE_ERR_INVALID_ARG, "m=%d, n=%d: too many tiles", m, n);
    if (m == 0) return ok();
    if (bad(a, 16) || bad(b, 16))
        return fail(MOE_ERR_INVALID_ARG, "a and b must be 16-byte aligned and not NULL");
    if (bad(a_scales, 4) || bad(b_scales, 4) || bad(out, type_size(out_dtype)))
        return fail(MOE_ERR_INVALID_ARG, "a pointer is NULL or not aligned to its type");
    if (a_stride < k || b_stride < k || a_stride % 16 || b_stride % 16 ||
        a_stride >= (1LL << 40) || b_stride >= (1LL << 40))
        return fail(MOE_ERR_INVALID_ARG,
                    "the row strides must be multiples of 16 of at least k=%d", k);
    const size_t no = (size_t)m * n * type_size(out_dtype), kb = (k + 127) / 128;
    if (overlap(out, no, a, span(m, a_stride, k, 1)) || overlap(out, no, b, span(n, b_stride, k, 1)) ||
        overlap(out, no, a_scales, m * kb * 4) ||
        overlap(out, no, b_scales, ((size_t)n + 127) / 128 * kb * 4))
        return fail(MOE_ERR_INVALID_ARG, "out overlaps an input");
    return launched(launch_matmul_fp8({a, m, k, a_stride}, a_scales, {b, n, k, b_stride}, b_scales,
                                      out, out_dtype, static_cast<cudaStream_t>(stream)),
                    "product launch");
}

size_t moeop_experts_workspace_size(const moeop_experts_config *cfg, int rows) {
    if (check_experts(cfg, rows) != MOE_OK) return 0;
    return ExpertsWs::make(*cfg, rows).total;
}

moe_status moeop_experts_fp8(const moeop_experts_config *cfg, const moeop_experts_weights *w,
                             const uint8_t *q, const float *scales, const int32_t *ids,
                             const float *wts, const uint16_t *addend, uint16_t *out, int rows,
                             void *ws, size_t ws_bytes, void *stream) {
    moe_status s;
    if ((s = check_experts(cfg, rows)) != MOE_OK) return s;
    if (!w) return fail(MOE_ERR_INVALID_ARG, "weights is NULL");
    if (bad(w->gate, 16) || bad(w->up, 16) || bad(w->down, 16))
        return fail(MOE_ERR_INVALID_ARG, "gate, up and down must be 16-byte aligned and not NULL");
    if (bad(w->gate_scales, 4) || bad(w->up_scales, 4) || bad(w->down_scales, 4))
        return fail(MOE_ERR_INVALID_ARG, "a weight scale array is NULL or misaligned");
    if (rows == 0) return ok();
    if (bad(q, 16) || bad(out, 16) || !aligned(addend, 16))
        return fail(MOE_ERR_INVALID_ARG, "q, out and addend must be 16-byte aligned (q, out not NULL)");
    if (bad(scales, 4) || bad(ids, 4) || bad(wts, 4))
        return fail(MOE_ERR_INVALID_ARG, "scales, ids or wts is NULL or misaligned");
    const ExpertsWs L = ExpertsWs::make(*cfg, rows);
    if (!ws) return fail(MOE_ERR_WORKSPACE, "workspace is NULL");
    if (!aligned(ws, 256)) return fail(MOE_ERR_WORKSPACE, "workspace is not 256-byte aligned");
    if (ws_bytes < L.total)
        return fail(MOE_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", ws_bytes, L.total);
    const size_t T = rows, H = cfg->hidden, I = cfg->inter, P = T * cfg->top_k;
    const size_t nw = (size_t)cfg->num_experts * H * I, nsc = nw / 16384 * 4;
    const struct { const void *p; size_t n; bool addend; } ins[] = {
        {q, T * H, false}, {scales, T * (H / 128) * 4, false}, {ids, P * 4, false},
        {wts, P * 4, false}, {addend, T * H * 2, true}, {w->gate, nw, false}, {w->up, nw, false},
        {w->down, nw, false}, {w->gate_scales, nsc, false}, {w->up_scales, nsc, false},
        {w->down_scales, nsc, false}};
    if (overlap(out, T * H * 2, ws, L.total))
        return fail(MOE_ERR_INVALID_ARG, "out overlaps the workspace");
    for (const auto &in : ins) {
        if (overlap(ws, L.total, in.p, in.n))
            return fail(MOE_ERR_INVALID_ARG, "the workspace overlaps an input");
        if (!(in.addend && in.p == out) && overlap(out, T * H * 2, in.p, in.n))
            return fail(MOE_ERR_INVALID_ARG, "out overlaps an input");
    }
    const ExpertsArgs a{*cfg, *w, q, scales, ids, wts, addend, out, rows, static_cast<char *>(ws)};
    return launched(launch_experts_fp8(a, static_cast<cudaStream_t>(stream)), "experts launch");
}

moe_status moeop_read_device_status(int *code, void *stream) {
    if (!code) return fail(MOE_ERR_INVALID_ARG, "code is NULL");
    uint32_t *word = nullptr, v = 0;
    cudaError_t e = cudaStreamSynchronize(static_cast<cudaStream_t>(stream));
    if (e == cudaSuccess) e = status_word(&word);
    if (e == cudaSuccess) e = cudaMemcpy(&v, word, sizeof v, cudaMemcpyDeviceToHost);
    if (e == cudaSuccess && v) e = cudaMemset(word, 0, sizeof v);
    if (e != cudaSuccess) return fail(MOE_ERR_CUDA, "status read: %s", cudaGetErrorString(e));
    *code = (int)v;
    if (v) return fail(MOE_ERR_DEVICE_STATUS, "device status %u", v);
    return ok();
}

}  // extern "C"

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

// Rows of `na` bytes every `sa` from a and of `nb` every `sb` from b share no byte:
// they lie apart, or in turn in strides of one size.
bool apart(const void *a, int64_t sa, int64_t na, const void *b, int64_t sb, int64_t nb,
           int64_t rows) {
    if (!overlap(a, span(rows, sa, na, 1), b, span(rows, sb, nb, 1))) return true;
    if (sa != sb || rows < 2) return false;
    int64_t d = (int64_t)(reinterpret_cast<intptr_t>(b) - reinterpret_cast<intptr_t>(a)) % sa;
    if (d < 0) d += sa;
    return d >= na && d + nb <= sa;
}
moe_status check_cache(const moeop_kv_cache *c) {
    if (!c) return fail(MOE_ERR_INVALID_ARG, "cache is NULL");
    if (c->type != MOEOP_BF16 && c->type != MOEOP_FP16 && c->type != MOEOP_E4M3)
        return fail(MOE_ERR_INVALID_ARG, "type=%d: must be bf16 (0), fp16 (1) or e4m3 (3)", c->type);
    if (c->dim != 64 && c->dim != 128 && c->dim != 256)
        return fail(MOE_ERR_INVALID_ARG, "dim=%d: must be 64, 128 or 256", c->dim);
    if (c->page < 16 || c->page > 1024 || c->page % 16)
        return fail(MOE_ERR_INVALID_ARG, "page=%d: must be a multiple of 16 in [16, 1024]", c->page);
    if (c->heads < 1 || c->heads > 1024)
        return fail(MOE_ERR_INVALID_ARG, "heads=%d: must be in [1, 1024]", c->heads);
    if (c->pages < 1 || (int64_t)c->pages * c->page > INT32_MAX)
        return fail(MOE_ERR_INVALID_ARG, "pages=%d: pages * page must be in [1, 2^31)", c->pages);
    const bool f8 = c->type == MOEOP_E4M3;
    const int64_t places = (int64_t)c->heads * c->page, es = f8 ? 1 : 2;
    if (bad(c->k, 16) || bad(c->v, 16))
        return fail(MOE_ERR_INVALID_ARG, "the cache's k and v must be 16-byte aligned and not NULL");
    for (const int64_t stride : {c->k_stride, c->v_stride})
        if (stride < places * c->dim || stride >= (1LL << 40) / es || stride * es % 16)
            return fail(MOE_ERR_INVALID_ARG,
                        "the cache's strides must be at least heads * page * dim and multiples of "
                        "16 bytes");
    const int64_t n = places * c->dim * es, kb = c->k_stride * es, vb = c->v_stride * es;
    if (!apart(c->k, kb, n, c->v, vb, n, c->pages))
        return fail(MOE_ERR_INVALID_ARG, "two arrays of the cache overlap");
    if (!f8) {
        if (c->k_scales || c->v_scales)
            return fail(MOE_ERR_INVALID_ARG, "a cache of 16 bits has no scales");
        return MOE_OK;
    }
    if (bad(c->k_scales, 16) || bad(c->v_scales, 16))
        return fail(MOE_ERR_INVALID_ARG,
                    "k_scales and v_scales must be 16-byte aligned and not NULL");
    for (const int64_t stride : {c->k_scales_stride, c->v_scales_stride})
        if (stride < places || stride % 4 || stride >= (1LL << 38))
            return fail(MOE_ERR_INVALID_ARG,
                        "the strides of the cache's scales must be at least heads * page and "
                        "multiples of 4");
    const int64_t ksb = c->k_scales_stride * 4, vsb = c->v_scales_stride * 4, ns = places * 4;
    if (!apart(c->k_scales, ksb, ns, c->v_scales, vsb, ns, c->pages) ||
        !apart(c->k, kb, n, c->k_scales, ksb, ns, c->pages) ||
        !apart(c->k, kb, n, c->v_scales, vsb, ns, c->pages) ||
        !apart(c->v, vb, n, c->k_scales, ksb, ns, c->pages) ||
        !apart(c->v, vb, n, c->v_scales, vsb, ns, c->pages))
        return fail(MOE_ERR_INVALID_ARG, "two arrays of the cache overlap");
    return MOE_OK;
}
struct Range {
    const void *p;
    size_t n;
};
// The cache's four arrays, as bytes from the first to the last element.
void cache_ranges(const moeop_kv_cache &c, Range (&r)[4]) {
    const int64_t places = (int64_t)c.heads * c.page;
    const size_t es = c.type == MOEOP_E4M3 ? 1 : 2;
    r[0] = {c.k, span(c.pages, c.k_stride, places * c.dim, es)};
    r[1] = {c.v, span(c.pages, c.v_stride, places * c.dim, es)};
    r[2] = {c.k_scales, span(c.pages, c.k_scales_stride, places, 4)};
    r[3] = {c.v_scales, span(c.pages, c.v_scales_stride, places, 4)};
}
bool meets(const void *p, size_t n, const Range (&r)[4]) {
    for (const Range &x : r)
        if (overlap(p, n, x.p, x.n)) return true;
    return false;
}
CacheParams cache_params(const moeop_kv_cache &c, int tokens, const int32_t *slots, int dtype) {
    CacheParams p{};
    p.k = c.k, p.v = c.v, p.k_scales = c.k_scales, p.v_scales = c.v_scales;
    p.k_stride = c.k_stride, p.v_stride = c.v_stride;
    p.k_scales_stride = c.k_scales_stride, p.v_scales_stride = c.v_scales_stride;
    p.slots = c.pages * c.page, p.heads = c.heads, p.page = c.page, p.dim = c.dim;
    p.cache_type = c.type, p.io_type = dtype, p.tokens = tokens, p.slots_of = slots;
    p.lanes_log2 = c.dim == 64 ? 2 : c.dim == 128 ? 3 : 4;
    p.by_page = Divisor(c.page), p.by_heads = Divisor(c.heads);
    return p;
}
moe_status check_tokens(const moeop_kv_cache &c, int tokens) {
    if (tokens < 0 || (int64_t)tokens * c.heads > (1 << 30))
        return fail(MOE_ERR_INVALID_ARG, "tokens=%d: tokens * heads must be in [0, 2^30]", tokens);
    return MOE_OK;
}
moe_status check_attend(int batch, int rows, int q_heads, int heads, int dim) {
    if (batch < 0 || batch > kAttendMaxBatch)
        return fail(MOE_ERR_INVALID_ARG, "batch=%d: must be in [0, %d]", batch, kAttendMaxBatch);
    if (rows < 1 || rows > 64)
        return fail(MOE_ERR_INVALID_ARG, "rows=%d: must be in [1, 64]", rows);
    if (heads < 1 || heads > 1024)
        return fail(MOE_ERR_INVALID_ARG, "heads=%d: must be in [1, 1024]", heads);
    if (dim != 64 && dim != 128 && dim != 256)
        return fail(MOE_ERR_INVALID_ARG, "dim=%d: must be 64, 128 or 256", dim);
    if (q_heads < 1 || q_heads % heads || (int64_t)(q_heads / heads) * rows > 256)
        return fail(MOE_ERR_INVALID_ARG,
                    "q_heads=%d: must be a multiple of heads=%d, rows * q_heads / heads at most 256",
                    q_heads, heads);
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

moe_status moeop_kv_write(const moeop_kv_cache *cache, const void *k, int64_t k_stride,
                          const void *v, int64_t v_stride, int dtype, const int32_t *slots,
                          int tokens, void *stream) {
    moe_status s;
    if ((s = check_cache(cache)) != MOE_OK || (s = check_dtype(dtype, "dtype")) != MOE_OK ||
        (s = check_tokens(*cache, tokens)) != MOE_OK)
        return s;
    if (cache->type != MOEOP_E4M3 && dtype != cache->type)
        return fail(MOE_ERR_INVALID_ARG, "dtype=%d: a cache of 16 bits takes its own type, %d",
                    dtype, cache->type);
    if (tokens == 0) return ok();
    const int64_t row = (int64_t)cache->heads * cache->dim, es = type_size(dtype);
    if (bad(k, 16) || bad(v, 16) || bad(slots, 4))
        return fail(MOE_ERR_INVALID_ARG,
                    "k and v must be 16-byte aligned, slots 4-byte, none of them NULL");
    for (const int64_t stride : {k_stride, v_stride})
        if (tokens > 1 && (stride < row || stride >= (1LL << 40) || stride * es % 16))
            return fail(MOE_ERR_INVALID_ARG,
                        "the row strides must be at least heads * dim and multiples of 16 bytes");
    Range r[4];
    cache_ranges(*cache, r);
    for (int i = 0; i < 4; ++i) {
        if (overlap(r[i].p, r[i].n, k, span(tokens, k_stride, row, es)) ||
            overlap(r[i].p, r[i].n, v, span(tokens, v_stride, row, es)) ||
            overlap(r[i].p, r[i].n, slots, (size_t)tokens * 4))
            return fail(MOE_ERR_INVALID_ARG, "the cache overlaps an input");
    }
    CacheParams p = cache_params(*cache, tokens, slots, dtype);
    p.k_io = const_cast<void *>(k), p.v_io = const_cast<void *>(v);
    p.k_io_stride = k_stride, p.v_io_stride = v_stride;
    return launched(launch_kv_write(p, static_cast<cudaStream_t>(stream)), "cache write launch");
}

moe_status moeop_kv_read(const moeop_kv_cache *cache, const int32_t *slots, int tokens, void *k,
                         void *v, int dtype, void *stream) {
    moe_status s;
    if ((s = check_cache(cache)) != MOE_OK || (s = check_dtype(dtype, "dtype")) != MOE_OK ||
        (s = check_tokens(*cache, tokens)) != MOE_OK)
        return s;
    if (tokens == 0) return ok();
    if (bad(k, 16) || bad(v, 16) || bad(slots, 4))
        return fail(MOE_ERR_INVALID_ARG,
                    "k and v must be 16-byte aligned, slots 4-byte, none of them NULL");
    const size_t n = (size_t)tokens * cache->heads * cache->dim * type_size(dtype);
    Range r[4];
    cache_ranges(*cache, r);
    if (overlap(k, n, v, n) || meets(k, n, r) || meets(v, n, r) ||
        overlap(k, n, slots, (size_t)tokens * 4) || overlap(v, n, slots, (size_t)tokens * 4))
        return fail(MOE_ERR_INVALID_ARG, "the outputs overlap each other or an input");
    CacheParams p = cache_params(*cache, tokens, slots, dtype);
    p.k_io = k, p.v_io = v;
    return launched(launch_kv_read(p, static_cast<cudaStream_t>(stream)), "cache read launch");
}

size_t moeop_attend_workspace_size(int batch, int rows, int q_heads, int heads, int dim) {
    if (check_attend(batch, rows, q_heads, heads, dim) != MOE_OK) return 0;
    return AttendWs::make(rows * (q_heads / heads), dim).total;
}

moe_status moeop_attend_workspace_init(void *ws, size_t ws_bytes, void *stream) {
    if (!ws || !aligned(ws, 256))
        return fail(MOE_ERR_WORKSPACE, "workspace is NULL or not 256-byte aligned");
    if (ws_bytes < kAttendCounters * 4)
        return fail(MOE_ERR_WORKSPACE, "workspace has %zu bytes, needs at least %d", ws_bytes,
                    kAttendCounters * 4);
    return launched(cudaMemsetAsync(ws, 0, kAttendCounters * 4, static_cast<cudaStream_t>(stream)),
                    "workspace initialisation");
}

moe_status moeop_attend_paged(const moeop_attend_config *cfg, const moeop_kv_cache *cache,
                              const void *q, int64_t q_batch_stride, int64_t q_row_stride,
                              const int32_t *table, int64_t table_stride, const int32_t *lengths,
                              void *out, void *ws, size_t ws_bytes, void *stream) {
    moe_status s;
    if (!cfg) return fail(MOE_ERR_INVALID_ARG, "cfg is NULL");
    const moeop_attend_config &c = *cfg;
    if ((s = check_cache(cache)) != MOE_OK ||
        (s = check_attend(c.batch, c.rows, c.q_heads, cache->heads, cache->dim)) != MOE_OK)
        return s;
    if (c.dtype != MOEOP_BF16 && c.dtype != MOEOP_FP16)
        return fail(MOE_ERR_INVALID_ARG, "dtype=%d: must be bf16 (0) or fp16 (1)", c.dtype);
    if (cache->type != MOEOP_E4M3 && c.dtype != cache->type)
        return fail(MOE_ERR_INVALID_ARG, "dtype=%d: a cache of 16 bits takes its own type, %d",
                    c.dtype, cache->type);
    if (c.width < 1 || (int64_t)c.width * cache->page > (1 << 30))
        return fail(MOE_ERR_INVALID_ARG, "width=%d: width * page must be in [1, 2^30]", c.width);
    if ((int64_t)c.batch * cache->heads * ((int64_t)c.width * cache->page / 16 + 2) > INT32_MAX)
        return fail(MOE_ERR_INVALID_ARG, "batch=%d: batch * heads * width * page / 16 must be below "
                    "2^31", c.batch);
    if (c.window < 0)
        return fail(MOE_ERR_INVALID_ARG, "window=%d: must not be negative", c.window);
    if (!(std::fabs(c.scale) < 0x1p127f))   // times log2(e) it is a finite number
        return fail(MOE_ERR_INVALID_ARG, "scale is not finite, or 2^127 or more");
    if (c.batch == 0) return ok();
    const int64_t row = (int64_t)c.q_heads * cache->dim;
    if (bad(q, 16) || bad(out, 16))
        return fail(MOE_ERR_INVALID_ARG, "q and out must be 16-byte aligned and not NULL");
    if (bad(table, 4) || bad(lengths, 4))
        return fail(MOE_ERR_INVALID_ARG, "table or lengths is NULL or misaligned");
    if ((c.rows > 1 && (q_row_stride < row || q_row_stride % 8 || q_row_stride >= (1LL << 40))) ||
        (c.batch > 1 && (q_batch_stride < row || q_batch_stride % 8 || q_batch_stride >= (1LL << 40))))
        return fail(MOE_ERR_INVALID_ARG,
                    "q's strides must be at least q_heads * dim and multiples of 8");
    if (c.batch > 1 && (table_stride < c.width || table_stride >= (1LL << 40)))
        return fail(MOE_ERR_INVALID_ARG, "the table's row stride is less than width=%d", c.width);
    const int group = c.q_heads / cache->heads, m = c.rows * group;
    const AttendWs L = AttendWs::make(m, cache->dim);
    if (!ws) return fail(MOE_ERR_WORKSPACE, "workspace is NULL");
    if (!aligned(ws, 256)) return fail(MOE_ERR_WORKSPACE, "workspace is not 256-byte aligned");
    if (ws_bytes < L.total)
        return fail(MOE_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", ws_bytes, L.total);
    Range r[4];
    cache_ranges(*cache, r);
    const size_t n = (size_t)c.batch * c.rows * row * 2;
    const size_t nq = ((size_t)(c.batch - 1) * (c.batch > 1 ? q_batch_stride : 0) +
                       (size_t)(c.rows - 1) * (c.rows > 1 ? q_row_stride : 0) + row) * 2;
    const size_t nt = span(c.batch, c.batch > 1 ? table_stride : 0, c.width, 4);
    if (meets(out, n, r) || overlap(out, n, q, nq) || overlap(out, n, table, nt) ||
        overlap(out, n, lengths, (size_t)c.batch * 4) || overlap(out, n, ws, L.total))
        return fail(MOE_ERR_INVALID_ARG, "out overlaps an input or the workspace");
    if (meets(ws, L.total, r) || overlap(ws, L.total, q, nq) || overlap(ws, L.total, table, nt) ||
        overlap(ws, L.total, lengths, (size_t)c.batch * 4))
        return fail(MOE_ERR_INVALID_ARG, "the workspace overlaps an input");
    AttendParams p{};
    p.k = cache->k, p.v = cache->v, p.k_scales = cache->k_scales, p.v_scales = cache->v_scales;
    p.k_stride = cache->k_stride, p.v_stride = cache->v_stride;
    p.k_scales_stride = cache->k_scales_stride, p.v_scales_stride = cache->v_scales_stride;
    p.pages = cache->pages, p.heads = cache->heads, p.page = cache->page;
    p.q = q, p.q_batch_stride = q_batch_stride, p.q_row_stride = q_row_stride;
    p.table = table, p.table_stride = table_stride, p.lengths = lengths, p.out = out;
    p.batch = c.batch, p.rows = c.rows, p.group = group, p.width = c.width, p.dtype = c.dtype;
    p.window = (int64_t)c.window >= (int64_t)c.width * cache->page ? 0 : c.window;  // sees all
    p.scale_log2 = (float)(c.scale * 1.4426950408889634);
    const int block = attend_block(cache->dim, m);
    p.blocks = (m + block - 1) / block;
    p.by_group = Divisor(group), p.by_page = Divisor(cache->page);
    p.counters = static_cast<uint32_t *>(ws);
    p.parts = reinterpret_cast<float *>(static_cast<char *>(ws) + L.parts);
    const auto launch = cache->type == MOEOP_E4M3  ? launch_attend_f8
                        : cache->type == MOEOP_BF16 ? launch_attend_bf
                                                    : launch_attend_hf;
    return launched(launch(p, cache->dim, static_cast<cudaStream_t>(stream)), "attention launch");
}

moe_status moeop_verify_draft(const moeop_verify_config *cfg, const int32_t *draft,
                              const float *target, const float *draft_probs, const float *accept_u,
                              const float *sample_u, int32_t *tokens, int32_t *accepted,
                              void *stream) {
    if (!cfg) return fail(MOE_ERR_INVALID_ARG, "cfg is NULL");
    const moeop_verify_config &c = *cfg;
    if (c.batch < 0 || c.batch > 65535)
        return fail(MOE_ERR_INVALID_ARG, "batch=%d: must be in [0, 65535]", c.batch);
    if (c.drafts < 0 || c.drafts > 31)
        return fail(MOE_ERR_INVALID_ARG, "drafts=%d: must be in [0, 31]", c.drafts);
    if (c.vocab < 1 || c.vocab > (1 << 19))
        return fail(MOE_ERR_INVALID_ARG, "vocab=%d: must be in [1, 2^19]", c.vocab);
    if (c.batch == 0) return ok();
    if (bad(target, 4) || bad(sample_u, 4) || bad(tokens, 4) || bad(accepted, 4))
        return fail(MOE_ERR_INVALID_ARG, "a pointer is NULL or not aligned to its type");
    if (c.drafts && (bad(draft, 4) || bad(accept_u, 4) || !aligned(draft_probs, 4)))
        return fail(MOE_ERR_INVALID_ARG, "a pointer is NULL or not aligned to its type");
    const int64_t rows = (int64_t)c.batch * (c.drafts + 1), drows = (int64_t)c.batch * c.drafts;
    const bool probs = draft_probs && c.drafts;
    if ((rows > 1 && (c.target_stride < c.vocab || c.target_stride >= (1LL << 40))) ||
        (probs && drows > 1 && (c.draft_stride < c.vocab || c.draft_stride >= (1LL << 40))))
        return fail(MOE_ERR_INVALID_ARG, "a row stride is less than vocab=%d", c.vocab);
    const size_t nt = (size_t)rows * 4, na = (size_t)c.batch * 4, nd = (size_t)drows * 4;
    const Range in[5] = {{target, span(rows, rows > 1 ? c.target_stride : 0, c.vocab, 4)},
                         {probs ? draft_probs : nullptr,
                          span(drows, drows > 1 ? c.draft_stride : 0, c.vocab, 4)},
                         {draft, nd}, {accept_u, nd}, {sample_u, na}};
    if (overlap(tokens, nt, accepted, na))
        return fail(MOE_ERR_INVALID_ARG, "the outputs overlap each other or an input");
    for (const Range &x : in)
        if (overlap(tokens, nt, x.p, x.n) || overlap(accepted, na, x.p, x.n))
            return fail(MOE_ERR_INVALID_ARG, "the outputs overlap each other or an input");
    const VerifyParams p{c, draft, target, probs ? draft_probs : nullptr, accept_u, sample_u,
                         tokens, accepted};
    return launched(launch_verify_draft(p, static_cast<cudaStream_t>(stream)), "verify launch");
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

// moeop.cuh -- what the FP8 layer operators' translation units share:
// parameter blocks, launchers, the device status word and e4m3 packing.
#pragma once

#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "moe_ops.h"

namespace moe {

moe_status set_error(moe_status s, const char *msg);  // moe_api.cu

namespace op {

constexpr float kFp8Max = 448.f;   // largest finite e4m3 value
constexpr float kFp8Tiny = 1e-30f; // least magnitude a scale is made of

struct NormParams {
    const void *x, *residual, *weight;
    int64_t x_stride, residual_stride;
    int rows, hidden, dtype;
    float eps;
    void *y, *residual_out;
    uint8_t *q;
    float *scales;
};
cudaError_t launch_rms_norm(const NormParams &p, bool vec, cudaStream_t st);

struct RouteParams {
    moeop_route_config c;
    const void *logits;
    int64_t stride;
    const float *bias;
    int rows;
    int32_t *ids;
    float *wts;
};
cudaError_t launch_route_topk(const RouteParams &p, cudaStream_t st);

// One FP8 matrix as the products read it: 128-byte columns of whole rows.
struct Fp8Mat {
    const uint8_t *p;
    int64_t rows, k, stride;
};
cudaError_t launch_matmul_fp8(const Fp8Mat &a, const float *sa, const Fp8Mat &b, const float *sb,
                              void *out, int out_dtype, cudaStream_t st);

// Rows up to which a product goes to moeop_few.cu, and pairs (row, slot).
constexpr int kFewRows = 16, kFewPairs = 32, kFewSmem = 160 << 10;
cudaError_t launch_few_dense(const Fp8Mat &a, const float *sa, const Fp8Mat &b, const float *sb,
                             void *out, int out_dtype, int sms, cudaStream_t st);

// Workspace of moeop_experts_fp8: the pairs (row, slot) in expert order, the
// tiles of 128 of them, the FP8 rows h and the products y in fp32.
struct ExpertsWs {
    size_t header, tiles, pair, token, h, h_scales, y, total;
    int max_tiles;
    static ExpertsWs make(const moeop_experts_config &c, int rows) {
        auto up = [](size_t v) { return (v + 255) / 256 * 256; };
        ExpertsWs w{};
        const size_t P = (size_t)rows * c.top_k;
        const size_t full = P / 128 + c.num_experts;
        w.max_tiles = (int)(P < full ? P : full);
        size_t o = 0;
        w.header = o, o += 256;
        w.tiles = o, o += up((size_t)w.max_tiles * 16);
        w.pair = o, o += up(P * 4);
        w.token = o, o += up(P * 4);
        w.h = o, o += up(P * c.inter);
        w.h_scales = o, o += up(P * (c.inter / 128) * 4);
        w.y = o, o += up(P * c.hidden * 4);
        // up to 32 pairs: h in fp32 and nothing else
        const size_t few = up((P < kFewPairs ? P : (size_t)kFewPairs) * c.inter * 4);
        w.total = o > few ? o : few;
        return w;
    }
};
struct ExpertsArgs {
    moeop_experts_config c;
    moeop_experts_weights w;
    const uint8_t *q;
    const float *scales;
    const int32_t *ids;
    const float *wts;
    const uint16_t *addend;
    uint16_t *out;
    int rows;
    char *ws;
};
cudaError_t launch_experts_fp8(const ExpertsArgs &a, cudaStream_t st);
cudaError_t launch_few_experts(const ExpertsArgs &a, float *h, cudaStream_t st);
bool few_experts(int64_t rows, const moeop_experts_config &c);
cudaError_t allow_few_smem();

cudaError_t status_word(uint32_t **p);  // the current device's status word

struct alignas(64) TensorMap {
    uint64_t v[16];
};
cudaError_t make_cache_map(TensorMap *m, const void *p, int row_bytes, int box_rows, int64_t rows,
                           int64_t page_bytes, int64_t pages);

// Quotients of numbers below 2^31 by one that many share: a multiplication
// (T. Granlund and P. Montgomery, "Division by invariant integers using
// multiplication", 1994).
struct Divisor {
    uint32_t d, mul, shift;
    Divisor() = default;
    explicit Divisor(uint32_t by) : d(by), shift(0) {
        while (shift < 31 && (1u << shift) < by) ++shift;
        mul = (uint32_t)((((uint64_t)1 << 32) * (((uint64_t)1 << shift) - by)) / by + 1);
    }
#ifdef __CUDACC__
    __device__ __forceinline__ uint32_t over(uint32_t n) const {
        return (__umulhi(n, mul) + n) >> shift;
    }
#endif
};

// moeop_kv_write and moeop_kv_read: the cache, and the rows outside of it.
struct CacheParams {
    void *k, *v;
    float *k_scales, *v_scales;
    int64_t k_stride, v_stride, k_scales_stride, v_scales_stride;
    int slots, heads, page, dim, cache_type;
    void *k_io, *v_io;
    int64_t k_io_stride, v_io_stride;
    int io_type, tokens, lanes_log2;  // 2^lanes_log2 = dim / 16 lanes to a row
    const int32_t *slots_of;
    Divisor by_page, by_heads;
};
cudaError_t launch_kv_write(const CacheParams &p, cudaStream_t st);
cudaError_t launch_kv_read(const CacheParams &p, cudaStream_t st);

// moeop_verify_draft.
struct VerifyParams {
    moeop_verify_config c;
    const int32_t *draft;
    const float *target, *draft_probs, *accept_u, *sample_u;
    int32_t *tokens, *accepted;
};
cudaError_t launch_verify_draft(const VerifyParams &p, cudaStream_t st);

// moeop_attend_paged.
struct AttendParams {
    const void *k, *v;
    const float *k_scales, *v_scales;
    int64_t k_stride, v_stride, k_scales_stride, v_scales_stride;
    int pages, heads, page;
    const void *q;
    int64_t q_batch_stride, q_row_stride;
    const int32_t *table;
    int64_t table_stride;
    const int32_t *lengths;
    void *out;
    int batch, rows, group, width, window, dtype;
    float scale_log2;          // of the scores, times log2(e)
    int blocks;                // of query rows of a key/value head
    Divisor by_group, by_page, by_grid;  // by_grid: thread blocks for a block of query rows
    uint32_t *counters;        // kAttendCounters, zero between calls
    float *parts;              // sums of a warp's or thread block's share of an item
    uint32_t *status;
    bool wide;                 // a tile never leaves its page
    bool apart;                // a kernel of its own joins what blocks have of an item
    int whole;                 // tiles up to which an item is not cut between blocks
    // it joins what warps have of an item: warps take shares of the whole work, in turn
    // from block to block, and blocks join nothing
    bool flat;
    Divisor by_warps;          // warps of the grid
};
// Query rows (row, head of the group) that a thread block takes together.
constexpr int attend_block(int dim, int m) { return dim == 256 || m <= 8 ? 8 : 16; }
// Thread blocks for each block of query rows: together one for every SM.
constexpr int kAttendSms = 152, kAttendCounters = 3 * 256, kAttendMaxBatch = 2048;
constexpr int attend_grid(int blocks) { return blocks < kAttendSms ? kAttendSms / blocks : 1; }
// Workspace of moeop_attend_paged: the counters, in every shape the same, then two
// partial sums for each warp (up to 8 in a thread block), or one for each warp and
// two for each thread block: three numbers for a row, and the row.
struct AttendWs {
    size_t parts, total;
    static AttendWs make(int m, int dim) {
        const int block = attend_block(dim, m), blocks = (m + block - 1) / block;
        const size_t part = (size_t)block * (3 + dim) * 4;
        AttendWs w{};
        w.parts = kAttendCounters * 4;
        w.total = w.parts + part * blocks * attend_grid(blocks) * (2 * 8);
        return w;
    }
};
cudaError_t launch_attend_f8(const AttendParams &p, int dim, cudaStream_t st);
cudaError_t launch_attend_bf(const AttendParams &p, int dim, cudaStream_t st);
cudaError_t launch_attend_hf(const AttendParams &p, int dim, cudaStream_t st);

#ifdef __CUDACC__
// Launch that may start while the kernel before it in the stream still runs; the
// kernel waits for that (pdl_wait) before its first read of memory.
template <typename... P, typename... A>
cudaError_t launch_early(void (*kernel)(P...), dim3 grid, int threads, size_t smem, int cluster,
                         cudaStream_t st, A... args) {
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute at[2];
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = at;
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.numAttrs = 1;
    if (cluster > 1) {
        at[1].id = cudaLaunchAttributeClusterDimension;
        at[1].val.clusterDim.x = cluster;
        at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
        cfg.numAttrs = 2;
    }
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Four values -> four e4m3 codes, nearest even, beyond +-448 the largest.
__device__ __forceinline__ uint32_t pack_e4m3x4(float a, float b, float c, float d) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    return lo | hi << 16;
}

// The scale of inputs of largest magnitude `amax`, and v / scale: the product
// with the reciprocal, corrected by its remainder (P. Markstein, "Computation
// of elementary functions on the IBM RISC System/6000 processor", 1990), which
// is the rounded quotient.  The product alone is up to 1.5 steps of fp32 off
// and takes the other code about once in 10^5 values.  Where amax is infinite,
// finite values become 0.
struct Fp8Scale {
    float scale, recip, divisor;
    __device__ __forceinline__ explicit Fp8Scale(float amax)
        : scale(fmaxf(amax, kFp8Tiny) / kFp8Max), recip(1.f / scale),
          divisor(recip > 0.f ? scale : 0.f) {}
    __device__ __forceinline__ float over(float v) const {
        const float q = v * recip;
        return fmaf(fmaf(-q, divisor, v), recip, q);
    }
    __device__ __forceinline__ uint32_t codes(float a, float b, float c, float d) const {
        return pack_e4m3x4(over(a), over(b), over(c), over(d));
    }
};
#endif

}  // namespace op
}  // namespace moe

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

#ifdef __CUDACC__
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

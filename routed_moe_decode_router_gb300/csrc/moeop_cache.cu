// moeop_cache.cu -- the paged cache written and read back (moeop_kv_write,
// moeop_kv_read).
//
//   scale = max(amax of a head's dim, 1e-30) / 448, code = e4m3(x / scale);
//   x = code * scale.
//
// Bound by memory: every row is read once and written once.  A thread holds 8
// elements of each half of a head's row, of the key and of the value: four
// loads under way, none of which waits for the slot, and accesses of 8, 16 or 32
// bytes beside those of the next lane.  A row's amax is a few shuffles among its
// dim / 16 lanes.  Quotients are computed two at a time (packed fp32: 13.3 -> 11.8
// million instructions for 16383 tokens, 21 -> 18 us).
//
// One GB300: 16383 tokens, 8 heads of 128, bf16 to e4m3 18 us in a stream of calls
// (5.6 TB/s), 15.7 with the inputs in L2; 65536 read back 61 us (6.6 TB/s), in fp32 120
// (5.6), a bf16 cache's 80 (6.7), those in fp32 128 (6.3); 61 tokens 1.8 us.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "moe_device.cuh"
#include "moeop.cuh"

namespace moe {
namespace op {

namespace {

struct Codes {
    uint8_t v;
};
template <int TYPE>
struct TypeOf;
template <>
struct TypeOf<MOEOP_BF16> {
    using T = __nv_bfloat16;
};
template <>
struct TypeOf<MOEOP_FP16> {
    using T = __half;
};
template <>
struct TypeOf<MOEOP_FP32> {
    using T = float;
};
template <>
struct TypeOf<MOEOP_E4M3> {
    using T = Codes;
};

// Eight elements as they lie in memory.
template <typename T>
struct alignas(sizeof(T) >= 2 ? 16 : 8) Eight {
    uint32_t u[sizeof(T) * 2];
};
__device__ __forceinline__ void widen(const Eight<__nv_bfloat16> &r, float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[2 * i] = bf16_lo(r.u[i]), v[2 * i + 1] = bf16_hi(r.u[i]);
}
__device__ __forceinline__ void halves(uint32_t u, float &a, float &b) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&u));
    a = f.x, b = f.y;
}
__device__ __forceinline__ void widen(const Eight<__half> &r, float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) halves(r.u[i], v[2 * i], v[2 * i + 1]);
}
__device__ __forceinline__ void widen(const Eight<float> &r, float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r.u[i]);
}
__device__ __forceinline__ void widen(const Eight<Codes> &r, float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
        halves(e4m3x2_to_f16x2(r.u[i / 2] >> (16 * (i % 2))), v[2 * i], v[2 * i + 1]);
}
__device__ __forceinline__ void narrow(const float (&v)[8], Eight<__nv_bfloat16> &r) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
        r.u[i] = (uint32_t)f2bf16_rn(v[2 * i]) | (uint32_t)f2bf16_rn(v[2 * i + 1]) << 16;
}
__device__ __forceinline__ void narrow(const float (&v)[8], Eight<__half> &r) {
#pragma unroll
    for (int i = 0; i < 4; ++i) r.u[i] = pack_f16x2(v[2 * i], v[2 * i + 1]);
}
__device__ __forceinline__ void narrow(const float (&v)[8], Eight<float> &r) {
#pragma unroll
    for (int i = 0; i < 8; ++i) r.u[i] = __float_as_uint(v[i]);
}

__device__ __forceinline__ uint64_t pair(float a, float b) {
    uint64_t v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b));
    return v;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
// Fp8Scale::over of two numbers at a time.
__device__ __forceinline__ float2 over2(const Fp8Scale &s, float a, float b) {
    const uint64_t v = pair(a, b), recip = pair(s.recip, s.recip), q = mul2(v, recip);
    const uint64_t r = fma2(fma2(q, pair(-s.divisor, -s.divisor), v), recip, q);
    float2 f;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(r));
    return f;
}
__device__ __forceinline__ uint32_t codes(const Fp8Scale &s, const float *v) {
    const float2 a = over2(s, v[0], v[1]), b = over2(s, v[2], v[3]);
    return pack_e4m3x4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ float largest(const float (&v)[8]) {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(v[i]));
    return m;
}

// Where a thread works: 8 elements at `col` and 8 at `col` + dim / 2 of a head's
// row of a token.
struct Place {
    int token, head, col, half;
    bool live;
    __device__ __forceinline__ Place(const CacheParams &p) {
        const int64_t i = blockIdx.x * 256LL + threadIdx.x;
        const int lane = (int)(i & ((1 << p.lanes_log2) - 1));
        const uint32_t row = (uint32_t)(i >> p.lanes_log2);
        token = (int)p.by_heads.over(row);
        head = (int)(row - (uint32_t)token * p.heads);
        col = lane * 8;
        half = 8 << p.lanes_log2;
        live = token < p.tokens;
    }
    // First element of the head's row in the cache; false for a slot outside.
    __device__ __forceinline__ bool row(const CacheParams &p, int slot, uint32_t *page,
                                        uint32_t *in_page) const {
        if ((uint32_t)slot >= (uint32_t)p.slots) return false;
        *page = p.by_page.over((uint32_t)slot);
        *in_page = (uint32_t)head * p.page + ((uint32_t)slot - *page * p.page);
        return true;
    }
};

// (A NaN does not count in amax: it becomes the code of NaN beside what the others are.)
template <int CACHE, int IN>
__global__ void __launch_bounds__(256, IN == MOEOP_FP32 ? 4 : 5) write_kernel(const CacheParams p) {
    using T = typename TypeOf<IN>::T;
    const Place at(p);
    pdl_trigger();
    pdl_wait();
    // the lanes of a row are all there or none is; those beyond the last token
    // take part in the shuffles
    Eight<T> raw[2][2] = {};
    int slot = -1;
    if (at.live) {
        slot = __ldg(p.slots_of + at.token);
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const T *x = static_cast<const T *>(s ? p.v_io : p.k_io) +
                         at.token * (s ? p.v_io_stride : p.k_io_stride) +
                         (int64_t)at.head * p.dim + at.col;
            raw[s][0] = *reinterpret_cast<const Eight<T> *>(x);
            raw[s][1] = *reinterpret_cast<const Eight<T> *>(x + at.half);
        }
    }
    uint32_t page = 0, in_page = 0;
    const bool put = at.row(p, slot, &page, &in_page);
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        const int64_t first = (int64_t)page * (s ? p.v_stride : p.k_stride) +
                              (int64_t)in_page * p.dim + at.col;
        if constexpr (CACHE != MOEOP_E4M3) {
            if (put) {
                T *y = static_cast<T *>(s ? p.v : p.k) + first;
                *reinterpret_cast<Eight<T> *>(y) = raw[s][0];
                *reinterpret_cast<Eight<T> *>(y + at.half) = raw[s][1];
            }
        } else {
            float v[2][8], amax = 0.f;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                widen(raw[s][h], v[h]);
                amax = fmaxf(amax, largest(v[h]));
            }
            for (int o = (1 << p.lanes_log2) / 2; o; o >>= 1)
                amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, o));
            const Fp8Scale q(amax);
            if (put) {
                uint8_t *y = static_cast<uint8_t *>(s ? p.v : p.k) + first;
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    *reinterpret_cast<uint2 *>(y + h * at.half) =
                        make_uint2(codes(q, v[h]), codes(q, v[h] + 4));
                if (at.col == 0)
                    (s ? p.v_scales : p.k_scales)[(int64_t)page * (s ? p.v_scales_stride
                                                                     : p.k_scales_stride) +
                                                  in_page] = q.scale;
            }
        }
    }
}

template <int CACHE, int OUT>
__global__ void __launch_bounds__(256) read_kernel(const CacheParams p) {
    using C = typename TypeOf<CACHE>::T;
    using T = typename TypeOf<OUT>::T;
    const Place at(p);
    pdl_trigger();
    pdl_wait();
    if (!at.live) return;
    uint32_t page, in_page;
    const bool got = at.row(p, __ldg(p.slots_of + at.token), &page, &in_page);
    Eight<C> raw[2][2] = {};
    float scale[2] = {1.f, 1.f};
    if (got) {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const C *x = static_cast<const C *>(s ? p.v : p.k) +
                         (int64_t)page * (s ? p.v_stride : p.k_stride) +
                         (int64_t)in_page * p.dim + at.col;
            raw[s][0] = *reinterpret_cast<const Eight<C> *>(x);
            raw[s][1] = *reinterpret_cast<const Eight<C> *>(x + at.half);
            if (CACHE == MOEOP_E4M3)
                scale[s] = __ldg((s ? p.v_scales : p.k_scales) +
                                 (int64_t)page * (s ? p.v_scales_stride : p.k_scales_stride) +
                                 in_page);
        }
    }
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        T *y = static_cast<T *>(s ? p.v_io : p.k_io) +
               ((int64_t)at.token * p.heads + at.head) * p.dim + at.col;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            Eight<T> r;
            if constexpr (CACHE == OUT) {
                r = raw[s][h];
            } else {
                float v[8];
                widen(raw[s][h], v);
                if (CACHE == MOEOP_E4M3 && got) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[i] *= scale[s];
                }
                narrow(v, r);
            }
            *reinterpret_cast<Eight<T> *>(y + h * at.half) = r;
        }
    }
}

template <typename K>
cudaError_t launch(K kernel, const CacheParams &p, cudaStream_t st) {
    const int64_t threads = (int64_t)p.tokens * p.heads << p.lanes_log2;
    return launch_early(kernel, dim3((unsigned)((threads + 255) / 256)), 256, 0, 1, st, p);
}

}  // namespace

cudaError_t launch_kv_write(const CacheParams &p, cudaStream_t st) {
    if (p.cache_type == MOEOP_BF16) return launch(write_kernel<MOEOP_BF16, MOEOP_BF16>, p, st);
    if (p.cache_type == MOEOP_FP16) return launch(write_kernel<MOEOP_FP16, MOEOP_FP16>, p, st);
    switch (p.io_type) {
        case MOEOP_BF16: return launch(write_kernel<MOEOP_E4M3, MOEOP_BF16>, p, st);
        case MOEOP_FP16: return launch(write_kernel<MOEOP_E4M3, MOEOP_FP16>, p, st);
        default: return launch(write_kernel<MOEOP_E4M3, MOEOP_FP32>, p, st);
    }
}

template <int CACHE>
static cudaError_t launch_read(const CacheParams &p, cudaStream_t st) {
    switch (p.io_type) {
        case MOEOP_BF16: return launch(read_kernel<CACHE, MOEOP_BF16>, p, st);
        case MOEOP_FP16: return launch(read_kernel<CACHE, MOEOP_FP16>, p, st);
        default: return launch(read_kernel<CACHE, MOEOP_FP32>, p, st);
    }
}
cudaError_t launch_kv_read(const CacheParams &p, cudaStream_t st) {
    switch (p.cache_type) {
        case MOEOP_BF16: return launch_read<MOEOP_BF16>(p, st);
        case MOEOP_FP16: return launch_read<MOEOP_FP16>(p, st);
        default: return launch_read<MOEOP_E4M3>(p, st);
    }
}

}  // namespace op
}  // namespace moe

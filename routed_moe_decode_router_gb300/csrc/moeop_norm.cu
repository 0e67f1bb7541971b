// moeop_norm.cu -- root-mean-square norm with the residual's addition and an
// FP8 output (moeop_rms_norm).
//
//   s = x (+ residual);  y = s * rsqrt(mean(s^2) + eps) * w;
//   q = e4m3(y / scale), scale = max(amax of 128 y, 1e-30) / 448.
//
// Bound by memory: every input is read once and every output written once.
// A thread owns 8 consecutive elements (16 bytes of a 16-bit type) per
// vector, 16 threads one group of 128, so a group's amax is four shuffles and
// the row is not read again for the second pass: it stays in registers, but
// for what the limits below make the compiler spill (at 2049 to 4096 elements
// 60 to 112 bytes a thread, which stay in L1).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "moeop.cuh"

namespace moe {
namespace op {

namespace {

template <typename T>
__device__ __forceinline__ float to_f(T v);
template <>
__device__ __forceinline__ float to_f(float v) { return v; }
template <>
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float to_f(__half v) { return __half2float(v); }

template <typename T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f(float v) { return __float2half_rn(v); }

// Eight elements from `col` on; VEC: 16-byte accesses (the caller has checked
// the alignment), else element by element.  Beyond `n`: zeros / not stored.
template <typename T, bool VEC>
__device__ __forceinline__ void load8(const T *p, int col, int n, float (&v)[8]) {
    if (VEC) {
        union {
            uint4 u[sizeof(T) / 2];
            T t[8];
        } r;
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i)
            r.u[i] = reinterpret_cast<const uint4 *>(p + col)[i];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = to_f(r.t[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = col + i < n ? to_f(p[col + i]) : 0.f;
    }
}
template <typename T, bool VEC>
__device__ __forceinline__ void store8(T *p, int col, int n, const float (&v)[8]) {
    if (VEC) {
        union {
            uint4 u[sizeof(T) / 2];
            T t[8];
        } r;
#pragma unroll
        for (int i = 0; i < 8; ++i) r.t[i] = from_f<T>(v[i]);
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i)
            reinterpret_cast<uint4 *>(p + col)[i] = r.u[i];
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (col + i < n) p[col + i] = from_f<T>(v[i]);
    }
}

// blockDim.x threads (a multiple of 32) per row, blockDim.y rows per block.
// A block loads, waits, computes and stores: what keeps the memory busy is
// the number of blocks on an SM, so up to 4096 elements the registers are
// held to 32 (8 blocks of 256).  8192 rows of 4096 bf16 with everything: 51 us
// (5.9 TB/s; 49 with codes by the reciprocal alone) against 66 us with 512
// threads of one vector and 3 blocks; fp32 92 us (6.2 TB/s).  Rows that do not
// start on 16 bytes go element by element: 8192 x 4095 bf16 200 us.
// WIDE, where there is an SM for every row: one vector per thread, and the
// weights are asked for together with the row (one row of 4096: 2.3 us
// against 3.0).
constexpr int kSms = 152;
constexpr int threads_of(int vpt, bool wide) { return wide ? 1024 : vpt == 8 ? 512 : 256; }
template <typename T, int VPT, bool VEC, bool WIDE>
__global__ void __launch_bounds__(threads_of(VPT, WIDE), WIDE       ? 1
                                                         : VPT <= 2 ? 8
                                                         : VPT == 4 ? 4
                                                                    : 1)
    rms_norm_kernel(NormParams p) {
    __shared__ float part[32];
    const int H = p.hidden, tpr = blockDim.x;
    const int row_raw = blockIdx.x * blockDim.y + threadIdx.y;
    const bool live = row_raw < p.rows;
    const int row = live ? row_raw : p.rows - 1;
    // x and residual may be written through residual_out: each element is
    // read and written by the same thread, reads first
    const T *x = static_cast<const T *>(p.x) + (size_t)row * p.x_stride;
    const T *res =
        p.residual ? static_cast<const T *>(p.residual) + (size_t)row * p.residual_stride : nullptr;
    const T *w = static_cast<const T *>(p.weight);
    float v[VPT][8], g[8];
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int col = (j * tpr + threadIdx.x) * 8;
        if (col < H) {
            if (WIDE) load8<T, VEC>(w, col, H, g);
            load8<T, VEC>(x, col, H, v[j]);
            if (res) {
                float r[8];
                load8<T, VEC>(res, col, H, r);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[j][i] += r[i];
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) sum = fmaf(v[j][i], v[j][i], sum);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[j][i] = 0.f;
        }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
    const int warps = tpr / 32, wid = threadIdx.y * warps + threadIdx.x / 32;
    if (warps > 1) {
        if (threadIdx.x % 32 == 0) part[wid] = sum;
        __syncthreads();
        const int lane = threadIdx.x % 32;
        sum = lane < warps ? part[threadIdx.y * warps + lane] : 0.f;
#pragma unroll
        for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
    }
    const float inv = 1.f / sqrtf(sum / (float)H + p.eps);
    const size_t base = (size_t)row * H;
    const int groups = (H + 127) / 128;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int col = (j * tpr + threadIdx.x) * 8;
        const bool in = live && col < H;
        if (col < H) {
            if (p.residual_out && in)
                store8<T, VEC>(static_cast<T *>(p.residual_out) + base, col, H, v[j]);
            if (!WIDE) load8<T, VEC>(w, col, H, g);
#pragma unroll
            for (int i = 0; i < 8; ++i) g[i] = v[j][i] * inv * g[i];
            if (p.y && in) store8<T, VEC>(static_cast<T *>(p.y) + base, col, H, g);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) g[i] = 0.f;
        }
        if (p.q) {
            float amax = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(g[i]));
#pragma unroll
            for (int o = 8; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, o));
            if (in) {
                const Fp8Scale s(amax);
                uint32_t c[2];
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    c[i] = s.codes(g[4 * i], g[4 * i + 1], g[4 * i + 2], g[4 * i + 3]);
                if (VEC) {
                    *reinterpret_cast<uint2 *>(p.q + base + col) = make_uint2(c[0], c[1]);
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (col + i < H) p.q[base + col + i] = (uint8_t)(c[i / 4] >> (8 * (i % 4)));
                }
                if (threadIdx.x % 16 == 0)
                    p.scales[(size_t)row * groups + col / 128] = s.scale;
            }
        }
    }
}

template <typename T, bool VEC>
cudaError_t launch_vpt(const NormParams &p, int vpt, dim3 grid, dim3 block, cudaStream_t st) {
    switch (vpt) {
        case 0: rms_norm_kernel<T, 1, VEC, true><<<grid, block, 0, st>>>(p); break;
        case 1: rms_norm_kernel<T, 1, VEC, false><<<grid, block, 0, st>>>(p); break;
        case 2: rms_norm_kernel<T, 2, VEC, false><<<grid, block, 0, st>>>(p); break;
        case 4: rms_norm_kernel<T, 4, VEC, false><<<grid, block, 0, st>>>(p); break;
        default: rms_norm_kernel<T, 8, VEC, false><<<grid, block, 0, st>>>(p); break;
    }
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rms_norm(const NormParams &p, bool vec, cudaStream_t st) {
    // Up to 256 threads of 1, 2 or 4 vectors of 8 elements, then 512 of 8;
    // short rows share a block.  Rows of at most 1024 vectors that have an SM
    // each: a thread per vector.
    const int nvec = (p.hidden + 7) / 8;
    int vpt = 1;
    while (nvec > threads_of(vpt, false) * vpt) vpt *= 2;
    if (p.rows <= kSms && nvec <= threads_of(1, true)) vpt = 0;  // WIDE
    const int per = vpt ? vpt : 1;
    const int tpr = ((nvec + per - 1) / per + 31) / 32 * 32;
    const int ry = tpr >= 256 || p.rows < 2 ? 1 : 256 / tpr;
    const dim3 block(tpr, ry), grid((p.rows + ry - 1) / ry);
    switch (p.dtype) {
        case MOEOP_BF16:
            return vec ? launch_vpt<__nv_bfloat16, true>(p, vpt, grid, block, st)
                       : launch_vpt<__nv_bfloat16, false>(p, vpt, grid, block, st);
        case MOEOP_FP16:
            return vec ? launch_vpt<__half, true>(p, vpt, grid, block, st)
                       : launch_vpt<__half, false>(p, vpt, grid, block, st);
        default:
            return vec ? launch_vpt<float, true>(p, vpt, grid, block, st)
                       : launch_vpt<float, false>(p, vpt, grid, block, st);
    }
}

}  // namespace op
}  // namespace moe

// moeop_few.cu -- the FP8 products for a few rows: moeop_matmul_fp8 up to 16
// rows, and moeop_experts_fp8 up to 32 pairs (row, slot).
//
// Few rows leave nothing to compute: the weights' bytes are the bound, and
// the time until they flow.  So there is no ring and no tensor memory here:
// every warp loads the 16 weight rows of its share of the inputs straight
// into registers as the left operand of mma.sync (m16n8k32, e4m3, fp32 sums),
// with all loads of a step under way at once, and the rows of x are the right
// one.  A lane's 16 bytes are cut into the fragments of two MMAs; the order
// of the inputs this makes is the same on both sides, and a sum does not
// depend on it.  Each block of 128 inputs is summed by itself, then scaled
// and added in fp32; the warps of a block split the inputs and add up in
// shared memory, in order.
//
// One GB300, in a CUDA graph: 1 x 4096 x 4096 4.5 us (3.7 TB/s with the launch),
// experts (hidden 2048, 128 x 768, top 8) of one row 14.1 us, against 8.5 and
// 24.2 us through tensor memory.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "moe_device.cuh"
#include "moeop.cuh"

namespace moe {
namespace op {

namespace {

// D[16 x 8] += A[16 x 32] B[8 x 32]^T, e4m3 in, fp32 sums.
__device__ __forceinline__ void mma_e4m3(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// 64 inputs: lo, hi are rows g and g + 8 of A, x row g of B.
__device__ __forceinline__ void mma64(float (&d)[4], uint4 lo, uint4 hi, uint4 x) {
    mma_e4m3(d, lo.x, hi.x, lo.y, hi.y, x.x, x.y);
    mma_e4m3(d, lo.z, hi.z, lo.w, hi.w, x.z, x.w);
}

__device__ __forceinline__ uint4 zero4() { return make_uint4(0, 0, 0, 0); }

// ---------------------------------------------------------------------------
// Dense: out[m][n0 .. n0 + 15] per block
// ---------------------------------------------------------------------------
struct DenseParams {
    const uint8_t *a, *b;
    int64_t a_stride, b_stride;
    const float *sa, *sb;
    int m, n, k, kb;
    void *out;
    int out_dtype;
};

// NT: groups of 8 rows of A.  A step is UNROLL blocks of 128 inputs.
template <int NT>
__global__ void __launch_bounds__(512, 1) few_dense_kernel(const DenseParams p) {
    constexpr int kUnroll = NT == 1 ? 2 : 1;
    __shared__ float part[16][NT][128];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, warps = blockDim.x / 32;
    const int g = lane / 4, t = lane % 4, n0 = blockIdx.x * 16;
    const bool lo_in = n0 + g < p.n, hi_in = n0 + 8 + g < p.n;
    const uint8_t *lo = p.b + (int64_t)min(n0 + g, p.n - 1) * p.b_stride + t * 16;
    const uint8_t *hi = p.b + (int64_t)min(n0 + 8 + g, p.n - 1) * p.b_stride + t * 16;
    const float *sb = p.sb + (size_t)(n0 / 128) * p.kb;
    float acc[NT][4];
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[j][i] = 0.f;
    const int b1 = (warp + 1) * p.kb / warps;
    for (int b0 = warp * p.kb / warps; b0 < b1; b0 += kUnroll) {
        uint4 w[kUnroll][2][2], x[kUnroll][NT][2];
        float s[kUnroll], sx[kUnroll][NT][2];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int b = b0 + u;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int64_t at = (int64_t)b * 128 + h * 64;
                const bool in = b < b1 && at + t * 16 < p.k;
                w[u][0][h] = in && lo_in ? ld_nc_v4(lo + at) : zero4();
                w[u][1][h] = in && hi_in ? ld_nc_v4(hi + at) : zero4();
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    const int row = j * 8 + g;
                    x[u][j][h] = in && row < p.m
                                     ? __ldg(reinterpret_cast<const uint4 *>(
                                           p.a + row * p.a_stride + at + t * 16))
                                     : zero4();
                }
            }
            s[u] = b < b1 ? __ldg(sb + b) : 0.f;
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const int row = j * 8 + t * 2 + c;
                    sx[u][j][c] = b < b1 && row < p.m ? __ldg(p.sa + (size_t)row * p.kb + b) : 0.f;
                }
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int h = 0; h < 2; ++h) mma64(d, w[u][0][h], w[u][1][h], x[u][j][h]);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    acc[j][i] = fmaf(d[i], s[u] * sx[u][j][i % 2], acc[j][i]);
            }
    }
    // part[..][row of A][weight row]
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) part[warp][j][(t * 2 + i % 2) * 16 + g + i / 2 * 8] = acc[j][i];
    __syncthreads();
    for (int i = threadIdx.x; i < NT * 128; i += blockDim.x) {
        const int row = i / 16, col = n0 + i % 16;
        if (row >= p.m || col >= p.n) continue;
        float v = 0.f;
        for (int q = 0; q < warps; ++q) v += part[q][i / 128][i % 128];
        const size_t at = (size_t)row * p.n + col;
        if (p.out_dtype == MOEOP_FP32) static_cast<float *>(p.out)[at] = v;
        else if (p.out_dtype == MOEOP_BF16) static_cast<uint16_t *>(p.out)[at] = f2bf16_rn(v);
        else static_cast<__half *>(p.out)[at] = __float2half_rn(v);
    }
}

// ---------------------------------------------------------------------------
// Experts: up to 32 pairs, one to a lane
// ---------------------------------------------------------------------------
// Every warp works out the same lists: the pairs of an expert in groups of 8
// (the columns of an MMA), the experts in the order of their first pair.
struct Groups {
    uint32_t peers;  // the lanes with this lane's expert
    int id, rank;    // this lane's expert; how many of its peers come before
    int start, n;    // of an expert's first lane: its first group; its groups
    int total;

    __device__ __forceinline__ Groups(const int32_t *ids, int pairs, int experts, int lane) {
        id = lane < pairs ? __ldg(ids + lane) : -1;
        const bool in = (unsigned)id < (unsigned)experts;
        if (!in) id = -1 - lane;
        peers = __match_any_sync(~0u, id);
        rank = __popc(peers & ((1u << lane) - 1));
        n = in && rank == 0 ? (__popc(peers) + 7) / 8 : 0;
        start = n;
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const int v = __shfl_up_sync(~0u, start, o);
            if (lane >= o) start += v;
        }
        total = __shfl_sync(~0u, start, 31);
        start -= n;
    }
    // Expert of group i; *pair: the pair in column lane / 4, or -1.
    __device__ __forceinline__ int at(int i, int lane, int *pair) const {
        const int first = __ffs(__ballot_sync(~0u, n > 0 && start <= i && i < start + n)) - 1;
        const int e = __shfl_sync(~0u, id, first);
        const int from = (i - __shfl_sync(~0u, start, first)) * 8;
        uint32_t m = __ballot_sync(~0u, id == e && rank >= from && rank < from + 8);
#pragma unroll
        for (int c = 0; c < 7; ++c)
            if (c < lane / 4) m &= m - 1;
        *pair = __ffs(m) - 1;
        return e;
    }
};

struct ExpertsParams {
    const uint8_t *q, *gate, *up, *down;
    const float *scales, *gate_scales, *up_scales, *down_scales;
    const int32_t *ids;
    const float *wts;
    const uint16_t *addend;
    uint16_t *out;
    float *h;  // [pair][inter], fp32
    int rows, pairs, top_k, experts, hidden, inter;
};

// Block: a group and 8 columns of h.  Rows 0-7 of the MMA are gate's, 8-15
// up's, so that a lane holds the gate and the up value of the same column and
// pair.
__global__ void __launch_bounds__(256, 3) few_gate_up_kernel(const ExpertsParams p) {
    __shared__ float part[8][128];
    pdl_trigger();
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, warps = blockDim.x / 32;
    const int g = lane / 4, t = lane % 4;
    const int cols = p.inter / 8, group = blockIdx.x / cols, c = blockIdx.x % cols;
    const Groups groups(p.ids, p.pairs, p.experts, lane);
    if (group >= groups.total) return;
    int pair;
    const int e = groups.at(group, lane, &pair);
    const int token = pair < 0 ? -1 : pair / p.top_k;
    const int tc[2] = {__shfl_sync(~0u, token, 8 * t), __shfl_sync(~0u, token, 8 * t + 4)};
    const int kb = p.hidden / 128;
    const int b1 = (warp + 1) * kb / warps;
    const size_t row = ((size_t)e * p.inter + c * 8 + g) * p.hidden + t * 16;
    const size_t sat = ((size_t)e * (p.inter / 128) + c / 16) * kb;
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    constexpr int kUnroll = 2;
    for (int b0 = warp * kb / warps; b0 < b1; b0 += kUnroll) {
        uint4 w[kUnroll][2][2], x[kUnroll][2];
        float sw[kUnroll][2], sx[kUnroll][2];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int b = b0 + u;
            const bool in = b < b1;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const size_t at = (size_t)b * 128 + h * 64;
                w[u][0][h] = in ? ld_nc_v4(p.gate + row + at) : zero4();
                w[u][1][h] = in ? ld_nc_v4(p.up + row + at) : zero4();
                x[u][h] = in && token >= 0
                              ? __ldg(reinterpret_cast<const uint4 *>(
                                    p.q + (size_t)token * p.hidden + at + t * 16))
                              : zero4();
            }
            sw[u][0] = in ? __ldg(p.gate_scales + sat + b) : 0.f;
            sw[u][1] = in ? __ldg(p.up_scales + sat + b) : 0.f;
#pragma unroll
            for (int i = 0; i < 2; ++i)
                sx[u][i] = in && tc[i] >= 0 ? __ldg(p.scales + (size_t)tc[i] * kb + b) : 0.f;
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int h = 0; h < 2; ++h) mma64(d, w[u][0][h], w[u][1][h], x[u][h]);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                acc[i] = fmaf(d[i], sx[u][i % 2] * sw[u][i / 2], acc[i]);
        }
    }
    // part[..][gate, up][pair of the group][column]
#pragma unroll
    for (int i = 0; i < 4; ++i) part[warp][i / 2 * 64 + (t * 2 + i % 2) * 8 + g] = acc[i];
    __syncthreads();
    if (warp < 2)
        for (int i = threadIdx.x; i < 64; i += 32 * min(warps, 2)) {
            const int to = __shfl_sync(~0u, pair, i / 8 * 4);
            float gv = 0.f, uv = 0.f;
            for (int q = 0; q < warps; ++q) gv += part[q][i], uv += part[q][64 + i];
            if (to >= 0)
                p.h[(size_t)to * p.inter + c * 8 + i % 8] =
                    __fdividef(gv, 1.f + __expf(-gv)) * uv;
        }
}

// Block: 16 columns of the output, for every pair, and their weighted sums.
// First h becomes e4m3 codes and scales in shared memory; then a unit of work
// is a group and a share of its inputs.  The first unit's weights do not
// depend on h and are asked for before it is there.  That overlaps little of
// the kernel before: 512 threads of 128 registers are all that an SM has, so a
// block starts only where no gate/up block is left.
constexpr int kDownWarps = 16;
// Row of codes: 64 bytes past a multiple of 128, so that the rows of two
// columns lie in different banks.
__host__ __device__ __forceinline__ int code_row(int inter) { return inter + 64; }
__host__ __device__ __forceinline__ size_t few_down_smem(int pairs, int inter) {
    return (size_t)pairs * (code_row(inter) + inter / 128 * 4);
}

__global__ void __launch_bounds__(kDownWarps * 32, 1) few_down_kernel(const ExpertsParams p) {
    extern __shared__ uint4 smem[];
    __shared__ float part[32][128], y[32][16], wts[32];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int g = lane / 4, t = lane % 4, n0 = blockIdx.x * 16;
    const int kb = p.inter / 128, pitch = code_row(p.inter);
    uint8_t *codes = reinterpret_cast<uint8_t *>(smem);
    float *scales = reinterpret_cast<float *>(codes + (size_t)p.pairs * pitch);
    const Groups groups(p.ids, p.pairs, p.experts, lane);
    // a weight of an id that is no expert: not used
    if (warp == 0) wts[lane] = lane < p.pairs ? __ldg(p.wts + lane) : 0.f;
    const uint32_t real = __ballot_sync(~0u, (unsigned)groups.id < (unsigned)p.experts);
    // shares: enough to give every warp a unit; at most 31 units, or the groups
    const int shares = groups.total ? min(kb, (kDownWarps + groups.total - 1) / groups.total) : 1;
    const int units = groups.total * shares;
    bool first = true;
    for (int u = warp; u < units || first; u += kDownWarps) {
        const bool work = u < units;
        int pair = -1, e = 0, b0 = 0, b1 = 0;
        if (work) {
            e = groups.at(u / shares, lane, &pair);
            b0 = u % shares * kb / shares, b1 = (u % shares + 1) * kb / shares;
        }
        const uint8_t *lo = p.down + ((size_t)e * p.hidden + n0 + g) * p.inter + t * 16;
        const uint8_t *hi = lo + (size_t)8 * p.inter;
        const float *sb = p.down_scales + ((size_t)e * (p.hidden / 128) + n0 / 128) * kb;
        const int row = max(pair, 0);
        const int p0 = __shfl_sync(~0u, row, 8 * t), p1 = __shfl_sync(~0u, row, 8 * t + 4);
        float acc[4] = {0.f, 0.f, 0.f, 0.f};
        constexpr int kUnroll = 4;
        do {
            uint4 w[kUnroll][2][2];
            float s[kUnroll];
#pragma unroll
            for (int i = 0; i < kUnroll; ++i) {
                const bool in = b0 + i < b1;
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const size_t at = (size_t)(b0 + i) * 128 + c * 64;
                    w[i][0][c] = in ? ld_nc_v4(lo + at) : zero4();
                    w[i][1][c] = in ? ld_nc_v4(hi + at) : zero4();
                }
                s[i] = in ? __ldg(sb + b0 + i) : 0.f;
            }
            if (first) {
                first = false;
                pdl_wait();
                // eight lanes to a block of 128 inputs
                for (int i0 = warp * 4; i0 < p.pairs * kb; i0 += 4 * kDownWarps) {
                    // (rows without an expert are read and not used)
                    const int i = min(i0 + lane / 8, p.pairs * kb - 1), r = i / kb, b = i % kb;
                    const int at = b * 128 + lane % 8 * 16;
                    float4 v[4];
                    float amax = 0.f;
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        v[j] = __ldcg(reinterpret_cast<const float4 *>(
                            p.h + (size_t)r * p.inter + at + j * 4));
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        amax = fmaxf(amax, fmaxf(fmaxf(fabsf(v[j].x), fabsf(v[j].y)),
                                                 fmaxf(fabsf(v[j].z), fabsf(v[j].w))));
#pragma unroll
                    for (int o = 4; o; o >>= 1)
                        amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, o));
                    const Fp8Scale scale(amax);
                    uint32_t q[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        q[j] = scale.codes(v[j].x, v[j].y, v[j].z, v[j].w);
                    *reinterpret_cast<uint4 *>(codes + r * pitch + at) =
                        make_uint4(q[0], q[1], q[2], q[3]);
                    if (lane % 8 == 0) scales[r * kb + b] = scale.scale;
                }
                __syncthreads();
            }
#pragma unroll
            for (int i = 0; i < kUnroll; ++i) {
                if (b0 + i >= b1) break;
                float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int c = 0; c < 2; ++c)
                    mma64(d, w[i][0][c], w[i][1][c],
                          *reinterpret_cast<const uint4 *>(codes + row * pitch +
                                                           (b0 + i) * 128 + c * 64 + t * 16));
                const float s0 = scales[p0 * kb + b0 + i] * s[i];
                const float s1 = scales[p1 * kb + b0 + i] * s[i];
#pragma unroll
                for (int c = 0; c < 4; ++c) acc[c] = fmaf(d[c], c % 2 ? s1 : s0, acc[c]);
            }
            b0 += kUnroll;
        } while (b0 < b1);
        // (columns without a pair hold another's sums: nobody reads them)
        if (work)
#pragma unroll
            for (int c = 0; c < 4; ++c) part[u][(t * 2 + c % 2) * 16 + g + c / 2 * 8] = acc[c];
    }
    __syncthreads();
    for (int i = warp; i < groups.total; i += kDownWarps) {
        int pair;
        groups.at(i, lane, &pair);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const int to = __shfl_sync(~0u, pair, (c * 2 + lane / 16) * 4);
            float v = 0.f;
            for (int q = 0; q < shares; ++q) v += part[i * shares + q][c * 32 + lane];
            if (to >= 0) y[to][lane % 16] = v;
        }
    }
    __syncthreads();
    const int row = threadIdx.x / 16, col = threadIdx.x % 16;
    if (row >= p.rows) return;
    const size_t at = (size_t)row * p.hidden + n0 + col;
    float v = p.addend ? bf16_lo(p.addend[at]) : 0.f;
    for (int j = 0; j < p.top_k; ++j) {
        const int pair = row * p.top_k + j;
        if (real >> pair & 1) v = fmaf(wts[pair], y[pair][col], v);
    }
    p.out[at] = f2bf16_rn(v);
}

}  // namespace

cudaError_t launch_few_dense(const Fp8Mat &a, const float *sa, const Fp8Mat &b, const float *sb,
                             void *out, int out_dtype, int sms, cudaStream_t st) {
    DenseParams p{a.p, b.p, a.stride, b.stride, sa, sb, (int)a.rows, (int)b.rows, (int)a.k,
                  (int)((a.k + 127) / 128), out, out_dtype};
    const int tiles = (p.n + 15) / 16;
    // a warp takes 4 blocks of inputs; fewer where there would not be 8 warps
    // to an SM
    int warps = (p.kb + 3) / 4;
    while (warps < p.kb && (int64_t)tiles * warps < 8 * sms) ++warps;
    if (warps > 16) warps = 16;
    if (p.m <= 8) few_dense_kernel<1><<<tiles, warps * 32, 0, st>>>(p);
    else few_dense_kernel<2><<<tiles, warps * 32, 0, st>>>(p);
    return cudaGetLastError();
}

bool few_experts(int64_t rows, const moeop_experts_config &c) {
    const int64_t pairs = rows * c.top_k;
    return pairs <= kFewPairs && few_down_smem((int)pairs, c.inter) <= kFewSmem;
}
cudaError_t allow_few_smem() {
    return cudaFuncSetAttribute(few_down_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                kFewSmem);
}

cudaError_t launch_few_experts(const ExpertsArgs &a, float *h, cudaStream_t st) {
    const int pairs = a.rows * a.c.top_k;
    const ExpertsParams p{a.q, a.w.gate, a.w.up, a.w.down, a.scales, a.w.gate_scales,
                          a.w.up_scales, a.w.down_scales, a.ids, a.wts, a.addend, a.out, h,
                          a.rows, pairs, a.c.top_k, a.c.num_experts, a.c.hidden, a.c.inter};
    // one warp for 4 blocks of inputs
    int warps = (a.c.hidden / 128 + 3) / 4;
    if (warps > 8) warps = 8;
    few_gate_up_kernel<<<(unsigned)pairs * (a.c.inter / 8), warps * 32, 0, st>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute at[1];
    cfg.gridDim = dim3(a.c.hidden / 16);
    cfg.blockDim = dim3(kDownWarps * 32);
    cfg.dynamicSmemBytes = few_down_smem(pairs, a.c.inter);
    cfg.stream = st;
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, few_down_kernel, p);
}

}  // namespace op
}  // namespace moe

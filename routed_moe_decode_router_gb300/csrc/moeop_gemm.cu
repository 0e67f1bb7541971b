// moeop_gemm.cu -- the FP8 products (moeop_matmul_fp8 and the two products of
// moeop_experts_fp8) on the 5th-generation tensor cores.
//
//   C[m][n] = sum_b sa[m][b] sb[n/128][b] (sum of the 128 inputs of block b
//             of A[m][i] B[n][i])
//
// The scales change every 128 inputs, so a block's sum leaves the tensor core
// before the next block is added: an A tile of 128 rows and a B tile of NB x
// 128 outputs are multiplied block by block into one of two halves of tensor
// memory (four MMAs of 32 inputs), and while the next block runs into the
// other half, eight warps read the finished one and add it, scaled, to fp32
// accumulators in registers (128 per thread for NB = 2).
//
// Roles: warp 8 loads (TMA, 128-byte swizzle, a ring of kStages), warp 9
// issues the MMAs, warps 0-7 accumulate and store.  Warp w reads lanes
// 32 (w % 4) .. + 31 (rows) and, of each 128-output block, columns
// 64 (w / 4) .. + 63, so that in the gate/up form a thread holds a gate value
// and the up value of the same column.
//
// Blocks are persistent over the tiles.  Where there are fewer tiles than
// SMs the inputs are split over a cluster of S blocks, whose partial sums are
// added through distributed shared memory in rank order: the result does not
// depend on timing.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <mutex>

#include "moeop.cuh"
#include "moeop_tc.cuh"

namespace moe {
namespace op {

__device__ uint32_t g_status;

namespace {

enum { kDense = 0, kGateUp = 1, kDown = 2 };
constexpr int kThreads = 320;
constexpr int kTile = 128 * 128;  // bytes of one operand tile

template <int NB>
constexpr int stages() { return NB == 2 ? 4 : 6; }
template <int NB>
constexpr size_t ring_bytes() { return (size_t)stages<NB>() * (1 + NB) * kTile; }

struct Params {
    int rows, n, kb;          // dense: rows of A; outputs; blocks of 128 inputs
    int tiles_m, tiles_n;     // dense: row tiles; column tiles (per expert)
    int nblocks;              // 128-output blocks of B (per expert)
    int split;                // blocks per cluster
    const float *sa, *sb, *sb2;
    void *out;
    int out_dtype;
    // experts
    const int *num_tiles;
    const int4 *tiles;        // expert, first position, rows
    const int *pair, *token;
    uint8_t *h;
    float *h_scales;
};

struct Tile {
    int e, pos, rows, nt;
};

template <int MODE>
__device__ __forceinline__ int tile_count(const Params &p) {
    return MODE == kDense ? p.tiles_m * p.tiles_n : __ldcg(p.num_tiles) * p.tiles_n;
}
template <int MODE>
__device__ __forceinline__ Tile tile_at(const Params &p, int t) {
    const int mt = t / p.tiles_n, nt = t % p.tiles_n;
    if (MODE == kDense) return {0, mt * 128, min(128, p.rows - mt * 128), nt};
    const int4 d = __ldcg(p.tiles + mt);
    return {d.x, d.y, d.z, nt};
}

// 16 consecutive outputs of one row.
__device__ __forceinline__ void store16(void *out, int dtype, size_t at, const float *v, int left) {
    if (dtype == MOEOP_FP32) {
        float *o = static_cast<float *>(out) + at;
        if (left >= 16 && (reinterpret_cast<uintptr_t>(o) & 15) == 0) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                reinterpret_cast<float4 *>(o)[i] =
                    make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (i < left) o[i] = v[i];
        }
        return;
    }
    uint16_t *o = static_cast<uint16_t *>(out) + at;
    uint32_t u[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (dtype == MOEOP_BF16) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            u[i] = *reinterpret_cast<const uint32_t *>(&b);
        } else {
            u[i] = pack_f16x2(v[2 * i], v[2 * i + 1]);
        }
    }
    if (left >= 16 && (reinterpret_cast<uintptr_t>(o) & 15) == 0) {
        reinterpret_cast<uint4 *>(o)[0] = make_uint4(u[0], u[1], u[2], u[3]);
        reinterpret_cast<uint4 *>(o)[1] = make_uint4(u[4], u[5], u[6], u[7]);
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (i < left) o[i] = (uint16_t)(u[i / 2] >> (16 * (i % 2)));
    }
}

template <int MODE, int NB>
__global__ void __launch_bounds__(kThreads, 1)
    gemm_kernel(const __grid_constant__ TensorMap ma, const __grid_constant__ TensorMap mb,
                const __grid_constant__ TensorMap mb2, const Params p) {
    constexpr int S = stages<NB>();
    constexpr int kStage = (1 + NB) * kTile;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t full[S], empty[S], tm_full[2], tm_empty[2];
    __shared__ float amax_s[2][128];
    __shared__ uint32_t tm_base;
    __shared__ int abort_s;
    const uint32_t ring = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int rank = p.split > 1 ? (int)cluster_rank() : 0;

    if (threadIdx.x == 0) {
        for (int i = 0; i < S; ++i) mbar_init(&full[i], 1), mbar_init(&empty[i], 1);
        for (int i = 0; i < 2; ++i) mbar_init(&tm_full[i], 1), mbar_init(&tm_empty[i], 8);
        abort_s = 0;
        fence_mbar_init();
    }
    if (warp == 8 && lane == 0) {
        tma_prefetch_map(&ma);
        tma_prefetch_map(&mb);
        if (MODE == kGateUp) tma_prefetch_map(&mb2);
    }
    if (warp == 9) tmem_alloc(&tm_base, 256 * NB);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = tm_base;

    const int first = blockIdx.x / p.split, step = gridDim.x / p.split;
    const int kb0 = rank * p.kb / p.split, kb1 = (rank + 1) * p.kb / p.split;
    const int total = tile_count<MODE>(p);
    int syncs = 0;  // of this thread with its cluster: two in every split block

    if (warp == 8) {
        // ---- loads
        int it = 0;
        bool ok = true;
        for (int t = first; t < total && ok; t += step) {
            const Tile T = tile_at<MODE>(p, t);
            int4 rows4 = make_int4(0, 0, 0, 0);
            if (MODE != kDense) {
                // rows 4 lane .. + 3 of the tile; past its end the last row again
                int *r = &rows4.x;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int pos = T.pos + min(4 * lane + i, T.rows - 1);
                    r[i] = MODE == kGateUp ? __ldcg(p.token + pos) : pos;
                }
            }
            const int b0 = (MODE == kGateUp ? T.e * p.n : MODE == kDown ? T.e * p.n : 0) +
                           T.nt * (MODE == kGateUp ? 128 : 128 * NB);
            const uint32_t bytes =
                NB * kTile + (MODE == kDense ? kTile : (T.rows + 3) / 4 * 512);
            for (int b = kb0; b < kb1 && ok; ++b, ++it) {
                const int s = it % S;
                ok = __all_sync(~0u, wait_bar(&empty[s], (it / S & 1) ^ 1, &abort_s));
                if (!ok) break;
                const uint32_t dst = ring + s * kStage;
                if (lane == 0) {
                    mbar_arrive_expect_tx(&full[s], bytes);
                    if (MODE == kDense) tma_box(dst, &ma, b * 128, T.pos, &full[s]);
                    tma_box(dst + kTile, &mb, b * 128, b0, &full[s]);
                    if (NB == 2)
                        tma_box(dst + 2 * kTile, MODE == kGateUp ? &mb2 : &mb, b * 128,
                                MODE == kGateUp ? b0 : b0 + 128, &full[s]);
                }
                __syncwarp();
                if (MODE != kDense && 4 * lane < T.rows)
                    tma_gather4(dst + lane * 512, &ma, b * 128, rows4, &full[s]);
            }
        }
        if (!ok && lane == 0)  // copies in flight end before the block does
            for (int i = it > S ? it - S : 0; i < it; ++i)
                mbar_wait(&full[i % S], i / S & 1);
    } else if (warp == 9) {
        // ---- MMAs
        if (lane == 0) {
            constexpr uint32_t idesc = tc_idesc(128, 128 * NB);
            int it = 0;
            bool ok = true;
            for (int t = first; t < total && ok; t += step) {
                for (int b = kb0; b < kb1; ++b, ++it) {
                    const int s = it % S, buf = it & 1;
                    ok = wait_bar(&tm_empty[buf], (it / 2 & 1) ^ 1, &abort_s) &&
                         wait_bar(&full[s], it / S & 1, &abort_s);
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t da = tc_desc(ring + s * kStage);
                    const uint64_t db = tc_desc(ring + s * kStage + kTile);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        tc_mma_e4m3(tm + buf * 128 * NB, da + 2 * k, db + 2 * k, idesc, k > 0);
                    tc_commit(&empty[s]);
                    tc_commit(&tm_full[buf]);
                }
            }
        }
        __syncwarp();
    } else {
        // ---- accumulation and stores
        const int wg = warp / 4, r = (warp % 4) * 32 + lane;
        const uint32_t tm_lane = tm + ((uint32_t)(warp % 4) * 32 << 16) + wg * 64;
        int it = 0;
        bool ok = true;  // false: an earlier wait gave up; nothing is stored any more
        for (int t = first; t < total; t += step) {
            const Tile T = tile_at<MODE>(p, t);
            const bool some = (warp % 4) * 32 < T.rows, live = r < T.rows;
            const int arow = MODE == kGateUp ? (live ? __ldcg(p.token + T.pos + r) : 0)
                                             : T.pos + (live ? r : 0);
            const float *sa = p.sa + (size_t)arow * p.kb;
            const int nb0 = MODE == kGateUp ? T.nt : T.nt * NB;
            const int nb1 = MODE == kGateUp ? nb0 : min(nb0 + NB - 1, p.nblocks - 1);
            const size_t eb = MODE == kDense ? 0 : (size_t)T.e * p.nblocks;
            const float *sb0 = p.sb + (eb + nb0) * p.kb;
            const float *sb1 = (MODE == kGateUp ? p.sb2 : p.sb) + (eb + nb1) * p.kb;
            uint64_t acc[32 * NB];
#pragma unroll
            for (int i = 0; i < 32 * NB; ++i) acc[i] = 0;
            float a_next = 0.f, b0_next = 0.f, b1_next = 0.f;
            if (kb0 < kb1 && some) {
                a_next = MODE == kDown ? __ldcg(sa + kb0) : __ldg(sa + kb0);
                b0_next = __ldg(sb0 + kb0);
                if (NB == 2) b1_next = __ldg(sb1 + kb0);
            }
            for (int b = kb0; b < kb1; ++b, ++it) {
                const int buf = it & 1;
                const float s0 = a_next * b0_next, s1 = a_next * b1_next;
                if (b + 1 < kb1 && some) {
                    a_next = MODE == kDown ? __ldcg(sa + b + 1) : __ldg(sa + b + 1);
                    b0_next = __ldg(sb0 + b + 1);
                    if (NB == 2) b1_next = __ldg(sb1 + b + 1);
                }
                if (ok) ok = __all_sync(~0u, wait_bar(&tm_full[buf], it / 2 & 1, &abort_s));
                tc_fence_after();
                if (some && ok) {
                    const uint64_t p0 = pack2(s0, s0), p1 = pack2(s1, s1);
#pragma unroll
                    for (int c = 0; c < 2 * NB; ++c) {
                        uint32_t v[32];
                        tmem_load32(tm_lane + buf * 128 * NB + (c / 2) * 128 + (c % 2) * 32, v);
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            fma2(acc[c * 16 + i], v[2 * i], v[2 * i + 1], c < 2 ? p0 : p1);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&tm_empty[buf]);
            }
            if (p.split > 1) {
                // Every load and MMA of this block is complete (the last
                // tm_full), so the ring holds the partial sums now; one tile
                // per cluster.
                float *part = reinterpret_cast<float *>(smem_raw + (ring - smem_u32(smem_raw)));
                if (rank && some && ok)
#pragma unroll
                    for (int i = 0; i < 32 * NB; ++i) {
                        const float2 f = unpack2(acc[i]);
                        const int col = (i / 32) * 128 + wg * 64 + (i % 32) * 2;
                        part[col * 128 + r] = f.x;
                        part[(col + 1) * 128 + r] = f.y;
                    }
                cluster_sync();
                if (rank == 0 && some && ok)
                    for (int q = 1; q < p.split; ++q) {
                        const uint32_t remote = map_rank(ring, q) + r * 4;
#pragma unroll
                        for (int i = 0; i < 32 * NB; ++i) {
                            const int col = (i / 32) * 128 + wg * 64 + (i % 32) * 2;
                            const float2 f = unpack2(acc[i]);
                            acc[i] = pack2(f.x + ld_cluster(remote + col * 512),
                                           f.y + ld_cluster(remote + (col + 1) * 512));
                        }
                    }
                cluster_sync();
                syncs = 2;
                if (rank) break;
            }
            if (MODE == kGateUp) {
                float amax = 0.f;
                if (some) {
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        const float2 g = unpack2(acc[i]), u = unpack2(acc[i + 32 * (NB - 1)]);
                        const float h0 = __fdividef(g.x, 1.f + __expf(-g.x)) * u.x;
                        const float h1 = __fdividef(g.y, 1.f + __expf(-g.y)) * u.y;
                        acc[i] = pack2(h0, h1);
                        amax = fmaxf(amax, fmaxf(fabsf(h0), fabsf(h1)));
                    }
                }
                amax_s[wg][r] = amax;
                named_bar(1, 256);
                amax = fmaxf(fmaxf(amax_s[0][r], amax_s[1][r]), kFp8Tiny);
                named_bar(1, 256);  // before the next tile writes amax_s
                if (live && ok) {
                    const float up = kFp8Max / amax;
                    const size_t at = (size_t)(T.pos + r) * p.n + T.nt * 128 + wg * 64;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t q[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float2 x = unpack2(acc[i * 8 + j * 2]);
                            const float2 y = unpack2(acc[i * 8 + j * 2 + 1]);
                            q[j] = pack_e4m3x4(x.x * up, x.y * up, y.x * up, y.y * up);
                        }
                        *reinterpret_cast<uint4 *>(p.h + at + i * 16) =
                            make_uint4(q[0], q[1], q[2], q[3]);
                    }
                    if (wg == 0)
                        p.h_scales[(size_t)(T.pos + r) * (p.n / 128) + T.nt] = amax / kFp8Max;
                }
            } else if (live && ok) {
                const size_t orow = MODE == kDown ? (size_t)__ldcg(p.pair + T.pos + r)
                                                  : (size_t)(T.pos + r);
#pragma unroll
                for (int c = 0; c < 4 * NB; ++c) {
                    const int col = (T.nt * NB + c / 4) * 128 + wg * 64 + (c % 4) * 16;
                    float v[16];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float2 f = unpack2(acc[c * 8 + i]);
                        v[2 * i] = f.x;
                        v[2 * i + 1] = f.y;
                    }
                    if (col < p.n)
                        store16(p.out, p.out_dtype, orow * p.n + col, v, p.n - col);
                }
            }
        }
    }
    // The accumulating warps have met their cluster twice; the other warps,
    // and all of a block without a tile, do so here.
    if (p.split > 1)
        for (; syncs < 2; ++syncs) cluster_sync();
    tc_fence_before();
    __syncthreads();
    if (warp == 9) tmem_free(tm, 256 * NB);
    if (threadIdx.x == 0 && abort_s) atomicCAS(&g_status, 0u, (uint32_t)MOE_DEV_WAIT_TIMEOUT);
}

// ---------------------------------------------------------------------------
// Pairs (row, slot) in expert order
// ---------------------------------------------------------------------------
// A counting sort in one launch: each block of a cluster counts its share of
// the ids in shared memory, reads the others' counts, and places its own
// pairs after those of the lower ranks.  The order inside an expert follows
// the shared-memory atomics and may differ from call to call; no result
// depends on it, for every row of a product is computed by itself and goes
// back to its pair's place.
struct IndexParams {
    const int32_t *ids;
    int pairs, top_k, experts;
    int *num_tiles, *pair, *token;
    int4 *tiles;
};

__global__ void __launch_bounds__(1024) index_kernel(IndexParams p) {
    __shared__ int hist[MOEOP_MAX_EXPERTS], cursor[MOEOP_MAX_EXPERTS];
    __shared__ int warp_rows[32], warp_tiles[32];
    const int rank = (int)cluster_rank(), ranks = (int)cluster_size();
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    hist[tid] = 0;
    __syncthreads();
    for (int64_t i = rank * 1024 + tid; i < p.pairs; i += ranks * 1024) {
        const int e = __ldg(p.ids + i);
        if ((unsigned)e < (unsigned)p.experts) atomicAdd(&hist[e], 1);
    }
    cluster_sync();
    int rows = 0, lower = 0;
    for (int q = 0; q < ranks; ++q) {
        const int v = ld_cluster_i(map_rank(smem_u32(&hist[tid]), q));
        if (q < rank) lower += v;
        rows += v;
    }
    // exclusive prefix sums of the rows and of the tiles of 128
    const int tiles = (rows + 127) / 128;
    int a = rows, b = tiles;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const int x = __shfl_up_sync(~0u, a, o), y = __shfl_up_sync(~0u, b, o);
        if (lane >= o) a += x, b += y;
    }
    if (lane == 31) warp_rows[warp] = a, warp_tiles[warp] = b;
    __syncthreads();
    if (warp == 0) {
        int x = warp_rows[lane], y = warp_tiles[lane];
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const int u = __shfl_up_sync(~0u, x, o), v = __shfl_up_sync(~0u, y, o);
            if (lane >= o) x += u, y += v;
        }
        warp_rows[lane] = x, warp_tiles[lane] = y;
    }
    __syncthreads();
    const int row0 = a - rows + (warp ? warp_rows[warp - 1] : 0);
    const int tile0 = b - tiles + (warp ? warp_tiles[warp - 1] : 0);
    cursor[tid] = row0 + lower;
    if (rank == 0) {
        if (tid == 0) *p.num_tiles = warp_tiles[31];
        for (int t = 0; t < tiles; ++t)
            p.tiles[tile0 + t] = make_int4(tid, row0 + t * 128, min(128, rows - t * 128), 0);
    }
    __syncthreads();
    for (int64_t i = rank * 1024 + tid; i < p.pairs; i += ranks * 1024) {
        const int e = __ldg(p.ids + i);
        if ((unsigned)e < (unsigned)p.experts) {
            const int at = atomicAdd(&cursor[e], 1);
            p.pair[at] = (int)i;
            p.token[at] = (int)(i / p.top_k);
        }
    }
    cluster_sync();  // the others have read this block's counts
}

// ---------------------------------------------------------------------------
// out[t] = sum_j wts[t][j] y[t * k + j] (+ addend[t]), in slot order
// ---------------------------------------------------------------------------
// Bound by memory: k bf16 rows in, one out.  A thread owns 8 outputs.
struct CombineParams {
    const int32_t *ids;
    const float *wts;
    const uint16_t *y, *addend;
    uint16_t *out;
    int rows, hidden, top_k, experts;
};

__global__ void __launch_bounds__(256) combine_kernel(CombineParams p) {
    const int per_row = p.hidden / 8;
    const int64_t n = (int64_t)p.rows * per_row;
    for (int64_t i = blockIdx.x * 256LL + threadIdx.x; i < n; i += gridDim.x * 256LL) {
        const int64_t t = i / per_row;
        const int col = (int)(i % per_row) * 8;
        float acc[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] = 0.f;
        if (p.addend) {
            const uint4 v = *reinterpret_cast<const uint4 *>(p.addend + t * p.hidden + col);
            const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[2 * j] = bf16_lo(u[j]), acc[2 * j + 1] = bf16_hi(u[j]);
        }
        for (int j = 0; j < p.top_k; ++j) {
            const int64_t pair = t * p.top_k + j;
            if ((unsigned)__ldg(p.ids + pair) >= (unsigned)p.experts) continue;
            const float w = __ldg(p.wts + pair);
            const uint4 v = ld_cg_v4(p.y + pair * p.hidden + col);
            const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                acc[2 * c] = fmaf(w, bf16_lo(u[c]), acc[2 * c]);
                acc[2 * c + 1] = fmaf(w, bf16_hi(u[c]), acc[2 * c + 1]);
            }
        }
        uint32_t o[4];
#pragma unroll
        for (int c = 0; c < 4; ++c)
            o[c] = (uint32_t)f2bf16_rn(acc[2 * c]) | (uint32_t)f2bf16_rn(acc[2 * c + 1]) << 16;
        *reinterpret_cast<uint4 *>(p.out + t * p.hidden + col) = make_uint4(o[0], o[1], o[2], o[3]);
    }
}

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------
using EncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                              const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                              const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
std::mutex g_mu;
EncodeFn g_encode = nullptr;
struct Dev {
    int sms = 0;
    uint32_t *status = nullptr;
} g_devs[64];

template <int MODE, int NB>
cudaError_t allow_smem() {
    return cudaFuncSetAttribute(gemm_kernel<MODE, NB>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)(ring_bytes<NB>() + 1024));
}

// Looked up once per device: SM count, the kernels' shared-memory limit, the
// status word and the driver's tensor-map encoder.
cudaError_t device(Dev **out) {
    int d = 0;
    cudaError_t e = cudaGetDevice(&d);
    if (e != cudaSuccess) return e;
    if (d < 0 || d >= 64) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lk(g_mu);
    Dev &v = g_devs[d];
    if (!v.status) {
        if (!g_encode) {
            void *fn = nullptr;
            cudaDriverEntryPointQueryResult r;
            if ((e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000,
                                                      cudaEnableDefault, &r)) != cudaSuccess)
                return e;
            if (r != cudaDriverEntryPointSuccess || !fn) return cudaErrorSymbolNotFound;
            g_encode = reinterpret_cast<EncodeFn>(fn);
        }
        void *sym = nullptr;
        if ((e = cudaDeviceGetAttribute(&v.sms, cudaDevAttrMultiProcessorCount, d)) != cudaSuccess ||
            (e = allow_smem<kDense, 1>()) != cudaSuccess ||
            (e = allow_smem<kDense, 2>()) != cudaSuccess ||
            (e = allow_smem<kGateUp, 2>()) != cudaSuccess ||
            (e = allow_smem<kDown, 1>()) != cudaSuccess ||
            (e = allow_smem<kDown, 2>()) != cudaSuccess ||
            (e = cudaGetSymbolAddress(&sym, g_status)) != cudaSuccess)
            return e;
        v.status = static_cast<uint32_t *>(sym);
    }
    *out = &v;
    return cudaSuccess;
}

// Map of an FP8 matrix in tiles of 128 bytes x box_rows, 128-byte swizzle;
// what lies outside the matrix reads as zero.
cudaError_t make_map(TensorMap *m, const Fp8Mat &a, uint32_t box_rows) {
    const cuuint64_t dims[2] = {(cuuint64_t)a.k, (cuuint64_t)a.rows};
    const cuuint64_t strides[1] = {(cuuint64_t)a.stride};
    const cuuint32_t box[2] = {128, box_rows}, elem[2] = {1, 1};
    const CUresult r = g_encode(
        reinterpret_cast<CUtensorMap *>(m), CU_TENSOR_MAP_DATA_TYPE_UINT8, 2,
        const_cast<uint8_t *>(a.p), dims, strides, box, elem, CU_TENSOR_MAP_INTERLEAVE_NONE,
        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int MODE, int NB>
cudaError_t launch(const TensorMap &ma, const TensorMap &mb, const TensorMap &mb2, const Params &p,
                   int grid, cudaStream_t st) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = ring_bytes<NB>() + 1024;
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    if (p.split > 1) {
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim.x = p.split;
        at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
        cfg.attrs = at;
        cfg.numAttrs = 1;
    }
    return cudaLaunchKernelEx(&cfg, gemm_kernel<MODE, NB>, ma, mb, mb2, p);
}

// Blocks per cluster that share one tile's inputs: as many as fill the SMs
// (at most 8, the portable cluster), each with two blocks of inputs or more.
int split_of(int sms, int64_t tiles, int kb) {
    int64_t s = sms / (tiles > 0 ? tiles : 1);
    if (s > 8) s = 8;
    if (s > kb / 2) s = kb / 2;
    return s < 1 ? 1 : (int)s;
}

}  // namespace

cudaError_t status_word(uint32_t **p) {
    Dev *d;
    const cudaError_t e = device(&d);
    if (e == cudaSuccess) *p = d->status;
    return e;
}

cudaError_t launch_matmul_fp8(const Fp8Mat &a, const float *sa, const Fp8Mat &b, const float *sb,
                              void *out, int out_dtype, cudaStream_t st) {
    Dev *d;
    cudaError_t e = device(&d);
    if (e != cudaSuccess) return e;
    Params p{};
    p.rows = (int)a.rows;
    p.n = (int)b.rows;
    p.kb = (int)((a.k + 127) / 128);
    p.nblocks = (p.n + 127) / 128;
    p.sa = sa;
    p.sb = p.sb2 = sb;
    p.out = out;
    p.out_dtype = out_dtype;
    p.tiles_m = (p.rows + 127) / 128;
    // Tiles of 128 x 256 feed the tensor core with fewer shared-memory reads
    // per MMA; tiles of 128 x 128 where they need fewer waves of the SMs.
    const int64_t t1 = (int64_t)p.tiles_m * p.nblocks;
    const int64_t t2 = (int64_t)p.tiles_m * ((p.nblocks + 1) / 2);
    const bool wide = 11 * ((t1 + d->sms - 1) / d->sms) >= 20 * ((t2 + d->sms - 1) / d->sms);
    p.tiles_n = wide ? (p.nblocks + 1) / 2 : p.nblocks;
    const int64_t tiles = wide ? t2 : t1;
    p.split = split_of(d->sms, tiles, p.kb);
    TensorMap ma, mb;
    if ((e = make_map(&ma, a, 128)) != cudaSuccess || (e = make_map(&mb, b, 128)) != cudaSuccess)
        return e;
    const int grid = p.split > 1 ? (int)tiles * p.split : (int)(tiles < d->sms ? tiles : d->sms);
    return wide ? launch<kDense, 2>(ma, mb, mb, p, grid, st)
                : launch<kDense, 1>(ma, mb, mb, p, grid, st);
}

cudaError_t launch_experts_fp8(const ExpertsArgs &a, cudaStream_t st) {
    Dev *d;
    cudaError_t e = device(&d);
    if (e != cudaSuccess) return e;
    const int H = a.c.hidden, I = a.c.inter, E = a.c.num_experts, k = a.c.top_k;
    const int64_t P = (int64_t)a.rows * k;
    const ExpertsWs w = ExpertsWs::make(a.c, a.rows);
    int *num_tiles = reinterpret_cast<int *>(a.ws + w.header);
    int4 *tiles = reinterpret_cast<int4 *>(a.ws + w.tiles);
    int *pair = reinterpret_cast<int *>(a.ws + w.pair);
    int *token = reinterpret_cast<int *>(a.ws + w.token);
    uint8_t *h = reinterpret_cast<uint8_t *>(a.ws + w.h);
    float *h_scales = reinterpret_cast<float *>(a.ws + w.h_scales);
    uint16_t *y = reinterpret_cast<uint16_t *>(a.ws + w.y);

    TensorMap mq, mg, mu, mh, md;
    if ((e = make_map(&mq, {a.q, a.rows, H, H}, 1)) != cudaSuccess ||
        (e = make_map(&mg, {a.w.gate, (int64_t)E * I, H, H}, 128)) != cudaSuccess ||
        (e = make_map(&mu, {a.w.up, (int64_t)E * I, H, H}, 128)) != cudaSuccess ||
        (e = make_map(&mh, {h, P, I, I}, 1)) != cudaSuccess ||
        (e = make_map(&md, {a.w.down, (int64_t)E * H, I, I}, 128)) != cudaSuccess)
        return e;

    // one block up to 4096 pairs, else a cluster of 8
    IndexParams ip{a.ids, (int)P, k, E, num_tiles, pair, token, tiles};
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute at[1];
    const int ranks = P <= 4096 ? 1 : 8;
    cfg.gridDim = dim3(ranks);
    cfg.blockDim = dim3(1024);
    cfg.stream = st;
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = ranks;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    if ((e = cudaLaunchKernelEx(&cfg, index_kernel, ip)) != cudaSuccess) return e;

    Params p{};
    p.num_tiles = num_tiles;
    p.tiles = tiles;
    p.pair = pair;
    p.token = token;
    p.h = h;
    p.h_scales = h_scales;
    p.sa = a.scales;
    p.sb = a.w.gate_scales;
    p.sb2 = a.w.up_scales;
    p.n = I;
    p.kb = H / 128;
    p.nblocks = p.tiles_n = I / 128;
    // the number of tiles is known on the device only: its upper bound
    int64_t most = (int64_t)w.max_tiles * p.tiles_n;
    p.split = split_of(d->sms, most, p.kb);
    int grid = p.split > 1 ? (int)most * p.split : (int)(most < d->sms ? most : d->sms);
    if ((e = launch<kGateUp, 2>(mq, mg, mu, p, grid, st)) != cudaSuccess) return e;

    p.sa = h_scales;
    p.sb = p.sb2 = a.w.down_scales;
    p.n = H;
    p.kb = I / 128;
    p.nblocks = H / 128;
    p.out = y;
    p.out_dtype = MOEOP_BF16;
    const bool wide = (int64_t)w.max_tiles * ((p.nblocks + 1) / 2) >= d->sms;
    p.tiles_n = wide ? (p.nblocks + 1) / 2 : p.nblocks;
    most = (int64_t)w.max_tiles * p.tiles_n;
    p.split = split_of(d->sms, most, p.kb);
    grid = p.split > 1 ? (int)most * p.split : (int)(most < d->sms ? most : d->sms);
    e = wide ? launch<kDown, 2>(mh, md, md, p, grid, st) : launch<kDown, 1>(mh, md, md, p, grid, st);
    if (e != cudaSuccess) return e;

    CombineParams cp{a.ids, a.wts, y, a.addend, a.out, a.rows, H, k, E};
    const int64_t blocks = ((int64_t)a.rows * (H / 8) + 255) / 256;
    combine_kernel<<<(int)(blocks < 65536 ? blocks : 65536), 256, 0, st>>>(cp);
    return cudaGetLastError();
}

}  // namespace op
}  // namespace moe

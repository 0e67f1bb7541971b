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
// other half, sixteen warps read the finished one and add it, scaled, to fp32
// accumulators in registers (64 per thread for NB = 2).
//
// Roles: warps 0-15 accumulate and store, warp 16 loads (TMA, 128-byte
// swizzle, a ring of 4 or 6 stages) with warps 18 and 19 where rows are
// gathered, warp 17 issues the MMAs.  Warp w reads lanes 32 (w % 4) .. + 31
// (rows) and, of each 128-output block, columns 32 (w / 4) .. + 31, so that
// in the gate/up form a thread holds a gate value and the up value of the
// same column.
//
// Blocks are persistent over the tiles.  Where there are fewer tiles than
// SMs the inputs are split over a cluster of S blocks.  Each 32 rows belong
// to one rank, into whose (by then idle) ring the others write their partial
// sums, and which adds them in rank order: the result does not depend on
// timing.
//
// Bound by the way out of tensor memory: 128 inputs of a 128 x 256 tile are
// 512 cycles of MMAs, but take 900.  Each of the 16 warps, four to a scheduler,
// has some 145 instructions for them and waits for its loads of 8 columns one
// at a time; no unit is saturated (8192 x 4096 x 4096: issue slots 54%, tensor
// pipe 52%, L1 46%).
// One GB300: 8192 x 4096 x 4096 119 us (2.3 PFLOP/s) in a short run, 127 when
// thousands in a row meet the power limit; 333 x 1000 x 2048 8.1 us; experts (hidden 2048, 128 x 768, top 8), 4096
// rows 322 us: gate/up 162, down 113, the weighted sum 47 (6.1 TB/s), lists
// 10; experts (hidden 4096, 160 x 1536, top 8), 61 rows 419 to 428 us.  The products y
// are fp32: rounded to bf16 on their way they would take 37 us less of the
// 4096 rows and 5 of the 61, and leave an error of 2^-9 of each product where
// slots cancel.
//
// Calls of a few rows go to moeop_few.cu.
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
constexpr int kColGroups = 4, kCols = 128 / kColGroups;  // of a 128-output block
constexpr int kAccWarps = 4 * kColGroups, kLoadWarp = kAccWarps, kMmaWarp = kAccWarps + 1;
constexpr int kThreads = (kAccWarps + 4) * 32;
constexpr int kBoxRows = 32;      // rows of A in one copy
constexpr int kMaxSplit = 7;      // six other ranks' sums of 32 rows fill the ring
constexpr int kTile = 128 * 128;  // bytes of one operand tile

// The ring: 192 KB.
template <int NB>
constexpr int stages() { return NB == 2 ? 4 : 6; }
constexpr size_t kRing = 12 * kTile;

struct Params {
    int rows, n, kb;          // dense: rows of A; outputs; blocks of 128 inputs
    int tiles_m, tiles_n;     // dense: row tiles; column tiles (per expert)
    int nblocks;              // 128-output blocks of B (per expert)
    int split;                // blocks per cluster
    const float *sa, *sb, *sb2;
    bool even;                // pairs of scales start on 8-byte boundaries
    void *out;
    int out_dtype;
    int out_align;            // 16 or 8 where rows of out start on such boundaries
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
__device__ __forceinline__ Tile tile_at(const Params &p, int t) {
    const int mt = t / p.tiles_n, nt = t % p.tiles_n;
    if (MODE == kDense) return {0, mt * 128, min(128, p.rows - mt * 128), nt};
    const int4 d = __ldcg(p.tiles + mt);
    return {d.x, d.y, d.z, nt};
}

// Scales of the A rows; h's were written by the kernel before.
template <int MODE, typename F>
__device__ __forceinline__ F ld_scales(const F *p) {
    return MODE == kDown ? __ldcg(p) : __ldg(p);
}

// Two fp32 sums -> two 16-bit outputs.
__device__ __forceinline__ uint32_t pack16(uint64_t v, int dtype) {
    const float2 f = unpack2(v);
    if (dtype != MOEOP_BF16) return pack_f16x2(f.x, f.y);
    const __nv_bfloat162 b = __floats2bfloat162_rn(f.x, f.y);
    return *reinterpret_cast<const uint32_t *>(&b);
}
__device__ __forceinline__ uint4 shfl_xor4(uint4 v, int m) {
    return make_uint4(__shfl_xor_sync(~0u, v.x, m), __shfl_xor_sync(~0u, v.y, m),
                      __shfl_xor_sync(~0u, v.z, m), __shfl_xor_sync(~0u, v.w, m));
}
// Among lanes 4q .. 4q + 3: u[j] of lane 4q + i becomes u[i] of lane 4q + j.
__device__ __forceinline__ void transpose4(uint4 (&u)[4], int lane) {
    const bool hi = lane & 2, odd = lane & 1;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint4 r = shfl_xor4(hi ? u[i] : u[i + 2], 2);
        if (hi) u[i] = r;
        else u[i + 2] = r;
    }
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
        const uint4 r = shfl_xor4(odd ? u[i] : u[i + 1], 1);
        if (odd) u[i] = r;
        else u[i + 1] = r;
    }
}
// Transposed units (16 bytes of outputs of SIZE bytes each) to the outputs
// from `col` on of rows orow of the lanes; `left`: valid rows from this warp's
// first on.  align: 16 or 8 where all rows start on such boundaries and all
// columns exist.  Else, all rows in one way (a warp would go all ways): 4-byte
// words, those of a row that starts on an odd 16-bit output shifted by one,
// the last output of the lane before in front.
template <int SIZE>
__device__ __forceinline__ void store_rows(const uint4 (&u)[4], void *out, int orow, int n, int col,
                                           int lane, int left, int align) {
    const int c = col + (lane & 3) * (16 / SIZE), have = n - c;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int src = (lane & ~3) + j;
        const size_t row = __shfl_sync(~0u, orow, src);
        char *to = static_cast<char *>(out) + (row * n + c) * SIZE;
        const uint32_t w[4] = {u[j].x, u[j].y, u[j].z, u[j].w};
        if (align == 16) {
            if (src < left) *reinterpret_cast<uint4 *>(to) = u[j];
            continue;
        }
        if (align == 8) {
            if (src < left) {
                reinterpret_cast<uint2 *>(to)[0] = make_uint2(w[0], w[1]);
                reinterpret_cast<uint2 *>(to)[1] = make_uint2(w[2], w[3]);
            }
            continue;
        }
        if (SIZE == 4) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (src < left && i < have) reinterpret_cast<uint32_t *>(to)[i] = w[i];
            continue;
        }
        const uint32_t before = __shfl_up_sync(~0u, w[3] >> 16, 1, 4);
        const int odd = reinterpret_cast<uintptr_t>(to) / 2 & 1;
        to -= odd * 2;
        int single = odd && (lane & 3) == 3 && have > 7 ? 8 : -1;  // of the word's halves
        uint32_t value = w[3] >> 16;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t lo = i ? w[i - 1] >> 16 : before;
            const uint32_t word = odd ? lo | w[i] << 16 : w[i];
            // the word's outputs are 2 i - odd and the next
            const bool first = 2 * i - odd < have && have >= 0 && (i || !odd || (lane & 3));
            const bool second = 2 * i - odd + 1 < have;
            if (src < left && first && second) reinterpret_cast<uint32_t *>(to)[i] = word;
            else if (first) single = 2 * i, value = word & 0xFFFFu;
            else if (second && !i && src < left)
                reinterpret_cast<uint16_t *>(to)[1] = (uint16_t)(word >> 16);
        }
        if (src < left && single >= 0)
            reinterpret_cast<uint16_t *>(to)[single] = (uint16_t)value;
    }
}

// SPLIT: the inputs are split over a cluster (its own kernel: the code for it
// costs the others registers that they have no spare of).
template <int MODE, int NB, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
    gemm_kernel(const __grid_constant__ TensorMap ma, const __grid_constant__ TensorMap mb,
                const __grid_constant__ TensorMap mb2, const Params p) {
    constexpr int S = stages<NB>();
    constexpr int kStage = (1 + NB) * kTile;
    constexpr int kBufs = 2;       // halves of tensor memory
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t full[S], empty[S], tm_full[kBufs], tm_empty[kBufs];
    __shared__ float amax_s[kColGroups][128];
    __shared__ uint32_t tm_base;
    __shared__ int abort_s;
    const uint32_t ring = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const int warp = uniform(threadIdx.x / 32), lane = threadIdx.x % 32;
    const int rank = SPLIT ? (int)cluster_rank() : 0;

    if (threadIdx.x == 0) {
        // a stage is free again when its MMAs are complete and, with three
        // loading warps, the other two are past it: none can be lapped
        for (int i = 0; i < S; ++i)
            mbar_init(&full[i], 1), mbar_init(&empty[i], MODE == kGateUp ? 3 : 1);
        for (int i = 0; i < kBufs; ++i)
            mbar_init(&tm_full[i], 1), mbar_init(&tm_empty[i], kAccWarps);
        abort_s = 0;
        fence_mbar_init();
    }
    if (warp == kLoadWarp && elect_one()) {
        tma_prefetch_map(&ma);
        tma_prefetch_map(&mb);
        if (MODE == kGateUp) tma_prefetch_map(&mb2);
    }
    if (warp == kMmaWarp) tmem_alloc(&tm_base, 256 * NB);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = tm_base;

    const int split = SPLIT ? p.split : 1;
    const int first = blockIdx.x / split, step = gridDim.x / split;
    const int kb0 = SPLIT ? rank * p.kb / split : 0;
    const int kb1 = SPLIT ? (rank + 1) * p.kb / split : p.kb;
    pdl_wait();
    const int total = (MODE == kDense ? p.tiles_m : __ldcg(p.num_tiles)) * p.tiles_n;
    int syncs = 0;  // of this thread with its cluster: two in every split block

    if (warp >= kLoadWarp && warp != kMmaWarp) {
        // ---- loads: warp 16 the weights and contiguous rows of A, the
        // gathered rows split over warps 16, 18 and 19
        const int part = warp == kLoadWarp ? 0 : warp - kMmaWarp;
        int it = 0;
        bool ok = true;
        for (int t = first; t < total && ok && (MODE == kGateUp || part == 0); t += step) {
            const Tile T = tile_at<MODE>(p, t);
            const int e = uniform(T.e), pos = uniform(T.pos), rows = uniform(T.rows);
            const int quads = (rows + 3) / 4, boxes = (rows + kBoxRows - 1) / kBoxRows;
            // Gathered: the tokens of rows 4 lane .. + 3, past the end the last
            // one again.  This warp's quads of them are held for all its
            // copies (a shuffle for each would wait behind the operands: 4096
            // rows in 310 us against 286), but for split tiles, which have
            // few rows and no registers to spare.
            constexpr bool kHold = MODE == kGateUp && !SPLIT;
            constexpr int kQuads = kHold ? (32 + 2) / 3 : 1;
            int mine[4], quad[kQuads][4];
            if (MODE == kGateUp) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    mine[j] = __ldcg(p.token + pos + min(4 * lane + j, rows - 1));
            }
            if (kHold) {
#pragma unroll
                for (int i = 0; i < kQuads; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        quad[i][j] = __shfl_sync(~0u, mine[j], min(part + 3 * i, 31));
            }
            const int b0 = e * p.n + T.nt * (MODE == kGateUp ? 128 : 128 * NB);
            const uint32_t bytes =
                NB * kTile + (MODE == kGateUp ? quads * 512 : boxes * kBoxRows * 128);
            for (int b = kb0; b < kb1; ++b, ++it) {
                const int s = it % S;
                ok = __all_sync(~0u, wait_bar(&empty[s], (it / S & 1) ^ 1, &abort_s));
                if (!ok) break;
                const uint32_t dst = ring + s * kStage;
                if (part == 0 && elect_one()) {
                    mbar_arrive_expect_tx(&full[s], bytes);
                    tma_box(dst + kTile, &mb, b * 128, b0, &full[s]);
                    if (NB == 2)
                        tma_box(dst + 2 * kTile, MODE == kGateUp ? &mb2 : &mb, b * 128,
                                MODE == kGateUp ? b0 : b0 + 128, &full[s]);
                    if (MODE != kGateUp)
                        for (int i = 0; i < boxes; ++i)
                            tma_box(dst + i * kBoxRows * 128, &ma, b * 128, pos + i * kBoxRows,
                                    &full[s]);
                }
                __syncwarp();
                if (kHold) {
                    if (elect_one())
#pragma unroll
                        for (int i = 0; i < kQuads; ++i)
                            if (part + 3 * i < quads)
                                tma_gather4(dst + (part + 3 * i) * 512, &ma, b * 128, quad[i],
                                            &full[s]);
                    __syncwarp();
                } else if (MODE == kGateUp) {
                    for (int i = part; i < quads; i += 3) {
                        int r[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) r[j] = __shfl_sync(~0u, mine[j], i);
                        if (elect_one()) tma_gather4(dst + i * 512, &ma, b * 128, r, &full[s]);
                    }
                }
                if (part && elect_one()) mbar_arrive(&empty[s]);
            }
        }
        if (!ok && part == 0)  // copies in flight end before the block does
            for (int i = it > S ? it - S : 0; i < it; ++i)
                mbar_wait(&full[i % S], i / S & 1);
    } else if (warp == kMmaWarp) {
        // ---- MMAs
        constexpr uint32_t idesc = tc_idesc(128, 128 * NB);
        const uint64_t desc0 = tc_desc(ring);
        int s = 0, buf = 0;
        uint32_t phase = 0, ring_phase = 0;
        bool ok = true;
        for (int t = first; t < total && ok; t += step) {
            for (int b = kb0; b < kb1; ++b) {
                const uint64_t da = desc0 + (uint64_t)(s * (kStage >> 4));
                const uint64_t db = da + (kTile >> 4);
                const uint32_t d = tm + buf * 128 * NB;
                ok = __all_sync(~0u, wait_bar(&tm_empty[buf], phase ^ 1, &abort_s) &&
                                         wait_bar(&full[s], ring_phase, &abort_s));
                if (!ok) break;
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        tc_mma_e4m3(d, da + 2 * k, db + 2 * k, idesc, k > 0);
                    tc_commit(&empty[s]);
                    tc_commit(&tm_full[buf]);
                }
                __syncwarp();
                if (++buf == kBufs) buf = 0, phase ^= 1;
                if (++s == S) s = 0, ring_phase ^= 1;
            }
        }
    } else {
        // ---- accumulation and stores
        const int wg = warp / 4, r = (warp % 4) * 32 + lane;
        const uint32_t tm_lane = tm + ((uint32_t)(warp % 4) * 32 << 16) + wg * kCols;
        constexpr int kAcc = kCols / 2 * NB;  // pairs of this thread's sums
        int arow = 0, brow = 0;               // where its scales are
        Tile T{};
        auto take = [&](int t) {
            T = tile_at<MODE>(p, t);
            const int row = min(r, T.rows - 1);  // past the end the last one again
            arow = MODE == kGateUp ? __ldcg(p.token + T.pos + row) : T.pos + row;
            brow = T.e * p.nblocks + T.nt * (MODE == kGateUp ? 1 : NB);
        };
        // The scales of input blocks b and b + 1: this row's, and those of the
        // tile's output blocks.  They come straight from global memory, two
        // blocks ahead: a read of shared memory, which is busy with the
        // operands, takes some 400 cycles and holds up the tensor-memory
        // loads behind it.
        float a0 = 0.f, a1 = 0.f, b00 = 0.f, b01 = 0.f, b10 = 0.f, b11 = 0.f;
        const bool even = p.even && kb0 % 2 == 0;
        auto fetch = [&](int b) {
            if ((warp % 4) * 32 >= T.rows) return;
            const float *sa = p.sa + (size_t)arow * p.kb + b;
            const float *sb0 = p.sb + (size_t)brow * p.kb + b;
            const float *sb1 = MODE == kGateUp ? p.sb2 + (size_t)brow * p.kb + b
                                               : sb0 + (T.nt * NB + 1 < p.nblocks ? p.kb : 0);
            if (even && b + 1 < kb1) {
                const float2 x = ld_scales<MODE>(reinterpret_cast<const float2 *>(sa));
                const float2 y = __ldg(reinterpret_cast<const float2 *>(sb0));
                a0 = x.x, a1 = x.y, b00 = y.x, b01 = y.y;
                if (NB == 2) {
                    const float2 z = __ldg(reinterpret_cast<const float2 *>(sb1));
                    b10 = z.x, b11 = z.y;
                }
            } else if (b < kb1) {
                const int n = b + 1 < kb1;
                a0 = ld_scales<MODE>(sa), a1 = ld_scales<MODE>(sa + n);
                b00 = __ldg(sb0), b01 = __ldg(sb0 + n);
                if (NB == 2) b10 = __ldg(sb1), b11 = __ldg(sb1 + n);
            }
        };
        int it = 0;
        bool ok = true;  // false: an earlier wait gave up; nothing is stored any more
        if (first < total) {
            take(first);
            fetch(kb0);
        }
        for (int t = first; t < total; t += step) {
            const int rows = T.rows;
            const bool some = (warp % 4) * 32 < rows;
            uint64_t acc[kAcc];
#pragma unroll
            for (int i = 0; i < kAcc; ++i) acc[i] = 0;
            bool hit = bar_done(&tm_full[it % kBufs], it / kBufs & 1);
            // (unrolled, the gate/up form spills 224 bytes of registers: 4096
            // rows of experts 286 -> 430 us with both forms unrolled)
#pragma unroll(MODE == kDense ? 2 : 1)
            for (int b = kb0; b < kb1; ++b, ++it) {
                const int buf = it % kBufs;
                const bool second = (b - kb0) & 1;
                const float s0 = second ? a1 * b01 : a0 * b00;
                const float s1 = second ? a1 * b11 : a0 * b10;
                const uint64_t p0 = pack2(s0, s0), p1 = pack2(s1, s1);
                if (second) fetch(b + 1);
                if (!__all_sync(~0u, hit) && ok)
                    ok = __all_sync(~0u, wait_bar(&tm_full[buf], it / kBufs & 1, &abort_s));
                tc_fence_after();
                // 8 columns at a time: registers are what these warps are short
                // of, and four of them to a scheduler hide each other's loads.
                // With the last columns in registers the half is given back,
                // and the next block's barrier is looked up while they are added.
                constexpr int kPart = kCols / 8, kChunks = kPart * NB;
                const uint32_t from = tm_lane + buf * 128 * NB;
                uint32_t v[8];
#pragma unroll
                for (int c = 0; c < kChunks; ++c) {
                    if (some && ok) tmem_load8(from + c / kPart * 128 + c % kPart * 8, v);
                    if (c + 1 == kChunks) {
                        tc_fence_before();
                        if (lane == 0) mbar_arrive(&tm_empty[buf]);
                        __syncwarp();
                        hit = b + 1 < kb1 &&
                              bar_done(&tm_full[(it + 1) % kBufs], (it + 1) / kBufs & 1);
                    }
                    if (some && ok)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            fma2(acc[c * 4 + i], v[2 * i], v[2 * i + 1], c < kPart ? p0 : p1);
                }
            }
            // the next tile's first scales come while this one is stored
            const Tile done = T;
            if (t + step < total) {
                take(t + step);
                fetch(kb0);
            }
            const bool live = r < rows;
            bool storing = some && ok;  // this warp stores its rows
            if (SPLIT) {
                // One tile per cluster.  After the first meeting every load
                // and MMA of the cluster is complete (each warp has seen its
                // last tm_full) and the rings are free; buffer q of a ring
                // holds the sums of the q-th other rank, column by column, so
                // that a warp's store to another block is 128 bytes in a row.
                const int block = warp % 4, owner = block % p.split;
                constexpr uint32_t kBuf = 128 * NB * 32 * 4;
                const uint32_t slot = (block / p.split * (p.split - 1)) * kBuf +
                                      (wg * kCols * 32 + lane) * 4;
                cluster_sync();
                if (rank != owner && some && ok) {
                    const uint32_t to =
                        map_rank(ring, owner) + slot + (rank - (rank > owner)) * kBuf;
#pragma unroll
                    for (int i = 0; i < kAcc; ++i) {
                        const float2 f = unpack2(acc[i]);
                        const uint32_t at =
                            to + ((i / (kCols / 2)) * 128 + (i % (kCols / 2)) * 2) * 128;
                        st_cluster(at, f.x);
                        st_cluster(at + 128, f.y);
                    }
                }
                cluster_sync();
                syncs = 2;
                storing = storing && rank == owner;
                if (storing) {
                    const float *part = reinterpret_cast<const float *>(
                        smem_raw + (ring - smem_u32(smem_raw)) + slot);
                    for (int q = 0; q < p.split - 1; ++q, part += kBuf / 4)
#pragma unroll
                        for (int i = 0; i < kAcc; ++i) {
                            const int at =
                                ((i / (kCols / 2)) * 128 + (i % (kCols / 2)) * 2) * 32;
                            const float2 f = unpack2(acc[i]);
                            acc[i] = pack2(f.x + part[at], f.y + part[at + 32]);
                        }
                }
            }
            if (MODE == kGateUp) {
                float amax = 0.f;
                if (some) {
#pragma unroll
                    for (int i = 0; i < kCols / 2; ++i) {
                        const float2 g = unpack2(acc[i]);
                        const float2 u = unpack2(acc[i + kCols / 2 * (NB - 1)]);
                        const float h0 = __fdividef(g.x, 1.f + __expf(-g.x)) * u.x;
                        const float h1 = __fdividef(g.y, 1.f + __expf(-g.y)) * u.y;
                        acc[i] = pack2(h0, h1);
                        amax = fmaxf(amax, fmaxf(fabsf(h0), fabsf(h1)));
                    }
                }
                amax_s[wg][r] = amax;
                named_bar(1, kAccWarps * 32);
#pragma unroll
                for (int i = 0; i < kColGroups; ++i) amax = fmaxf(amax, amax_s[i][r]);
                named_bar(1, kAccWarps * 32);  // before the next tile writes amax_s
                if (storing && live) {
                    const Fp8Scale scale(amax);
                    const size_t at = (size_t)(done.pos + r) * p.n + done.nt * 128 + wg * kCols;
#pragma unroll
                    for (int i = 0; i < kCols / 16; ++i) {
                        uint32_t q[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float2 x = unpack2(acc[i * 8 + j * 2]);
                            const float2 y = unpack2(acc[i * 8 + j * 2 + 1]);
                            q[j] = scale.codes(x.x, x.y, y.x, y.y);
                        }
                        *reinterpret_cast<uint4 *>(p.h + at + i * 16) =
                            make_uint4(q[0], q[1], q[2], q[3]);
                    }
                    if (wg == 0)
                        p.h_scales[(size_t)(done.pos + r) * (p.n / 128) + done.nt] = scale.scale;
                }
            } else if (storing) {
                // A lane has 32 consecutive outputs of one row; four lanes
                // exchange them so that a store covers 64 bytes of each of 8
                // rows (rows apart cost a store one cycle each).
                const int row = min(r, rows - 1);
                const int orow = MODE == kDown ? __ldcg(p.pair + done.pos + row) : done.pos + row;
#pragma unroll
                for (int c = 0; c < NB; ++c) {
                    const int col = (done.nt * NB + c) * 128 + wg * kCols;
                    if (col >= p.n) continue;
                    const int align = MODE == kDown ? 16 : col + kCols <= p.n ? p.out_align : 0;
                    const int left = rows - (warp % 4) * 32;
                    uint4 u[4];
                    if (MODE == kDense && p.out_dtype != MOEOP_FP32) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const uint64_t *v = acc + c * 16 + i * 4;
                            u[i] = make_uint4(pack16(v[0], p.out_dtype), pack16(v[1], p.out_dtype),
                                              pack16(v[2], p.out_dtype), pack16(v[3], p.out_dtype));
                        }
                        transpose4(u, lane);
                        store_rows<2>(u, p.out, orow, p.n, col, lane, left, align);
                        continue;
                    }
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float2 x = unpack2(acc[c * 16 + h * 8 + i * 2]);
                            const float2 y = unpack2(acc[c * 16 + h * 8 + i * 2 + 1]);
                            u[i] = make_uint4(__float_as_uint(x.x), __float_as_uint(x.y),
                                              __float_as_uint(y.x), __float_as_uint(y.y));
                        }
                        transpose4(u, lane);
                        store_rows<4>(u, p.out, orow, p.n, col + h * 16, lane, left, align);
                    }
                }
            }
        }
    }
    // The accumulating warps have met their cluster twice; the other warps,
    // and all of a block without a tile, do so here.
    if (SPLIT)
        for (; syncs < 2; ++syncs) cluster_sync();
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) tmem_free(tm, 256 * NB);
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

template <int RANKS>
__global__ void __launch_bounds__(1024) index_kernel(IndexParams p) {
    __shared__ int hist[MOEOP_MAX_EXPERTS], cursor[MOEOP_MAX_EXPERTS];
    __shared__ int warp_rows[32], warp_tiles[32];
    pdl_trigger();
    const int rank = RANKS > 1 ? (int)cluster_rank() : 0, ranks = RANKS;
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    hist[tid] = 0;
    __syncthreads();
    for (int64_t i = rank * 1024 + tid; i < p.pairs; i += ranks * 1024) {
        const int e = __ldg(p.ids + i);
        if ((unsigned)e < (unsigned)p.experts) atomicAdd(&hist[e], 1);
    }
    if (RANKS > 1) cluster_sync();
    else __syncthreads();
    int counts[RANKS], rows = 0, lower = 0;
#pragma unroll
    for (int q = 0; q < RANKS; ++q)
        counts[q] = RANKS > 1 ? ld_cluster_i(map_rank(smem_u32(&hist[tid]), q)) : hist[tid];
#pragma unroll
    for (int q = 0; q < RANKS; ++q) {
        if (q < rank) lower += counts[q];
        rows += counts[q];
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
    if (RANKS > 1) cluster_sync();  // the others have read this block's counts
}

// ---------------------------------------------------------------------------
// out[t] = sum_j wts[t][j] y[t * k + j] (+ addend[t]), in slot order
// ---------------------------------------------------------------------------
// Bound by memory: k rows of fp32 in, one of bf16 out.  A thread owns 8 outputs
// and has the loads of kSlots slots under way at a time.
struct CombineParams {
    const int32_t *ids;
    const float *wts;
    const float *y;
    const uint16_t *addend;
    uint16_t *out;
    int rows, hidden, top_k, experts;
};

__global__ void __launch_bounds__(256) combine_kernel(CombineParams p) {
    constexpr int kSlots = 4;
    pdl_wait();
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
        for (int j0 = 0; j0 < p.top_k; j0 += kSlots) {
            // a slot without an expert has no row y: what lies there is read
            // and not used
            uint4 v[kSlots][2];
            float w[kSlots];
            bool in[kSlots];
#pragma unroll
            for (int j = 0; j < kSlots; ++j) {
                const int64_t pair = t * p.top_k + min(j0 + j, p.top_k - 1);
                in[j] = j0 + j < p.top_k &&
                        (unsigned)__ldg(p.ids + pair) < (unsigned)p.experts;
                w[j] = __ldg(p.wts + pair);
                const float *y = p.y + pair * p.hidden + col;
                v[j][0] = ld_cg_v4(y);
                v[j][1] = ld_cg_v4(y + 4);
            }
#pragma unroll
            for (int j = 0; j < kSlots; ++j) {
                if (!in[j]) continue;
                const uint4 a = v[j][0], b = v[j][1];
                const uint32_t u[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
                for (int c = 0; c < 8; ++c) acc[c] = fmaf(w[j], __uint_as_float(u[c]), acc[c]);
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
    int clusters[kMaxSplit + 1] = {};  // clusters of a size that run at a time
    uint32_t *status = nullptr;
} g_devs[64];

// A launch of `grid` blocks in clusters of `size`; `early`: it may start while
// the kernel before it still runs (and waits for it before its first read).
struct Launch {
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute at[2];
    Launch(int64_t grid, int size, int threads, size_t smem, bool early, cudaStream_t st) {
        cfg.gridDim = dim3((unsigned)grid);
        cfg.blockDim = dim3(threads);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = st;
        cfg.attrs = at;
        if (size > 1) {
            at[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
            at[cfg.numAttrs].val.clusterDim.x = size;
            at[cfg.numAttrs].val.clusterDim.y = at[cfg.numAttrs].val.clusterDim.z = 1;
            ++cfg.numAttrs;
        }
        if (early) {
            at[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
            at[cfg.numAttrs].val.programmaticStreamSerializationAllowed = 1;
            ++cfg.numAttrs;
        }
    }
};

template <int MODE, int NB, bool SPLIT>
cudaError_t allow_smem() {
    return cudaFuncSetAttribute(gemm_kernel<MODE, NB, SPLIT>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize, (int)(kRing + 1024));
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
            (e = allow_smem<kDense, 1, false>()) != cudaSuccess ||
            (e = allow_smem<kDense, 1, true>()) != cudaSuccess ||
            (e = allow_smem<kDense, 2, false>()) != cudaSuccess ||
            (e = allow_smem<kGateUp, 2, false>()) != cudaSuccess ||
            (e = allow_smem<kGateUp, 2, true>()) != cudaSuccess ||
            (e = allow_smem<kDown, 1, false>()) != cudaSuccess ||
            (e = allow_smem<kDown, 1, true>()) != cudaSuccess ||
            (e = allow_smem<kDown, 2, false>()) != cudaSuccess ||
            (e = allow_few_smem()) != cudaSuccess ||
            (e = cudaGetSymbolAddress(&sym, g_status)) != cudaSuccess)
            return e;
        for (int s = 2; s <= kMaxSplit; ++s) {
            Launch l(s * v.sms, s, kThreads, kRing + 1024, false, nullptr);
            if ((e = cudaOccupancyMaxActiveClusters(&v.clusters[s],
                                                    gemm_kernel<kGateUp, 2, true>, &l.cfg)) != cudaSuccess)
                return e;
        }
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
cudaError_t launch(const TensorMap &ma, const TensorMap &mb, const TensorMap &mb2, Params p,
                   int64_t grid, bool early, cudaStream_t st) {
    p.even = p.kb % 2 == 0 && (reinterpret_cast<uintptr_t>(p.sa) | reinterpret_cast<uintptr_t>(p.sb) |
                               reinterpret_cast<uintptr_t>(p.sb2)) % 8 == 0;
    Launch l(grid, p.split, kThreads, kRing + 1024, early, st);
    // two blocks of outputs to a tile only come without a split, but for the
    // gate and up products
    if (p.split > 1)
        return cudaLaunchKernelEx(&l.cfg, gemm_kernel<MODE, MODE == kGateUp ? NB : 1, true>, ma, mb,
                                  mb2, p);
    return cudaLaunchKernelEx(&l.cfg, gemm_kernel<MODE, NB, false>, ma, mb, mb2, p);
}

// Blocks per cluster that share one tile's inputs: as many as still let all
// tiles run at a time, each with four blocks of inputs or more (250 x 2048 x
// 512 takes 7.0 us whole and 8.4 split in two).  The GPCs do
// not divide evenly (46 clusters of 3 fit 152 SMs, 28 of 5, 23 of 6): the
// counts are the driver's.
int split_of(const Dev &d, int64_t tiles, int kb) {
    int s = kMaxSplit < kb / 4 ? kMaxSplit : kb / 4;
    while (s > 1 && d.clusters[s] < tiles) --s;
    return s < 1 ? 1 : s;
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
    if (a.rows <= kFewRows) return launch_few_dense(a, sa, b, sb, out, out_dtype, d->sms, st);
    Params p{};
    p.rows = (int)a.rows;
    p.n = (int)b.rows;
    p.kb = (int)((a.k + 127) / 128);
    p.nblocks = (p.n + 127) / 128;
    p.sa = sa;
    p.sb = p.sb2 = sb;
    p.out = out;
    p.out_dtype = out_dtype;
    const uintptr_t starts = reinterpret_cast<uintptr_t>(out) |
                             (uintptr_t)p.n * (out_dtype == MOEOP_FP32 ? 4 : 2);
    p.out_align = starts % 16 == 0 ? 16 : starts % 8 == 0 ? 8 : 0;
    p.tiles_m = (p.rows + 127) / 128;
    // Tiles of 128 x 256 read less per product, tiles of 128 x 128 fill the SMs
    // better.  By the cycles that a tile takes, measured: 900 per 128 inputs
    // and 4500 besides, or 620 and 3500, and 5000 to join a split.  At 8192 x
    // 4096 x 4096 they take 121 and 170 us, at 2000 x 5000 x 1024 21 and 25
    // (3 waves, 5 waves), at 700 x 1500 x 3600 23 and 14 (36 tiles, 72 split
    // in two).
    const int64_t t1 = (int64_t)p.tiles_m * p.nblocks;
    const int64_t t2 = (int64_t)p.tiles_m * ((p.nblocks + 1) / 2);
    const int split = split_of(*d, t1, p.kb);
    const int64_t c1 = split > 1 ? (p.kb + split - 1) / split * 620 + 8500
                                 : (t1 + d->sms - 1) / d->sms * ((int64_t)p.kb * 620 + 3500);
    const int64_t c2 = (t2 + d->sms - 1) / d->sms * ((int64_t)p.kb * 900 + 4500);
    const bool wide = c2 < c1;
    p.tiles_n = wide ? (p.nblocks + 1) / 2 : p.nblocks;
    const int64_t tiles = wide ? t2 : t1;
    p.split = wide ? 1 : split;
    TensorMap ma, mb;
    if ((e = make_map(&ma, a, kBoxRows)) != cudaSuccess || (e = make_map(&mb, b, 128)) != cudaSuccess)
        return e;
    const int64_t grid = p.split > 1 ? tiles * p.split : tiles < d->sms ? tiles : d->sms;
    return wide ? launch<kDense, 2>(ma, mb, mb, p, grid, false, st)
                : launch<kDense, 1>(ma, mb, mb, p, grid, false, st);
}

cudaError_t launch_experts_fp8(const ExpertsArgs &a, cudaStream_t st) {
    Dev *d;
    cudaError_t e = device(&d);
    if (e != cudaSuccess) return e;
    const int H = a.c.hidden, I = a.c.inter, E = a.c.num_experts, k = a.c.top_k;
    const int64_t P = (int64_t)a.rows * k;
    if (few_experts(a.rows, a.c))
        return launch_few_experts(a, reinterpret_cast<float *>(a.ws), st);
    const ExpertsWs w = ExpertsWs::make(a.c, a.rows);
    int *num_tiles = reinterpret_cast<int *>(a.ws + w.header);
    int4 *tiles = reinterpret_cast<int4 *>(a.ws + w.tiles);
    int *pair = reinterpret_cast<int *>(a.ws + w.pair);
    int *token = reinterpret_cast<int *>(a.ws + w.token);
    uint8_t *h = reinterpret_cast<uint8_t *>(a.ws + w.h);
    float *h_scales = reinterpret_cast<float *>(a.ws + w.h_scales);
    float *y = reinterpret_cast<float *>(a.ws + w.y);

    TensorMap mq, mg, mu, mh, md;
    if ((e = make_map(&mq, {a.q, a.rows, H, H}, 1)) != cudaSuccess ||
        (e = make_map(&mg, {a.w.gate, (int64_t)E * I, H, H}, 128)) != cudaSuccess ||
        (e = make_map(&mu, {a.w.up, (int64_t)E * I, H, H}, 128)) != cudaSuccess ||
        (e = make_map(&mh, {h, P, I, I}, kBoxRows)) != cudaSuccess ||
        (e = make_map(&md, {a.w.down, (int64_t)E * H, I, I}, 128)) != cudaSuccess)
        return e;

    // one block up to 4096 pairs, else a cluster of 8
    const IndexParams ip{a.ids, (int)P, k, E, num_tiles, pair, token, tiles};
    const int ranks = P <= 4096 ? 1 : 8;
    Launch li(ranks, ranks, 1024, 0, false, st);
    e = ranks == 1 ? cudaLaunchKernelEx(&li.cfg, index_kernel<1>, ip)
                   : cudaLaunchKernelEx(&li.cfg, index_kernel<8>, ip);
    if (e != cudaSuccess) return e;

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
    p.split = split_of(*d, most, p.kb);
    int64_t grid = p.split > 1 ? most * p.split : most < d->sms ? most : d->sms;
    if ((e = launch<kGateUp, 2>(mq, mg, mu, p, grid, true, st)) != cudaSuccess) return e;

    p.sa = h_scales;
    p.sb = p.sb2 = a.w.down_scales;
    p.n = H;
    p.kb = I / 128;
    p.nblocks = H / 128;
    p.out = y;
    const bool wide = (int64_t)w.max_tiles * ((p.nblocks + 1) / 2) >= d->sms;
    p.tiles_n = wide ? (p.nblocks + 1) / 2 : p.nblocks;
    most = (int64_t)w.max_tiles * p.tiles_n;
    p.split = wide ? 1 : split_of(*d, most, p.kb);
    grid = p.split > 1 ? most * p.split : most < d->sms ? most : d->sms;
    e = wide ? launch<kDown, 2>(mh, md, md, p, grid, true, st)
             : launch<kDown, 1>(mh, md, md, p, grid, true, st);
    if (e != cudaSuccess) return e;

    const CombineParams cp{a.ids, a.wts, y, a.addend, a.out, a.rows, H, k, E};
    const int64_t blocks = ((int64_t)a.rows * (H / 8) + 255) / 256;
    Launch l(blocks < 65536 ? blocks : 65536, 1, 256, 0, true, st);
    return cudaLaunchKernelEx(&l.cfg, combine_kernel, cp);
}

}  // namespace op
}  // namespace moe

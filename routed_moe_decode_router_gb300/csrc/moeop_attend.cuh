// moeop_attend.cuh -- attention of new tokens over a paged cache
// (moeop_attend_paged): the kernel, instantiated per cache type.
//
//   s_j = scale q.k_j over the tokens j that a row sees;  m = max s_j;
//   out = sum_j exp(s_j - m) v_j / sum_j exp(s_j - m),
// one pass over the cache with the running maximum.
//
// Bound by memory: a token's key and value are read once for all query rows of
// their head (rows x group of them), 4 dim operations a row.  What keeps the
// memory busy is bytes under way, so every warp has a ring of its own, filled by
// 16-byte cp.async two or more tiles ahead, and no warp waits for another.
//
// - Work.  A sequence's tokens for one key/value head are an item, cut into
//   tiles of 16 tokens (a tile never leaves its page).  The tiles of all items
//   in a row are dealt to the warps of the grid in equal contiguous shares, so
//   lengths may differ as they like, one long sequence fills the GPU as well as
//   many short ones, and the ring runs on from one item into the next.
// - Product.  The 16 tokens are the rows of mma.sync (m16n8k16), the query rows
//   its 8 columns: S = K Q^T, then O^T = V^T P^T with the d's as rows.  So a group
//   of up to 8 rows pays for 8, not 16.  Which inputs of a sum stand in which
//   place of a fragment is free as long as both operands agree: a lane's place
//   for the d's of K and the d's of V is what 16 contiguous bytes of a row hold,
//   so fragments are cut from what the lane itself copied, without ldmatrix and
//   without a bank conflict, and e4m3 pairs become f16 pairs by one conversion.
//   (tcgen05 would want 64 rows or more: here there are 8 or 16, and the tensor
//   cores are idle most of the time as it is.)
// - P is turned by movmatrix.  It enters as two 16-bit numbers, hi + lo.
// - e4m3: the scale of a key multiplies its score, that of a value its weight.
//   A weight is exp(s_j - m) vs_j, so the sums O have a running maximum of their
//   own, of s_j + log vs_j, and keep the range of f16 whatever the scales are.
// - Maxima are raised only where a score exceeds them by 2^8, so that most tiles
//   need one vote and no reduction.
// - Join.  A warp's share of an item goes to shared memory (its last item) or to
//   the workspace (an item begun by another warp), then the block adds its warps
//   up, then the last block to finish an item adds the blocks' sums, in order.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "moe_device.cuh"
#include "moeop.cuh"

namespace moe {
namespace op {
namespace attend {

constexpr int kTile = 16;        // tokens
constexpr int kMaxSmem = 227 << 10;
constexpr float kSlack = 8.f;    // what a score may exceed the running maximum by (log2)

// TYPE of the cache, D: dim, NT: groups of 8 query rows.
// A tile is 32 rows of D elements; warps x stages of them fill shared memory.
// Warps as the registers allow (Q: NT D / 8, O: NT D / 4 a thread).
template <int TYPE, int D, int NT>
struct Shape {
    static constexpr bool F8 = TYPE == MOEOP_E4M3;
    static constexpr int kSize = F8 ? 1 : 2;
    static constexpr int kRow = D * kSize;                // bytes of a row
    static constexpr int E = 16 / kSize;                  // elements of 16 bytes
    static constexpr int kStage = 2 * kTile * kRow + (F8 ? 128 : 0);
    static constexpr int kWarps = kRow == 512 ? 4 : kRow == 256 ? 8 : NT * D > 128 ? 12 : 16;
    static constexpr int kStages = kRow == 64 ? 5 : NT * D > 128 && kRow == 128 ? 4 : 3;
    static constexpr int M = 8 * NT;
    // a partial sum: m, l and the sums' own maximum of each row, then O
    static constexpr int kStats = 3 * M, kPart = kStats + M * D;
    static constexpr int kRing = kWarps * kStages * kStage;
    static constexpr int KC = kRow / 64;                  // 16-byte pieces of a key per lane
    static constexpr int VB = kRow / 8;                   // bytes of a value per lane
    static_assert(kPart * 4 <= kStages * kStage, "a partial sum lies in its warp's ring");
    static_assert(kStage % 16 == 0, "");
};

__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool in) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                 "r"(in ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void copy8(uint32_t dst, const void *src, bool in) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src),
                 "r"(in ? 8 : 0)
                 : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void *src, bool in) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src),
                 "r"(in ? 4 : 0)
                 : "memory");
}
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float lg2(float x) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t transposed(uint32_t v) {
    uint32_t d;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(v));
    return d;
}
template <int TYPE>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if (TYPE == MOEOP_BF16)
        mma_bf16_16816(d, a[0], a[1], a[2], a[3], b0, b1);
    else
        mma_f16_16816(d, a[0], a[1], a[2], a[3], b0, b1);
}
// Two numbers as 16-bit pairs hi and lo: hi + lo is within 2^-16 (bf16) or 2^-22
// (f16) of them.
template <int TYPE>
__device__ __forceinline__ void split(float x, float y, uint32_t &hi, uint32_t &lo) {
    if (TYPE == MOEOP_BF16) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
        const __nv_bfloat162 l =
            __floats2bfloat162_rn(x - __low2float(h), y - __high2float(h));
        hi = *reinterpret_cast<const uint32_t *>(&h);
        lo = *reinterpret_cast<const uint32_t *>(&l);
    } else {
        const __half2 h = __floats2half2_rn(x, y);
        const __half2 l = __floats2half2_rn(x - __low2float(h), y - __high2float(h));
        hi = *reinterpret_cast<const uint32_t *>(&h);
        lo = *reinterpret_cast<const uint32_t *>(&l);
    }
}
// Some element of a word of the cache is an infinity or NaN.
template <int TYPE>
__device__ __forceinline__ uint32_t not_finite(uint32_t w) {
    if (TYPE == MOEOP_E4M3) return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
    if (TYPE == MOEOP_BF16) return ((w & 0x7F807F80u) + 0x00800080u) & 0x80008000u;
    return ((w & 0x7C007C00u) + 0x04000400u) & 0x80008000u;
}
// exp2(a - b), 0 where a is -inf.
__device__ __forceinline__ float ratio(float a, float b) {
    return a == -INFINITY ? 0.f : ex2(a - b);
}

// The tiles of a batch in a row: sequence by sequence, head by head.
struct Tiles {
    const int *first;    // [batch + 1] of a sequence, divided by heads
    const int *length;   // [batch]
    int heads;
    // the item that tile x belongs to
    __device__ __forceinline__ int sequence(int64_t x, int batch) const {
        int lo = 0, hi = batch;
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if ((int64_t)first[mid] * heads <= x) lo = mid;
            else hi = mid;
        }
        return lo;
    }
    __device__ __forceinline__ int count(int b) const { return first[b + 1] - first[b]; }
};
struct Item {
    int b, h, tiles;      // sequence, head, tiles of the item
    int64_t start;        // its first tile among all
    __device__ __forceinline__ Item(const Tiles &t, int64_t x, int batch) {
        b = t.sequence(x, batch);
        tiles = t.count(b);
        const int64_t base = (int64_t)t.first[b] * t.heads;
        h = (int)(x - base) / tiles;
        start = base + (int64_t)h * tiles;
    }
    __device__ __forceinline__ void next(const Tiles &t) {
        start += tiles;
        if (++h == t.heads) h = 0, ++b, tiles = t.count(b);
    }
};
// Equal shares of `tiles` tiles for `workers` warps.
struct Shares {
    int64_t tiles;
    int workers;
    __device__ __forceinline__ int64_t begin(int w) const {
        return w >= workers ? tiles : tiles * w / workers;
    }
    __device__ __forceinline__ int owner(int64_t x) const {
        return (int)(((x + 1) * workers - 1) / tiles);
    }
};

// First tile of a sequence of n tokens that some row sees (0 without a window).
__device__ __forceinline__ int first_tile(const AttendParams &p, int n) {
    return p.window ? max(0, n - p.rows - p.window + 1) / kTile : 0;
}

template <int TYPE, int D, int NT>
__global__ void __launch_bounds__(Shape<TYPE, D, NT>::kWarps * 32, 1)
    attend_kernel(const AttendParams p) {
    using S = Shape<TYPE, D, NT>;
    constexpr bool F8 = S::F8;
    constexpr int W = S::kWarps, E = S::E, KC = S::KC, VB = S::VB, M = S::M;
    constexpr int kSteps = D / 16;              // of 16 inputs in Q K^T
    extern __shared__ __align__(128) char smem[];
    __shared__ int scan[32];
    __shared__ int64_t starts[W + 1];
    __shared__ int joins[2];
    int *first = reinterpret_cast<int *>(smem + S::kRing);
    int *length = first + p.batch + 1;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int g = lane / 4, t = lane % 4;
    const int mb = blockIdx.y;                  // block of query rows
    const int m_all = p.rows * p.group;

    // Tiles of the sequences before each one
    int sum = 0;
    for (int b0 = 0; b0 < p.batch; b0 += W * 32) {
        const int b = b0 + threadIdx.x;
        int n = 0, c = 0;
        if (b < p.batch) {
            n = min(max(__ldg(p.lengths + b), 0), p.width * p.page);
            c = max(1, (n + kTile - 1) / kTile - first_tile(p, n));
            length[b] = n;
        }
        int run = c;
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const int left = __shfl_up_sync(~0u, run, o);
            if (lane >= o) run += left;
        }
        if (lane == 31) scan[warp] = run;
        __syncthreads();
        int before = sum;
        for (int w = 0; w < W; ++w) {
            if (w < warp) before += scan[w];
            sum += scan[w];
        }
        if (b < p.batch) first[b] = before + run - c;
        __syncthreads();
    }
    if (threadIdx.x == 0) first[p.batch] = sum;
    Shares shares;
    shares.tiles = (int64_t)sum * p.heads;
    shares.workers = (int)min((int64_t)gridDim.x * W, shares.tiles);
    if ((int64_t)blockIdx.x * W >= shares.workers) return;
    if (threadIdx.x <= W) starts[threadIdx.x] = shares.begin(blockIdx.x * W + threadIdx.x);
    __syncthreads();
    const Tiles all{first, length, p.heads};
    const int64_t begin = starts[warp], end = starts[warp + 1];

    char *ring = smem + warp * (S::kStages * S::kStage);
    const uint32_t ring_addr = smem_u32(ring);
    float *const tail = reinterpret_cast<float *>(ring);
    // sums of items begun by another warp: one for each warp of the grid, then two
    // for each block
    float *const heads_at =
        p.parts + ((int64_t)mb * gridDim.x * (W + 2) + (int64_t)blockIdx.x * W) * S::kPart;
    float *const blocks_at =
        p.parts + ((int64_t)mb * gridDim.x * (W + 2) + (int64_t)gridDim.x * W) * S::kPart;

    if (begin < end) {
        // -------------------------------------------------------------------
        // Loads: the item, tile and page that are next
        // -------------------------------------------------------------------
        Item li(all, begin, p.batch);
        int64_t lx = begin;                        // next tile to load
        int ltile, lpage, lplace;                  // in its sequence; of its page
        const int page_tiles = p.page / kTile;
        int lid = -1;                              // page number
        uint32_t valid = 0;                        // bit 0: the tile loaded last is in the cache
        auto seek = [&]() {
            ltile = first_tile(p, length[li.b]) + (int)(lx - li.start);
            lpage = ltile / page_tiles;
            lplace = ltile - lpage * page_tiles;
        };
        auto look = [&]() {                        // the page number, a tile ahead of its use
            lid = lpage < p.width ? __ldg(p.table + li.b * p.table_stride + lpage) : -1;
        };
        seek();
        look();
        int stage_in = 0;
        auto load = [&]() {
            if (lx < end) {
                const bool in = (unsigned)lid < (unsigned)p.pages;
                valid = valid << 1 | (in ? 1u : 0u);
                if (in) {
                    const int n = length[li.b], tok = ltile * kTile;
                    const int from = p.window ? max(0, n - p.rows - p.window + 1) : 0;
                    const uint32_t dst = ring_addr + stage_in * S::kStage;
                    const int64_t place = (int64_t)li.h * p.page + lplace * kTile;
                    const char *k = static_cast<const char *>(p.k) +
                                    (lid * p.k_stride + place * D) * S::kSize;
                    const char *v = static_cast<const char *>(p.v) +
                                    (lid * p.v_stride + place * D) * S::kSize;
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const int at = g + 8 * r;
                        const bool there = tok + at < n && tok + at >= from;
#pragma unroll
                        for (int c = 0; c < KC; ++c)
                            copy16(dst + (r * KC + c) * 512 + lane * 16,
                                   k + at * S::kRow + (c * 4 + t) * 16, there);
                    }
                    const uint32_t vdst = dst + kTile * S::kRow;
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int at = 2 * t + (r & 1) + (r & 2) * 4;
                        const bool there = tok + at < n && tok + at >= from;
                        if constexpr (VB == 8) {
                            copy8(vdst + r * 256 + lane * 8, v + at * S::kRow + g * 8, there);
                        } else {
#pragma unroll
                            for (int c = 0; c < VB / 16; ++c)
                                copy16(vdst + (r * (VB / 16) + c) * 512 + lane * 16,
                                       v + at * S::kRow + (c * 8 + g) * 16, there);
                        }
                    }
                    if constexpr (F8) {
                        const int at = lane % 16;
                        const float *s =
                            lane < 16 ? p.k_scales + lid * p.k_scales_stride + place
                                      : p.v_scales + lid * p.v_scales_stride + place;
                        copy4(dst + 2 * kTile * S::kRow + lane * 4, s + at,
                              tok + at < n && tok + at >= from);
                    }
                }
                ++lx;
                if (++stage_in == S::kStages) stage_in = 0;
                if (lx < end) {
                    if (lx == li.start + li.tiles) {
                        li.next(all);
                        seek();
                    } else {
                        ++ltile;
                        if (++lplace == page_tiles) lplace = 0, ++lpage;
                    }
                    look();
                }
            } else {
                valid <<= 1;
            }
            copies_end();
        };
#pragma unroll
        for (int i = 0; i < S::kStages - 1; ++i) load();

        // -------------------------------------------------------------------
        // Items
        // -------------------------------------------------------------------
        int stage = 0;
        Item it(all, begin, p.batch);
        for (int64_t x = begin; x < end;) {
            const int n = length[it.b];
            const int s0 = (int)(x - it.start);
            const int s1 = (int)(min(end, it.start + it.tiles) - it.start);
            const int tile0 = first_tile(p, n);

            // Q as the right operand; e4m3: in f16, a bf16 row by the power of two
            // that brings it there (exact within 2^-28 of its largest)
            uint32_t q[NT][kSteps][2];
            float qmul[NT][2];
            int pos[NT][2];                       // of the rows of this lane's columns
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const int m = mb * M + j * 8 + g;
                const uint16_t *row = nullptr;
                if (m < m_all) {
                    const int r = m / p.group;
                    row = static_cast<const uint16_t *>(p.q) + it.b * p.q_batch_stride +
                          r * p.q_row_stride +
                          ((int64_t)it.h * p.group + (m - r * p.group)) * D;
                }
#pragma unroll
                for (int c = 0; c < KC; ++c)
#pragma unroll
                    for (int e = 0; e < E / 8; ++e) {
                        uint4 w = make_uint4(0, 0, 0, 0);
                        if (row)
                            w = __ldg(reinterpret_cast<const uint4 *>(row + (c * 4 + t) * E + e * 8));
                        const int k = c * (E / 4) + e * 2;
                        q[j][k][0] = w.x, q[j][k][1] = w.y;
                        q[j][k + 1][0] = w.z, q[j][k + 1][1] = w.w;
                    }
                float f = p.scale_log2;
                if (F8 && p.dtype == MOEOP_BF16) {
                    float big = 0.f;
#pragma unroll
                    for (int k = 0; k < kSteps; ++k)
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            big = fmaxf(big, fmaxf(fabsf(bf16_lo(q[j][k][i])),
                                                   fabsf(bf16_hi(q[j][k][i]))));
                    big = fmaxf(big, __shfl_xor_sync(~0u, big, 1));
                    big = fmaxf(big, __shfl_xor_sync(~0u, big, 2));
                    const int e = f16_block_exponent(big);
                    const float up = exp2i(e);
#pragma unroll
                    for (int k = 0; k < kSteps; ++k)
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            q[j][k][i] = pack_f16x2(bf16_lo(q[j][k][i]) * up,
                                                    bf16_hi(q[j][k][i]) * up);
                    f *= exp2i(-e);
                }
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    qmul[j][c] = F8 ? __shfl_sync(~0u, f, (2 * t + c) * 4) : f;
                    pos[j][c] = n - p.rows + min(mb * M + j * 8 + 2 * t + c, m_all - 1) / p.group;
                }
            }

            float o[D / 16][NT][4];
            float top[NT][2], sums[NT][2], otop[NT][2], lift[NT][2];
#pragma unroll
            for (int j = 0; j < NT; ++j) {
#pragma unroll
                for (int c = 0; c < 2; ++c)
                    top[j][c] = otop[j][c] = -INFINITY, sums[j][c] = 0.f, lift[j][c] = 1.f;
#pragma unroll
                for (int i = 0; i < D / 16; ++i)
#pragma unroll
                    for (int c = 0; c < 4; ++c) o[i][j][c] = 0.f;
            }

            for (int s = s0; s < s1; ++s) {
                load();
                copies_wait<S::kStages - 1>();
                __syncwarp();
                const char *at = ring + stage * S::kStage;
                if (++stage == S::kStages) stage = 0;
                if (!(valid >> (S::kStages - 1) & 1)) continue;
                const int tok = (tile0 + s) * kTile;

                // scores
                float x2[NT][4] = {}, y2[NT][4] = {};
#pragma unroll
                for (int c = 0; c < KC; ++c) {
                    const uint4 lo = *reinterpret_cast<const uint4 *>(at + c * 512 + lane * 16);
                    const uint4 hi =
                        *reinterpret_cast<const uint4 *>(at + (KC + c) * 512 + lane * 16);
                    const uint32_t a[4] = {lo.x, lo.y, lo.z, lo.w}, b[4] = {hi.x, hi.y, hi.z, hi.w};
#pragma unroll
                    for (int k = 0; k < E / 4; ++k) {
                        uint32_t f[4];
                        if (F8) {
                            f[0] = e4m3x2_to_f16x2(a[k]), f[2] = e4m3x2_to_f16x2(a[k] >> 16);
                            f[1] = e4m3x2_to_f16x2(b[k]), f[3] = e4m3x2_to_f16x2(b[k] >> 16);
                        } else {
                            f[0] = a[(2 * k) % 4], f[2] = a[(2 * k + 1) % 4];
                            f[1] = b[(2 * k) % 4], f[3] = b[(2 * k + 1) % 4];
                        }
                        // two sums in turn: an MMA need not wait for the one before
#pragma unroll
                        for (int j = 0; j < NT; ++j)
                            mma<TYPE>(k % 2 ? y2[j] : x2[j], f, q[j][c * (E / 4) + k][0],
                                      q[j][c * (E / 4) + k][1]);
                    }
                }
                float ks[2] = {1.f, 1.f}, vs[2] = {1.f, 1.f}, lv[2] = {0.f, 0.f};
                if (F8) {
                    const float *sc = reinterpret_cast<const float *>(at + 2 * kTile * S::kRow);
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        ks[r] = sc[g + 8 * r], vs[r] = sc[16 + g + 8 * r];
                        lv[r] = fmaxf(lg2(vs[r]), -120.f);
                    }
                }
                const bool partly = tok + kTile - 1 > n - p.rows ||
                                    (p.window && tok < n - p.window);
                bool up = false;
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        float v = (x2[j][c] + y2[j][c]) * (F8 ? ks[c / 2] * qmul[j][c % 2]
                                                              : qmul[j][c % 2]);
                        if (partly) {
                            const int token = tok + g + c / 2 * 8, last = pos[j][c % 2];
                            if (token > last || (p.window && token <= last - p.window))
                                v = -INFINITY;
                        }
                        x2[j][c] = v;
                        up |= v > top[j][c % 2] + kSlack;
                        if (F8) up |= v + lv[c / 2] > otop[j][c % 2] + kSlack;
                    }
                if (__any_sync(~0u, up)) {
#pragma unroll
                    for (int j = 0; j < NT; ++j)
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            float a = fmaxf(x2[j][c], x2[j][c + 2]);
                            float b = fmaxf(x2[j][c] + lv[0], x2[j][c + 2] + lv[1]);
#pragma unroll
                            for (int d = 4; d < 32; d *= 2) {
                                a = fmaxf(a, __shfl_xor_sync(~0u, a, d));
                                if (F8) b = fmaxf(b, __shfl_xor_sync(~0u, b, d));
                            }
                            a = fmaxf(a, top[j][c]);
                            const float fade = ratio(top[j][c], a);
                            sums[j][c] *= fade;
                            top[j][c] = a;
                            float ofade = fade;
                            if (F8) {
                                b = fmaxf(b, otop[j][c]);
                                ofade = ratio(otop[j][c], b);
                                otop[j][c] = b;
                                lift[j][c] = a == -INFINITY || b == -INFINITY ? 1.f : ex2(a - b);
                            }
#pragma unroll
                            for (int i = 0; i < D / 16; ++i)
                                o[i][j][c] *= ofade, o[i][j][c + 2] *= ofade;
                        }
                }

                // weights
                uint32_t ph[NT][2], pl[NT][2];
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    float w[4];
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const float from = top[j][c % 2] == -INFINITY ? 0.f : top[j][c % 2];
                        const float e = ex2(x2[j][c] - from);
                        sums[j][c % 2] += e;
                        w[c] = e;
                        // a token that is not seen has e = 0 whatever its scale holds
                        if (F8) w[c] = x2[j][c] == -INFINITY ? 0.f : e * vs[c / 2] * lift[j][c % 2];
                    }
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        split<TYPE>(w[2 * r], w[2 * r + 1], ph[j][r], pl[j][r]);
                        ph[j][r] = transposed(ph[j][r]);
                        pl[j][r] = transposed(pl[j][r]);
                    }
                }

                // sums of the values
                const char *vat = at + kTile * S::kRow;
                uint32_t odd = 0;
                auto values = [&](auto use) {
#pragma unroll
                    for (int c = 0; c < (VB + 15) / 16; ++c) {
                        constexpr int kWords = VB < 16 ? 2 : 4;
                        uint32_t v[4][4];
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            if constexpr (VB == 8) {
                                const uint2 w =
                                    *reinterpret_cast<const uint2 *>(vat + r * 256 + lane * 8);
                                v[r][0] = w.x, v[r][1] = w.y;
                            } else {
                                const uint4 w = *reinterpret_cast<const uint4 *>(
                                    vat + (r * (VB / 16) + c) * 512 + lane * 16);
                                v[r][0] = w.x, v[r][1] = w.y, v[r][2] = w.z, v[r][3] = w.w;
                            }
                        }
#pragma unroll
                        for (int k = 0; k < kWords; ++k) {
                            if (F8) {
#pragma unroll
                                for (int h = 0; h < 2; ++h) {
                                    const uint32_t a =
                                        __byte_perm(v[0][k], v[1][k], h ? 0x7362 : 0x5140);
                                    const uint32_t b =
                                        __byte_perm(v[2][k], v[3][k], h ? 0x7362 : 0x5140);
                                    const uint32_t f[4] = {
                                        e4m3x2_to_f16x2(a), e4m3x2_to_f16x2(a >> 16),
                                        e4m3x2_to_f16x2(b), e4m3x2_to_f16x2(b >> 16)};
                                    use((c * kWords + k) * 2 + h, f);
                                }
                            } else {
                                const uint32_t f[4] = {__byte_perm(v[0][k], v[1][k], 0x5410),
                                                       __byte_perm(v[0][k], v[1][k], 0x7632),
                                                       __byte_perm(v[2][k], v[3][k], 0x5410),
                                                       __byte_perm(v[2][k], v[3][k], 0x7632)};
                                use(c * kWords + k, f);
                            }
                        }
                    }
                };
                if (partly && p.rows > 1) {
                    // a value that one row sees and another does not
#pragma unroll
                    for (int r = 0; r < 4 * VB / 4; ++r)
                        odd |= not_finite<TYPE>(*reinterpret_cast<const uint32_t *>(
                            vat + (r * 32 + lane) * 4));
                }
                if (!__any_sync(~0u, odd != 0)) {
                    values([&](int i, const uint32_t (&f)[4]) {
#pragma unroll
                        for (int j = 0; j < NT; ++j) {
                            mma<TYPE>(o[i][j], f, ph[j][0], ph[j][1]);
                            mma<TYPE>(o[i][j], f, pl[j][0], pl[j][1]);
                        }
                    });
                } else {
                    // 0 times an infinity would reach the rows that do not see it:
                    // row by row, with the values that it sees
                    for (int r = 0; r < p.rows; ++r) {
                        const int last = n - p.rows + r;
                        uint32_t keep[2] = {0, 0};
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int token = tok + 2 * t + (i & 1) + (i & 2) * 4;
                            if (token <= last && !(p.window && token <= last - p.window))
                                keep[i / 2] |= i & 1 ? 0xFFFF0000u : 0xFFFFu;
                        }
                        values([&](int i, const uint32_t (&f)[4]) {
                            const uint32_t a[4] = {f[0] & keep[0], f[1] & keep[0], f[2] & keep[1],
                                                   f[3] & keep[1]};
#pragma unroll
                            for (int j = 0; j < NT; ++j) {
                                float d[4] = {0.f, 0.f, 0.f, 0.f};
                                mma<TYPE>(d, a, ph[j][0], ph[j][1]);
                                mma<TYPE>(d, a, pl[j][0], pl[j][1]);
#pragma unroll
                                for (int c = 0; c < 4; ++c)
                                    if (pos[j][c % 2] == last) o[i][j][c] += d[c];
                            }
                        });
                    }
                }
            }

            // the sums of the rows' weights over the lanes
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int c = 0; c < 2; ++c)
#pragma unroll
                    for (int d = 4; d < 32; d *= 2)
                        sums[j][c] += __shfl_xor_sync(~0u, sums[j][c], d);

            // d of a lane's i-th value of a row
            constexpr int kRun = VB < 16 ? 8 : E;
            if (s0 == 0 && s1 == it.tiles) {
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const int m = mb * M + j * 8 + 2 * t + c;
                        if (m >= m_all) continue;
                        const float l = sums[j][c];
                        float f = l == 0.f ? 0.f : 1.f / l;
                        if (F8 && l != 0.f) f /= lift[j][c];
                        const int r = m / p.group;
                        uint16_t *row = static_cast<uint16_t *>(p.out) +
                                        (((int64_t)it.b * p.rows + r) * p.heads + it.h) *
                                            p.group * D +
                                        (int64_t)(m - r * p.group) * D;
#pragma unroll
                        for (int u = 0; u < D / 8; u += 8) {   // runs of 8
                            uint32_t w[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const float a = o[u / 2 + i][j][c] * f,
                                            b = o[u / 2 + i][j][c + 2] * f;
                                w[i] = p.dtype == MOEOP_BF16
                                           ? (uint32_t)f2bf16_rn(a) | (uint32_t)f2bf16_rn(b) << 16
                                           : pack_f16x2(a, b);
                            }
                            *reinterpret_cast<uint4 *>(row + (u / kRun * 8 + g) * kRun + u % kRun) =
                                make_uint4(w[0], w[1], w[2], w[3]);
                        }
                    }
            } else {
                // the last item's sums go to the ring, which is empty then
                const bool last = it.start + s1 == end;
                if (last) {
                    copies_wait<0>();
                    __syncwarp();
                }
                float *part = last ? tail : heads_at + (int64_t)warp * S::kPart;
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const int m = j * 8 + 2 * t + c;
                        if (g == 0) {
                            part[m] = top[j][c];
                            part[M + m] = sums[j][c];
                            part[2 * M + m] = F8 ? otop[j][c] : top[j][c];
                        }
                        float *row = part + S::kStats + m * D;
#pragma unroll
                        for (int u = 0; u < D / 8; u += 4)
                            *reinterpret_cast<float4 *>(row + (u / kRun * 8 + g) * kRun + u % kRun) =
                                make_float4(o[u / 2][j][c], o[u / 2][j][c + 2], o[u / 2 + 1][j][c],
                                            o[u / 2 + 1][j][c + 2]);
                    }
            }
            x = it.start + s1;
            if (x < end) it.next(all);
        }
        copies_wait<0>();
    }
    __syncthreads();

    // -----------------------------------------------------------------------
    // Join: the block's warps, then the blocks
    // -----------------------------------------------------------------------
    // what a sum's rows are worth: to the common maximum, and at the end
    auto store = [&](const Item &x, int m, int d, float4 v, float f) {
        const int row = mb * M + m;
        if (row >= m_all) return;
        const int r = row / p.group;
        uint16_t *to = static_cast<uint16_t *>(p.out) +
                       (((int64_t)x.b * p.rows + r) * p.heads + x.h) * p.group * D +
                       (int64_t)(row - r * p.group) * D + d;
        uint2 w;
        if (p.dtype == MOEOP_BF16) {
            w.x = (uint32_t)f2bf16_rn(v.x * f) | (uint32_t)f2bf16_rn(v.y * f) << 16;
            w.y = (uint32_t)f2bf16_rn(v.z * f) | (uint32_t)f2bf16_rn(v.w * f) << 16;
        } else {
            w.x = pack_f16x2(v.x * f, v.y * f);
            w.y = pack_f16x2(v.z * f, v.w * f);
        }
        *reinterpret_cast<uint2 *>(to) = w;
    };
    auto worth = [](float l, float top, float otop) {  // 2^(otop - top) / l
        if (l == 0.f) return 0.f;
        return F8 && top != -INFINITY && otop != -INFINITY ? ex2(otop - top) / l : 1.f / l;
    };
    const int64_t cs = starts[0], ce = starts[W];
    int crosses = 0;
    Item cross0(all, cs, p.batch), cross1 = cross0;
    int64_t done = cs;                    // items up to here are joined
    for (int w0 = -1; w0 < W; ++w0) {
        // the block's first item where another block began it, then the last one
        // of each warp
        if (w0 >= 0 && starts[w0] >= starts[w0 + 1]) break;
        if (w0 < 0 && cross0.start == cs) continue;
        const Item x(all, w0 < 0 ? cs : starts[w0 + 1] - 1, p.batch);
        const int64_t xe = x.start + x.tiles;
        if (xe <= done || (w0 >= 0 && x.start < done)) continue;
        const bool inside = x.start >= cs && xe <= ce;
        const int64_t from = max(x.start, cs), to = min(xe, ce);
        int a = 0, b = 0;
        while (starts[a + 1] <= from) ++a;
        b = a;
        while (starts[b + 1] < to) ++b;
        done = to;
        if (inside && a == b) continue;   // written by its warp
        float *out = blocks_at + (2 * blockIdx.x + (x.start >= cs ? 1 : 0)) * (int64_t)S::kPart;
        for (int i = threadIdx.x; i < M * D / 4; i += W * 32) {
            const int m = i / (D / 4), d = i % (D / 4) * 4;
            auto part = [&](int w) -> const float * {
                return starts[w + 1] <= xe ? reinterpret_cast<const float *>(
                                                 smem + w * (S::kStages * S::kStage))
                                           : heads_at + (int64_t)w * S::kPart;
            };
            float top = -INFINITY, otop = -INFINITY, l = 0.f;
            for (int w = a; w <= b; ++w) {
                top = fmaxf(top, part(w)[m]);
                otop = fmaxf(otop, part(w)[2 * M + m]);
            }
            const float tref = top == -INFINITY ? 0.f : top, oref = otop == -INFINITY ? 0.f : otop;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int w = a; w <= b; ++w) {
                const float *q = part(w);
                l = fmaf(q[M + m], ex2(q[m] - tref), l);
                const float f = ex2(q[2 * M + m] - oref);
                const float4 u = *reinterpret_cast<const float4 *>(q + S::kStats + m * D + d);
                v.x = fmaf(u.x, f, v.x), v.y = fmaf(u.y, f, v.y);
                v.z = fmaf(u.z, f, v.z), v.w = fmaf(u.w, f, v.w);
            }
            if (inside) {
                store(x, m, d, v, worth(l, top, otop));
            } else {
                if (d == 0) out[m] = top, out[M + m] = l, out[2 * M + m] = otop;
                *reinterpret_cast<float4 *>(out + S::kStats + m * D + d) = v;
            }
        }
        if (!inside) (crosses++ ? cross1 : cross0) = x;
    }
    if (!crosses) return;
    // the last block to reach an item joins it; atomicInc leaves the counter zero
    __syncthreads();
    if ((int)threadIdx.x < crosses) {
        const Item &x = threadIdx.x ? cross1 : cross0;
        const int first_block = shares.owner(x.start) / W,
                  last_block = shares.owner(x.start + x.tiles - 1) / W;
        __threadfence();
        // an item's counter is its first block's: no other item goes on from there
        uint32_t *counter = p.counters + mb * gridDim.x + first_block;
        joins[threadIdx.x] =
            atomicInc(counter, last_block - first_block) == (uint32_t)(last_block - first_block);
        __threadfence();
    }
    __syncthreads();
    float *const stats = reinterpret_cast<float *>(smem);      // the ring is free
    for (int k = 0; k < crosses; ++k) {
        if (!joins[k]) continue;
        const Item &x = k ? cross1 : cross0;
        const int c0 = shares.owner(x.start) / W;
        const int parts = shares.owner(x.start + x.tiles - 1) / W - c0 + 1;
        // a block's share is its second sum where the item begins in it
        auto part = [&](int i) {
            return blocks_at + (2 * (c0 + i) + (i == 0 ? 1 : 0)) * (int64_t)S::kPart;
        };
        // stats: the three numbers of each part's rows, then what the part is worth
        for (int i = threadIdx.x; i < parts * S::kStats; i += W * 32)
            stats[i] = __ldcg(part(i / S::kStats) + i % S::kStats);
        float *const final = stats + parts * S::kStats;
        __syncthreads();
        for (int m = warp; m < M; m += W) {
            float top = -INFINITY, otop = -INFINITY, l = 0.f;
            for (int i = lane; i < parts; i += 32) {
                top = fmaxf(top, stats[i * S::kStats + m]);
                otop = fmaxf(otop, stats[i * S::kStats + 2 * M + m]);
            }
#pragma unroll
            for (int o = 16; o; o >>= 1) {
                top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
                otop = fmaxf(otop, __shfl_xor_sync(~0u, otop, o));
            }
            const float tref = top == -INFINITY ? 0.f : top, oref = otop == -INFINITY ? 0.f : otop;
            for (int i = lane; i < parts; i += 32) {
                float *s = stats + i * S::kStats;
                l = fmaf(s[M + m], ex2(s[m] - tref), l);
                s[m] = ex2(s[2 * M + m] - oref);
            }
#pragma unroll
            for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(~0u, l, o);
            if (lane == 0) final[m] = worth(l, top, otop);
        }
        __syncthreads();
        for (int i = threadIdx.x; i < M * D / 4; i += W * 32) {
            const int m = i / (D / 4), d = i % (D / 4) * 4;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
            for (int w = 0; w < parts; ++w) {
                const float f = stats[w * S::kStats + m];
                const float4 u = __ldcg(
                    reinterpret_cast<const float4 *>(part(w) + S::kStats + m * D + d));
                v.x = fmaf(u.x, f, v.x), v.y = fmaf(u.y, f, v.y);
                v.z = fmaf(u.z, f, v.z), v.w = fmaf(u.w, f, v.w);
            }
            store(x, m, d, v, final[m]);
        }
        __syncthreads();
    }
}

template <int TYPE, int D, int NT>
cudaError_t launch(const AttendParams &p, cudaStream_t st) {
    using S = Shape<TYPE, D, NT>;
    const auto kernel = attend_kernel<TYPE, D, NT>;
    // every call: the attribute is the device's, and costs less than a lookup
    const int smem = S::kRing + (2 * p.batch + 1) * 4;
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem - 1024);
    if (e != cudaSuccess) return e;
    // no more blocks than there can be tiles for their warps
    int64_t tiles = (int64_t)p.width * p.page / kTile;
    if (p.window && (p.window + p.rows) / kTile + 2 < tiles) tiles = (p.window + p.rows) / kTile + 2;
    const int64_t most = (tiles * p.batch * p.heads + S::kWarps - 1) / S::kWarps;
    const int grid = attend_grid(p.blocks);
    kernel<<<dim3((unsigned)(most < grid ? most : grid), p.blocks), S::kWarps * 32, smem, st>>>(p);
    return cudaGetLastError();
}
template <int TYPE>
cudaError_t launch_type(const AttendParams &p, int dim, cudaStream_t st) {
    const bool wide = attend_block(dim, p.rows * p.group) == 16;
    switch (dim) {
        case 64: return wide ? launch<TYPE, 64, 2>(p, st) : launch<TYPE, 64, 1>(p, st);
        case 128: return wide ? launch<TYPE, 128, 2>(p, st) : launch<TYPE, 128, 1>(p, st);
        default: return launch<TYPE, 256, 1>(p, st);
    }
}

}  // namespace attend
}  // namespace op
}  // namespace moe

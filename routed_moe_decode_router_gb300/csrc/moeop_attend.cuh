// moeop_attend.cuh -- attention of new tokens over a paged cache
// (moeop_attend_paged): the kernel, instantiated per cache type.
//
//   s_j = scale q.k_j over the tokens j that a row sees;  m = max s_j;
//   out = sum_j exp(s_j - m) v_j / sum_j exp(s_j - m),
// one pass over the cache with the running maximum.
//
// Bound by memory: a token's key and value are read once for all query rows of
// their head (rows x group of them), 4 dim operations a row.  What keeps the
// memory busy is bytes under way, and what may keep it waiting is instructions
// (a tile of 32 tokens of 128 e4m3 has 350 cycles of its SM at the memory's rate; its
// conversions to f16 alone take 256), so every warp has a ring of its own, filled by
// TMA two or more tiles ahead at a few instructions a tile, and no warp waits for
// another.
//
// - Work.  A sequence's tokens for one key/value head are an item, cut into
//   tiles of 16 or 32 tokens (16 never leave their page).  The tiles of all items
//   in a row are dealt to the warps of the grid in equal contiguous shares, so
//   lengths may differ as they like, one long sequence fills the GPU as well as
//   many short ones, and the ring runs on from one item into the next.
// - Product.  16 tokens are the rows of mma.sync, the query rows its 8 columns:
//   S = K Q^T, then O^T = V^T P^T with the d's as rows.  So a group of up to 8
//   rows pays for 8, not 16.  (tcgen05 would want the tokens as its 128 rows, and P
//   through shared memory; at 8 rows the tensor pipe is busy 22% of the time as it
//   is.)  Fragments come by ldmatrix from the swizzled tiles, V transposed on the way.
// - e4m3 is widened to f16, exactly.  A key's scale multiplies its score, a value's
//   its weight: weights are exp(s_j - m) vs_j, so the sums O have a running maximum
//   of their own, of s_j + log |vs_j|, and keep the range of f16 whatever the scales.
//   It is held as what it exceeds m by, and thresholds are on differences of scores:
//   a sum of a score of 2^24 and a logarithm would be off by more than f16 has room.
//   (mma.sync on e4m3 itself, Q in two e4m3 numbers, takes 80 instructions a tile more.)
// - P is turned by movmatrix.  It enters as two 16-bit numbers, hi + lo (one f16
//   number for e4m3 would be 2^-11 off, and saves no time).  f16 ends at 2^-24, and a
//   long row's weights may all be below that beside its largest, so there they count
//   from 2^15 down, and lo is 2^12 times what hi left, summed apart and added at 2^-12:
//   hi + lo is within 2^-22 of the weight, or 2^-44 of the row's largest.  (The sums
//   apart take 16 x <= 4000, 32 query rows, e4m3 from 41.5 to 44.7 us, 96 x 16384 from
//   258.0 to 258.3, against weights of one scale.)
// - Maxima are raised only where a score exceeds them by 2^8, so that most tiles
//   need one vote and no reduction.
// - Join.  A warp's share of an item goes to shared memory (its last item) or to
//   the workspace (an item begun by another warp), then the block adds its warps
//   up, then the last block to finish an item adds the blocks' sums, in order, or
//   where items are few a kernel of its own does.
//
// One GB300, calls in a stream: 96 sequences of up to 16384 tokens, 64/8 heads of 128,
// e4m3 260 us (6.5 TB/s); one of 131071, 16/2 of 256, fp16 55 us (4.9 TB/s); 9 of up to
// 6007, 4 rows, 64/8 of 128, bf16 37.5 us (two passes of 16 query rows; fp16 39); one of
// 901, e4m3 8.7 us, 6000 cycles of which are waits for lengths, table, tiles, one after
// the other.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <atomic>

#include "moe_device.cuh"
#include "moeop.cuh"
#include "moeop_tc.cuh"

namespace moe {
namespace op {
namespace attend {

constexpr float kSlack = 8.f;    // what a score may exceed the running maximum by (log2)
// f16 weights: at most 2^(kSlack + kRoom), hi off by 2^3 there, and 2^3 kLow = 2^15
constexpr float kRoom = 7.f, kLow = 4096.f;
static_assert(kRoom == 7.f, "2^-kRoom in worth()");

// TYPE of the cache, D: dim, NT: groups of 8 query rows.
// A tile is kTok tokens, 8 KB of keys and values where it can be; warps x stages of
// them fill shared memory.  Eight warps: with more the registers of O (NT D / 4 a
// thread) spill, and what every warp does once costs more.
template <int TYPE, int D, int NT>
struct Shape {
    static constexpr bool F8 = TYPE == MOEOP_E4M3;
    static constexpr int kSize = F8 ? 1 : 2;
    static constexpr int kRow = D * kSize;                // bytes of a row
    static constexpr int kSubs = kRow <= 128 ? 2 : 1;     // a tile's groups of 16 tokens
    static constexpr int kTok = 16 * kSubs;
    static constexpr int kSub = 16 * kRow, kHalf = kSubs * kSub, kStage = 2 * kHalf;
    static constexpr int kWarps = kRow == 512 ? 4 : 8;
    static constexpr int kStages = kRow == 64 ? 6 : 3;
    static constexpr int M = 8 * NT;
    // a partial sum: m, l and what the sums' own maximum is above m (0 without e4m3) of
    // each row, then O^T
    static constexpr int kStats = 3 * M, kPart = kStats + M * D;
    static constexpr int kRing = kWarps * kStages * kStage;
    static constexpr int smem(int batch) { return 1024 + kRing + (2 * batch + 1) * 4; }
    static constexpr int kSteps = kRow / 32;              // 32 bytes of a row: an MMA's
    static_assert(2 * M * D * 4 <= kStages * kStage, "two shares' sums lie in their warp's ring");
    static_assert(kWarps <= 16, "two shares of each warp: a lane for each");
    static_assert(kStage % 1024 == 0 && kSub % 1024 == 0, "the swizzle's period");
};

__device__ __forceinline__ void copy16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }
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
template <bool TRANS>
__device__ __forceinline__ void load_matrices(uint32_t (&r)[4], uint32_t addr) {
    if (TRANS)
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                     : "r"(addr)
                     : "memory");
    else
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                     : "r"(addr)
                     : "memory");
}
template <int TYPE>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if (TYPE == MOEOP_BF16)
        mma_bf16_16816(d, a[0], a[1], a[2], a[3], b0, b1);
    else
        mma_f16_16816(d, a[0], a[1], a[2], a[3], b0, b1);
}
template <int TYPE>
__device__ __forceinline__ uint32_t pair(float x, float y) {
    if (TYPE == MOEOP_BF16) return (uint32_t)f2bf16_rn(x) | (uint32_t)f2bf16_rn(y) << 16;
    return pack_f16x2(x, y);
}
template <int TYPE>
__device__ __forceinline__ float2 unpair(uint32_t v) {
    if (TYPE == MOEOP_BF16) return make_float2(bf16_lo(v), bf16_hi(v));
    return __half22float2(*reinterpret_cast<const __half2 *>(&v));
}
// Some element of a pair is an infinity or NaN.
template <int TYPE>
__device__ __forceinline__ uint32_t not_finite(uint32_t w) {
    if (TYPE == MOEOP_BF16) return ((w & 0x7F807F80u) + 0x00800080u) & 0x80008000u;
    return ((w & 0x7C007C00u) + 0x04000400u) & 0x80008000u;
}
__device__ __forceinline__ float inverse(float x) {    // within 2^-23
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// mbar_wait of all lanes together: none goes on where another gave up.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity) {
    if (__all_sync(~0u, mbar_try_wait(bar, parity))) return true;
    const long long t0 = clock64();
    while (!__all_sync(~0u, mbar_try_wait(bar, parity)))
        if (__any_sync(~0u, clock64() - t0 > kWaitLimitCycles)) return false;
    return true;
}
// exp2(a - b), 0 where a is -inf.
__device__ __forceinline__ float ratio(float a, float b) {
    return a == -INFINITY ? 0.f : ex2(a - b);
}

// What sums are worth in the end: 2^above / l, with e4m3 (whose weights alone have the
// factor 2^kRoom; above is -120 and more).
template <bool F8>
__device__ __forceinline__ float worth(float l, float above) {
    if (l == 0.f) return 0.f;
    return F8 && above != -INFINITY ? ex2(above) * (inverse(l) * 0x1p-7f) : inverse(l);
}

// An item begins with kEmpty tiles of nothing: what a warp does once for an item takes
// as long as two tiles, and the shares are to be equal in time (128 sequences of up to
// 500 tokens, 8 heads of e4m3: without 29.6 us, with 1, 2, 3, 4 of them 22.7, 20.3, 21.2,
// 22.8; 33 sequences, window 1024: 15.4, then 14.9, 13.5, 13.7, 13.7).
constexpr int kEmpty = 2;
// An item among the tiles of a batch: sequence by sequence, head by head.
struct alignas(16) Item {
    int b, h, tiles;      // sequence, head, tiles of the item
    int start;            // its first tile among all
    Item() = default;
    // the item of tile x (the same in all lanes); first: tiles of the sequences before
    // each, for one head.  A warp looks at 32 of them at a time.
    __device__ __forceinline__ Item(const int *first, int heads, int batch, int x) {
        const int lane = threadIdx.x % 32;
        int lo = 0;
        for (int step = batch > 1024 ? 1024 : batch > 32 ? 32 : 1; step; step /= 32) {
            const int at = lo + lane * step;
            lo += (__popc(__ballot_sync(~0u, at < batch && first[at] * heads <= x)) - 1) * step;
        }
        b = lo;
        tiles = first[lo + 1] - first[lo];
        const int base = first[lo] * heads;
        // the quotient is below 1024: one off at most
        h = (int)((float)(x - base) * inverse((float)tiles));
        if (h * tiles > x - base) --h;
        if ((h + 1) * tiles <= x - base) ++h;
        start = base + h * tiles;
    }
    __device__ __forceinline__ void next(const int *first, int heads) {
        start += tiles;
        if (++h == heads) h = 0, ++b, tiles = first[b + 1] - first[b];
    }
    __device__ __forceinline__ int end() const { return start + tiles; }
};
// Where the share of thread block c of n begins: equal shares of `tiles`.
struct Shares {
    int each, more;       // the first `more` blocks take one tile more
    __device__ __forceinline__ Shares(int tiles, const Divisor &n)
        : each((int)n.over(tiles)), more(tiles - each * (int)n.d) {}
    __device__ __forceinline__ int begin(int c) const { return c * each + min(c, more); }
    __device__ __forceinline__ int owner(int x) const {
        const int big = more * (each + 1);
        return x < big ? x / (each + 1) : more + (x - big) / max(each, 1);
    }
};
// An item of up to `whole` tiles is not cut between blocks: the cut goes to its
// nearer end.
__device__ __forceinline__ int cut(const int *first, int heads, int batch, int tiles, int whole,
                                   int x) {
    if (x <= 0 || x >= tiles) return min(x, tiles);
    const Item i(first, heads, batch, x);
    return i.tiles > whole ? x : x - i.start < i.end() - x ? i.start : i.end();
}

// First tile of a sequence of n tokens that some row sees (0 without a window).
template <int TOK>
__device__ __forceinline__ int first_tile(const AttendParams &p, int n) {
    return p.window ? max(0, n - p.rows - p.window + 1) / TOK : 0;
}

template <int TYPE, int D, int NT>
__global__ void __launch_bounds__(Shape<TYPE, D, NT>::kWarps * 32, 1)
    attend_kernel(const __grid_constant__ TensorMap kmap, const __grid_constant__ TensorMap vmap,
                  const AttendParams p) {
    using S = Shape<TYPE, D, NT>;
    constexpr bool F8 = S::F8, kHalf = TYPE != MOEOP_BF16;    // weights in f16
    constexpr int W = S::kWarps, M = S::M, kStages = S::kStages, kSteps = S::kSteps;
    constexpr int kTok = S::kTok, kSubs = S::kSubs;
    extern __shared__ char raw[];
    __shared__ uint64_t bars[W][kStages];
    __shared__ int2 places[W][kStages][kSubs];   // of a tile's tokens: page, row in the page
    __shared__ int scan[W], joined[2];
    // the shares of an item that a warp has and others too, in the order of their
    // tiles: the item it did not begin (2 w) and its last one (2 w + 1)
    __shared__ Item lasts[W], fronts[W];
    __shared__ float stats[2 * W][3][M];
    __shared__ __align__(16) float worth_of[2 * W > 16 ? 2 * W : 16][M];
    __shared__ int shares_of[W];         // which of its two shares a warp has, as bits
    char *const smem = raw + (1024 - smem_u32(raw) % 1024) % 1024;
    int *const first = reinterpret_cast<int *>(smem + S::kRing);
    int *const length = first + p.batch + 1;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int g = lane / 4, t = lane % 4;
    const int mb = blockIdx.y;                  // block of query rows
    const int m_all = p.rows * p.group;

    // Tiles of the sequences before each one.  Up to 32 every warp counts them for
    // itself (and all write the same): no barrier.
    int sum = 0;
    const bool few = p.batch <= 32;
    if (lane == 0) {
#pragma unroll
        for (int i = 0; i < kStages; ++i) mbar_init(&bars[warp][i], 1);
        fence_mbar_init();
        if (warp == W - 1) tma_prefetch_map(&kmap), tma_prefetch_map(&vmap);
    }
    pdl_wait();
    for (int b0 = 0; b0 < p.batch; b0 += W * 32) {
        const int b = b0 + (few ? lane : threadIdx.x);
        int n = 0, c = 0;
        if (b < p.batch) {
            n = min(max(__ldg(p.lengths + b), 0), p.width * p.page);
            c = kEmpty + max(1, (n + kTok - 1) / kTok - first_tile<kTok>(p, n));
            length[b] = n;
        }
        int run = c;
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const int left = __shfl_up_sync(~0u, run, o);
            if (lane >= o) run += left;
        }
        int before = sum;
        if (few) {
            sum = __shfl_sync(~0u, run, 31);
        } else {
            if (lane == 31) scan[warp] = run;
            __syncthreads();
            for (int w = 0; w < W; ++w) {
                if (w < warp) before += scan[w];
                sum += scan[w];
            }
        }
        if (b < p.batch) first[b] = before + run - c;
        if (!few) __syncthreads();
    }
    if (lane == 0) first[p.batch] = sum;
    if (few) __syncwarp();
    else __syncthreads();
    const int tiles = sum * p.heads;
    const Shares shares(tiles, p.flat ? p.by_warps : p.by_grid);
    const int worker = warp * gridDim.x + blockIdx.x;          // of a flat grid
    int begin, end, cs = 0, ce = 0;
    if (p.flat) {
        begin = shares.begin(worker), end = shares.begin(worker + 1);
    } else {
        cs = cut(first, p.heads, p.batch, tiles, p.whole, shares.begin(blockIdx.x));
        ce = cut(first, p.heads, p.batch, tiles, p.whole, shares.begin(blockIdx.x + 1));
        if (cs >= ce) return;
        // equal shares for the block's warps
        const int each = (ce - cs) / W, more = (ce - cs) % W;
        begin = cs + warp * each + min(warp, more);
        end = begin + each + (warp < more ? 1 : 0);
    }
    const int used = min(W, ce - cs);

    char *const ring = smem + warp * (kStages * S::kStage);
    const uint32_t ring_addr = smem_u32(ring);
    // partial sums: of items begun by another warp, one for each warp of the grid; of
    // items begun or ended by another block, two for each block
    float *const mb_at = p.parts + (int64_t)mb * gridDim.x * (W + 2) * S::kPart;
    float *const heads_at = mb_at + (int64_t)blockIdx.x * W * S::kPart;
    float *const blocks_at = mb_at + (int64_t)gridDim.x * W * S::kPart;

    int has = 0;
    if (begin < end) {
        // -------------------------------------------------------------------
        // Q of an item, as it is
        // -------------------------------------------------------------------
        Item it(first, p.heads, p.batch, begin);
        if (lane == 0) fronts[warp] = it;
        uint32_t q[NT][D / 16][2];
        auto load_q = [&]() {
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const int m = mb * M + j * 8 + g;
                const uint16_t *row = nullptr;
                if (m < m_all) {
                    const int r = p.by_group.over(m);
                    row = static_cast<const uint16_t *>(p.q) + it.b * p.q_batch_stride +
                          r * p.q_row_stride + ((int64_t)it.h * p.group + (m - r * p.group)) * D;
                }
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    if constexpr (F8) {
                        // a lane's bytes of a key are four in a row: so its numbers of Q
                        const uint2 w = row ? __ldg(reinterpret_cast<const uint2 *>(
                                                  row + k * 16 + t * 4))
                                            : make_uint2(0, 0);
                        q[j][k][0] = w.x, q[j][k][1] = w.y;
                    } else {
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            q[j][k][i] = row ? __ldg(reinterpret_cast<const uint32_t *>(
                                                   row + k * 16 + i * 8 + t * 2))
                                             : 0u;
                    }
                }
            }
        };
        // -------------------------------------------------------------------
        // Loads: the item, tile and page that are next
        // -------------------------------------------------------------------
        Item li = it;
        int lx = begin;                            // next tile to load
        int lpage, lplace;                         // its page in the sequence, place in the page
        int page0 = 0, ids = -1;                   // lane i: the number of page page0 + i
        // which groups of the tiles under way are in the cache: the last loaded lowest
        uint32_t valid = 0;
        bool lost = false;                         // a wait ran out: no more loads
        auto pages = [&]() {                       // a tile ahead of their use
            page0 = lpage;
            ids = page0 + lane < p.width
                      ? __ldg(p.table + li.b * p.table_stride + page0 + lane)
                      : -1;
        };
        auto seek = [&]() {
            const int tok = (first_tile<kTok>(p, length[li.b]) + max(0, lx - li.start - kEmpty)) *
                            kTok;
            lpage = p.by_page.over(tok);
            lplace = tok - lpage * p.page;
            pages();
        };
        seek();
        load_q();
        int stage_in = 0;
        auto load = [&]() {
            const bool empty = lx - li.start < kEmpty, live = lx < end && !lost && !empty;
            int id[kSubs], row[kSubs];
            uint32_t in = 0;
#pragma unroll
            for (int u = 0; u < kSubs; ++u) {
                const bool next = lplace + 16 * u >= p.page;
                id[u] = __shfl_sync(~0u, ids, lpage - page0 + next);
                row[u] = li.h * p.page + lplace + 16 * u - (next ? p.page : 0);
                if (!live || (unsigned)id[u] >= (unsigned)p.pages) id[u] = -1;
                else in |= 1u << u;
                if (F8 && lane == u) places[warp][stage_in][u] = make_int2(id[u], row[u]);
            }
            valid = valid << kSubs | in;
            if (in) {
                const uint32_t dst = ring_addr + stage_in * S::kStage;
                uint64_t *bar = &bars[warp][stage_in];
                if (elect_one()) {
                    mbar_arrive_expect_tx(bar, __popc(in) * 2 * S::kSub);
                    if (p.wide) {
                        tma_rows(dst, &kmap, row[0], id[0], bar);
                        tma_rows(dst + S::kHalf, &vmap, row[0], id[0], bar);
                    } else {
#pragma unroll
                        for (int u = 0; u < kSubs; ++u)
                            if (id[u] >= 0) {
                                tma_rows(dst + u * S::kSub, &kmap, row[u], id[u], bar);
                                tma_rows(dst + S::kHalf + u * S::kSub, &vmap, row[u], id[u], bar);
                            }
                    }
                }
                __syncwarp();
            }
            if (++stage_in == kStages) stage_in = 0;
            if (++lx < end) {
                if (lx == li.end()) {
                    li.next(first, p.heads);
                    seek();
                } else if (!empty) {
                    lplace += kTok;
                    while (lplace >= p.page) lplace -= p.page, ++lpage;
                    if (lpage - page0 >= 31) pages();
                }
            }
        };
#pragma unroll 1
        for (int i = 0; i < kStages - 1; ++i) load();
        // the scales of the next tile: lane i's of token i
        float ks_next = 1.f, vs_next = 1.f;
        auto scales = [&](int at) {
            if constexpr (F8) {
                __syncwarp();
                const int2 w = places[warp][at][lane / 16 % kSubs];
                const int64_t i = w.y + lane % 16;
                ks_next = __ldg(p.k_scales + (w.x < 0 ? 0 : w.x * p.k_scales_stride + i));
                vs_next = __ldg(p.v_scales + (w.x < 0 ? 0 : w.x * p.v_scales_stride + i));
            }
        };
        scales(0);

        // where a lane's rows of the matrices lie in a tile: K and e4m3 V have the
        // tokens 8..15 in the second matrix, V in 16 bits in the third
        const int row_k = lane % 16, col_k = lane / 16;
        const int row_v = F8 ? row_k : lane % 8 + lane / 16 * 8, col_v = F8 ? col_k : lane / 8 % 2;
        auto offset = [](int row, int col) {
            return S::kRow == 64 ? row * 64 + ((col ^ (row / 2 % 4)) * 16)
                                 : row * 128 + ((col ^ (row % 8)) * 16);
        };
        const uint32_t off_k = offset(row_k, col_k), off_v = S::kHalf + offset(row_v, col_v);

        // -------------------------------------------------------------------
        // Items
        // -------------------------------------------------------------------
        int stage = 0;
        uint32_t phases = 0;
        for (int x = begin; x < end;) {
            const int n = length[it.b];
            const int s0 = x - it.start, s1 = min(end, it.end()) - it.start;
            const int tile0 = first_tile<kTok>(p, n);

            // Q as the right operand: with e4m3 a bf16 row goes to f16 by the power of
            // two that brings it there, exact within 2^-28 of its largest
            float qmul[NT][2];
            int pos[NT][2];                       // of the rows of this lane's columns
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                float f = p.scale_log2;
                if (F8 && p.dtype == MOEOP_BF16) {
                    uint32_t most = 0;            // magnitudes order as whole numbers do
#pragma unroll
                    for (int k = 0; k < D / 16; ++k)
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            most = __vmaxu2(most, q[j][k][i] & 0x7FFF7FFFu);
                    most = __vmaxu2(most, __shfl_xor_sync(~0u, most, 1));
                    most = __vmaxu2(most, __shfl_xor_sync(~0u, most, 2));
                    const float big = __uint_as_float(max(most << 16, most & 0xFFFF0000u));
                    const int e = f16_block_exponent(big);
                    const float by = exp2i(e);
#pragma unroll
                    for (int k = 0; k < D / 16; ++k)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const float2 v = unpair<MOEOP_BF16>(q[j][k][i]);
                            q[j][k][i] = pack_f16x2(v.x * by, v.y * by);
                        }
                    f *= exp2i(-e);
                }
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    qmul[j][c] = F8 ? __shfl_sync(~0u, f, (2 * t + c) * 4) : f;
                    pos[j][c] = p.rows == 1 ? n - 1
                                            : n - p.rows + (int)p.by_group.over(min(
                                                  mb * M + j * 8 + 2 * t + c, m_all - 1));
                }
            }

            float o[D / 16][NT][4];
            // m, l, with e4m3 what the sums' own maximum is above m, 2^(kRoom - that)
            float top[NT][2], sums[NT][2], above[NT][2], lift[NT][2];
#pragma unroll
            for (int j = 0; j < NT; ++j) {
#pragma unroll
                for (int c = 0; c < 2; ++c)
                    top[j][c] = above[j][c] = -INFINITY, sums[j][c] = 0.f, lift[j][c] = 1.f;
#pragma unroll
                for (int i = 0; i < D / 16; ++i)
#pragma unroll
                    for (int c = 0; c < 4; ++c) o[i][j][c] = 0.f;
            }

            for (int s = s0; s < s1; ++s) {
                const float ks_now = ks_next, vs_now = vs_next;
                load();
                const uint32_t at = ring_addr + stage * S::kStage;
                const int now = stage;
                if (++stage == kStages) stage = 0;
                scales(stage);
                const uint32_t there = valid >> (kSubs * (kStages - 1)) & ((1u << kSubs) - 1);
                if (!there) continue;
                if (!warp_wait(&bars[warp][now], phases >> now & 1)) {
                    lost = true;
                    if (lane == 0) atomicExch(p.status, (uint32_t)MOE_DEV_WAIT_TIMEOUT);
                }
                phases ^= 1u << now;
                const int tok = (tile0 + s - kEmpty) * kTok;

                // scores
                float x2[kSubs][NT][4];
#pragma unroll
                for (int u = 0; u < kSubs; ++u) {
                    // two sums in turn: an MMA need not wait for the one before
                    float acc[NT][2][4] = {};
#pragma unroll
                    for (int k = 0; k < kSteps; ++k) {
                        uint32_t r[4];
                        load_matrices<false>(
                            r, (at + off_k + u * S::kSub + k / 4 * 2048) ^ (k % 4 * 32));
                        if constexpr (F8) {
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const uint32_t f[4] = {
                                    e4m3x2_to_f16x2(r[2 * h]), e4m3x2_to_f16x2(r[2 * h + 1]),
                                    e4m3x2_to_f16x2(r[2 * h] >> 16),
                                    e4m3x2_to_f16x2(r[2 * h + 1] >> 16)};
#pragma unroll
                                for (int j = 0; j < NT; ++j)
                                    mma<TYPE>(acc[j][h], f, q[j][2 * k + h][0], q[j][2 * k + h][1]);
                            }
                        } else {
#pragma unroll
                            for (int j = 0; j < NT; ++j)
                                mma<TYPE>(acc[j][k % 2], r, q[j][k][0], q[j][k][1]);
                        }
                    }
#pragma unroll
                    for (int j = 0; j < NT; ++j)
#pragma unroll
                        for (int c = 0; c < 4; ++c) x2[u][j][c] = acc[j][0][c] + acc[j][1][c];
                }
                float vs[kSubs][2], lv[kSubs][2];
#pragma unroll
                for (int u = 0; u < kSubs; ++u)
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        float ks = 1.f;
                        vs[u][r] = 1.f, lv[u][r] = 0.f;
                        if (F8) {
                            ks = __shfl_sync(~0u, ks_now, 16 * u + 8 * r + g);
                            vs[u][r] = __shfl_sync(~0u, vs_now, 16 * u + 8 * r + g);
                            lv[u][r] = fmaxf(lg2(fabsf(vs[u][r])), -120.f);
                        }
#pragma unroll
                        for (int j = 0; j < NT; ++j)
#pragma unroll
                            for (int c = 0; c < 2; ++c)
                                x2[u][j][2 * r + c] *= F8 ? ks * qmul[j][c] : qmul[j][c];
                    }
                const bool partly = tok + kTok - 1 > n - p.rows ||
                                    (p.window && tok < n - p.window) || there + 1 != 1u << kSubs;
                if (partly) {
#pragma unroll
                    for (int u = 0; u < kSubs; ++u)
#pragma unroll
                        for (int j = 0; j < NT; ++j)
#pragma unroll
                            for (int c = 0; c < 4; ++c) {
                                const int token = tok + 16 * u + g + c / 2 * 8, last = pos[j][c % 2];
                                if (token > last || (p.window && token <= last - p.window) ||
                                    !(there >> u & 1))
                                    x2[u][j][c] = -INFINITY;
                            }
                }
                bool up = false;
#pragma unroll
                for (int u = 0; u < kSubs; ++u)
#pragma unroll
                    for (int j = 0; j < NT; ++j)
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            const float m = top[j][c % 2];
                            if (F8)
                                up |= x2[u][j][c] - m >
                                      fminf(kSlack, above[j][c % 2] + kSlack - lv[u][c / 2]);
                            else      // (rounded down: a weight in f16 has no room above)
                                up |= x2[u][j][c] > (kHalf ? __fadd_rd(m, kSlack) : m + kSlack);
                        }
                if (__any_sync(~0u, up)) {
#pragma unroll
                    for (int j = 0; j < NT; ++j)
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            float a = -INFINITY;
#pragma unroll
                            for (int u = 0; u < kSubs; ++u)
                                a = fmaxf(a, fmaxf(x2[u][j][c], x2[u][j][c + 2]));
#pragma unroll
                            for (int d = 4; d < 32; d *= 2)
                                a = fmaxf(a, __shfl_xor_sync(~0u, a, d));
                            a = fmaxf(a, top[j][c]);
                            const float fade = ratio(top[j][c], a);
                            sums[j][c] *= fade;
                            float ofade = fade;
                            if (F8) {
                                const float from = a == -INFINITY ? 0.f : a;
                                float b = -INFINITY;
#pragma unroll
                                for (int u = 0; u < kSubs; ++u)
                                    b = fmaxf(b, fmaxf(x2[u][j][c] - from + lv[u][0],
                                                       x2[u][j][c + 2] - from + lv[u][1]));
#pragma unroll
                                for (int d = 4; d < 32; d *= 2)
                                    b = fmaxf(b, __shfl_xor_sync(~0u, b, d));
                                const float old = above[j][c] + (top[j][c] - from);
                                b = fmaxf(b, old);
                                ofade = ratio(old, b);
                                above[j][c] = b;
                                lift[j][c] = b == -INFINITY ? 1.f : ex2(kRoom - b);
                            }
                            top[j][c] = a;
#pragma unroll
                            for (int i = 0; i < D / 16; ++i)
                                o[i][j][c] *= ofade, o[i][j][c + 2] *= ofade;
                        }
                }

                // weights
                uint32_t ph[kSubs][NT][2], pl[kSubs][NT][2];
#pragma unroll
                for (int u = 0; u < kSubs; ++u)
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
                        float w[4];
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            const float from = top[j][c % 2] == -INFINITY ? 0.f : top[j][c % 2];
                            const float x = x2[u][j][c] - from;
                            w[c] = ex2(kHalf && !F8 ? x + kRoom : x);
                            sums[j][c % 2] += w[c];
                            // a token that is not seen weighs 0 whatever its scale holds
                            if (F8)
                                w[c] = x2[u][j][c] == -INFINITY
                                           ? 0.f
                                           : w[c] * (vs[u][c / 2] * lift[j][c % 2]);
                        }
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            const uint32_t hi = pair<TYPE>(w[2 * r], w[2 * r + 1]);
                            ph[u][j][r] = transposed(hi);
                            const float2 h = unpair<TYPE>(hi);
                            float l0 = w[2 * r] - h.x, l1 = w[2 * r + 1] - h.y;
                            if (kHalf) l0 *= kLow, l1 *= kLow;
                            pl[u][j][r] = transposed(pair<TYPE>(l0, l1));
                        }
                    }

                // sums of the values: use(i, fragment of 16 d's and the 16 tokens)
                auto values_at = [&](int u, int k, auto use) {
                    uint32_t v[4];
                    load_matrices<true>(v, (at + off_v + u * S::kSub + k / 4 * 2048) ^
                                               (k % 4 * 32));
                    if constexpr (F8) {
                        // pairs of d's of two tokens -> pairs of tokens of two d's
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const uint32_t a = __byte_perm(v[2 * h], 0, 0x3120);
                            const uint32_t b = __byte_perm(v[2 * h + 1], 0, 0x3120);
                            const uint32_t f[4] = {e4m3x2_to_f16x2(a), e4m3x2_to_f16x2(a >> 16),
                                                   e4m3x2_to_f16x2(b), e4m3x2_to_f16x2(b >> 16)};
                            use(2 * k + h, f);
                        }
                    } else {
                        use(k, v);
                    }
                };
                auto values = [&](int u, auto use) {
#pragma unroll
                    for (int k = 0; k < kSteps; ++k) values_at(u, k, use);
                };
                if (!partly) {
#pragma unroll
                    for (int k = 0; k < kSteps; ++k) {
                        constexpr int kEach = D / 16 / kSteps;      // d fragments of a step
                        float low[kEach][NT][4] = {};
#pragma unroll
                        for (int u = 0; u < kSubs; ++u)
                            values_at(u, k, [&](int i, const uint32_t (&f)[4]) {
#pragma unroll
                                for (int j = 0; j < NT; ++j) {
                                    mma<TYPE>(o[i][j], f, ph[u][j][0], ph[u][j][1]);
                                    mma<TYPE>(kHalf ? low[i % kEach][j] : o[i][j], f, pl[u][j][0],
                                              pl[u][j][1]);
                                }
                            });
                        if (!kHalf) continue;
#pragma unroll
                        for (int h = 0; h < kEach; ++h)
#pragma unroll
                            for (int j = 0; j < NT; ++j)
#pragma unroll
                                for (int c = 0; c < 4; ++c)
                                    o[k * kEach + h][j][c] =
                                        fmaf(low[h][j][c], 1.f / kLow, o[k * kEach + h][j][c]);
                    }
                } else {
                    // Values that no row sees are taken out: 0 times what lies there
                    // may be NaN.  Where a value that some rows see and others do not
                    // is none, row by row, with the values that each sees.
#pragma unroll 1
                    for (int u = 0; u < kSubs; ++u) {
                        if (!(there >> u & 1)) continue;
                        uint32_t any[2] = {0, 0}, some[2] = {0, 0}, p0[NT][2], p1[NT][2];
#pragma unroll
                        for (int j = 0; j < NT; ++j)
#pragma unroll
                            for (int r = 0; r < 2; ++r) {
                                p0[j][r] = u ? ph[kSubs - 1][j][r] : ph[0][j][r];
                                p1[j][r] = u ? pl[kSubs - 1][j][r] : pl[0][j][r];
                            }
                        const int tok_u = tok + 16 * u + 2 * t;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int token = tok_u + (i & 1) + (i & 2) * 4;
                            const uint32_t bits = i & 1 ? 0xFFFF0000u : 0xFFFFu;
                            if (token < n && !(p.window && token <= n - p.rows - p.window)) {
                                any[i / 2] |= bits;
                                if (token > n - p.rows || (p.window && token < n - p.window))
                                    some[i / 2] |= bits;
                            }
                        }
                        uint32_t odd = 0;
                        if (p.rows > 1)
                            values(u, [&](int, const uint32_t (&f)[4]) {
                                odd |= not_finite<TYPE>(f[0] & some[0]) |
                                       not_finite<TYPE>(f[1] & some[0]) |
                                       not_finite<TYPE>(f[2] & some[1]) |
                                       not_finite<TYPE>(f[3] & some[1]);
                            });
                        const bool each = __any_sync(~0u, odd != 0);
#pragma unroll 1
                        for (int r = 0; r < (each ? p.rows : 1); ++r) {
                            const int last = n - p.rows + r;
                            uint32_t keep[2] = {any[0], any[1]};
                            if (each) {
                                keep[0] = keep[1] = 0;
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    const int token = tok_u + (i & 1) + (i & 2) * 4;
                                    if (token <= last && !(p.window && token <= last - p.window))
                                        keep[i / 2] |= i & 1 ? 0xFFFF0000u : 0xFFFFu;
                                }
                            }
                            values(u, [&](int i, const uint32_t (&f)[4]) {
                                const uint32_t a[4] = {f[0] & keep[0], f[1] & keep[0],
                                                       f[2] & keep[1], f[3] & keep[1]};
#pragma unroll
                                for (int j = 0; j < NT; ++j) {
                                    float d[4] = {0.f, 0.f, 0.f, 0.f}, low[4] = {0.f, 0.f, 0.f, 0.f};
                                    mma<TYPE>(d, a, p0[j][0], p0[j][1]);
                                    mma<TYPE>(kHalf ? low : d, a, p1[j][0], p1[j][1]);
#pragma unroll
                                    for (int c = 0; c < 4; ++c) {
                                        if (kHalf) d[c] = fmaf(low[c], 1.f / kLow, d[c]);
                                        if (!each || pos[j][c % 2] == last) o[i][j][c] += d[c];
                                    }
                                }
                            });
                        }
                    }
                }
                __syncwarp();                  // the stage may be filled again
            }

            // no copy may still be on its way when the ring is used for sums, or left
            if (lost)
                for (int i = 0; i < kStages; ++i) warp_wait(&bars[warp][i], ~phases >> i & 1);

            // the sums of the rows' weights over the lanes
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int c = 0; c < 2; ++c)
#pragma unroll
                    for (int d = 4; d < 32; d *= 2)
                        sums[j][c] += __shfl_xor_sync(~0u, sums[j][c], d);

            // the next item's Q is asked for here, to come while this one is written
            const Item was = it;
            x = it.start + s1;
            if (x < end) {
                it.next(first, p.heads);
                load_q();
            }
            // o[i][j][2 h + c] is of d = 16 i + 2 g + h (e4m3) or 16 i + 8 h + g
            if (s0 == 0 && s1 == was.tiles) {
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const int m = mb * M + j * 8 + 2 * t + c;
                        if (m >= m_all) continue;
                        // (not 1 / (l lift): that ends where values are below 2^-100)
                        const float f = worth<F8>(sums[j][c], above[j][c]);
                        const int r = p.by_group.over(m);
                        uint16_t *row = static_cast<uint16_t *>(p.out) +
                                        (((int64_t)was.b * p.rows + r) * p.heads + was.h) *
                                            p.group * D +
                                        (int64_t)(m - r * p.group) * D;
#pragma unroll
                        for (int i = 0; i < D / 16; ++i) {
                            const float a = o[i][j][c] * f, b = o[i][j][c + 2] * f;
                            const uint32_t w = p.dtype == MOEOP_BF16 ? pair<MOEOP_BF16>(a, b)
                                                                     : pair<MOEOP_FP16>(a, b);
                            if (F8) {
                                *reinterpret_cast<uint32_t *>(row + 16 * i + 2 * g) = w;
                            } else {
                                row[16 * i + g] = (uint16_t)w;
                                row[16 * i + 8 + g] = (uint16_t)(w >> 16);
                            }
                        }
                    }
            } else {
                // the last item's sums go to the ring, which is empty then
                const bool last = was.start + s1 == end;
                float *of_rows = &stats[2 * warp + (last ? 1 : 0)][0][0];
                float *part = last ? reinterpret_cast<float *>(ring)
                                   : heads_at + (int64_t)warp * S::kPart;
                if (p.flat) {
                    of_rows = p.parts + (((int64_t)mb * gridDim.x * W + worker) * 2 + (last ? 1 : 0)) *
                                            S::kPart;
                    part = of_rows + S::kStats;
                }
                has |= last ? 2 : 1;
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    if (g == 0) {
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            const int m = j * 8 + 2 * t + c;
                            of_rows[m] = top[j][c];
                            of_rows[M + m] = sums[j][c];
                            of_rows[2 * M + m] = F8 ? above[j][c] : 0.f;
                        }
                    }
#pragma unroll
                    for (int i = 0; i < D / 16; ++i)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int d = 16 * i + (F8 ? 2 * g + h : 8 * h + g);
                            *reinterpret_cast<float2 *>(part + d * M + j * 8 + 2 * t) =
                                make_float2(o[i][j][2 * h], o[i][j][2 * h + 1]);
                        }
                }
            }
        }
        if (lane == 0) lasts[warp] = it;
        // what the warp has of the item it did not begin follows into the ring
        if ((has & 1) && !p.flat) {
            const float *from = heads_at + (int64_t)warp * S::kPart;
            __syncwarp();
#pragma unroll 1
            for (int i = lane * 4; i < M * D; i += 128)
                copy16(ring_addr + (M * D + i) * 4, from + i);
            copies_wait();
        }
    }
    if (p.flat) return;
    if (lane == 0) shares_of[warp] = has;
    // The next kernel may come (calls in a row, 9 x 6007: 44 us, so 41); the one that
    // joins reads the lengths before it waits, and would only take room (32768 tokens
    // of one sequence 20.1 us, so 19.0).
    if (!p.apart) pdl_trigger();
    __syncthreads();

    // -----------------------------------------------------------------------
    // Join: the block's warps, then the blocks
    // -----------------------------------------------------------------------
    // Four numbers of a partial sum O^T from number i on are of d = i / M and the rows
    // i % M ..: where those rows of the output are (NULL: nowhere), and the numbers.
    auto rows_from = [&](const Item &x, int m, uint16_t *(&to)[4]) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const int row = mb * M + m + c, r = p.by_group.over(row);
            to[c] = row < m_all ? static_cast<uint16_t *>(p.out) +
                                      ((((int64_t)x.b * p.rows + r) * p.heads + x.h) * p.group +
                                       (row - r * p.group)) * D
                                : nullptr;
        }
    };
    auto store = [&](uint16_t *const (&to)[4], int i, const float (&v)[4]) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const uint32_t w = p.dtype == MOEOP_BF16 ? pair<MOEOP_BF16>(v[c], 0.f)
                                                     : pair<MOEOP_FP16>(v[c], 0.f);
            if (to[c]) to[c][i / M] = (uint16_t)w;
        }
    };
    auto finite = [](float v) { return v == -INFINITY ? 0.f : v; };
    // Lane e looks at share e.  A share that is not there counts to the item of the
    // next one, with nothing.
    Item mine;
    mine.start = -1, mine.tiles = 0;
    const bool there = lane < 2 * W && (shares_of[lane / 2] >> (lane & 1) & 1);
    const uint32_t present = __ballot_sync(~0u, there);
    if (lane < 2 * used) mine = !(lane & 1) && there ? fronts[lane / 2] : lasts[lane / 2];
    const int before = __shfl_up_sync(~0u, mine.start, 1);
    const uint32_t begins = __ballot_sync(~0u, lane == 0 || before != mine.start);
    const uint32_t later = begins & ~((2u << lane) - 1);
    const int from = 31 - __clz(begins & ((2u << lane) - 1)), to = later ? __ffs(later) - 2 : 31;
    const bool inside = mine.start >= cs && mine.end() <= ce;
    const uint32_t those = present >> from & ((2u << (to - from)) - 1);
    // an item with one share here, all of it, was written by its warp: it has none
    const uint32_t need = __ballot_sync(~0u, lane == from && those != 0);
    float *const blocks_out = blocks_at + 2 * blockIdx.x * (int64_t)S::kPart;
    // what each share's rows are worth: to the common maximum, or in the end
#pragma unroll 1
    for (int m = warp; m < M; m += W) {
        const float top = there ? stats[lane][0][m] : -INFINITY, l = there ? stats[lane][1][m] : 0.f;
        float tall = top;
#pragma unroll
        for (int d = 1; d < 2 * W; d *= 2) {          // to the end of the item's shares
            const float a = __shfl_down_sync(~0u, tall, d);
            if (lane + d <= to) tall = fmaxf(tall, a);
        }
        tall = __shfl_sync(~0u, tall, from);
        // what the sums' own maxima are above the common one
        const float below = top - finite(tall), otop = there ? below + stats[lane][2][m] : -INFINITY;
        float oall = otop, sum_l = there ? l * ex2(below) : 0.f;
#pragma unroll
        for (int d = 1; d < 2 * W; d *= 2) {
            const float a = __shfl_down_sync(~0u, sum_l, d), b = __shfl_down_sync(~0u, oall, d);
            if (lane + d <= to) sum_l += a, oall = fmaxf(oall, b);
        }
        sum_l = __shfl_sync(~0u, sum_l, from), oall = __shfl_sync(~0u, oall, from);
        const float f = ex2(otop - finite(oall));
        if (there) worth_of[lane][m] = inside ? f * worth<F8>(sum_l, oall) : f;
        if (there && !inside && lane == from + __ffs(those) - 1) {
            float *out = blocks_out + (mine.start >= cs ? S::kPart : 0);
            out[m] = tall, out[M + m] = sum_l, out[2 * M + m] = oall;
        }
    }
    __syncthreads();
    // the warps share the items out
    const int groups = __popc(need), slices = groups > 0 && groups < W ? W / groups : 1;
#pragma unroll 1
    for (int k = warp / slices; k < groups; k += W / slices) {
        uint32_t rest = need;
        for (int i = 0; i < k; ++i) rest &= rest - 1;
        const int e0 = __ffs(rest) - 1;
        const bool here = __shfl_sync(~0u, inside ? 1 : 0, e0);
        const uint32_t bits = __shfl_sync(~0u, those, e0) << e0;
        Item x;
        x.b = __shfl_sync(~0u, mine.b, e0), x.h = __shfl_sync(~0u, mine.h, e0);
        x.start = __shfl_sync(~0u, mine.start, e0);
        float *const out = blocks_out + (x.start >= cs ? S::kPart : 0) + S::kStats;
        // share by share, four of a lane's places at a time: finding a share takes as
        // long as adding it
        const int stride = slices * 128;                  // places keep their row
        uint16_t *to[4];
        rows_from(x, lane * 4 % M, to);
#pragma unroll 1
        for (int i0 = (warp % slices * 32 + lane) * 4; i0 < M * D; i0 += 4 * stride) {
            float v[4][4] = {};
#pragma unroll 1
            for (uint32_t left = bits; left; left &= left - 1) {
                // a warp's last item, and behind it the one that another began
                const int e = __ffs(left) - 1;
                const float *part = reinterpret_cast<const float *>(
                                        smem + e / 2 * (kStages * S::kStage)) + (~e & 1) * M * D;
                const float4 f = *reinterpret_cast<const float4 *>(&worth_of[e][i0 % M]);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    if (i0 + c * stride >= M * D) break;
                    const float4 u = *reinterpret_cast<const float4 *>(part + i0 + c * stride);
                    v[c][0] = fmaf(u.x, f.x, v[c][0]), v[c][1] = fmaf(u.y, f.y, v[c][1]);
                    v[c][2] = fmaf(u.z, f.z, v[c][2]), v[c][3] = fmaf(u.w, f.w, v[c][3]);
                }
            }
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int i = i0 + c * stride;
                if (i >= M * D) break;
                if (here)
                    store(to, i, v[c]);
                else
                    *reinterpret_cast<float4 *>(out + i) =
                        make_float4(v[c][0], v[c][1], v[c][2], v[c][3]);
            }
        }
    }
    // -----------------------------------------------------------------------
    // The last block to reach an item joins it; beyond kJoin blocks the last of
    // each kJoin of them joins theirs, the last of those the whole.  atomicInc
    // leaves the counters zero.
    // -----------------------------------------------------------------------
    constexpr int kJoin = 16;
    const Item head = fronts[0], back = lasts[used - 1];
    const bool from_before = head.start < cs, goes_on = back.start >= cs && back.end() > ce;
    const int crosses = (from_before ? 1 : 0) + (goes_on ? 1 : 0);
    if (!crosses || p.apart) return;
    // counters by a block that no other item has in this place: the one where the
    // item begins, or where one of its groups does
    uint32_t *const counters = p.counters + mb * gridDim.x;
    // true for the last; what the blocks wrote before their barrier is then visible
    auto arrive = [&](uint32_t *counter, int parts) {
        uint32_t before = 0;
        if (parts > 1)
            asm volatile("atom.acq_rel.gpu.global.inc.u32 %0, [%1], %2;"
                         : "=r"(before)
                         : "l"(counter), "r"(parts - 1)
                         : "memory");
        return before == (uint32_t)parts - 1;
    };
    float *const all = reinterpret_cast<float *>(smem);        // the ring is free
    auto crossing = [&](int k) { return from_before && k == 0 ? head : back; };
    __syncthreads();
    if ((int)threadIdx.x < crosses) {
        const Item x = crossing(threadIdx.x);
        const int c0 = shares.owner(x.start), count = shares.owner(x.end() - 1) - c0 + 1;
        const int group = (blockIdx.x - c0) / kJoin, from = c0 + group * kJoin;
        joined[threadIdx.x] =
            arrive(counters + from + (group ? 256 : 0), min(count - group * kJoin, kJoin));
    }
    __syncthreads();
#pragma unroll 1
    for (int k = 0; k < crosses; ++k) {
        if (!joined[k]) continue;
        const Item x = crossing(k);
        const int c0 = shares.owner(x.start), count = shares.owner(x.end() - 1) - c0 + 1;
        const int group = (blockIdx.x - c0) / kJoin, groups = (count + kJoin - 1) / kJoin;
        int parts = min(count - group * kJoin, kJoin), from = c0 + group * kJoin, step = 1;
#pragma unroll 1
        while (true) {
            // a block's share is its second sum where the item begins in it
            auto part = [&](int i) {
                const int c = from + i * step;
                return blocks_at + (2 * c + (c == c0 ? 1 : 0)) * (int64_t)S::kPart;
            };
            const bool whole = step > 1 || groups == 1;
            // the three numbers of each part's rows, then what the part is worth
            for (int i = threadIdx.x; i < parts * S::kStats; i += W * 32)
                all[i] = __ldcg(part(i / S::kStats) + i % S::kStats);
            __syncthreads();
#pragma unroll 1
            for (int m = warp; m < M; m += W) {
                const float *s = all + lane * S::kStats;
                const bool in = lane < parts;
                const float top = in ? s[m] : -INFINITY;
                float tall = top;
#pragma unroll
                for (int d = kJoin / 2; d; d >>= 1)
                    tall = fmaxf(tall, __shfl_xor_sync(~0u, tall, d));
                const float below = top - finite(tall), otop = in ? below + s[2 * M + m] : -INFINITY;
                float oall = otop, l = in ? s[M + m] * ex2(below) : 0.f;
#pragma unroll
                for (int d = kJoin / 2; d; d >>= 1) {
                    l += __shfl_xor_sync(~0u, l, d);
                    oall = fmaxf(oall, __shfl_xor_sync(~0u, oall, d));
                }
                if (in) {
                    const float f = ex2(otop - finite(oall));
                    worth_of[lane][m] = whole ? f * worth<F8>(l, oall) : f;
                }
                if (lane == 0 && !whole) {
                    float *out = part(0);
                    out[m] = tall, out[M + m] = l, out[2 * M + m] = oall;
                }
            }
            __syncthreads();
            uint16_t *to[4];
            rows_from(x, threadIdx.x * 4 % M, to);
#pragma unroll 1
            for (int i = threadIdx.x * 4; i < M * D; i += W * 128) {
                float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
                for (int w = 0; w < parts; ++w) {
                    const float4 u =
                        __ldcg(reinterpret_cast<const float4 *>(part(w) + S::kStats + i));
                    const float4 f = *reinterpret_cast<const float4 *>(&worth_of[w][i % M]);
                    v[0] = fmaf(u.x, f.x, v[0]), v[1] = fmaf(u.y, f.y, v[1]);
                    v[2] = fmaf(u.z, f.z, v[2]), v[3] = fmaf(u.w, f.w, v[3]);
                }
                if (whole)
                    store(to, i, v);
                else
                    *reinterpret_cast<float4 *>(part(0) + S::kStats + i) =
                        make_float4(v[0], v[1], v[2], v[3]);
            }
            if (whole) break;
            __syncthreads();
            parts = groups, from = c0, step = kJoin;
            if (threadIdx.x == 0) joined[k] = arrive(counters + c0 + 512, parts);
            __syncthreads();
            if (!joined[k]) break;
        }
    }
}

// The sums of an item's blocks added up: where items are few, so that many blocks
// share one, and the last of them would be long at it alone.  A block of this kernel
// takes 32 d's of an item and a block of query rows; its threads share the parts.
// One sequence of 32768 tokens, 8 heads: 27 us with the join in the kernel above.
template <int TYPE, int D, int NT>
__global__ void __launch_bounds__(256) join_kernel(const AttendParams p) {
    using S = Shape<TYPE, D, NT>;
    constexpr bool F8 = S::F8;
    constexpr int M = S::M, kStats = S::kStats, kEach = 32 * M / 4, kGroups = 256 / kEach;
    __shared__ float all[kAttendSms * kStats];
    __shared__ float4 sums[256];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, mb = blockIdx.y;
    const int b = blockIdx.x / p.heads, h = blockIdx.x - b * p.heads;
    int c = 0;
    if (lane < p.batch) {
        const int n = min(max(__ldg(p.lengths + lane), 0), p.width * p.page);
        c = kEmpty + max(1, (n + S::kTok - 1) / S::kTok - first_tile<S::kTok>(p, n));
    }
    int run = c;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const int left = __shfl_up_sync(~0u, run, o);
        if (lane >= o) run += left;
    }
    const Shares shares(__shfl_sync(~0u, run, 31) * p.heads, p.flat ? p.by_warps : p.by_grid);
    c = __shfl_sync(~0u, c, b);
    const int start = (__shfl_sync(~0u, run, b) - c) * p.heads + h * c;
    pdl_wait();
    pdl_trigger();
    if (c <= p.whole) return;
    const int c0 = shares.owner(start), parts = shares.owner(start + c - 1) - c0 + 1;
    if (parts == 1) return;
    const int W = S::kWarps, grid = p.by_grid.d;
    const bool goes_on = shares.begin(c0 + parts) > start + c;     // its last owner does
    const float *const parts_at =
        p.parts + (p.flat ? (int64_t)mb * grid * W * 2
                          : (int64_t)mb * grid * (W + 2) + (int64_t)grid * W) * S::kPart;
    // a warp's second sum is that of its last item, a block's of one that begins in it
    auto part = [&](int i) {
        const bool second = p.flat ? i < parts - 1 || !goes_on : i == 0;
        return parts_at + (2 * (c0 + i) + (second ? 1 : 0)) * (int64_t)S::kPart;
    };
    static_assert(140 <= kAttendSms, "an item's warps, and its blocks, fit");
    const int mine = threadIdx.x % kEach * 4, group = threadIdx.x / kEach;
    const int at = blockIdx.z * 32 * M + mine;          // number of a partial sum
    float4 u[8];
#pragma unroll
    for (int k = 0; k < 8; ++k)
        if (group + k * kGroups < parts)
            u[k] = __ldcg(reinterpret_cast<const float4 *>(part(group + k * kGroups) + kStats + at));
    for (int i = threadIdx.x; i < parts * kStats; i += 256)
        all[i] = __ldcg(part(i / kStats) + i % kStats);
    __syncthreads();
    for (int m = warp; m < M; m += 8) {
        float top = -INFINITY, otop = -INFINITY, l = 0.f;
        for (int i = lane; i < parts; i += 32) top = fmaxf(top, all[i * kStats + m]);
#pragma unroll
        for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
        const float tref = top == -INFINITY ? 0.f : top;
        // what the sums' own maxima are above the common one
        for (int i = lane; i < parts; i += 32) {
            float *s = all + i * kStats;
            const float below = s[m] - tref;
            l = fmaf(s[M + m], ex2(below), l);
            s[2 * M + m] += below;
            otop = fmaxf(otop, s[2 * M + m]);
        }
#pragma unroll
        for (int d = 16; d; d >>= 1) {
            l += __shfl_xor_sync(~0u, l, d);
            otop = fmaxf(otop, __shfl_xor_sync(~0u, otop, d));
        }
        const float w = worth<F8>(l, otop), oref = otop == -INFINITY ? 0.f : otop;
        for (int i = lane; i < parts; i += 32) {
            float *s = all + i * kStats;
            s[m] = ex2(s[2 * M + m] - oref) * w;
        }
    }
    __syncthreads();
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](const float4 &x, int i) {
        const float *f = all + i * kStats + mine % M;
        v.x = fmaf(x.x, f[0], v.x), v.y = fmaf(x.y, f[1], v.y);
        v.z = fmaf(x.z, f[2], v.z), v.w = fmaf(x.w, f[3], v.w);
    };
#pragma unroll
    for (int k = 0; k < 8; ++k)
        if (group + k * kGroups < parts) add(u[k], group + k * kGroups);
#pragma unroll 4
    for (int i = group + 8 * kGroups; i < parts; i += kGroups)
        add(__ldcg(reinterpret_cast<const float4 *>(part(i) + kStats + at)), i);
    sums[threadIdx.x] = v;
    __syncthreads();
    // a number for each thread, the groups' sums in order
    const float *const of = reinterpret_cast<const float *>(sums);
    for (int i = threadIdx.x; i < kEach * 4; i += 256) {
        float f = 0.f;
#pragma unroll
        for (int k = 0; k < kGroups; ++k) f += of[k * kEach * 4 + i];
        const int row = mb * M + i % M, d = blockIdx.z * 32 + i / M;
        if (row >= p.rows * p.group) continue;
        const int r = p.by_group.over(row);
        static_cast<uint16_t *>(p.out)[((((int64_t)b * p.rows + r) * p.heads + h) * p.group +
                                        (row - r * p.group)) * D + d] =
            (uint16_t)(p.dtype == MOEOP_BF16 ? pair<MOEOP_BF16>(f, 0.f) : pair<MOEOP_FP16>(f, 0.f));
    }
}

template <int TYPE, int D, int NT>
cudaError_t launch(AttendParams p, cudaStream_t st) {
    using S = Shape<TYPE, D, NT>;
    const auto kernel = attend_kernel<TYPE, D, NT>;
    // the limit of shared memory is set once on each device
    static std::atomic<uint64_t> allowed{0};
    int device = 0;
    cudaError_t e = cudaGetDevice(&device);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (device & 63);
    if (!(allowed.load(std::memory_order_relaxed) & bit)) {
        if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      S::smem(kAttendMaxBatch))) != cudaSuccess)
            return e;
        allowed.fetch_or(bit, std::memory_order_relaxed);
    }
    TensorMap kmap, vmap;
    const int64_t rows = (int64_t)p.heads * p.page;
    p.wide = p.page % S::kTok == 0;
    if ((e = status_word(&p.status)) != cudaSuccess ||
        (e = make_cache_map(&kmap, p.k, S::kRow, p.wide ? S::kTok : 16, rows,
                            p.k_stride * S::kSize, p.pages)) != cudaSuccess ||
        (e = make_cache_map(&vmap, p.v, S::kRow, p.wide ? S::kTok : 16, rows,
                            p.v_stride * S::kSize, p.pages)) != cudaSuccess)
        return e;
    // no more blocks than there can be tiles for their warps
    int64_t tiles = (int64_t)p.width * p.page / S::kTok + 1;
    if (p.window && (p.window + p.rows) / S::kTok + 2 < tiles)
        tiles = (p.window + p.rows) / S::kTok + 2;
    tiles += kEmpty;
    const int grid = attend_grid(p.blocks);
    // The plan is made of the table's width and the window, for the lengths are on the
    // device: one sequence of 901 takes 8.7 us with a table of its 15 pages, 10.8 with
    // one of 256 or 2048.
    // Where there is a block for every item, the blocks share the items out, short ones
    // too, and a kernel of its own joins them (8 sequences of up to 2000 tokens, 8
    // heads: 14.5 -> 12.5 us; 32768 tokens of one: 21.3 -> 18.4); where all sequences are
    // of up to 140 tiles (what that kernel can hold of an item) it joins the warps' sums,
    // and warps may be spread over all SMs (901 tokens of one: 10.2 -> 8.5; 4 of up to
    // 901: 10.2 -> 9.0); up to 512 tokens one block takes an item (300 tokens: 7.9, with
    // the kernel that joins 7.8).  With more items than blocks they stay whole up to 1536
    // tokens (33 sequences, window 1024: up to 800 18.2, 1536 13.5 us).
    p.apart = p.batch <= 32 && p.batch * p.heads <= grid && tiles > 512 / S::kTok + kEmpty + 1;
    p.flat = p.apart && tiles <= 140;
    p.whole = p.flat ? 0 : (p.apart ? 256 : 1536) / S::kTok + kEmpty;
    const int64_t all = tiles * p.batch * p.heads;
    const int64_t most = p.flat ? all : (all + S::kWarps - 1) / S::kWarps;
    p.by_grid = Divisor((uint32_t)(most < grid ? most : grid));
    p.by_warps = Divisor(p.by_grid.d * S::kWarps);
    e = launch_early(kernel, dim3(p.by_grid.d, p.blocks), S::kWarps * 32, S::smem(p.batch), 1, st,
                     kmap, vmap, p);
    if (e != cudaSuccess || !p.apart) return e;
    return launch_early(join_kernel<TYPE, D, NT>, dim3(p.batch * p.heads, p.blocks, D / 32), 256, 0,
                        1, st, p);
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

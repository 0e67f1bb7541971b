// moeop_verify.cu -- verification of drafted tokens against the target's
// probabilities, and the draw of the token after them (moeop_verify_draft).
//
//   draft i stays while u_i q_i(x_i) < p_i(x_i);
//   the next token: the lowest id with  sum_{j <= id} w_j > u sum_j w_j,
//   w = max(p - q, 0) at a refusal, p after the last draft.
//
// A sequence has one row to read, of p and with a refusal of q: bound by memory
// where there are many sequences, by latency (two round trips for the decision,
// one for the row, one to find the place) where there are few.  So a cluster of
// thread blocks shares a row: each warp sums one contiguous piece of it, the
// sums meet in distributed shared memory, and the warp in whose piece the number
// falls goes over it once more.
//
// Which id a number falls to must not depend on rounding: a vocabulary of 10^5
// has as many borders, and sums in fp32 would take a neighbour once in 40 draws.
// So weights are counted in steps of 2^-44, in whole numbers, whose sums are
// exact in any order.  64-bit floating point would do too, but an SM adds two a
// cycle; whole numbers come out of fp32 additions of a constant whose last bit
// is the step wanted (its sum's lower bits are the number), two at a time.
//
// One GB300: 1 sequence, 3 drafts, 32768 ids 5.0 us (launch, draft, its probability,
// the row, the clusters' meeting, the id); 64 sequences, 131072 ids 20.3 us (3.3 TB/s),
// 15.7 with the rows in L2; with a 64-bit sum per id 31.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include "moe_device.cuh"
#include "moeop.cuh"

namespace cg = cooperative_groups;

namespace moe {
namespace op {

namespace {

constexpr int kMaxWarps = 16, kBlocks = 8;

__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t both(float a, float b) {
    uint64_t v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b));
    return v;
}
__device__ __forceinline__ int low(uint64_t v) { return (int)(uint32_t)v; }
__device__ __forceinline__ int high(uint64_t v) { return (int)(v >> 32); }

// What weights count so far: hi 2^-22 + lo 2^-44.  A lane's share is at most 260 of
// them (2^19 ids, 8 blocks of 256 lanes, whole fours), and both stay below 2^31.
struct Count {
    int hi = 0, lo = 0;
    // The weight of an id: p, or what p has more than q.  A number w in [0, 1] is
    // rounded to whole steps: the lower bits of w + 3 (last bit 2^-22), and of what
    // that left + 3 * 2^-22 (last bit 2^-44).  p and q go together, and the
    // constants fall away in their difference.
    template <bool REST>
    __device__ __forceinline__ void add(float p, float q) {
        constexpr float c1 = 3.f, c2 = 3.f / (1 << 22);
        p = __saturatef(p), q = REST ? __saturatef(q) : 0.f;   // NaN: 0
        const uint64_t w = both(p, q), t = add2(w, both(c1, c1));
        const uint64_t left = fma2(add2(t, both(-c1, -c1)), both(-1.f, -1.f), w);
        const uint64_t l = add2(left, both(c2, c2));
        if (!REST || p > q) hi += low(t) - high(t), lo += low(l) - high(l);
    }
    __device__ __forceinline__ uint64_t steps() const {
        return (uint64_t)(((int64_t)hi << 22) + lo);
    }
};

// u * total of a u in [0, 1), rounded down, exactly: a whole sum exceeds u * total
// where it exceeds this.  (In 64-bit floating point the product of 24 and 44 bits or
// more may be rounded up to a whole number, and the next id would be drawn.)
__device__ __forceinline__ uint64_t share_of(float u, uint64_t total) {
    const uint32_t bits = __float_as_uint(fabsf(u)), e = bits >> 23;   // (-0: 0)
    const uint64_t m = (bits & 0x7FFFFFu) | (e ? 0x800000u : 0u);     // u = m 2^-shift
    const uint32_t shift = 150 - (e ? e : 1);                         // 24 .. 149
    const uint64_t lo = m * total, hi = __umul64hi(m, total);         // hi < 2^24
    if (shift < 64) return hi << (64 - shift) | lo >> shift;
    return shift < 128 ? hi >> (shift - 64) : 0;
}

__device__ __forceinline__ uint64_t warp_sum(uint64_t v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
    return v;
}
__device__ __forceinline__ uint64_t warp_scan(uint64_t v, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const uint64_t left = __shfl_up_sync(~0u, v, o);
        if (lane >= o) v += left;
    }
    return v;
}

struct Row {
    const float *p, *q;  // q: may be NULL
    int refused;         // without q: the id that is certain to have been drafted; -1: none
    int vocab;
    template <bool REST>
    __device__ __forceinline__ void at(int i, Count &c) const {
        c.add<REST>(__ldg(p + i), !REST ? 0.f : q ? __ldg(q + i) : i == refused ? 1.f : 0.f);
    }
    // Ids i .. i + 3, p and q on 16 bytes.
    template <bool REST>
    __device__ __forceinline__ void four(int i, Count &c) const {
        const float4 a = __ldg(reinterpret_cast<const float4 *>(p + i));
        float4 b = make_float4(0.f, 0.f, 0.f, 0.f);
        if (REST && q) b = __ldg(reinterpret_cast<const float4 *>(q + i));
        if (REST && !q) {
            b.x = i == refused, b.y = i + 1 == refused;
            b.z = i + 2 == refused, b.w = i + 3 == refused;
        }
        c.add<REST>(a.x, b.x), c.add<REST>(a.y, b.y), c.add<REST>(a.z, b.z), c.add<REST>(a.w, b.w);
    }
};

// A lane's share of the ids from i0 to i1 (multiples of 4 apart from vocab itself).
template <bool REST, bool VEC>
__device__ __forceinline__ uint64_t sum_piece(const Row &r, int i0, int i1, int lane) {
    Count c;
    if (VEC) {
#pragma unroll 4
        for (int i = i0 + lane * 4; i < i1; i += 128) r.four<REST>(i, c);
    } else {
#pragma unroll 8
        for (int i = i0 + lane; i < i1; i += 32) r.at<REST>(i, c);
    }
    return c.steps();
}

// The lowest id from i0 to i1 whose running sum exceeds `target`; the sum of all of
// them does.  First the lane in whose part of them it is, then the id.
template <bool REST>
__device__ __forceinline__ int find(const Row &r, int i0, int i1, uint64_t target, int lane) {
    const int each = (i1 - i0 + 31) / 32;
    Count c;
#pragma unroll 8
    for (int i = i0 + lane * each; i < min(i0 + (lane + 1) * each, i1); ++i) r.at<REST>(i, c);
    uint64_t run = warp_scan(c.steps(), lane);
    int who = __ffs(__ballot_sync(~0u, run > target)) - 1;
    target -= __shfl_sync(~0u, run - c.steps(), who);
    const int from = i0 + who * each, to = min(from + each, i1);
    for (int i = from;; i += 32) {
        Count one;
        if (i + lane < to) r.at<REST>(i + lane, one);
        run = warp_scan(one.steps(), lane);
        const unsigned over = __ballot_sync(~0u, run > target);
        if (over) return i + __ffs(over) - 1;
        if (i + 32 >= to) return to - 1;  // not reached
        target -= __shfl_sync(~0u, run, 31);
    }
}

template <bool VEC>
__device__ __forceinline__ void draw(const VerifyParams &p, const Row &row, bool rest, int b,
                                     int accepted, uint64_t *warp_total, uint64_t *block_total) {
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = cluster.block_rank();
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, warps = blockDim.x / 32;
    // equal pieces of whole fours, one for each warp of the cluster
    const int fours = (p.c.vocab + 3) / 4, pieces = kBlocks * warps, piece = rank * warps + warp;
    const int i0 = (int)((int64_t)fours * piece / pieces) * 4;
    const int i1 = min((int)((int64_t)fours * (piece + 1) / pieces) * 4, p.c.vocab);
    uint64_t before, total;
    while (true) {
        uint64_t s = rest ? sum_piece<true, VEC>(row, i0, i1, lane)
                          : sum_piece<false, VEC>(row, i0, i1, lane);
        s = warp_sum(s);
        if (lane == 0) warp_total[warp] = s;
        __syncthreads();
        if (warp == 0) {
            const uint64_t t = warp_sum(lane < warps ? warp_total[lane] : 0);
            if (lane == 0) *block_total = t;
        }
        cluster.sync();
        const uint64_t own = lane < kBlocks ? *cluster.map_shared_rank(block_total, lane) : 0;
        total = warp_sum(own);
        before = warp_sum(lane < rank ? own : 0);
        cluster.barrier_arrive();  // block_total was read here
        if (total || !rest) break;
        rest = false;  // p has nowhere more than q
        cluster.barrier_wait();
    }
    int32_t *out = p.tokens + (size_t)b * (p.c.drafts + 1) + accepted;
    if (!total && rank == 0 && threadIdx.x == 0) *out = -1;
    before += warp_sum(lane < warp ? warp_total[lane] : 0);
    const uint64_t own = warp_total[warp];
    const float u = fminf(fmaxf(__ldg(p.sample_u + b), 0.f), 1.f - 0x1p-24f);
    const uint64_t target = share_of(u, total);
    if (target >= before && target < before + own) {
        const int id = rest ? find<true>(row, i0, i1, target - before, lane)
                            : find<false>(row, i0, i1, target - before, lane);
        if (lane == 0) *out = id;
    }
    cluster.barrier_wait();        // block_total may go
}

__global__ void __launch_bounds__(kMaxWarps * 32, 2) verify_kernel(const VerifyParams p) {
    __shared__ uint64_t warp_total[kMaxWarps], block_total;
    const int rank = cg::this_cluster().block_rank();
    const int b = blockIdx.x / kBlocks, lane = threadIdx.x % 32, n = p.c.drafts;
    // no trigger: the next kernel's blocks would only take room while they wait (calls in
    // a row, 64 x 131072: 16.5 us, so 15.5)
    pdl_wait();
    // lane i decides about draft i; every warp does, which saves a barrier
    int x = -1;
    bool good = false;
    if (lane < n) {
        x = __ldg(p.draft + (size_t)b * n + lane);
        const float u = __ldg(p.accept_u + (size_t)b * n + lane);
        if ((unsigned)x < (unsigned)p.c.vocab) {
            const float t =
                __ldg(p.target + ((size_t)b * (n + 1) + lane) * p.c.target_stride + x);
            const float q = p.draft_probs
                                ? __ldg(p.draft_probs + ((size_t)b * n + lane) * p.c.draft_stride + x)
                                : 1.f;
            // from 0 to 1, NaN 0, as in the draw
            good = (double)u * (double)__saturatef(q) < (double)__saturatef(t);
        }
    }
    const int accepted = __ffs(__ballot_sync(~0u, !good)) - 1;  // lane 31 has no draft
    const int last = __shfl_sync(~0u, x, accepted);
    const bool rest = accepted < n && last >= 0;
    if (rank == 0 && threadIdx.x <= n && (int)threadIdx.x != accepted)
        p.tokens[(size_t)b * (n + 1) + threadIdx.x] = (int)threadIdx.x < accepted ? x : -1;
    if (rank == 0 && threadIdx.x == 0) p.accepted[b] = accepted;
    Row row;
    row.p = p.target + ((size_t)b * (n + 1) + accepted) * p.c.target_stride;
    row.q = rest && p.draft_probs ? p.draft_probs + ((size_t)b * n + accepted) * p.c.draft_stride
                                  : nullptr;
    row.refused = last;
    row.vocab = p.c.vocab;
    const uintptr_t starts = reinterpret_cast<uintptr_t>(row.p) | reinterpret_cast<uintptr_t>(row.q);
    if (starts % 16 == 0 && p.c.vocab % 4 == 0)
        draw<true>(p, row, rest, b, accepted, warp_total, &block_total);
    else
        draw<false>(p, row, rest, b, accepted, warp_total, &block_total);
}

}  // namespace

cudaError_t launch_verify_draft(const VerifyParams &p, cudaStream_t st) {
    // 512 threads where the clusters of all sequences run at once (two blocks on each
    // of 152 SMs), else 256 (four)
    const int threads = p.c.batch * kBlocks <= 2 * 152 ? 512 : 256;
    return launch_early(verify_kernel, dim3((unsigned)p.c.batch * kBlocks), threads, 0, kBlocks, st,
                        p);
}

}  // namespace op
}  // namespace moe

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
// is the step wanted (its sum's lower bits are the number), all at full rate.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include "moe_device.cuh"
#include "moeop.cuh"

namespace cg = cooperative_groups;

namespace moe {
namespace op {

namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32, kBlocks = 8;

// w in [0, 1] as hi 2^-22 + lo 2^-44, rounded to the nearest: the lower bits of
// w + 3 (last bit 2^-22) and of what it left + 3 * 2^-22 (last bit 2^-44).
__device__ __forceinline__ void steps(float w, int &hi, int &lo) {
    constexpr float c1 = 3.f, c2 = 3.f / (1 << 22);
    w = fminf(fmaxf(w, 0.f), 1.f);  // NaN: 0
    const float t = w + c1;
    hi = __float_as_int(t) - __float_as_int(c1);
    lo = __float_as_int(w - (t - c1) + c2) - __float_as_int(c2);
}
// The weight of an id in steps of 2^-44: p, or what p has more than q.
template <bool REST>
__device__ __forceinline__ uint64_t weight(float p, float q) {
    int hi, lo;
    steps(p, hi, lo);
    int64_t n = ((int64_t)hi << 22) + lo;
    if (REST) {
        steps(q, hi, lo);
        n -= ((int64_t)hi << 22) + lo;
    }
    return n > 0 ? (uint64_t)n : 0;
}

__device__ __forceinline__ uint64_t warp_sum(uint64_t v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
    return v;
}

struct Row {
    const float *p, *q;  // q: may be NULL
    int refused;         // without q: the id that is certain to have been drafted; -1: none
    int vocab;
    template <bool REST>
    __device__ __forceinline__ uint64_t at(int i) const {
        if (i >= vocab) return 0;
        return weight<REST>(__ldg(p + i), !REST ? 0.f : q ? __ldg(q + i) : i == refused ? 1.f : 0.f);
    }
    // Ids i .. i + 3, p and q on 16 bytes.
    template <bool REST>
    __device__ __forceinline__ uint64_t four(int i, uint64_t (&w)[4]) const {
        const float4 a = __ldg(reinterpret_cast<const float4 *>(p + i));
        float4 b = make_float4(0.f, 0.f, 0.f, 0.f);
        if (REST && q) b = __ldg(reinterpret_cast<const float4 *>(q + i));
        if (REST && !q) {
            b.x = i == refused, b.y = i + 1 == refused;
            b.z = i + 2 == refused, b.w = i + 3 == refused;
        }
        w[0] = weight<REST>(a.x, b.x), w[1] = weight<REST>(a.y, b.y);
        w[2] = weight<REST>(a.z, b.z), w[3] = weight<REST>(a.w, b.w);
        return w[0] + w[1] + w[2] + w[3];
    }
};

// Sum of a lane's share of the ids from i0 to i1 (a multiple of 4 apart from
// vocab itself).
template <bool REST, bool VEC>
__device__ __forceinline__ uint64_t sum_piece(const Row &r, int i0, int i1, int lane) {
    uint64_t s = 0;
    if (VEC) {
#pragma unroll 4
        for (int i = i0 + lane * 4; i < i1; i += 128) {
            uint64_t w[4];
            s += r.four<REST>(i, w);
        }
    } else {
#pragma unroll 8
        for (int i = i0 + lane; i < i1; i += 32) s += r.at<REST>(i);
    }
    return s;
}

// The lowest id from i0 to i1 whose running sum exceeds `target`; the sum of
// all of them does.
template <bool REST, bool VEC>
__device__ __forceinline__ int find(const Row &r, int i0, int i1, uint64_t target, int lane) {
    constexpr int kEach = VEC ? 4 : 1;
    uint64_t before = 0;
    for (int i = i0; i < i1; i += 32 * kEach) {
        uint64_t w[4] = {0, 0, 0, 0};
        const int own = i + lane * kEach;
        uint64_t s = 0;
        if (own < i1) s = VEC ? r.four<REST>(own, w) : r.at<REST>(own);
        if (!VEC) w[0] = s;
        uint64_t run = s;
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const uint64_t left = __shfl_up_sync(~0u, run, o);
            if (lane >= o) run += left;
        }
        const unsigned over = __ballot_sync(~0u, before + run > target);
        if (over) {
            const int who = __ffs(over) - 1;
            int id = own;
            uint64_t c = before + run - s;
#pragma unroll
            for (int j = 0; j < kEach - 1; ++j) {
                c += w[j];
                if (c <= target && id == own + j) id = own + j + 1;
            }
            return __shfl_sync(~0u, id, who);
        }
        before += __shfl_sync(~0u, run, 31);
    }
    return -1;  // not reached
}

template <bool VEC>
__device__ __forceinline__ void draw(const VerifyParams &p, const Row &row, bool rest, int b,
                                     int accepted, uint64_t *warp_total, uint64_t *block_total) {
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = cluster.block_rank(), blocks = cluster.num_blocks();
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    // equal pieces of whole fours, one for each warp of the cluster
    const int fours = (p.c.vocab + 3) / 4, pieces = blocks * kWarps, piece = rank * kWarps + warp;
    const int i0 = (int)((int64_t)fours * piece / pieces) * 4;
    const int i1 = min((int)((int64_t)fours * (piece + 1) / pieces) * 4, p.c.vocab);
    uint64_t before, total;
    while (true) {
        uint64_t s = rest ? sum_piece<true, VEC>(row, i0, i1, lane)
                          : sum_piece<false, VEC>(row, i0, i1, lane);
        s = warp_sum(s);
        if (lane == 0) warp_total[warp] = s;
        __syncthreads();
        if (threadIdx.x == 0) {
            uint64_t t = 0;
            for (int w = 0; w < kWarps; ++w) t += warp_total[w];
            *block_total = t;
        }
        cluster.sync();
        before = total = 0;
        for (int k = 0; k < blocks; ++k) {
            const uint64_t t = *cluster.map_shared_rank(block_total, k);
            total += t;
            if (k < rank) before += t;
        }
        cluster.sync();  // block_total may go, or be written again
        if (total || !rest) break;
        rest = false;  // p has nowhere more than q
    }
    int32_t *out = p.tokens + (size_t)b * (p.c.drafts + 1) + accepted;
    if (!total) {
        if (rank == 0 && threadIdx.x == 0) *out = -1;
        return;
    }
    for (int w = 0; w < warp; ++w) before += warp_total[w];
    const uint64_t own = warp_total[warp];
    // u * total < total, rounded down: a whole sum exceeds u * total where it
    // exceeds this.  The product is rounded at 2^-53 of itself.
    const float u = fminf(fmaxf(__ldg(p.sample_u + b), 0.f), 1.f - 0x1p-24f);
    const uint64_t target = (uint64_t)((double)u * (double)total);
    if (own && target >= before && target < before + own) {
        const int id = rest ? find<true, VEC>(row, i0, i1, target - before, lane)
                            : find<false, VEC>(row, i0, i1, target - before, lane);
        if (lane == 0) *out = id;
    }
}

__global__ void __launch_bounds__(kThreads, 2) verify_kernel(const VerifyParams p) {
    __shared__ uint64_t warp_total[kWarps], block_total;
    const int blocks = cg::this_cluster().num_blocks(), rank = cg::this_cluster().block_rank();
    const int b = blockIdx.x / blocks, lane = threadIdx.x % 32, n = p.c.drafts;
    pdl_trigger();
    pdl_wait();
    // lane i decides about draft i; every warp does, which saves a barrier
    int x = -1;
    bool good = false;
    if (lane < n) {
        x = __ldg(p.draft + (size_t)b * n + lane);
        if ((unsigned)x < (unsigned)p.c.vocab) {
            const float u = __ldg(p.accept_u + (size_t)b * n + lane);
            const float t =
                __ldg(p.target + ((size_t)b * (n + 1) + lane) * p.c.target_stride + x);
            const float q = p.draft_probs
                                ? __ldg(p.draft_probs + ((size_t)b * n + lane) * p.c.draft_stride + x)
                                : 1.f;
            good = (double)u * (double)q < (double)t;
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
    return launch_early(verify_kernel, dim3((unsigned)p.c.batch * kBlocks), kThreads, 0, kBlocks, st,
                        p);
}

}  // namespace op
}  // namespace moe

// moeop_route.cu -- routing of any number of token rows to experts
// (moeop_route_topk): softmax or sigmoid scores, a balance bias, groups,
// top-k, renormalised weights.
//
// One warp per row; lane l holds experts l, l + 32, ... in registers.  The
// logits are read once (4 E bytes a row, the bound of large calls); a row is
// otherwise a chain of warp reductions (the bound of small ones): softmax
// maximum and sum, the group scores, and top_k + 1 rounds of a maximum over
// order-preserving 32-bit keys.
//
// Which of two experts comes first must not depend on fp32 rounding, so the
// row is checked after the fp32 selection: where two neighbours of the
// descending order (or the last group taken and the first left out) are
// nearer than the error bound of their fp32 values, or the weights' sum is
// too small for fp32, the warp decides the row again in 64 bits.  The bound:
// with u = 2^-24, expf, the divisions and the sum of E terms (E/32 serial, 5
// in the tree) leave p within (E/32 + 16) u of its value, relative to the
// largest p of the row; a sigmoid within 8 u; adding the bias rounds by u
// |key|.  About one row in a hundred takes the second way with N(0, 1.5)
// logits, 256 experts and a bias.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>

#include "moeop.cuh"

namespace moe {
namespace op {

namespace {

constexpr int kWarps = 4;  // rows per block
constexpr float kUlp = 5.9604645e-8f;

__device__ __forceinline__ float load_logit(const void *p, int dtype, int64_t i) {
    if (dtype == MOEOP_FP32) return __ldg(static_cast<const float *>(p) + i);
    if (dtype == MOEOP_BF16)
        return __uint_as_float((uint32_t)__ldg(static_cast<const uint16_t *>(p) + i) << 16);
    return __half2float(__ushort_as_half(__ldg(static_cast<const uint16_t *>(p) + i)));
}

// Order-preserving map of finite or infinite floats to unsigned; 0 is below
// all, and -0 equals 0.
__device__ __forceinline__ uint32_t order_key(float f) {
    const uint32_t b = __float_as_uint(f + 0.f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float order_value(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

template <typename F>
__device__ __forceinline__ F warp_max(F v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v = fmax(v, __shfl_xor_sync(~0u, v, o));
    return v;
}
template <typename F>
__device__ __forceinline__ F warp_sum(F v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
    return v;
}

// Scores of the groups from s[0..E) (dead experts -inf), in lane g for group
// g; -inf beyond the groups and for groups with nothing left.  `lanes` lanes
// (a power of two, lanes * groups <= 32) read one group together.
template <typename F>
__device__ __forceinline__ F group_scores(const F *s, int E, int groups, int top2, int lane) {
    const int size = E / groups;
    int lanes = 1;
    while (lanes * 2 * groups <= 32) lanes *= 2;
    const int g = lane / lanes, sub = lane % lanes;
    const F none = -INFINITY;
    F a = none, b = none;  // the two largest
    if (g < groups) {
        // every lane's list starts at another place, so that the lanes' reads
        // fall into different banks
        const int n = size > sub ? (size - sub + lanes - 1) / lanes : 0;
        int i = n ? g % n : 0;
        for (int t = 0; t < n; ++t) {
            const F v = s[g * size + sub + i * lanes];
            if (v > a) { b = a; a = v; }
            else if (v > b) b = v;
            if (++i == n) i = 0;
        }
    }
    for (int o = 1; o < lanes; o *= 2) {
        const F oa = __shfl_xor_sync(~0u, a, o), ob = __shfl_xor_sync(~0u, b, o);
        const F lo = fmin(a, oa);
        a = fmax(a, oa);
        b = fmax(lo, fmax(b, ob));
    }
    F score = a;
    if (top2 && b > none) score += b;
    const F mine = __shfl_sync(~0u, score, (lane * lanes) & 31);
    return lane < groups ? mine : none;
}

// Bit g: group g is among the `limit` best (ties: lower index first).
// *gap: the smallest taken score minus the largest left out.
template <typename F>
__device__ __forceinline__ uint32_t take_groups(F score, int groups, int limit, int lane, F *gap) {
    int rank = 0;
    for (int g = 0; g < groups; ++g) {
        const F o = __shfl_sync(~0u, score, g);
        rank += o > score || (o == score && g < lane);
    }
    const bool in = lane < groups && rank < limit;
    const F none = -INFINITY;
    const F worst = -warp_max(in ? -score : none);
    const F best = warp_max(lane < groups && !in ? score : none);
    *gap = worst - best;  // NaN where both are -inf: then nothing is left in either
    return __ballot_sync(~0u, in);
}

__device__ __forceinline__ bool is_dead(float l) { return !(l > -INFINITY); }

__device__ __forceinline__ double prob_wide(float l, bool soft, double mx, double sum) {
    if (is_dead(l)) return 0.0;
    return soft ? exp((double)l - mx) / sum : 1.0 / (1.0 + exp(-(double)l));
}

// The row again in 64 bits, its keys in `key` (E doubles of this warp): few
// rows come here, and registers for them would cost all rows occupancy.
__device__ __noinline__ void route_row_wide(const RouteParams &p, int row, int lane, double *key) {
    const moeop_route_config &c = p.c;
    const int E = c.num_experts, k = c.top_k;
    const int64_t base = (int64_t)row * p.stride;
    const bool soft = c.scoring == MOE_SCORING_SOFTMAX;
    double mx = -INFINITY, sum = 0.0;
    if (soft) {
        for (int e = lane; e < E; e += 32) {
            const float l = load_logit(p.logits, c.dtype, base + e);
            if (!is_dead(l)) mx = fmax(mx, (double)l);
        }
        mx = warp_max(mx);
        for (int e = lane; e < E; e += 32) {
            const float l = load_logit(p.logits, c.dtype, base + e);
            if (!is_dead(l)) sum += exp((double)l - mx);
        }
        sum = warp_sum(sum);
    }
    __syncwarp();
    for (int e = lane; e < E; e += 32) {
        const float l = load_logit(p.logits, c.dtype, base + e);
        const double biased =
            prob_wide(l, soft, mx, sum) + (p.bias ? (double)__ldg(p.bias + e) : 0.0);
        key[e] = is_dead(l) ? -INFINITY : biased;
    }
    __syncwarp();
    uint32_t in = ~0u;
    const int size = E / c.groups;
    if (c.groups > 1) {
        double gap;
        const double s =
            group_scores<double>(key, E, c.groups, c.group_score == MOEOP_GROUP_TOP2, lane);
        in = take_groups<double>(s, c.groups, c.group_limit, lane, &gap);
        __syncwarp();
    }
    for (int e = lane; e < E; e += 32) {
        const float l = load_logit(p.logits, c.dtype, base + e);
        if (!(in >> (e / size) & 1)) key[e] = -INFINITY;
        else if (!p.bias) key[e] = is_dead(l) ? -INFINITY : (double)l;
    }
    int my_id[2] = {-1, -1};
    double my_p[2] = {0.0, 0.0};
    for (int s = 0; s < k; ++s) {
        double best = -INFINITY;
        int be = 1 << 30;
        for (int e = lane; e < E; e += 32)
            if (key[e] > best) { best = key[e]; be = e; }
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            const double ob = __shfl_xor_sync(~0u, best, o);
            const int oe = __shfl_xor_sync(~0u, be, o);
            if (ob > best || (ob == best && oe < be)) { best = ob; be = oe; }
        }
        if (!(best > -INFINITY)) break;
        if (lane == be % 32) key[be] = -INFINITY;   // the lane that reads it
        if (lane == s % 32) {
            const double bp =
                prob_wide(load_logit(p.logits, c.dtype, base + be), soft, mx, sum);
            if (s < 32) { my_id[0] = be; my_p[0] = bp; }
            else { my_id[1] = be; my_p[1] = bp; }
        }
    }
    double f = c.routed_scaling_factor;
    if (c.norm_topk_prob) {
        const double total = warp_sum(my_p[0] + my_p[1]);
        f = total > 0.0 ? f / total : 0.0;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
        if (lane + 32 * h < k) {
            p.ids[(size_t)row * k + lane + 32 * h] = my_id[h];
            p.wts[(size_t)row * k + lane + 32 * h] = (float)(my_p[h] * f);
        }
}

// The largest of this lane's keys, and which: the first among equals.
template <int VPT>
__device__ __forceinline__ uint32_t local_best(const uint32_t (&ord)[VPT], int *at) {
    uint32_t best = ord[0];
    int j = 0;
#pragma unroll
    for (int i = 1; i < VPT; ++i)
        if (ord[i] > best) { best = ord[i]; j = i; }
    *at = j;
    return best;
}

// VPT: experts per lane.  A round of the selection is one maximum over the
// lanes' best keys; only the lane that held it looks through its keys again.
template <int VPT>
__global__ void __launch_bounds__(kWarps * 32) route_topk_kernel(RouteParams p) {
    __shared__ double sm_all[kWarps][VPT * 32];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int row = blockIdx.x * kWarps + warp;
    if (row >= p.rows) return;
    const moeop_route_config &c = p.c;
    const int E = c.num_experts, k = c.top_k;
    const int64_t base = (int64_t)row * p.stride;
    const bool soft = c.scoring == MOE_SCORING_SOFTMAX;
    float prob[VPT], key[VPT];
    float mx = -INFINITY;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int e = j * 32 + lane;
        const float l = e < E ? load_logit(p.logits, c.dtype, base + e) : -INFINITY;
        key[j] = is_dead(l) ? -INFINITY : l;
        mx = fmaxf(mx, key[j]);
    }
    float perr = 8 * kUlp;
    if (soft) {
        mx = warp_max(mx);
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            prob[j] = key[j] > -INFINITY ? expf(key[j] - mx) : 0.f;
            sum += prob[j];
        }
        sum = warp_sum(sum);
        const float inv = 1.f / sum;  // the largest p of the row
        perr = (VPT + 16) * kUlp * inv;
#pragma unroll
        for (int j = 0; j < VPT; ++j) prob[j] = key[j] > -INFINITY ? prob[j] * inv : 0.f;
    } else {
#pragma unroll
        for (int j = 0; j < VPT; ++j)
            prob[j] = key[j] > -INFINITY ? __fdividef(1.f, 1.f + expf(-key[j])) : 0.f;
    }
    bool wide = false;
    uint32_t ord[VPT];
    uint32_t in = ~0u;
    int size = E;
    if (c.groups > 1) {
        float *sm = reinterpret_cast<float *>(sm_all[warp]);
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int e = j * 32 + lane;
            const bool dead = !(key[j] > -INFINITY);
            const float biased = prob[j] + (p.bias && e < E ? __ldg(p.bias + e) : 0.f);
            if (p.bias && !dead) key[j] = biased;
            if (e < E) sm[e] = dead ? -INFINITY : biased;
        }
        __syncwarp();
        float gap;
        const float s =
            group_scores<float>(sm, E, c.groups, c.group_score == MOEOP_GROUP_TOP2, lane);
        in = take_groups<float>(s, c.groups, c.group_limit, lane, &gap);
        const float mag = warp_max(lane < c.groups && s > -INFINITY ? fabsf(s) : 0.f);
        wide |= gap <= 4.f * perr + 6.f * kUlp * mag;
        size = E / c.groups;
    } else if (p.bias) {
#pragma unroll
        for (int j = 0; j < VPT; ++j)
            if (key[j] > -INFINITY) key[j] = prob[j] + __ldg(p.bias + j * 32 + lane);
    }
    // e / size for e up to 1023, exact: e * (2^20 / size rounded up) >> 20
    const uint32_t div = ((1u << 20) + size - 1) / size;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const uint32_t e = j * 32 + lane;
        const bool out = !(key[j] > -INFINITY) || !(in >> (e * div >> 20) & 1);
        ord[j] = out ? 0u : order_key(key[j]);
    }
    int my_id[2] = {-1, -1};
    float my_p[2] = {0.f, 0.f};
    float before = 0.f;
    // one round more than top_k with a bias: the last one taken against the
    // first left out.  Without a bias the keys are the logits and exact.
    const int rounds = p.bias ? k + 1 : k;
    int mine_at;
    uint32_t mine = local_best<VPT>(ord, &mine_at);
    for (int s = 0; s < rounds; ++s) {
        const uint32_t best = __reduce_max_sync(~0u, mine);
        if (best == 0) break;
        if (p.bias) {
            const float v = order_value(best);
            if (s) wide |= before - v <= 2.f * perr + 4.f * kUlp * fabsf(before);
            before = v;
            if (s == k) break;
        }
        uint32_t who = __ballot_sync(~0u, mine == best);
        if (who & (who - 1))  // equal keys in several lanes: the lowest expert
            who = 1u << (__reduce_min_sync(~0u, mine == best ? mine_at * 32 + lane : 1 << 30) & 31);
        const int from = __ffs(who) - 1;
        const int be = __shfl_sync(~0u, mine_at * 32 + lane, from);
        float bp = 0.f;
        if (lane == from) {
#pragma unroll
            for (int j = 0; j < VPT; ++j)
                if (j == mine_at) { ord[j] = 0u; bp = prob[j]; }
            mine = local_best<VPT>(ord, &mine_at);
        }
        bp = __shfl_sync(~0u, bp, from);
        if (lane == s % 32) {
            if (s < 32) { my_id[0] = be; my_p[0] = bp; }
            else { my_id[1] = be; my_p[1] = bp; }
        }
    }
    float f = c.routed_scaling_factor;
    if (c.norm_topk_prob) {
        const float total = warp_sum(my_p[0] + my_p[1]);
        // under 2^-60 of the row's unit the p that fp32 holds are too small
        wide |= __any_sync(~0u, my_id[0] >= 0) && !(total > 8.7e-19f);
        f = total > 0.f ? f / total : 0.f;
    }
    if (wide) {
        route_row_wide(p, row, lane, sm_all[warp]);
        return;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
        if (lane + 32 * h < k) {
            p.ids[(size_t)row * k + lane + 32 * h] = my_id[h];
            p.wts[(size_t)row * k + lane + 32 * h] = my_p[h] * f;
        }
}

}  // namespace

cudaError_t launch_route_topk(const RouteParams &p, cudaStream_t st) {
    const int grid = (p.rows + kWarps - 1) / kWarps, E = p.c.num_experts;
    if (E <= 128) route_topk_kernel<4><<<grid, kWarps * 32, 0, st>>>(p);
    else if (E <= 256) route_topk_kernel<8><<<grid, kWarps * 32, 0, st>>>(p);
    else if (E <= 512) route_topk_kernel<16><<<grid, kWarps * 32, 0, st>>>(p);
    else route_topk_kernel<32><<<grid, kWarps * 32, 0, st>>>(p);
    return cudaGetLastError();
}

}  // namespace op
}  // namespace moe

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
// |key|, and a group's sum of two by u of their magnitudes.  About one row in a
// thousand takes the second way with N(0, 1.5) fp32 logits, 256 experts and a
// bias that tells them apart.  Equal keys count as near: of bf16 logits with a
// constant bias a third of the rows does.  64-bit arithmetic is slow here (an SM does
// two such operations a cycle): where only the order of the keys is in doubt,
// as nearly always, just the candidates' keys are computed, one to a lane, and
// the same for a sigmoid group's place; else the block's threads share the
// row's experts out.
//
// Bound by instructions: with 256 experts, sigmoid, bias and 8 groups some
// 1270 a row, six in ten issue slots taken.  One GB300: 16384 rows 24 us, 1 row
// 3.9 us (5.2 where the biases are asked for after the scores), 777 rows of 160
// experts by softmax 3.6 us.  16384 x 256 by softmax: 17 us; with a bias of
// zeros 27 us, of bf16 logits 102; 8 groups by the largest 29 us, bf16 65.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>

#include "moeop.cuh"

namespace moe {
namespace op {

namespace {

// Rows per block: 8, at most 48 KB of shared memory for them.
constexpr int warps_of(int vpt) { return vpt == 32 ? 4 : 8; }
constexpr float kUlp = 5.9604645e-8f;

// What the kernel needs beside the caller's arguments, worked out once.
struct Args {
    RouteParams p;
    int size;        // experts per group
    int lane_shift;  // 2^lane_shift lanes score one group (2^lane_shift * groups <= 32)
    uint32_t div;    // e / size == e * div >> 20 for e up to 1023
};

template <int DT>
__device__ __forceinline__ float load_logit(const void *p, int64_t i) {
    if (DT == MOEOP_FP32) return __ldg(static_cast<const float *>(p) + i);
    if (DT == MOEOP_BF16)
        return __uint_as_float((uint32_t)__ldg(static_cast<const uint16_t *>(p) + i) << 16);
    return __half2float(__ushort_as_half(__ldg(static_cast<const uint16_t *>(p) + i)));
}
// A logit or bias that takes its expert out: -inf or NaN.
__device__ __forceinline__ bool is_dead(float l) { return !(l > -INFINITY); }

// Order-preserving maps of finite or infinite floats to unsigned; 0 is below
// all, and -0 equals 0.
__device__ __forceinline__ uint32_t order_key(float f) {
    const uint32_t b = __float_as_uint(f + 0.f);
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float order_value(uint32_t k) {
    return __uint_as_float(k ^ (~(uint32_t)((int32_t)k >> 31) | 0x80000000u));
}
__device__ __forceinline__ uint64_t order_key(double f) {
    const uint64_t b = (uint64_t)__double_as_longlong(f + 0.0);
    return b ^ ((uint64_t)((int64_t)b >> 63) | 0x8000000000000000ull);
}

template <typename F>
__device__ __forceinline__ F warp_max(F v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v = fmax(v, __shfl_xor_sync(~0u, v, o));
    return v;
}
__device__ __forceinline__ float warp_max(float v) {
    return order_value(__reduce_max_sync(~0u, order_key(v)));
}
template <typename F>
__device__ __forceinline__ F warp_sum(F v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
    return v;
}

// Scores of the groups from s[0..E) (dead experts -inf), in lane g for group
// g; -inf beyond the groups and for groups with nothing left.  *least: the
// smallest of the values that make the score; *size: the sum of their
// magnitudes, 0 where one is infinite (the score is exact then).
template <typename F>
__device__ __forceinline__ F group_scores(const F *s, const Args &q, int lane, F *least, F *size) {
    const int sh = q.lane_shift, lanes = 1 << sh, g = lane >> sh, sub = lane & (lanes - 1);
    const F none = -INFINITY;
    F a = none, b = none;  // the two largest
    if (g < q.p.c.groups) {
        // every lane's list starts at another place, so that the lanes' reads
        // fall into different banks
        const int n = (q.size - sub + lanes - 1) >> sh;
        const F *from = s + g * q.size + sub;
        int i = g;
        while (i >= n && n) i -= n;
#pragma unroll 4
        for (int t = 0; t < n; ++t) {
            const F v = from[i << sh];
            b = fmax(b, fmin(a, v));
            a = fmax(a, v);
            if (++i == n) i = 0;
        }
    }
    for (int o = 1; o < lanes; o *= 2) {
        const F oa = __shfl_xor_sync(~0u, a, o), ob = __shfl_xor_sync(~0u, b, o);
        b = fmax(fmin(a, oa), fmax(b, ob));
        a = fmax(a, oa);
    }
    const bool two = q.p.c.group_score == MOEOP_GROUP_TOP2 && b > none;
    *least = __shfl_sync(~0u, two ? b : a, (lane << sh) & 31);
    const F sum = a < INFINITY ? fabs(a) + (two ? fabs(b) : F(0)) : F(0);
    *size = __shfl_sync(~0u, sum, (lane << sh) & 31);
    const F mine = __shfl_sync(~0u, two ? a + b : a, (lane << sh) & 31);
    return lane < q.p.c.groups ? mine : none;
}

// Bit g: group g is among the `limit` best (ties: lower index first).
template <typename F>
__device__ __forceinline__ uint32_t take_groups(F score, const Args &q, int lane) {
    int rank = 0;
    for (int g = 0; g < q.p.c.groups; ++g) {
        const F o = __shfl_sync(~0u, score, g);
        rank += o > score || (o == score && g < lane);
    }
    return __ballot_sync(~0u, lane < q.p.c.groups && rank < q.p.c.group_limit);
}

__device__ __forceinline__ double prob_wide(float l, bool soft, double mx, double sum) {
    if (is_dead(l)) return 0.0;
    return soft ? exp((double)l - mx) / sum : 1.0 / (1.0 + exp(-(double)l));
}

// A row again in 64 bits, by the whole block: few rows come here, but an SM
// does two 64-bit operations a cycle and an exp takes a warp a microsecond,
// so the experts are spread over all threads.  The keys are compared as
// integers.  key, prob: E doubles each; lane and warp of the calling thread;
// `owner`: the warp that selects.  The block's threads call it together.
template <int DT>
__device__ __noinline__ void route_row_wide(const Args &q, int row, int lane, int warp, int owner,
                                            double *key, double *prob, double *sums) {
    const RouteParams &p = q.p;
    const moeop_route_config &c = p.c;
    const int E = c.num_experts, k = c.top_k, threads = blockDim.x;
    const int64_t base = (int64_t)row * p.stride;
    const bool soft = c.scoring == MOE_SCORING_SOFTMAX;
    __syncthreads();  // the arrays are free
    double sum = 1.0;
    if (soft) {
        float m = -INFINITY;
        for (int e = lane; e < E; e += 32) {
            const float l = load_logit<DT>(p.logits, base + e);
            if (!is_dead(l)) m = fmaxf(m, l);
        }
        const double mx = warp_max(m);
        sum = 0.0;
        for (int e = threadIdx.x; e < E; e += threads) {
            const float l = load_logit<DT>(p.logits, base + e);
            prob[e] = is_dead(l) ? 0.0 : exp((double)l - mx);
            sum += prob[e];
        }
        sum = warp_sum(sum);
        if (lane == 0) sums[warp] = sum;
        __syncthreads();
        sum = 0.0;
        for (int w = 0; w < threads / 32; ++w) sum += sums[w];
    }
    for (int e = threadIdx.x; e < E; e += threads) {
        const float l = load_logit<DT>(p.logits, base + e);
        const float b = p.bias ? __ldg(p.bias + e) : 0.f;
        const bool dead = is_dead(l);
        const double v = dead ? 0.0 : soft ? prob[e] / sum : 1.0 / (1.0 + exp(-(double)l));
        prob[e] = v;
        key[e] = dead || is_dead(b) ? -INFINITY : v + (double)b;
    }
    __syncthreads();
    if (warp != owner) return;
    uint32_t in = ~0u;
    if (c.groups > 1) {
        double least, size;
        const double score = group_scores<double>(key, q, lane, &least, &size);
        in = take_groups<double>(score, q, lane);
    }
    __syncwarp();
    uint64_t *ord = reinterpret_cast<uint64_t *>(key);
    uint64_t mine = 0;
    int mine_at = lane;
    for (int e = lane; e < E; e += 32) {
        const float l = load_logit<DT>(p.logits, base + e);
        const bool out = key[e] == -INFINITY || !(in >> ((uint32_t)e * q.div >> 20) & 1);
        const uint64_t o = out ? 0 : order_key(p.bias ? key[e] : (double)l);
        ord[e] = o;
        if (o > mine) { mine = o; mine_at = e; }
    }
    int my_id[2] = {-1, -1};
    for (int s = 0; s < k; ++s) {
        const uint32_t hi = __reduce_max_sync(~0u, (uint32_t)(mine >> 32));
        if (hi == 0) break;
        const bool top = (uint32_t)(mine >> 32) == hi;
        const uint32_t lo = __reduce_max_sync(~0u, top ? (uint32_t)mine : 0u);
        const int be = __reduce_min_sync(~0u, top && (uint32_t)mine == lo ? mine_at : 1 << 30);
        if (be == mine_at) {
            ord[be] = 0;
            mine = 0;
            for (int e = lane; e < E; e += 32)
                if (ord[e] > mine) { mine = ord[e]; mine_at = e; }
        }
        __syncwarp();
        if (lane == s % 32) {
            if (s < 32) my_id[0] = be;
            else my_id[1] = be;
        }
    }
    double my_p[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) my_p[h] = my_id[h] < 0 ? 0.0 : prob[my_id[h]];
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

// Lane i holds the i-th of n candidates for the top k (-1: none): their
// order and weights in 64 bits.  The sum of a softmax takes the whole row.
template <int DT>
__device__ __noinline__ void route_row_close(const Args &q, int row, int lane, int id, int n) {
    const RouteParams &p = q.p;
    const moeop_route_config &c = p.c;
    const int E = c.num_experts, k = c.top_k;
    const int64_t base = (int64_t)row * p.stride;
    const bool soft = c.scoring == MOE_SCORING_SOFTMAX;
    double mx = 0.0, sum = 0.0;
    if (soft) {
        float m = -INFINITY;
        for (int e = lane; e < E; e += 32) {
            const float l = load_logit<DT>(p.logits, base + e);
            if (!is_dead(l)) m = fmaxf(m, l);
        }
        mx = warp_max(m);
#pragma unroll 4
        for (int e = lane; e < E; e += 32) {
            const float l = load_logit<DT>(p.logits, base + e);
            sum += is_dead(l) ? 0.0 : exp((double)l - mx);
        }
        sum = warp_sum(sum);
    }
    double prob = 0.0;
    uint64_t ord = 0;
    if (id >= 0) {
        prob = prob_wide(load_logit<DT>(p.logits, base + id), soft, mx, sum);
        ord = order_key(prob + (double)__ldg(p.bias + id));
    }
    int rank = 0;
    for (int i = 0; i < n; ++i) {
        const uint64_t o = __shfl_sync(~0u, ord, i);
        const int oid = __shfl_sync(~0u, id, i);
        rank += o > ord || (o == ord && oid < id);
    }
    const bool in = id >= 0 && rank < k;
    double f = c.routed_scaling_factor;
    if (c.norm_topk_prob) {
        const double total = warp_sum(in ? prob : 0.0);
        f = total > 0.0 ? f / total : 0.0;
    }
    if (in) {
        p.ids[(size_t)row * k + rank] = id;
        p.wts[(size_t)row * k + rank] = (float)(prob * f);
    }
    // slots that no expert is left for
    const int have = __popc(__ballot_sync(~0u, in));
    if (lane >= have && lane < k) {
        p.ids[(size_t)row * k + lane] = -1;
        p.wts[(size_t)row * k + lane] = 0.f;
    }
}

// The largest of the lanes' keys and the first lane that has it.
__device__ __forceinline__ uint64_t warp_max_key(uint64_t v, int *who) {
    const uint32_t hi = __reduce_max_sync(~0u, (uint32_t)(v >> 32));
    const bool top = (uint32_t)(v >> 32) == hi;
    const uint32_t lo = __reduce_max_sync(~0u, top ? (uint32_t)v : 0u);
    *who = __ffs(__ballot_sync(~0u, top && (uint32_t)v == lo)) - 1;
    return (uint64_t)hi << 32 | lo;
}

// Sigmoid scores: which of the `contested` groups (bits) come in beside the
// `sure` ones, in 64 bits.  s: the biased fp32 scores; `from` in lane g: the
// least fp32 value that may be among those that make group g's score.
// 0 where there are more candidates than lanes.
template <int VPT, int DT>
__device__ __noinline__ uint32_t settle_groups(const Args &q, int row, int lane, const float *s,
                                               uint32_t contested, uint32_t sure, float from) {
    const RouteParams &p = q.p;
    const int E = p.c.num_experts;
    int id = -1, n = 0;
    for (int j = 0; j < VPT; ++j) {
        const int e = j * 32 + lane, g = min((int)((uint32_t)e * q.div >> 20), 31);
        const float low = __shfl_sync(~0u, from, g);
        const bool may = e < E && (contested >> g & 1) && s[e] >= low;
        for (uint32_t m = __ballot_sync(~0u, may); m; m &= m - 1, ++n)
            if (lane == n) id = j * 32 + __ffs(m) - 1;
    }
    if (n > 32) return 0;
    double v = 0.0;
    if (id >= 0) {
        v = prob_wide(load_logit<DT>(p.logits, (int64_t)row * p.stride + id), false, 0.0, 1.0);
        if (p.bias) v += (double)__ldg(p.bias + id);
    }
    const int group = id >= 0 ? (int)((uint32_t)id * q.div >> 20) : -1;
    uint64_t score = 0;
    for (uint32_t m = contested; m; m &= m - 1) {
        const int g = __ffs(m) - 1;
        uint64_t key = group == g ? order_key(v) : 0;
        int who;
        warp_max_key(key, &who);
        double total = __shfl_sync(~0u, v, who);
        if (lane == who) key = 0;
        if (p.c.group_score == MOEOP_GROUP_TOP2 && warp_max_key(key, &who))
            total += __shfl_sync(~0u, v, who);
        if (lane == g) score = order_key(total);
    }
    int rank = 0;
    for (uint32_t m = contested; m; m &= m - 1) {
        const int g = __ffs(m) - 1;
        const uint64_t o = __shfl_sync(~0u, score, g);
        rank += o > score || (o == score && g < lane);
    }
    return sure | __ballot_sync(~0u, (contested >> lane & 1) &&
                                         rank < p.c.group_limit - __popc(sure));
}

__device__ __forceinline__ float prob_of(float l, bool soft, float mx, float inv) {
    if (is_dead(l)) return 0.f;
    return soft ? expf(l - mx) * inv : __fdividef(1.f, 1.f + expf(-l));
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

// VPT: experts per lane.  The result: true where the row has to be decided in 64 bits by the block.
template <int VPT, int DT>
__device__ __forceinline__ bool route_row(const Args &q, int row, int lane, float *sm) {
    const RouteParams &p = q.p;
    const moeop_route_config &c = p.c;
    const int E = c.num_experts, k = c.top_k;
    const int64_t base = (int64_t)row * p.stride;
    const bool soft = c.scoring == MOE_SCORING_SOFTMAX;
    float key[VPT], bias[VPT];
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int e = j * 32 + lane;
        const float l = e < E ? load_logit<DT>(p.logits, base + e) : -INFINITY;
        key[j] = is_dead(l) ? -INFINITY : l;
        bias[j] = p.bias && e < E ? __ldg(p.bias + e) : 0.f;
    }
    float perr = 8 * kUlp, mx = 0.f, inv = 1.f;
    if (soft) {
        mx = key[0];
#pragma unroll
        for (int j = 1; j < VPT; ++j) mx = fmaxf(mx, key[j]);
        mx = warp_max(mx);
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < VPT; ++j) sum += key[j] > -INFINITY ? expf(key[j] - mx) : 0.f;
        sum = warp_sum(sum);
        inv = 1.f / sum;  // the largest p of the row
        perr = (VPT + 16) * kUlp * inv;
    }
    bool wide = false;
    uint32_t in = ~0u;
    if (p.bias || c.groups > 1) {
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int e = j * 32 + lane;
            const bool dead = is_dead(key[j]) || is_dead(bias[j]);
            const float biased = prob_of(key[j], soft, mx, inv) + bias[j];
            if (p.bias) key[j] = dead ? -INFINITY : biased;
            if (c.groups > 1 && e < E) sm[e] = dead ? -INFINITY : biased;
        }
        if (c.groups > 1) {
            __syncwarp();
            float least, size;
            const float s = group_scores<float>(sm, q, lane, &least, &size);
            in = take_groups<float>(s, q, lane);
            // the last group taken against the first left out; where nothing
            // is left in either there is nothing to decide
            const bool taken = in >> lane & 1, some = lane < c.groups && least > -INFINITY;
            const float worst = -warp_max(taken ? -s : -INFINITY);
            const float best = warp_max(!taken && some ? s : -INFINITY);
            // each term of a score is off by perr and u of its magnitude, the
            // sum by u of theirs; of two large terms that cancel the score
            // itself says nothing.  Finite terms may sum to more than fp32 holds.
            const float most = warp_max(some ? size : 0.f);
            const float near = 4.f * perr + 6.f * kUlp * most;
            if (worst - best <= near || most == INFINITY) {
                uint32_t settled = 0;
                if (!soft && most < INFINITY)
                    settled = settle_groups<VPT, DT>(
                        q, row, lane, sm,
                        __ballot_sync(~0u, some && s >= worst - near && s <= best + near),
                        __ballot_sync(~0u, some && s > best + near),
                        least - 2.f * perr - 4.f * kUlp * fabsf(least));
                wide = settled == 0;
                if (!wide) in = settled;
            }
            __syncwarp();
        }
    }
    uint32_t ord[VPT];
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const uint32_t e = j * 32 + lane;
        const bool out = !(key[j] > -INFINITY) || !(in >> (e * q.div >> 20) & 1);
        ord[j] = out ? 0u : order_key(key[j]);
    }
    // At most 32 wanted: the k-th largest of the lanes' best keys bounds the
    // k-th largest of all from below; the keys from it on (hardly more than
    // k) go to a list, one to a lane, and are ranked against each other.  One
    // more than top_k with a bias: the last one taken against the first left
    // out.  Without a bias the keys are the logits and exact.
    const int rounds = p.bias ? k + 1 : k;
    uint2 *list = reinterpret_cast<uint2 *>(sm);
    auto collect = [&](uint32_t from) {  // keys >= from, at most 32; their number
        int n = 0;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const bool has = ord[j] >= from;
            const uint32_t m = __ballot_sync(~0u, has);
            const int at = n + __popc(m & ((1u << lane) - 1));
            if (has && at < 32) list[at] = make_uint2(ord[j], j * 32 + lane);
            n += __popc(m);
        }
        __syncwarp();
        return n;
    };
    if (rounds <= 32 && !wide) {
        uint32_t cur = ord[0], from = 1;
#pragma unroll
        for (int j = 1; j < VPT; ++j) cur = max(cur, ord[j]);
        int s = 0;
        for (; s < rounds; ++s) {
            const uint32_t best = __reduce_max_sync(~0u, cur);
            if (best == 0) break;
            from = best;
            if (cur == best) cur = 0;
        }
        const int n = collect(s < rounds ? 1u : from);
        if (n <= 32) {
            uint2 mine = make_uint2(0, 0);
            if (lane < n) mine = list[lane];
            int rank = 0;
            for (int i = 0; i < n; ++i) {
                const uint2 o = list[i];
                rank += o.x > mine.x || (o.x == mine.x && o.y < mine.y);
            }
            const bool in_k = lane < n && rank < k;
            if (p.bias) {
                __syncwarp();
                if (lane < n) list[rank].x = mine.x;
                __syncwarp();
                const float v = order_value(mine.x);
                const bool next = in_k && rank + 1 < n;
                // (beside an infinite key nothing is in doubt)
                if (__any_sync(~0u, next && v < INFINITY &&
                                        v - order_value(list[next ? rank + 1 : 0].x) <=
                                            2.f * perr + 4.f * kUlp * fabsf(v))) {
                    // every expert that may belong to the top k: those taken,
                    // and those whose keys are as near to the last taken
                    const float last = order_value(list[min(n, k) - 1].x);
                    __syncwarp();
                    const int m = collect(order_key(last - 2.f * perr - 4.f * kUlp * fabsf(last)));
                    if (m > 32) return true;
                    route_row_close<DT>(q, row, lane, lane < m ? (int)list[lane].y : -1, m);
                    return false;
                }
            }
            const float prob =
                in_k ? prob_of(load_logit<DT>(p.logits, base + mine.y), soft, mx, inv) : 0.f;
            float f = c.routed_scaling_factor;
            if (c.norm_topk_prob) {
                const float total = warp_sum(prob);
                // under 2^-60 of the row's unit the p that fp32 holds are too small
                if (n && !(total > 8.7e-19f)) return true;
                f = n ? __fdividef(f, total) : 0.f;
            }
            if (in_k) {
                p.ids[(size_t)row * k + rank] = (int)mine.y;
                p.wts[(size_t)row * k + rank] = prob * f;
            }
            if (lane >= n && lane < k) {  // no expert is left for these slots
                p.ids[(size_t)row * k + lane] = -1;
                p.wts[(size_t)row * k + lane] = 0.f;
            }
            return false;
        }
    }
    // More than 32 wanted, or too many equal keys: one by one.
    int my_id[2] = {-1, -1};
    float before = 0.f;
    bool close = false;
    int mine_at;
    uint32_t mine = local_best<VPT>(ord, &mine_at);
    for (int s = 0; s < rounds; ++s) {
        const uint32_t best = __reduce_max_sync(~0u, mine);
        if (best == 0) break;
        if (p.bias) {
            const float v = order_value(best);
            if (s)
                close |= before < INFINITY && before - v <= 2.f * perr + 4.f * kUlp * fabsf(before);
            before = v;
            if (s == k) break;
        }
        uint32_t who = __ballot_sync(~0u, mine == best);
        if (who & (who - 1))  // equal keys in several lanes: the lowest expert
            who = 1u << (__reduce_min_sync(~0u, mine == best ? mine_at * 32 + lane : 1 << 30) & 31);
        const int from = __ffs(who) - 1;
        const int be = __shfl_sync(~0u, mine_at * 32 + lane, from);
        if (lane == from) {
#pragma unroll
            for (int j = 0; j < VPT; ++j)
                if (j == mine_at) ord[j] = 0u;
            mine = local_best<VPT>(ord, &mine_at);
        }
        if (lane == s % 32) {
            if (s < 32) my_id[0] = be;
            else my_id[1] = be;
        }
    }
    float my_p[2];
#pragma unroll
    for (int h = 0; h < 2; ++h)
        my_p[h] = my_id[h] < 0 ? 0.f
                               : prob_of(load_logit<DT>(p.logits, base + my_id[h]), soft, mx, inv);
    float f = c.routed_scaling_factor;
    if (c.norm_topk_prob) {
        const float total = warp_sum(my_p[0] + my_p[1]);
        // under 2^-60 of the row's unit the p that fp32 holds are too small
        wide |= __any_sync(~0u, my_id[0] >= 0) && !(total > 8.7e-19f);
        f = total > 0.f ? __fdividef(f, total) : 0.f;
    }
    if (wide || close) return true;
#pragma unroll
    for (int h = 0; h < 2; ++h)
        if (lane + 32 * h < k) {
            p.ids[(size_t)row * k + lane + 32 * h] = my_id[h];
            p.wts[(size_t)row * k + lane + 32 * h] = my_p[h] * f;
        }
    return false;
}

template <int VPT, int DT>
__global__ void __launch_bounds__(warps_of(VPT) * 32) route_topk_kernel(const Args q) {
    constexpr int kWarps = warps_of(VPT);
    __shared__ float sm[kWarps][VPT * 32];
    __shared__ double key[VPT * 32], prob[VPT * 32], sums[kWarps];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int row = blockIdx.x * kWarps + warp;
    const bool wide = row < q.p.rows && route_row<VPT, DT>(q, row, lane, sm[warp]);
    if (!__syncthreads_or(wide)) return;
    // by every warp in turn, so that all threads know whose row it is
    for (int w = 0; w < kWarps; ++w)
        if (__syncthreads_or(wide && warp == w))
            route_row_wide<DT>(q, blockIdx.x * kWarps + w, lane, warp, w, key, prob, sums);
}

template <int DT>
cudaError_t launch_typed(const Args &q, cudaStream_t st) {
    const int E = q.p.c.num_experts, w = E <= 512 ? 8 : 4, grid = (q.p.rows + w - 1) / w;
    if (E <= 128) route_topk_kernel<4, DT><<<grid, w * 32, 0, st>>>(q);
    else if (E <= 256) route_topk_kernel<8, DT><<<grid, w * 32, 0, st>>>(q);
    else if (E <= 512) route_topk_kernel<16, DT><<<grid, w * 32, 0, st>>>(q);
    else route_topk_kernel<32, DT><<<grid, w * 32, 0, st>>>(q);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_route_topk(const RouteParams &p, cudaStream_t st) {
    Args q{p, p.c.num_experts / p.c.groups, 0, 0};
    while ((2 << q.lane_shift) * p.c.groups <= 32) ++q.lane_shift;
    q.div = ((1u << 20) + q.size - 1) / q.size;
    switch (p.c.dtype) {
        case MOEOP_BF16: return launch_typed<MOEOP_BF16>(q, st);
        case MOEOP_FP16: return launch_typed<MOEOP_FP16>(q, st);
        default: return launch_typed<MOEOP_FP32>(q, st);
    }
}

}  // namespace op
}  // namespace moe

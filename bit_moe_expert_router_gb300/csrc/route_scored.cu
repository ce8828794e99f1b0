// Routing by scores: softmax or sigmoid of the router's logits, a bias that moves
// the choice but not the weights, groups of experts of which some are kept,
// and the k best experts.
//
// Per token: s_e = softmax_e(x) or 1 / (1 + e^-x); r_e = s_e + bias_e, or x_e itself without a bias
// (s grows with x, so the order is the same); a group's value is its largest r, or the sum of its two
// largest (of s where there is no bias); of the groups the best, of their experts the k best by (r desc,
// index asc); w = s of those, divided by their sum if asked for, times the scale.
//
// Which experts are chosen is decided as in exact arithmetic on the given logits and fp32 biases: the
// choice is made in fp32, and where two candidates whose order matters lie closer together than the error
// bounds below, the token is taken again in fp64 (one in some hundred to a thousand tokens with a bias;
// without one the logits themselves are compared).
//
// Bound: HBM for many tokens (the logits, read once), in fact the instructions of a warp per token.  A lane
// holds J consecutive experts of one group (32 / groups lanes a group), so lane order is expert order.  It
// sorts them once, by a network on 32-bit keys whose low bits are the expert's place in the lane; the k best
// of the warp are then k rounds of a warp-wide maximum and one ballot, in which the winner moves its list up.
// 8192 tokens of 256 experts, 8 of 4 groups of 8, sigmoid with a bias: 11.4 us, where the logits alone take 1.3 at HBM's rate;
// without groups 9.7, without a bias 7.5.  64 tokens of 160 experts 3.2 us, 4 of 512 with 10 chosen 4.0: the launch and the
// chain of a warp's steps.
//
// Errors, with u = 2^-24 and d = |x - c|, c the largest logit for softmax and 0 for the sigmoid.  A fast exponential is off by 2^-22 of
// itself and, from the argument's three roundings, 1.4e-7 d.  The softmax's sum of them is off by the mean of that over its terms, in which d
// is ln E at most (the entropy), and (log2 J + 5) u for the additions, pairs of pairs: kSum.  A fast score is off by kFast times the largest score at
// most, its own exponential, the quotient and the product counted (the part in d is largest at d = 0, as e^-d falls faster than d grows; a
// sigmoid has no sum and stays below).  For the experts on the list s is computed anew with expf and a correctly rounded
// quotient, off by 4e-7 s and, for softmax, by d u and kSum, as it has the same sum: that factor is the same for all experts
// of a token, but does not cancel against a bias.  Below the smallest normal number fp32 is off by more than a part of s; 1e-37 covers that.
#include <algorithm>

#include "attention_common.cuh"
#include "route_scored.h"

namespace moe {
namespace {

constexpr int kWarps = 4;  // tokens of a block

// An order-preserving key: absent 0, then NaN, then the numbers (-0 and 0 the same).
template <int MAXJ>
__device__ __forceinline__ uint32_t key_of(float v) {
    if (v != v) return 2 * MAXJ;
    const uint32_t u = __float_as_uint(v + 0.0f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float key_number(uint32_t k) { return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k); }
__device__ __forceinline__ unsigned long long key_of(double v) {
    if (v != v) return 1;
    const unsigned long long u = __double_as_longlong(v + 0.0);
    return (u >> 63) ? ~u : (u | 1ull << 63);
}

__device__ __forceinline__ float widen(uint32_t h, int dtype) { return dtype == 1 ? __uint_as_float(h << 16) : Elem<__half>::unpack(h).x; }
__device__ __forceinline__ float logit(const RouteScoredArgs& a, int64_t at) {
    if (a.dtype == 0) return __ldg(static_cast<const float*>(a.logits) + at);
    return widen(__ldg(static_cast<const unsigned short*>(a.logits) + at), a.dtype);
}

// The place of a lane: its group, its first expert and how many it has.
struct Lane {
    int group, first, n;
    __device__ __forceinline__ Lane(const RouteScoredArgs& a) {
        const int lane = threadIdx.x & 31, sub = lane & ((1 << a.lanes_log2) - 1);
        group = lane >> a.lanes_log2;
        first = group * a.group_size + sub * a.per_lane;
        n = min(max(a.group_size - sub * a.per_lane, 0), a.per_lane);
    }
};

// What one expert's choice goes by in fp64: s with its bias if there is one; top, sum: of the softmax (sum 1 where the scores are
// only compared with one another).
__device__ __forceinline__ double exact_score(const RouteScoredArgs& a, int64_t row, int e, double top, double sum) {
    const double x = logit(a, row + e);
    const double s = a.sigmoid ? 1.0 / (1.0 + exp(-x)) : a.bias ? exp(x - top) / sum : exp(x - top);
    return a.bias ? s + static_cast<double>(__ldg(a.bias + e)) : s;
}
__device__ __noinline__ double exact_sum(const RouteScoredArgs& a, int64_t row, const Lane& me, double top) {
    double sum = 0.0;
#pragma unroll 1
    for (int i = 0; i < me.n; ++i) {
        const double x = logit(a, row + me.first + i);
        if (x == x) sum += exp(x - top);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
    return sum;
}

// The whole choice in fp64 (of which a warp does little at a time: about 10 us for 8 experts a lane), where the kernel's shorter
// ways do not settle it: expert of rank `lane` (lane < k).
template <int MAXJ>
__device__ __noinline__ int choose_exactly(const RouteScoredArgs& a, int64_t row) {
    const int lane = threadIdx.x & 31, lanes = 1 << a.lanes_log2;
    const Lane me(a);
    const bool softmax = a.sigmoid == 0, groups = a.topk_groups < a.n_groups;
    double top = -INFINITY, sum = 1.0;
    if (softmax) {
        float m = -INFINITY;
        for (int i = 0; i < me.n; ++i) m = fmaxf(m, logit(a, row + me.first + i));
#pragma unroll
        for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
        top = m;
        if (a.bias) sum = exact_sum(a, row, me, top);
    }
    unsigned long long key[MAXJ];
    double b1 = -INFINITY, b2 = -INFINITY;  // the two largest
#pragma unroll
    for (int i = 0; i < MAXJ; ++i) {
        key[i] = 0;
        if (i >= me.n) continue;
        const double x = logit(a, row + me.first + i);
        double r = x, g = x;
        if (a.bias || (groups && a.group_top == 2)) {
            g = exact_score(a, row, me.first + i, top, sum);
            if (a.bias) r = g;
        }
        key[i] = key_of(r);
        if (g > b1) b2 = b1, b1 = g;
        else if (g > b2) b2 = g;
    }
    if (groups) {
        for (int o = 1; o < lanes; o <<= 1) {
            const double o1 = __shfl_xor_sync(~0u, b1, o), o2 = __shfl_xor_sync(~0u, b2, o);
            b2 = fmax(fmin(b1, o1), fmax(b2, o2));
            b1 = fmax(b1, o1);
        }
        const unsigned long long g = key_of(a.group_top == 2 ? b1 + b2 : b1);
        int better = 0;
        for (int i = 0; i < a.n_groups; ++i) {
            const unsigned long long o = __shfl_sync(~0u, g, i * lanes);
            better += o > g || (o == g && i < me.group);
        }
        if (better >= a.topk_groups)
#pragma unroll
            for (int i = 0; i < MAXJ; ++i) key[i] = 0;
    }
    int mine = 0;
    for (int r = 0; r < a.k; ++r) {
        unsigned long long best = 0;
        int at = 0;
#pragma unroll
        for (int i = 0; i < MAXJ; ++i)
            if (key[i] > best) best = key[i], at = i;
        unsigned long long m = best;
#pragma unroll
        for (int o = 16; o; o >>= 1) m = max(m, __shfl_xor_sync(~0u, m, o));
        const int win = __ffs(__ballot_sync(~0u, best == m)) - 1;
        const int e = __shfl_sync(~0u, me.first + at, win);
        if (lane == r) mine = e;
        if (lane == win)
#pragma unroll
            for (int i = 0; i < MAXJ; ++i)
                if (i == at) key[i] = 0;
    }
    return mine;
}

__device__ __forceinline__ float sigmoid_of(float x) {
    const float t = expf(-fabsf(x));
    return __fdiv_rn(x >= 0.f ? 1.f : t, 1.f + t);  // (NaN of a NaN, by t)
}

// The sum of f(FROM) to f(FROM + N - 1), pairs of pairs: log2 N roundings deep.  (One after another they are N, and more pairs of experts
// come closer than the sum's bound: 8192 tokens of 1024 experts, 16 chosen, with a softmax and a bias 62.9 us, so 57.9.)
template <int FROM, int N, typename F>
__device__ __forceinline__ float pair_sum(const F& f) {
    if constexpr (N == 1) return f(FROM);
    else return pair_sum<FROM, N / 2>(f) + pair_sum<FROM + N / 2, N / 2>(f);
}

// Sorts a lane's keys, the largest first: odd-even merges of runs of P, the comparisons K apart.  (The steps are template arguments, because
// as loops of one another they leave 16 and 32 keys in local memory: 8192 tokens of 512
// experts, 10 of them chosen, 21.7 us, so 14.8; of 1024 experts 55 and 28.6.)
template <int MAXJ, int P = 1, int K = 1>
__device__ __forceinline__ void sort_down(uint32_t (&s)[MAXJ]) {
    if constexpr (P < MAXJ) {
#pragma unroll
        for (int i = K % P; i + K < MAXJ; ++i)
            if ((i - K % P) % (2 * K) < K && i / (2 * P) == (i + K) / (2 * P)) {
                const uint32_t lo = min(s[i], s[i + K]);
                s[i] = max(s[i], s[i + K]);
                s[i + K] = lo;
            }
        if constexpr (K > 1) sort_down<MAXJ, P, K / 2>(s);
        else sort_down<MAXJ, 2 * P, 2 * P>(s);
    }
}

// The bounds on registers, blocks an SM: 8192 tokens of 256 experts in groups with 8 11.0 us, with 10 12.1, with 6 11.4; of 512 with 7 16.7, with 5
// 17.2, of 1024 with 4 28.6, with 3 33.6.
template <int MAXJ>
__global__ void __launch_bounds__(32 * kWarps, MAXJ <= 8 ? 8 : MAXJ == 16 ? 7 : 4) route_scored_kernel(const __grid_constant__ RouteScoredArgs a) {
    constexpr int kBits = MAXJ == 1 ? 0 : MAXJ == 2 ? 1 : MAXJ == 4 ? 2 : MAXJ == 8 ? 3 : MAXJ == 16 ? 4 : 5;
    // the errors of the head of this file; ln E <= ln (32 MAXJ) = 3.47 + 0.694 kBits
    constexpr float kSum = 2.4e-7f + 1.4e-7f * (3.5f + 0.7f * kBits) + (kBits + 5) * 6e-8f, kFast = kSum + 5.4e-7f;
    const int lane = threadIdx.x & 31, lanes = 1 << a.lanes_log2;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    wait_for_stream();
    if (t >= a.T) return;
    const int64_t row = t * a.stride;
    const Lane me(a);
    const bool softmax = a.sigmoid == 0, groups = a.topk_groups < a.n_groups;
    float x[MAXJ];
    if (MAXJ >= 4 && a.vec) {
        if (a.dtype == 0) {
#pragma unroll
            for (int i = 0; i + 3 < MAXJ; i += 4) {
                const float4 v = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(a.logits) + row + me.first + i));
                x[i] = v.x, x[i + 1] = v.y, x[i + 2] = v.z, x[i + 3] = v.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i + 3 < MAXJ; i += 4) {
                const uint2 v = __ldg(reinterpret_cast<const uint2*>(static_cast<const unsigned short*>(a.logits) + row + me.first + i));
                x[i] = widen(v.x & 0xFFFFu, a.dtype), x[i + 1] = widen(v.x >> 16, a.dtype);
                x[i + 2] = widen(v.y & 0xFFFFu, a.dtype), x[i + 3] = widen(v.y >> 16, a.dtype);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < MAXJ; ++i) x[i] = i < me.n ? logit(a, row + me.first + i) : -INFINITY;
    }
    // what the choice is made by: r (with a bias or for sums), else x
    const bool scores = a.bias || (groups && a.group_top == 2) || (softmax && !a.renormalise);
    float r[MAXJ], m = 0.f, sum = 1.f, big = 1.f;  // big: no score is larger
    if (softmax) {
        m = x[0];
#pragma unroll
        for (int i = 1; i < MAXJ; ++i) m = fmaxf(m, x[i]);
#pragma unroll
        for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
    }
    if (scores) {
        if (softmax) {
#pragma unroll
            for (int i = 0; i < MAXJ; ++i) r[i] = exp2_fast((x[i] - m) * kLog2e);
            sum = pair_sum<0, MAXJ>([&](int i) { return i < me.n && x[i] == x[i] ? r[i] : 0.f; });
#pragma unroll
            for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
            big = __fdividef(1.f, sum);
#pragma unroll
            for (int i = 0; i < MAXJ; ++i) r[i] *= big;
        } else {
#pragma unroll
            for (int i = 0; i < MAXJ; ++i) {
                const float e = exp2_fast(-fabsf(x[i]) * kLog2e);
                r[i] = __fdividef(x[i] >= 0.f ? 1.f : e, 1.f + e);
            }
        }
        if (a.bias) {
            if (MAXJ >= 4 && a.vec) {
#pragma unroll
                for (int i = 0; i + 3 < MAXJ; i += 4) {
                    const float4 v = __ldg(reinterpret_cast<const float4*>(a.bias + me.first + i));
                    r[i] += v.x, r[i + 1] += v.y, r[i + 2] += v.z, r[i + 3] += v.w;
                }
            } else {
#pragma unroll
                for (int i = 0; i < MAXJ; ++i)
                    if (i < me.n) r[i] += __ldg(a.bias + me.first + i);
            }
        }
    }
    bool doubt = false, kept = true, settled = true;  // settled: the groups are
    double esum = 0.0;                                // the softmax's sum in fp64, once it is needed
    if (groups) {
        const bool by_r = a.bias || a.group_top == 2;
        float b1 = -INFINITY, b2 = -INFINITY;
#pragma unroll
        for (int i = 0; i < MAXJ; ++i) {
            const float g = i < me.n ? fmaxf(by_r ? r[i] : x[i], -INFINITY) : -INFINITY;  // (of a NaN and b1 the smaller would be b1, twice)
            b2 = fmaxf(b2, fminf(b1, g));
            b1 = fmaxf(b1, g);
        }
        for (int o = 1; o < lanes; o <<= 1) {
            const float o1 = __shfl_xor_sync(~0u, b1, o), o2 = __shfl_xor_sync(~0u, b2, o);
            b2 = fmaxf(fminf(b1, o1), fmaxf(b2, o2));
            b1 = fmaxf(b1, o1);
        }
        const uint32_t g = key_of<MAXJ>(a.group_top == 2 ? b1 + b2 : b1);
        int better = 0;
        for (int i = 0; i < a.n_groups; ++i) {
            const uint32_t o = __shfl_sync(~0u, g, i * lanes);
            better += o > g || (o == g && i < me.group);
        }
        kept = better < a.topk_groups;
        if (by_r) {
            const float in = key_number(__reduce_min_sync(~0u, kept ? g : ~0u)), out = key_number(__reduce_max_sync(~0u, kept ? 0u : g));
            const float size = __uint_as_float(__reduce_max_sync(~0u, __float_as_uint(fabsf(b1) + fabsf(b2))));
            // two scores each: the sum's and the quotient's factor moves their difference by 2 (kSum + 2.4e-7) big at most, the rest four
            // scores by 3e-7 big; size: the roundings of the additions
            static_assert(2 * (kSum + 2.4e-7f) + 4 * 3e-7f < 1e-5f, "the border's width");
            const float near = 1e-5f * big + 5e-7f * size;
            if (!(in - out > near)) {
                // The groups' values in fp64, of the experts that make them: the largest, and the largest of the others.  Where the next
                // one is too close to the last of these in a group at the border, the long way.
                auto largest = [&](int but, float& v) {  // of the group but expert `but`: the first
                    int e = 1 << 30;
                    v = -INFINITY;
#pragma unroll
                    for (int i = 0; i < MAXJ; ++i)
                        if (i < me.n && me.first + i != but && r[i] > v) v = r[i], e = me.first + i;
                    for (int o = 1; o < lanes; o <<= 1) {
                        const float ov = __shfl_xor_sync(~0u, v, o);
                        const int oe = __shfl_xor_sync(~0u, e, o);
                        if (ov > v || (ov == v && oe < e)) v = ov, e = oe;
                    }
                    return e;
                };
                float v1, v2, v3 = -INFINITY;
                const int e1 = largest(-1, v1), e2 = largest(e1, v2);
                if (a.group_top == 2) {  // (the third: whatever is below the second and not it)
#pragma unroll
                    for (int i = 0; i < MAXJ; ++i)
                        if (i < me.n && me.first + i != e1 && me.first + i != e2) v3 = fmaxf(v3, r[i]);
                    for (int o = 1; o < lanes; o <<= 1) v3 = fmaxf(v3, __shfl_xor_sync(~0u, v3, o));
                }
                const float value = key_number(g);
                const bool border = !(value - out > 4.f * near) && !(in - value > 4.f * near);
                settled = lanes >= a.group_top && !__any_sync(~0u, border && !((a.group_top == 2 ? v2 - v3 : v1 - v2) > near));
                if (settled) {
                    if (softmax && a.bias) esum = exact_sum(a, row, me, m);
                    const int sub = lane & (lanes - 1), e = sub == 0 ? e1 : e2;
                    double x = -INFINITY;
                    if (sub < a.group_top && e < (1 << 30)) x = exact_score(a, row, e, m, esum);
                    if (a.group_top == 2) x += __shfl_xor_sync(~0u, x, 1);
                    const unsigned long long own = __shfl_sync(~0u, key_of(x), lane - sub);
                    better = 0;
                    for (int i = 0; i < a.n_groups; ++i) {
                        const unsigned long long o = __shfl_sync(~0u, own, i * lanes);
                        better += o > own || (o == own && i < me.group);
                    }
                    kept = better < a.topk_groups;
                }
            }
        }
    }
    uint32_t s[MAXJ];
#pragma unroll
    for (int i = 0; i < MAXJ; ++i) s[i] = i < me.n && kept ? (key_of<MAXJ>(a.bias ? r[i] : x[i]) & ~(MAXJ - 1u)) | (MAXJ - 1 - i) : 0u;
    sort_down<MAXJ>(s);
    int e = -1;           // of rank `lane`, and of the one behind the last
    uint32_t bucket = 0;  // of its key
    const int places = min(a.k + 1, 32);
    for (int q = 0; q < places; ++q) {
        const uint32_t own = s[0] >> kBits, best = __reduce_max_sync(~0u, own);
        const int win = __ffs(__ballot_sync(~0u, own == best)) - 1;
        const int we = __shfl_sync(~0u, me.first + (MAXJ - 1 - static_cast<int>(s[0] & (MAXJ - 1u))), win);
        if (lane == q) {
            e = best ? we : -1;
            bucket = best;
        }
        if (lane == win) {
#pragma unroll
            for (int i = 0; i + 1 < MAXJ; ++i) s[i] = s[i + 1];
            s[MAXJ - 1] = 0;
        }
    }
    // (with k = 32 the best of the rest has no lane)
    const uint32_t rest = a.k == 32 ? __reduce_max_sync(~0u, s[0] >> kBits) : 0u;

    float xe = -INFINITY, be = 0.f, se = 0.f;
    auto score = [&]() {
        xe = -INFINITY, be = 0.f, se = 0.f;
        if (e < 0) return;
        xe = logit(a, row + e);
        if (a.bias) be = __ldg(a.bias + e);
        se = softmax ? __fdiv_rn(expf(xe - m), sum) : sigmoid_of(xe);
    };
    score();
    const int next_e = __shfl_down_sync(~0u, e, 1);
    const bool last = lane == a.k - 1;
    if (a.bias) {
        // Each place against the next: what stands in the wrong order is close to its neighbour; what should be on the list and
        // is not has a key no better than the first one's behind it.
        constexpr float kCut = (MAXJ + 1) * 1.2e-7f;  // the keys' low bits, and the sums with a bias
        const float far = fminf(fabsf(xe - m), 128.f);  // (from 104 on s is zero)
        const float re = se + be, err = se * (softmax ? 4e-7f + kSum + 6e-8f * far : 4e-7f) + 1.2e-7f * fabsf(re) + 1e-37f;
        const float loose = kFast * big + se * (2e-6f + 1.2e-7f * far) + kCut * fabsf(re);
        float up = __shfl_down_sync(~0u, re + (lane == a.k ? loose : err), 1);
        const float next_x = __shfl_down_sync(~0u, xe, 1), next_b = __shfl_down_sync(~0u, be, 1);
        bool there = next_e >= 0;
        if (lane == 31) {
            there = rest != 0;
            up = key_number((rest + 1) << kBits);
            up += kFast * big + 1.2e-7f * fabsf(up);
        }
        const bool same = !last && next_x == xe && next_b == be && next_e > e;
        doubt |= lane < a.k && there && !same && !(re - err > up);
    } else if (a.dtype == 0) {
        // (16-bit logits in one bucket are the same)
        const uint32_t next = __shfl_down_sync(~0u, bucket, 1);
        const float next_x = __shfl_down_sync(~0u, xe, 1);
        const bool one = bucket == (lane == 31 ? rest : next) && bucket != 0;
        doubt |= lane < a.k && one && (last || !(xe > next_x || (xe == next_x && next_e > e)));
    }
    if (__any_sync(~0u, doubt || !settled)) {
        // What could be on the list goes to a lane each, is taken in fp64 and put in order.
        int n = 32;
        if (settled && a.k < 24) {
            const float low = __shfl_sync(~0u, a.bias ? se + be : xe, a.k - 1);
            // (nothing with a key below it can be among the best: two fast scores' errors and the difference of a fast and a listed one)
            static_assert(2 * kFast + 1e-6f < 1e-5f, "the limit's width");
            const float limit = a.bias ? low - (1e-5f * big + 4.f * MAXJ * 1.2e-7f * fabsf(low)) : low;
            for (n = a.k + 1; n < 32; ++n) {  // the lanes' lists go on
                const uint32_t own = s[0] >> kBits, best = __reduce_max_sync(~0u, own);
                if (best == 0 || !(key_number((best << kBits) + (MAXJ - 1)) >= limit)) break;
                const int win = __ffs(__ballot_sync(~0u, own == best)) - 1;
                const int we = __shfl_sync(~0u, me.first + (MAXJ - 1 - static_cast<int>(s[0] & (MAXJ - 1u))), win);
                if (lane == n) e = we;
                if (lane == win) {
#pragma unroll
                    for (int i = 0; i + 1 < MAXJ; ++i) s[i] = s[i + 1];
                    s[MAXJ - 1] = 0;
                }
            }
        }
        int got;
        if (n < 32) {
            if (softmax && a.bias && esum == 0.0) esum = exact_sum(a, row, me, m);
            unsigned long long key = 0;
            if (e >= 0) key = key_of(a.bias ? exact_score(a, row, e, m, esum) : static_cast<double>(logit(a, row + e)));
            int rank = 0;
            for (int i = 0; i < n; ++i) {
                const unsigned long long o = __shfl_sync(~0u, key, i);
                const int oe = __shfl_sync(~0u, e, i);
                rank += o > key || (o == key && oe < e);
            }
            __shared__ int places[kWarps][32];
            int* place = places[threadIdx.x >> 5];
            if (lane < n && e >= 0) place[rank] = e;
            __syncwarp();
            got = lane < a.k ? place[lane] : -1;
        } else {
            got = choose_exactly<MAXJ>(a, row);
        }
        e = lane < a.k ? got : -1;
        score();
    }

    if (lane >= a.k) xe = -INFINITY, se = 0.f;
    float w = se;
    if (a.renormalise) {
        float top = xe;
#pragma unroll
        for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
        // relative to the largest logit where the scores themselves could vanish (a sigmoid far below zero is an exponential)
        if (softmax || top < -60.f) w = lane < a.k ? expf(xe - top) : 0.f;
        float all = w;
#pragma unroll
        for (int o = 16; o; o >>= 1) all += __shfl_xor_sync(~0u, all, o);
        w = __fdiv_rn(w, all);
    }
    if (lane < a.k) {
        a.ids[t * a.k + lane] = e;
        a.wts[t * a.k + lane] = w * a.scale;
    }
}

template <int MAXJ>
cudaError_t launch_j(RouteScoredArgs a, cudaStream_t st) {
    // four at a time where every lane is full and begins on a multiple of four
    a.vec = a.per_lane == MAXJ && a.group_size == MAXJ << a.lanes_log2 && a.stride % 4 == 0;
    return launch_in_stream(route_scored_kernel<MAXJ>, dim3(static_cast<unsigned>((a.T + kWarps - 1) / kWarps)), 32 * kWarps, 0, 1, st, a);
}

}  // namespace

cudaError_t launch_route_scored(RouteScoredArgs a, cudaStream_t st) {
    a.lanes_log2 = 5;
    while ((a.n_groups << a.lanes_log2) > 32) --a.lanes_log2;
    a.group_size = static_cast<int>(a.E) / a.n_groups;
    a.per_lane = (a.group_size + (1 << a.lanes_log2) - 1) >> a.lanes_log2;
    if (a.per_lane <= 1) return launch_j<1>(a, st);
    if (a.per_lane <= 2) return launch_j<2>(a, st);
    if (a.per_lane <= 4) return launch_j<4>(a, st);
    if (a.per_lane <= 8) return launch_j<8>(a, st);
    if (a.per_lane <= 16) return launch_j<16>(a, st);
    return launch_j<32>(a, st);
}

}  // namespace moe

// Norms of queries and keys per head, rotation by position, and the store of
// keys and values into the paged cache: one kernel over the rows of the fused
// projection.
//
// Per (token, head): y = x rsqrt(mean(x^2) + eps) (w + offset) for queries and
// keys, then the first R components are turned in pairs by the position's
// angle, (a, b) -> (a c - b s, b c + a s); values are copied.  All of it is
// fp32 with one rounding at the store.
//
// Bound: HBM, each input element read once and each output element written
// once.  A head of D components is D / 8 lanes' 16-byte loads, padded to 8, 16
// or 32 lanes, so a warp carries 4, 2 or 1 heads and a norm is a reduction of
// 3 to 5 shuffles.  A rotated pair lies in one lane (interleaved) or in two
// lanes whose distance is the same for the whole head (halves), which costs
// four shuffles of the packed elements.
#include <algorithm>

#include "attention_common.cuh"

namespace moe {
namespace {

constexpr int kAppendThreads = 128;
constexpr int kRoundsPerWarp = 8;
constexpr int64_t kManyRounds = 64 * 152;

// The sequence that token t belongs to (its index b with q_start[b] <= t < q_start[b + 1]), or -1.
// A decoding batch has one token per sequence, so b = t is tried first; else a 32-way search.
__device__ __forceinline__ int find_seq(const KvArgs& a, int t) {
    const int lane = threadIdx.x & 31;
    const int guess = min(t, a.n_seqs - 1);
    if (__ldg(a.q_start + guess) <= t && t < __ldg(a.q_start + guess + 1)) return guess;
    int lo = 0, n = a.n_seqs;  // the first b of [lo, lo + n) with q_start[b + 1] > t
    while (n > 0) {
        const int step = (n + 31) / 32;
        const int j = min((lane + 1) * step, n) - 1;
        const unsigned past = __ballot_sync(~0u, __ldg(a.q_start + lo + j + 1) > t);
        if (!past) return -1;
        const int f = __ffs(past) - 1;
        const int at = f * step;
        n = min(step, n - at);
        lo += at;
        if (step == 1) break;
    }
    return __ldg(a.q_start + lo) <= t ? lo : -1;
}

// How the rotation finds a component's partner and its angle.
enum Turn {
    kPairs,    // neighbours, whole 8-component chunks rotated: the partner is in the lane
    kHalves,   // halves of whole chunks: the partner is in a lane at a fixed distance
    kAnywhere  // either layout, a rotated width that cuts chunks: partners are read again (they are in L1)
};

// A warp takes rounds of 32 / LPH heads, all of one kind (queries, keys or values), of one token: rounds
// [first, last) of the token's.  What a head's norm weights and angles come to is the same for every round of
// a kind, so they are put together once: component e of the result is r (x_e a_e + x_p b_e) with its
// partner p, a_e = w_e cos, b_e = -+ w_p sin (a_e = w_e past the rotated part), r the norm's factor.
template <typename T, int LPH, int BATCH, Turn TURN>
__global__ void __launch_bounds__(kAppendThreads, BATCH > 1 ? 6 : 4) kv_append_kernel(const AppendArgs a, int rounds_per_warp) {
    constexpr int kPerWarp = 32 / LPH;  // heads of a round
    const int lane = threadIdx.x & 31;
    const int t = blockIdx.x * (kAppendThreads / 32) + (threadIdx.x >> 5);
    if (t >= a.kv.n_tokens) return;
    const int e0 = (lane % LPH) * 8;  // this lane's first component
    const bool on = e0 < a.kv.d;
    const int rq = (a.kv.hq + kPerWarp - 1) / kPerWarp, rk = (a.kv.hkv + kPerWarp - 1) / kPerWarp;
    const int last = min(static_cast<int>(blockIdx.y + 1) * rounds_per_warp, rq + 2 * rk);
    int i = blockIdx.y * rounds_per_warp;
    int kind, end, begin, heads;  // of the rounds that run: [begin, end) and `heads` are the kind's
    const T* src;                 // this lane's chunk of the kind's head lane / LPH
    int64_t src_step;             // from one round to the next
    auto enter = [&]() {
        kind = i < rq ? 0 : i < rq + rk ? 1 : 2;
        begin = kind == 0 ? 0 : kind == 1 ? rq : rq + rk;
        end = min(last, kind == 0 ? rq : begin + rk);
        heads = kind == 0 ? a.kv.hq : a.kv.hkv;
        const int64_t hs = kind == 0 ? a.q_hs : kind == 1 ? a.k_hs : a.v_hs;
        const int64_t ts = kind == 0 ? a.q_ts : kind == 1 ? a.k_ts : a.v_ts;
        src = static_cast<const T*>(kind == 0 ? a.q : kind == 1 ? a.k : a.v) + t * ts + (lane / LPH) * hs + e0;
        src_step = kPerWarp * hs;
    };
    uint4 raw[BATCH];
    auto load = [&]() {
#pragma unroll
        for (int x = 0; x < BATCH; ++x) {
            const int n = i + x - begin;
            raw[x] = make_uint4(0, 0, 0, 0);
            if (i + x < end && on && n * kPerWarp + lane / LPH < heads) raw[x] = *reinterpret_cast<const uint4*>(src + n * src_step);
        }
    };
    enter();
    load();  // under way while the token's place is looked up

    const int b = find_seq(a.kv, t);
    int pos = -1;
    if (b >= 0) {  // q_start[b] <= t < q_start[b + 1]; entries past the tokens count as their end
        const int stop = min(__ldg(a.kv.q_start + b + 1), a.kv.n_tokens);
        pos = max(__ldg(a.kv.kv_len + b), 0) - (stop - t);
    }
    const int turn = a.positions && pos >= 0 ? __ldg(a.positions + t) : pos;
    if (a.rot > 0 && (turn < 0 || turn >= a.table_rows)) pos = -1;
    int64_t row = 0;
    int id = -1;
    if (pos >= 0 && pos < a.kv.cap) {
        const int p = static_cast<unsigned>(pos) / static_cast<unsigned>(a.kv.page);
        id = page_id(a.kv, b, p);
        row = pos - p * a.kv.page;
    }
    const int half = a.rot / 2;
    const bool turned = pos >= 0 && e0 < a.rot && on;
    const bool low = e0 < half;  // (kHalves)
    const int away = low ? half : -half;
    const float* tab = a.cos_sin + static_cast<int64_t>(turn) * a.rot;

    while (i < last) {
        float ca[8], cb[8];
        const float* weight = kind == 0 ? a.q_weight : a.k_weight;
        T* dst;
        int64_t dst_step;
        if (kind == 0) {
            dst = static_cast<T*>(a.q_out) + t * a.o_ts + (lane / LPH) * a.o_hs + e0;
            dst_step = kPerWarp * a.o_hs;
        } else {
            const int64_t hs = kind == 1 ? a.kv.k_hs : a.kv.v_hs;
            dst = static_cast<T*>(kind == 1 ? a.kv.k : a.kv.v) + max(id, 0) * (kind == 1 ? a.kv.k_ps : a.kv.v_ps) +
                  row * (kind == 1 ? a.kv.k_rs : a.kv.v_rs) + (lane / LPH) * hs + e0;
            dst_step = kPerWarp * hs;
        }
        const bool store = on && (kind == 0 || id >= 0);
        if (kind != 2) {
            auto load8 = [](const float* p, float* v) {
                const float4 x = __ldg(reinterpret_cast<const float4*>(p)), y = __ldg(reinterpret_cast<const float4*>(p) + 1);
                v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w, v[4] = y.x, v[5] = y.y, v[6] = y.z, v[7] = y.w;
            };
            float w[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j] = 1.f;
            if (weight && on) {
                load8(weight + e0, w);
#pragma unroll
                for (int j = 0; j < 8; ++j) w[j] += a.weight_offset;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) ca[j] = w[j], cb[j] = 0.f;
            if (turned) {
                if constexpr (TURN == kPairs) {
                    const float4 c = __ldg(reinterpret_cast<const float4*>(tab + e0 / 2)), s = __ldg(reinterpret_cast<const float4*>(tab + half + e0 / 2));
                    const float cs[4] = {c.x, c.y, c.z, c.w}, sn[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        ca[2 * j] = w[2 * j] * cs[j];
                        cb[2 * j] = -w[2 * j + 1] * sn[j];
                        ca[2 * j + 1] = w[2 * j + 1] * cs[j];
                        cb[2 * j + 1] = w[2 * j] * sn[j];
                    }
                } else if constexpr (TURN == kHalves) {
                    float c[8], s[8], wp[8];
                    load8(tab + (low ? e0 : e0 - half), c);
                    load8(tab + (low ? e0 : e0 - half) + half, s);
#pragma unroll
                    for (int j = 0; j < 8; ++j) wp[j] = 1.f;
                    if (weight) {
                        load8(weight + e0 + away, wp);
#pragma unroll
                        for (int j = 0; j < 8; ++j) wp[j] += a.weight_offset;
                    }
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        ca[j] = w[j] * c[j];
                        cb[j] = (low ? -wp[j] : wp[j]) * s[j];
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const int e = e0 + j;
                        if (e >= a.rot) continue;
                        const bool lo = a.interleaved ? (j & 1) == 0 : e < half;
                        const int p = a.interleaved ? e ^ 1 : lo ? e + half : e - half;
                        const int x = a.interleaved ? e / 2 : lo ? e : e - half;
                        const float wp = weight ? __ldg(weight + p) + a.weight_offset : 1.f;
                        ca[j] = w[j] * __ldg(tab + x);
                        cb[j] = (lo ? -wp : wp) * __ldg(tab + half + x);
                    }
                }
            }
        }
        for (;;) {
#pragma unroll
            for (int x = 0; x < BATCH; ++x) {
                const int n = i + x - begin;
                const bool in = i + x < end && n * kPerWarp + lane / LPH < heads;
                uint4 out = raw[x];  // values go as they came
                if (kind != 2) {
                    const uint32_t w4[4] = {raw[x].x, raw[x].y, raw[x].z, raw[x].w};
                    float v[8], y[8];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 f = Elem<T>::unpack(w4[j]);
                        v[2 * j] = f.x;
                        v[2 * j + 1] = f.y;
                    }
                    float r = 1.f;
                    if (weight) {
                        float sum = 0.f;
#pragma unroll
                        for (int j = 0; j < 8; ++j) sum += v[j] * v[j];
#pragma unroll
                        for (int o = LPH / 2; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
                        r = rsqrtf(sum * a.inv_d + a.eps);
                    }
                    if constexpr (TURN == kPairs) {
#pragma unroll
                        for (int j = 0; j < 8; ++j) y[j] = v[j ^ 1];
                    } else if constexpr (TURN == kHalves) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float2 f = Elem<T>::unpack(__shfl_sync(~0u, w4[j], lane + away / 8));
                            y[2 * j] = f.x;
                            y[2 * j + 1] = f.y;
                        }
                    } else {
                        const T* head = src + n * src_step - e0;
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const int e = e0 + j;
                            y[j] = in && turned && e < a.rot ? static_cast<float>(head[a.interleaved ? e ^ 1 : e < half ? e + half : e - half]) : 0.f;
                        }
                    }
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] *= ca[j];
                    if (turned) {
#pragma unroll
                        for (int j = 0; j < 8; ++j) v[j] += y[j] * cb[j];
                    }
                    if (weight) {
#pragma unroll
                        for (int j = 0; j < 8; ++j) v[j] *= r;
                    }
                    out = make_uint4(Elem<T>::pack(v[0], v[1]), Elem<T>::pack(v[2], v[3]), Elem<T>::pack(v[4], v[5]), Elem<T>::pack(v[6], v[7]));
                    if (kind == 0 && pos < 0) out = make_uint4(0, 0, 0, 0);
                }
                if constexpr (TURN == kAnywhere) __syncwarp();  // a head is read before any of it is written (q_out may be q)
                if (in && store) *reinterpret_cast<uint4*>(dst + n * dst_step) = out;
            }
            i += BATCH;
            if (i >= end) break;
            load();
        }
        i = end;
        if (i < last) {
            enter();
            load();
        }
    }
}

template <typename T, int LPH, Turn TURN>
cudaError_t launch_m(const AppendArgs& a, cudaStream_t st) {
    constexpr int kPerWarp = 32 / LPH;
    const int rounds = (a.kv.hq + kPerWarp - 1) / kPerWarp + 2 * ((a.kv.hkv + kPerWarp - 1) / kPerWarp);
    // A round per warp while the GPU has warps to spare (few tokens: latency); else up to eight, so that a
    // token's position and angles are looked up by few warps.
    const bool many = static_cast<int64_t>(a.kv.n_tokens) * rounds >= kManyRounds;
    const int parts = many ? (rounds + kRoundsPerWarp - 1) / kRoundsPerWarp : rounds;
    const int per = (rounds + parts - 1) / parts;
    const dim3 grid((a.kv.n_tokens + kAppendThreads / 32 - 1) / (kAppendThreads / 32), parts);
    if (many) kv_append_kernel<T, LPH, 4, TURN><<<grid, kAppendThreads, 0, st>>>(a, per);
    else kv_append_kernel<T, LPH, 1, TURN><<<grid, kAppendThreads, 0, st>>>(a, per);
    return cudaGetLastError();
}

template <typename T, int LPH>
cudaError_t launch_t(const AppendArgs& a, cudaStream_t st) {
    if (a.interleaved && a.rot % 8 == 0) return launch_m<T, LPH, kPairs>(a, st);
    if (!a.interleaved && a.rot % 16 == 0) return launch_m<T, LPH, kHalves>(a, st);
    return launch_m<T, LPH, kAnywhere>(a, st);
}

}  // namespace

cudaError_t launch_kv_append(const AppendArgs& a, int dtype, cudaStream_t st) {
    const int lanes = a.kv.d / 8;
    if (dtype == 0)
        return lanes <= 8 ? launch_t<__nv_bfloat16, 8>(a, st) : lanes <= 16 ? launch_t<__nv_bfloat16, 16>(a, st) : launch_t<__nv_bfloat16, 32>(a, st);
    return lanes <= 8 ? launch_t<__half, 8>(a, st) : lanes <= 16 ? launch_t<__half, 16>(a, st) : launch_t<__half, 32>(a, st);
}

}  // namespace moe

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
// once.  A head of D components is 8 lanes' 16-byte loads (D <= 64), 16 (D <= 128)
// or 16 lanes' two, so a warp carries 4 or 2 heads and a norm is a reduction of
// 3 or 4 shuffles.  A rotated pair lies in one lane (interleaved, and halves of 128) or in
// two lanes whose distance is the same for the whole head (halves), which
// costs four shuffles of the packed elements.
//
// Measured: 8192 tokens 40.6 us, 4.2 TB/s; a copy of as many bytes takes 26.7 us.  Other shapes (64 threads a
// block, 5 to 24 rounds a warp, 2 chunks in flight, 5 to 8 blocks an SM) took 39.4 to 48.5.  Streaming stores
// would give 2048 mixed tokens 0.7 us, but the keys are read next.
#include <algorithm>

#include "attention_common.cuh"

namespace moe {
namespace {

constexpr int kAppendThreads = 128;
constexpr int kRoundsPerWarp = 12;
constexpr int kBatch = 4;  // chunks a lane has in flight, and as many of the next rounds
// From this many rounds on warps take several: 1024 tokens of 16 / 2 heads of 256 7.3 us, one each 10.0 (8192
// 40.6 and 66); below it 64 tokens take 2.6 us with one each, 6.4 with several.
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
    kPairs,    // neighbours, whole chunks rotated: the partner is in the same chunk
    kHalves,   // halves of whole chunks, all in the lanes' first chunks: the partner is in a lane at a fixed distance
    kWhole,    // halves of a head of two chunks per lane, rotated as a whole: the partner is in the lane's other chunk
    kAnywhere  // any layout and width: partners are read again (they are in L1)
};

// A lane holds C chunks of 8 components of a head, LPH lanes make a head; a warp takes rounds of 32 / LPH
// heads, all of one kind (queries, keys or values), of one token: rounds [first, last) of the token's.  What a
// head's norm weights and angles come to is the same for every round of a kind, so they are put together once:
// component e of the result is r (x_e a_e + x_p b_e) with its partner p, a_e = w_e cos, b_e = -+ w_p sin (past the
// rotated part r x_e w_e), r the norm's factor.  The next rounds' loads are under way while these are computed.
template <typename T, int LPH, int C, int BATCH, Turn TURN>
__global__ void __launch_bounds__(kAppendThreads, 4) kv_append_kernel(const AppendArgs a, int rounds_per_warp) {
    constexpr int kPerWarp = 32 / LPH;  // heads of a round
    constexpr int kB = TURN == kHalves ? 1 : C;  // chunks that may be rotated
    const int lane = threadIdx.x & 31;
    const int t = blockIdx.x * (kAppendThreads / 32) + (threadIdx.x >> 5);
    if (t >= a.kv.n_tokens) return;
    auto at = [&](int c) { return (lane % LPH + LPH * c) * 8; };  // first component of this lane's chunk c
    const int rq = (a.kv.hq + kPerWarp - 1) / kPerWarp, rk = (a.kv.hkv + kPerWarp - 1) / kPerWarp;
    const int last = min(static_cast<int>(blockIdx.y + 1) * rounds_per_warp, rq + 2 * rk);
    int i = blockIdx.y * rounds_per_warp;
    int kind, end, head;      // of the rounds that run: their kind, its last, this lane's head of round i
    int heads;                // the kind's heads
    const T* src;             // that head's first component
    int64_t src_step;         // from one round to the next
    auto enter = [&]() {
        kind = i < rq ? 0 : i < rq + rk ? 1 : 2;
        const int begin = kind == 0 ? 0 : kind == 1 ? rq : rq + rk;
        end = min(last, kind == 0 ? rq : begin + rk);
        heads = kind == 0 ? a.kv.hq : a.kv.hkv;
        head = (i - begin) * kPerWarp + lane / LPH;
        const int64_t hs = kind == 0 ? a.q_hs : kind == 1 ? a.k_hs : a.v_hs;
        const int64_t ts = kind == 0 ? a.q_ts : kind == 1 ? a.k_ts : a.v_ts;
        src = static_cast<const T*>(kind == 0 ? a.q : kind == 1 ? a.k : a.v) + t * ts + head * hs;
        src_step = kPerWarp * hs;
    };
    // Chunk c of round i + x; zeros where there is none.
    auto load = [&](uint4 (&raw)[BATCH][C], int ahead) {
#pragma unroll
        for (int x = 0; x < BATCH; ++x)
#pragma unroll
            for (int c = 0; c < C; ++c) {
                raw[x][c] = make_uint4(0, 0, 0, 0);
                if (i + ahead + x < end && head + (ahead + x) * kPerWarp < heads && at(c) < a.kv.d)
                    raw[x][c] = *reinterpret_cast<const uint4*>(src + (ahead + x) * src_step + at(c));
            }
    };
    uint4 raw[BATCH][C];
    enter();
    wait_for_stream();
    load(raw, 0);  // under way while the token's place is looked up

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
        const int p = div_by(pos, a.kv.by_page);
        id = page_id(a.kv, b, p);
        row = pos - p * a.kv.page;
    }
    const int half = a.rot / 2;
    const bool any_turn = pos >= 0 && a.rot > 0;
    const bool low = at(0) < half;  // (kHalves)
    const int partner = (TURN == kHalves && at(0) < a.rot) ? lane + (low ? half / 8 : -(half / 8)) : lane;
    const float* tab = a.cos_sin + static_cast<int64_t>(turn) * a.rot;

    while (i < last) {
        uint64_t ca[C][4], cb[kB][4];
        const float* weight = kind == 0 ? a.q_weight : a.k_weight;
        T* dst;
        int64_t dst_step;
        if (kind == 0) {
            dst = static_cast<T*>(a.q_out) + t * a.o_ts + head * a.o_hs;
            dst_step = kPerWarp * a.o_hs;
        } else {
            const int64_t hs = kind == 1 ? a.kv.k_hs : a.kv.v_hs;
            dst = static_cast<T*>(kind == 1 ? a.kv.k : a.kv.v) + max(id, 0) * (kind == 1 ? a.kv.k_ps : a.kv.v_ps) +
                  row * (kind == 1 ? a.kv.k_rs : a.kv.v_rs) + head * hs;
            dst_step = kPerWarp * hs;
        }
        const bool store = kind == 0 || id >= 0;
        if (kind != 2) {
            auto load8 = [](const float* p, float* v) {
                const float4 x = __ldg(reinterpret_cast<const float4*>(p)), y = __ldg(reinterpret_cast<const float4*>(p) + 1);
                v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w, v[4] = y.x, v[5] = y.y, v[6] = y.z, v[7] = y.w;
            };
            auto weights = [&](int e, float* w) {
#pragma unroll
                for (int j = 0; j < 8; ++j) w[j] = 1.f;
                if (weight && e < a.kv.d) {
                    load8(weight + e, w);
#pragma unroll
                    for (int j = 0; j < 8; ++j) w[j] += a.weight_offset;
                }
            };
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const int e0 = at(c);
                float w[8], wb[8];
                weights(e0, w);
#pragma unroll
                for (int j = 0; j < 8; ++j) wb[j] = 0.f;
                if (any_turn && e0 < a.rot && c < kB) {
                    if constexpr (TURN == kPairs) {
                        const float4 cv = __ldg(reinterpret_cast<const float4*>(tab + e0 / 2)), sv = __ldg(reinterpret_cast<const float4*>(tab + half + e0 / 2));
                        const float cs[4] = {cv.x, cv.y, cv.z, cv.w}, sn[4] = {sv.x, sv.y, sv.z, sv.w};
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            wb[2 * j] = -w[2 * j + 1] * sn[j];
                            wb[2 * j + 1] = w[2 * j] * sn[j];
                            w[2 * j] *= cs[j];
                            w[2 * j + 1] *= cs[j];
                        }
                    } else if constexpr (TURN == kHalves || TURN == kWhole) {
                        const bool lo = e0 < half;
                        float cs[8], sn[8], wp[8];
                        load8(tab + (lo ? e0 : e0 - half), cs);
                        load8(tab + (lo ? e0 : e0 - half) + half, sn);
                        weights(lo ? e0 + half : e0 - half, wp);
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            wb[j] = (lo ? -wp[j] : wp[j]) * sn[j];
                            w[j] *= cs[j];
                        }
                    } else {
                        float own[8];
#pragma unroll
                        for (int j = 0; j < 8; ++j) own[j] = w[j];
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const int e = e0 + j;
                            if (e >= a.rot) continue;
                            const bool lo = a.interleaved ? (j & 1) == 0 : e < half;
                            const int p = a.interleaved ? e ^ 1 : lo ? e + half : e - half;
                            const int x = a.interleaved ? e / 2 : lo ? e : e - half;
                            const float wp = weight ? __ldg(weight + p) + a.weight_offset : 1.f;
                            w[j] = own[j] * __ldg(tab + x);
                            wb[j] = (lo ? -wp : wp) * __ldg(tab + half + x);
                        }
                    }
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    ca[c][j] = pair(w[2 * j], w[2 * j + 1]);
                    if (c < kB) cb[c < kB ? c : 0][j] = pair(wb[2 * j], wb[2 * j + 1]);
                }
            }
        }
        for (;;) {
            uint4 next[BATCH][C];
            load(next, BATCH);
#pragma unroll
            for (int x = 0; x < BATCH; ++x) {
                const bool in = i + x < end && head + x * kPerWarp < heads;
                uint4 out[C];
#pragma unroll
                for (int c = 0; c < C; ++c) out[c] = raw[x][c];  // values go as they came
                if (kind != 2) {
                    uint64_t v[C][4];
#pragma unroll
                    for (int c = 0; c < C; ++c) {
                        const uint32_t w4[4] = {raw[x][c].x, raw[x][c].y, raw[x][c].z, raw[x][c].w};
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float2 f = Elem<T>::unpack(w4[j]);
                            v[c][j] = pair(f.x, f.y);
                        }
                    }
                    float r = 1.f;
                    if (weight) {
                        uint64_t sq = mul2(v[0][0], v[0][0]);
#pragma unroll
                        for (int j = 1; j < 4 * C; ++j) sq = fma2(v[j / 4][j % 4], v[j / 4][j % 4], sq);
                        const float2 s2 = unpair(sq);
                        float sum = s2.x + s2.y;
#pragma unroll
                        for (int o = LPH / 2; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
                        r = rsqrtf(sum * a.inv_d + a.eps);
                    }
                    const uint64_t r2 = pair(r, r);
#pragma unroll
                    for (int c = 0; c < C; ++c) {
                        uint64_t y[4], z[4];
                        if constexpr (TURN == kHalves) {
                            if (c == 0) {
                                const uint32_t w4[4] = {raw[x][c].x, raw[x][c].y, raw[x][c].z, raw[x][c].w};
#pragma unroll
                                for (int j = 0; j < 4; ++j) {
                                    const float2 f = Elem<T>::unpack(__shfl_sync(~0u, w4[j], partner));
                                    y[j] = pair(f.x, f.y);
                                }
                            }
                        } else if constexpr (TURN == kPairs) {
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const float2 f = unpair(v[c][j]);
                                y[j] = pair(f.y, f.x);
                            }
                        } else if constexpr (TURN == kWhole) {
#pragma unroll
                            for (int j = 0; j < 4; ++j) y[j] = v[C - 1 - c][j];
                        } else {
                            const T* from = src + x * src_step;
                            float f[8];
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                const int e = at(c) + j;
                                f[j] = in && any_turn && e < a.rot ? static_cast<float>(from[a.interleaved ? e ^ 1 : e < half ? e + half : e - half]) : 0.f;
                            }
#pragma unroll
                            for (int j = 0; j < 4; ++j) y[j] = pair(f[2 * j], f[2 * j + 1]);
                        }
#pragma unroll
                        for (int j = 0; j < 4; ++j) z[j] = mul2(v[c][j], ca[c][j]);
                        if (c < kB && any_turn && at(c) < a.rot) {
#pragma unroll
                            for (int j = 0; j < 4; ++j) z[j] = fma2(y[j], cb[c < kB ? c : 0][j], z[j]);
                        }
                        uint32_t o4[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float2 f = unpair(weight ? mul2(z[j], r2) : z[j]);
                            o4[j] = Elem<T>::pack(f.x, f.y);
                        }
                        out[c] = make_uint4(o4[0], o4[1], o4[2], o4[3]);
                        if (kind == 0 && pos < 0) out[c] = make_uint4(0, 0, 0, 0);
                    }
                }
                if constexpr (TURN == kAnywhere) __syncwarp();  // a head is read before any of it is written (q_out may be q)
                if (in && store) {
#pragma unroll
                    for (int c = 0; c < C; ++c)
                        if (at(c) < a.kv.d) *reinterpret_cast<uint4*>(dst + x * dst_step + at(c)) = out[c];
                }
            }
            i += BATCH;
            if (i >= end) break;
            head += BATCH * kPerWarp;
            src += BATCH * src_step;
            dst += BATCH * dst_step;
#pragma unroll
            for (int x = 0; x < BATCH; ++x)
#pragma unroll
                for (int c = 0; c < C; ++c) raw[x][c] = next[x][c];
        }
        i = end;
        if (i < last) {
            enter();
            load(raw, 0);
        }
    }
}

template <typename T, int LPH, int C, Turn TURN>
cudaError_t launch_m(const AppendArgs& a, cudaStream_t st) {
    constexpr int kPerWarp = 32 / LPH;
    const int rounds = (a.kv.hq + kPerWarp - 1) / kPerWarp + 2 * ((a.kv.hkv + kPerWarp - 1) / kPerWarp);
    // A round per warp while the GPU has warps to spare (few tokens: latency); else up to twelve, so that a
    // token's position and angles are looked up by few warps.
    const bool many = static_cast<int64_t>(a.kv.n_tokens) * rounds >= kManyRounds;
    const int parts = many ? (rounds + kRoundsPerWarp - 1) / kRoundsPerWarp : rounds;
    const int per = (rounds + parts - 1) / parts;
    const dim3 grid((a.kv.n_tokens + kAppendThreads / 32 - 1) / (kAppendThreads / 32), parts);
    auto kernel = many ? kv_append_kernel<T, LPH, C, kBatch / C, TURN> : kv_append_kernel<T, LPH, C, 1, TURN>;
    return launch_in_stream(kernel, grid, kAppendThreads, 0, 1, st, a, per);
}

template <typename T, int LPH, int C>
cudaError_t launch_c(const AppendArgs& a, cudaStream_t st) {
    if (a.interleaved && a.rot % 8 == 0) return launch_m<T, LPH, C, kPairs>(a, st);
    if (!a.interleaved && a.rot % 16 == 0 && a.rot <= 8 * LPH) return launch_m<T, LPH, C, kHalves>(a, st);
    if constexpr (C == 2)
        if (!a.interleaved && a.rot == 16 * LPH) return launch_m<T, LPH, C, kWhole>(a, st);
    return launch_m<T, LPH, C, kAnywhere>(a, st);
}

template <typename T>
cudaError_t launch_t(const AppendArgs& a, cudaStream_t st) {
    if (a.kv.d <= 64) return launch_c<T, 8, 1>(a, st);
    if (a.kv.d <= 128) return launch_c<T, 16, 1>(a, st);
    return launch_c<T, 16, 2>(a, st);
}

}  // namespace

cudaError_t launch_kv_append(const AppendArgs& a, int dtype, cudaStream_t st) {
    return dtype == 0 ? launch_t<__nv_bfloat16>(a, st) : launch_t<__half>(a, st);
}

}  // namespace moe

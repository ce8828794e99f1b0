// The row of a latent cache and the rotated query parts: the norm of a token's
// latent vector, the rotation of the key part that all heads share and of
// every head's query part, and the store into the paged cache, in one kernel.
//
// Per token: c' = c rsqrt(mean(c^2) + eps) (w + offset) over Dc components; R
// components of the key and of each query head are turned in pairs by the
// position's angle, (a, b) -> (a c - b s, b c + a s).  All of it is fp32 with one
// rounding at the store.
//
// Bound: HBM, each element read once and written once.  A warp takes one
// token: the row, whose up to 512 components are two 16-byte chunks a lane (the
// norm five shuffles) and whose key part goes to the first lanes, and rounds of as
// many query heads as their chunks fill the warp with (R = 64: 8 lanes a
// head, 4 heads).  A lane has the same chunk of every head, so its cosines and
// sines are loaded once.  Several rounds' loads are under way together.
// 8192 tokens of 16 heads, 512 + 64: 13.3 us with inputs that L2 does not hold, 52 MB in and out, 3.9 TB/s (a copy of as many
// bytes takes 18.6); of 128 heads 46.2 us, 287 MB, 6.2 TB/s.  Single tokens 2.5 us, the launch and the chain of lookups.
#include <algorithm>

#include "attention_common.cuh"
#include "latent.h"

namespace moe {
namespace {

constexpr int kThreads = 64;  // 2048 tokens of 16 heads 3.7 us, with 128 threads 3.9, with 256 3.8; 64 tokens of 128 heads 2.5, 2.6, 2.8
constexpr int kRounds = 4;  // rounds of heads whose loads are under way together

// How a lane finds the partners of its chunk's components.
enum LatentTurn {
    kPairs,    // neighbours
    kHalves,   // halves of whole chunks: the partners are one other chunk
    kAnywhere  // halves of 4, 12, .. components: the partners lie in two chunks
};

// The angles of a lane's chunk, and the chunk turned by them.
template <typename T, LatentTurn TURN>
struct Turner {
    float cs[8], sn[8];  // kPairs: the first four
    int e0, half;
    __device__ __forceinline__ void init(const float* tab, int chunk, int rot) {
        e0 = chunk * 8;
        half = rot / 2;
        auto load4 = [](const float* p, float* v) {
            const float4 x = __ldg(reinterpret_cast<const float4*>(p));
            v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
        };
        if constexpr (TURN == kPairs) {
            load4(tab + e0 / 2, cs);
            load4(tab + half + e0 / 2, sn);
        } else if constexpr (TURN == kHalves) {
            const int x = e0 < half ? e0 : e0 - half;
            load4(tab + x, cs);
            load4(tab + x + 4, cs + 4);
            load4(tab + half + x, sn);
            load4(tab + half + x + 4, sn + 4);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int e = e0 + j, x = e < half ? e : e - half;
                cs[j] = __ldg(tab + x);
                sn[j] = __ldg(tab + half + x);
            }
        }
    }
    // head: the first component, own: this lane's chunk.  Reads the partners from memory (they are in L1).
    __device__ __forceinline__ uint4 partners(const T* head) const {
        if constexpr (TURN == kPairs) {
            return make_uint4(0, 0, 0, 0);
        } else if constexpr (TURN == kHalves) {
            return *reinterpret_cast<const uint4*>(head + (e0 < half ? e0 + half : e0 - half));
        } else {
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float f[2];
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const int e = e0 + 2 * j + x;
                    f[x] = static_cast<float>(head[e < half ? e + half : e - half]);
                }
                w[j] = Elem<T>::pack(f[0], f[1]);  // (exact: they are of this type)
            }
            return make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
    __device__ __forceinline__ uint4 turn(const uint4& own, const uint4& other) const {
        const uint32_t a4[4] = {own.x, own.y, own.z, own.w}, b4[4] = {other.x, other.y, other.z, other.w};
        uint32_t o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 v = Elem<T>::unpack(a4[j]);
            if constexpr (TURN == kPairs) {
                o[j] = Elem<T>::pack(v.x * cs[j] - v.y * sn[j], v.y * cs[j] + v.x * sn[j]);
            } else {
                const float2 p = Elem<T>::unpack(b4[j]);
                const float s0 = e0 + 2 * j < half ? -sn[2 * j] : sn[2 * j], s1 = e0 + 2 * j + 1 < half ? -sn[2 * j + 1] : sn[2 * j + 1];
                o[j] = Elem<T>::pack(v.x * cs[2 * j] + p.x * s0, v.y * cs[2 * j + 1] + p.y * s1);
            }
        }
        return make_uint4(o[0], o[1], o[2], o[3]);
    }
};

// lanes: of a head, a power of two with room for its R / 8 chunks.  per: rounds of query heads of a warp; few: the row has a
// warp (blockIdx.y = 0) of its own, else it goes with the first rounds.
template <typename T, LatentTurn TURN>
__global__ void __launch_bounds__(kThreads) latent_append_kernel(const LatentAppendArgs a, int lanes_log2, int per, int few) {
    const int lane = threadIdx.x & 31;
    const int t = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    if (t >= a.kv.n_tokens) return;
    const int lanes = 1 << lanes_log2, heads = 32 >> lanes_log2;  // heads of a round
    const int chunk = lane & (lanes - 1), chunks = a.rot / 8;
    const bool on = chunk < chunks;
    const bool row = blockIdx.y == 0;
    const int first = max(static_cast<int>(blockIdx.y) - few, 0) * per;
    const int h0 = first * heads + (lane >> lanes_log2), h1 = row && few ? 0 : min((first + per) * heads, a.kv.hq);
    wait_for_stream();
    // the inputs are under way while the token's place is looked up
    uint4 c[2], kr = make_uint4(0, 0, 0, 0);
    if (row) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            c[x] = make_uint4(0, 0, 0, 0);
            if ((lane + 32 * x) * 8 < a.kv.d) c[x] = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.latent) + t * a.c_ts + (lane + 32 * x) * 8);
        }
        if (lane < chunks) kr = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.k_rot) + t * a.k_ts + lane * 8);
    }
    const T* src = static_cast<const T*>(a.q_rot) + t * a.q_ts;
    uint4 q[kRounds];
    auto load = [&](int h) {
#pragma unroll
        for (int x = 0; x < kRounds; ++x)
            if (on && h + x * heads < h1) q[x] = *reinterpret_cast<const uint4*>(src + (h + x * heads) * a.q_hs + chunk * 8);
    };
    load(h0);

    const int b = find_seq(a.kv, t);
    int pos = -1;
    if (b >= 0) {  // q_start[b] <= t < q_start[b + 1]; entries past the tokens count as their end
        const int stop = min(__ldg(a.kv.q_start + b + 1), a.kv.n_tokens);
        pos = max(__ldg(a.kv.kv_len + b), 0) - (stop - t);
    }
    const int at = a.positions && pos >= 0 ? __ldg(a.positions + t) : pos;
    if (a.rot > 0 && (at < 0 || at >= a.table_rows)) pos = -1;
    const float* tab = a.cos_sin + static_cast<int64_t>(at) * a.rot;
    Turner<T, TURN> turner;

    if (row && pos >= 0 && pos < a.kv.cap) {
        const int p = div_by(pos, a.kv.by_page), id = page_id(a.kv, b, p);
        if (id >= 0) {
            T* dst = static_cast<T*>(a.kv.k) + id * a.kv.k_ps + static_cast<int64_t>(pos - p * a.kv.page) * a.kv.k_rs;
            float v[2][8], r = 1.f;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const uint32_t w4[4] = {c[x].x, c[x].y, c[x].z, c[x].w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 f = Elem<T>::unpack(w4[j]);
                    v[x][2 * j] = f.x;
                    v[x][2 * j + 1] = f.y;
                }
            }
            if (a.weight) {
                float sum = 0.f;
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int j = 0; j < 8; ++j) sum += v[x][j] * v[x][j];
#pragma unroll
                for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
                r = rsqrtf(sum * a.inv_d + a.eps);
            }
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int e = (lane + 32 * x) * 8;
                if (e >= a.kv.d) continue;
                if (a.weight) {
                    const float4 w0 = __ldg(reinterpret_cast<const float4*>(a.weight + e)), w1 = __ldg(reinterpret_cast<const float4*>(a.weight + e) + 1);
                    const float w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
                    uint32_t o[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        o[j] = Elem<T>::pack(v[x][2 * j] * r * (w[2 * j] + a.weight_offset), v[x][2 * j + 1] * r * (w[2 * j + 1] + a.weight_offset));
                    c[x] = make_uint4(o[0], o[1], o[2], o[3]);
                }
                *reinterpret_cast<uint4*>(dst + e) = c[x];
            }
            if (lane < chunks) {
                turner.init(tab, lane, a.rot);
                *reinterpret_cast<uint4*>(dst + a.kv.d + lane * 8) = turner.turn(kr, turner.partners(static_cast<const T*>(a.k_rot) + t * a.k_ts));
            }
        }
    }

    if (pos >= 0 && on && h0 < h1) turner.init(tab, chunk, a.rot);
    T* dst = static_cast<T*>(a.q_out) + t * a.o_ts;
    for (int h = h0; h - h0 + first * heads < h1; h += kRounds * heads) {  // (the same turns in every lane)
        uint4 o[kRounds];
#pragma unroll
        for (int x = 0; x < kRounds; ++x) {
            o[x] = make_uint4(0, 0, 0, 0);
            if (pos >= 0 && on && h + x * heads < h1) o[x] = turner.turn(q[x], turner.partners(src + (h + x * heads) * a.q_hs));
        }
        if constexpr (TURN != kPairs) __syncwarp();  // a head is read before any of it is written (q_out may be q_rot)
#pragma unroll
        for (int x = 0; x < kRounds; ++x)
            if (on && h + x * heads < h1) *reinterpret_cast<uint4*>(dst + (h + x * heads) * a.o_hs + chunk * 8) = o[x];
        load(h + kRounds * heads);
    }
}

template <typename T, LatentTurn TURN>
cudaError_t launch_m(const LatentAppendArgs& a, cudaStream_t st) {
    int log2 = 0;
    while ((1 << log2) < a.rot / 8) ++log2;
    const int heads = 32 >> log2, rounds = a.rot == 0 ? 0 : (a.kv.hq + heads - 1) / heads;
    // A warp for each round and one for the row while the GPU has warps to spare (latency), else a warp for a token's row and
    // four rounds, or eight once there are more of these than run at a time.  128 heads of 64, us with one | four | eight
    // rounds: 64 tokens 2.6 | - | 3.5, 128 tokens 3.1 | 3.1 | 3.6, 256 4.5 | 3.5 | 3.8, 512 7.6 | 4.8 | 5.1, 2048 29.5 | 14.4 | 14.3,
    // 8192 110.8 | 48.4 | 46.5 (sixteen: 46.5, but 4.6 of 256).
    const int64_t tokens = a.kv.n_tokens;
    const bool few = tokens * (1 + rounds) <= 152 * 16;
    const int per = few ? 1 : tokens * ((rounds + kRounds - 1) / kRounds) <= 152 * 64 ? kRounds : 2 * kRounds;
    const int parts = std::max((rounds + per - 1) / per, few ? 0 : 1) + (few ? 1 : 0);
    const dim3 grid((a.kv.n_tokens + kThreads / 32 - 1) / (kThreads / 32), parts);
    return launch_in_stream(latent_append_kernel<T, TURN>, grid, kThreads, 0, 1, st, a, log2, per, few ? 1 : 0);
}

template <typename T>
cudaError_t launch_t(const LatentAppendArgs& a, cudaStream_t st) {
    if (a.interleaved) return launch_m<T, kPairs>(a, st);
    return a.rot % 16 == 0 ? launch_m<T, kHalves>(a, st) : launch_m<T, kAnywhere>(a, st);
}

}  // namespace

cudaError_t launch_latent_append(const LatentAppendArgs& a, int dtype, cudaStream_t st) {
    return dtype == 0 ? launch_t<__nv_bfloat16>(a, st) : launch_t<__half>(a, st);
}

}  // namespace moe

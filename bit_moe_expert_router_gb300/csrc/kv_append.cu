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
// four shuffles of the packed elements; where half the rotated width is not a
// multiple of 8 the partners are read again instead (they are in L1).
#include "attention_common.cuh"

namespace moe {
namespace {

constexpr int kAppendThreads = 128;

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

template <typename T, int LPH, int HEADS>
__global__ void __launch_bounds__(kAppendThreads) kv_append_kernel(const AppendArgs a, int groups) {
    constexpr int kPerWarp = 32 / LPH;  // heads a warp carries at a time
    const int lane = threadIdx.x & 31;
    const int64_t item = static_cast<int64_t>(blockIdx.x) * (kAppendThreads / 32) + (threadIdx.x >> 5);
    const int t = static_cast<int>(item / groups);
    if (t >= a.kv.n_tokens) return;
    const int slot0 = static_cast<int>(item - static_cast<int64_t>(t) * groups) * (kPerWarp * HEADS) + lane / LPH;
    const int e0 = (lane % LPH) * 8;  // this lane's first component
    const bool on = e0 < a.kv.d;
    const int heads = a.kv.hq + 2 * a.kv.hkv;

    uint4 raw[HEADS];
    const T* src[HEADS];
#pragma unroll
    for (int i = 0; i < HEADS; ++i) {
        const int s = slot0 + i * kPerWarp;
        src[i] = nullptr;
        raw[i] = make_uint4(0, 0, 0, 0);
        if (s < a.kv.hq) src[i] = static_cast<const T*>(a.q) + t * a.q_ts + s * a.q_hs;
        else if (s < a.kv.hq + a.kv.hkv) src[i] = static_cast<const T*>(a.k) + t * a.k_ts + (s - a.kv.hq) * a.k_hs;
        else if (s < heads) src[i] = static_cast<const T*>(a.v) + t * a.v_ts + (s - a.kv.hq - a.kv.hkv) * a.v_hs;
        if (src[i] && on) raw[i] = *reinterpret_cast<const uint4*>(src[i] + e0);
    }

    const int b = find_seq(a.kv, t);
    int pos = -1;
    if (b >= 0) {  // q_start[b] <= t < q_start[b + 1]; entries past the tokens count as their end
        const int end = min(__ldg(a.kv.q_start + b + 1), a.kv.n_tokens);
        pos = max(__ldg(a.kv.kv_len + b), 0) - (end - t);
    }
    int turn = a.positions && pos >= 0 ? __ldg(a.positions + t) : pos;
    if (a.rot > 0 && (turn < 0 || turn >= a.table_rows)) pos = -1;
    int64_t row = 0;
    int id = -1;
    if (pos >= 0 && pos < a.kv.cap) {
        id = page_id(a.kv, b, pos / a.kv.page);
        row = pos % a.kv.page;
    }

    // this lane's cosines and sines: one for each pair (interleaved) or each component (halves)
    float cs[8], sn[8];
    const int half = a.rot / 2;
    if (pos >= 0 && e0 < a.rot) {
        const float* tab = a.cos_sin + static_cast<int64_t>(turn) * a.rot;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int e = e0 + j;
            const int x = a.interleaved ? e / 2 : (e < half ? e : e - half);
            const bool in = e < a.rot;
            cs[j] = in ? __ldg(tab + x) : 1.f;
            sn[j] = in ? __ldg(tab + half + x) : 0.f;
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) cs[j] = 1.f, sn[j] = 0.f;
    }
    const bool shuffled = !a.interleaved && (half & 7) == 0;
    const int partner = lane + (e0 < half ? half / 8 : -(half / 8));

#pragma unroll
    for (int i = 0; i < HEADS; ++i) {
        const int s = slot0 + i * kPerWarp;
        const bool is_q = s < a.kv.hq, is_v = s >= a.kv.hq + a.kv.hkv;
        const float* weight = is_v ? nullptr : is_q ? a.q_weight : a.k_weight;
        const uint32_t w4[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
        float x[8];
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 f = Elem<T>::unpack(w4[j]);
            x[2 * j] = f.x;
            x[2 * j + 1] = f.y;
            sum += f.x * f.x + f.y * f.y;
        }
#pragma unroll
        for (int o = LPH / 2; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
        const float r = weight ? rsqrtf(sum / a.kv.d + a.eps) : 1.f;
        float y[8];  // the partners of a rotation by halves, not yet normed
        if (shuffled) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 f = Elem<T>::unpack(__shfl_sync(~0u, w4[j], partner));
                y[2 * j] = f.x;
                y[2 * j + 1] = f.y;
            }
        } else if (!a.interleaved && src[i] && on) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int e = e0 + j;
                y[j] = e < a.rot ? static_cast<float>(src[i][e < half ? e + half : e - half]) : 0.f;
            }
        }
        __syncwarp();  // all of the head is read before any of it is written (q_out may be q)
        if (s >= heads || !on) continue;
        if (weight) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int e = e0 + j;
                x[j] *= r * (__ldg(weight + e) + a.weight_offset);
                if (!a.interleaved && e < a.rot) y[j] *= r * (__ldg(weight + (e < half ? e + half : e - half)) + a.weight_offset);
            }
        }
        if (!is_v && e0 < a.rot) {
            if (a.interleaved) {
#pragma unroll
                for (int j = 0; j < 8; j += 2) {
                    const float p = x[j], q = x[j + 1];
                    x[j] = p * cs[j] - q * sn[j];
                    x[j + 1] = q * cs[j] + p * sn[j];
                }
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int e = e0 + j;
                    if (e < a.rot) x[j] = x[j] * cs[j] + (e < half ? -y[j] : y[j]) * sn[j];
                }
            }
        }
        uint4 w = raw[i];  // values go as they came
        if (!is_v) w = make_uint4(Elem<T>::pack(x[0], x[1]), Elem<T>::pack(x[2], x[3]), Elem<T>::pack(x[4], x[5]), Elem<T>::pack(x[6], x[7]));
        if (is_q) {
            if (pos < 0) w = make_uint4(0, 0, 0, 0);
            *reinterpret_cast<uint4*>(static_cast<T*>(a.q_out) + t * a.o_ts + s * a.o_hs + e0) = w;
        } else if (id >= 0) {
            if (is_v)
                *reinterpret_cast<uint4*>(static_cast<T*>(a.kv.v) + id * a.kv.v_ps + row * a.kv.v_rs + (s - a.kv.hq - a.kv.hkv) * a.kv.v_hs + e0) = w;
            else
                *reinterpret_cast<uint4*>(static_cast<T*>(a.kv.k) + id * a.kv.k_ps + row * a.kv.k_rs + (s - a.kv.hq) * a.kv.k_hs + e0) = w;
        }
    }
}

template <typename T, int LPH>
cudaError_t launch_t(const AppendArgs& a, cudaStream_t st) {
    constexpr int kPerWarp = 32 / LPH;
    const int heads = a.kv.hq + 2 * a.kv.hkv;
    const int rounds = (heads + kPerWarp - 1) / kPerWarp;
    constexpr int kMany = 4;
    const bool many = static_cast<int64_t>(a.kv.n_tokens) * rounds >= 64 * 152;
    const int groups = many ? (rounds + kMany - 1) / kMany : rounds;
    const int64_t items = static_cast<int64_t>(a.kv.n_tokens) * groups;
    const unsigned grid = static_cast<unsigned>((items + kAppendThreads / 32 - 1) / (kAppendThreads / 32));
    if (many) kv_append_kernel<T, LPH, kMany><<<grid, kAppendThreads, 0, st>>>(a, groups);
    else kv_append_kernel<T, LPH, 1><<<grid, kAppendThreads, 0, st>>>(a, groups);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv_append(const AppendArgs& a, int dtype, cudaStream_t st) {
    const int lanes = a.kv.d / 8;
    if (dtype == 0)
        return lanes <= 8 ? launch_t<__nv_bfloat16, 8>(a, st) : lanes <= 16 ? launch_t<__nv_bfloat16, 16>(a, st) : launch_t<__nv_bfloat16, 32>(a, st);
    return lanes <= 8 ? launch_t<__half, 8>(a, st) : lanes <= 16 ? launch_t<__half, 16>(a, st) : launch_t<__half, 32>(a, st);
}

}  // namespace moe

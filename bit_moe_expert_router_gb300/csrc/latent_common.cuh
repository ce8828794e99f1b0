// Device helpers of latent attention: the exact row, and the rows of no
// sequence.
#pragma once

#include "attention_common.cuh"
#include "latent.h"

namespace moe {

// One (token, head) row over the positions it sees and no others, by one warp: 16-byte chunks of a row go to lanes in turn.
// See attend_row for when it is needed.  Writes components [col0, col1), and lse with component 0.
template <typename T>
__device__ __noinline__ void latent_row(const LatentArgs& a, int b, int token, int head, int pos, int col0 = 0, int col1 = kMaxLatent) {
    constexpr int kC = (kMaxLatent + kMaxLatentRot + 255) / 256, kV = kMaxLatent / 256;  // chunks of a lane: of the row, of its latent part
    const int lane = threadIdx.x & 31;
    const T* qp = static_cast<const T*>(a.q) + token * a.q_ts + head * a.q_hs;
    float q[kC][8] = {}, o[kV][8] = {};
#pragma unroll
    for (int x = 0; x < kC; ++x) {
        const int e = (lane + 32 * x) * 8;
        if (e >= a.dk) continue;
        const uint4 w = *reinterpret_cast<const uint4*>(qp + e);
        const uint32_t w4[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = Elem<T>::unpack(w4[i]);
            q[x][2 * i] = f.x;
            q[x][2 * i + 1] = f.y;
        }
    }
    const int hi = min(pos, a.kv.cap - 1) + 1;
    const float c = a.scale * kLog2e;
    float m = kNegInf, l = 0.f, z = 0.f;  // z: NaN if some score is
    for (int j = 0; j < hi; ++j) {
        const int at = div_by(j, a.kv.by_page), id = page_id(a.kv, b, at);
        const T* row = static_cast<const T*>(a.kv.k) + max(id, 0) * a.kv.k_ps + static_cast<int64_t>(j - at * a.kv.page) * a.kv.k_rs;
        float s = 0.f, v[kV][8] = {};
#pragma unroll
        for (int x = 0; x < kC; ++x) {
            const int e = (lane + 32 * x) * 8;
            if (e >= a.dk || id < 0) continue;
            const uint4 w = *reinterpret_cast<const uint4*>(row + e);
            const uint32_t w4[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 f = Elem<T>::unpack(w4[i]);
                s += q[x][2 * i] * f.x + q[x][2 * i + 1] * f.y;
                if (x < kV && e < a.kv.d) v[x < kV ? x : 0][2 * i] = f.x, v[x < kV ? x : 0][2 * i + 1] = f.y;
            }
        }
#pragma unroll
        for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(~0u, s, x);
        s *= c;
        if (s != s) z = s;
        const float mn = fmaxf(m, s);  // a NaN score is not the maximum, but it reaches l below
        const float base = mn == kNegInf ? 0.f : mn;
        const float f = exp2f(m - base), p = exp2f(s - base);
        m = mn;
        l = l * f + p;
#pragma unroll
        for (int x = 0; x < kV; ++x)
#pragma unroll
            for (int i = 0; i < 8; ++i) o[x][i] = o[x][i] * f + p * v[x][i];
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    T* dst = static_cast<T*>(a.out) + token * a.o_ts + head * a.o_hs;
#pragma unroll
    for (int x = 0; x < kV; ++x) {
        const int e = (lane + 32 * x) * 8;
        if (e >= a.kv.d || e < col0 || e >= col1) continue;
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = Elem<T>::pack(o[x][2 * i] * inv, o[x][2 * i + 1] * inv);
        *reinterpret_cast<uint4*>(dst + e) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    // (a score of +inf makes the weights NaN, but the sum of the exponentials is infinite)
    if (lane == 0 && col0 == 0 && a.lse) a.lse[static_cast<int64_t>(token) * a.kv.hq + head] = l == 0.f ? kNegInf : m == -kNegInf ? m + z : (m + log2f(l)) * kLn2;
}

}  // namespace moe

// The join of the pieces of row tiles that CTA boundaries cut: both attention
// engines' second kernel.
#pragma once

#include "attention_common.cuh"

namespace moe {

constexpr int kJoinWarps = 8;

// Block (c, y) stands for the boundary before CTA c + 1; the rows of a tile that several boundaries cut
// are dealt over their blocks.  A row is taken by WPR warps, which share its pieces (few rows and many
// pieces: 8; many rows and two or three pieces: 1).  The sums' order is that of the pieces' CTAs, whatever
// order they were finished in, so two runs give the same bits.
template <typename T, int ROWS, int DH, int WPR>
__global__ void __launch_bounds__(kJoinWarps * 32) attend_join_kernel(const AttendArgs a) {
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    constexpr int kGroups = kJoinWarps / WPR;
    constexpr int kVec = DH / 32;  // components per lane: 2 lane + 64 x, + 1
    __shared__ float2 part[WPR > 1 ? kJoinWarps : 1][WPR > 1 ? DH / 2 : 1];
    __shared__ float part_l[kJoinWarps];
    const int cta = blockIdx.x + 1;
    const BoundaryRec rec = a.recs[cta];
    if (!rec.cut) return;
    const KvArgs& kv = a.kv;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int group = warp / WPR, wi = warp % WPR;
    const int c0 = static_cast<int>(rec.begin / rec.per), c1 = static_cast<int>((rec.begin + rec.n - 1) / rec.per);
    const SeqInfo s = seq_info(kv, rec.b);
    const int r0 = rec.rt * ROWS, rows = min(s.q_len * kv.group - r0, ROWS);
    auto slot_of = [&](int p) { return 2 * static_cast<int64_t>(p) + (p * rec.per >= rec.begin ? 0 : 1); };
    const int step = c1 - c0;
    for (int k = blockIdx.y * kGroups; cta - (c0 + 1) + k * step < rows; k += gridDim.y * kGroups) {
        const int r = cta - (c0 + 1) + (k + group) * step;
        float mm = kNegInf, ll = 0.f;
        float2 acc[kVec / 2];
#pragma unroll
        for (int x = 0; x < kVec / 2; ++x) acc[x] = make_float2(0.f, 0.f);
        if (r < rows) {
            for (int p = c0 + lane; p <= c1; p += 32) mm = fmaxf(mm, a.part_ml[slot_of(p) * ROWS + r].x);
#pragma unroll
            for (int x = 16; x; x >>= 1) mm = fmaxf(mm, __shfl_xor_sync(~0u, mm, x));
            const float base = mm == kNegInf ? 0.f : mm;
#pragma unroll 4
            for (int p = c0 + wi; p <= c1; p += WPR) {
                const int64_t slot = slot_of(p);
                const float2 v = a.part_ml[slot * ROWS + r];
                const float f = exp2_fast(v.x - base);
                const float2* o = reinterpret_cast<const float2*>(a.part_o + (slot * ROWS + r) * DH) + lane;
                ll += v.y * f;
#pragma unroll
                for (int x = 0; x < kVec / 2; ++x) {
                    const float2 w = o[32 * x];
                    acc[x].x += w.x * f;
                    acc[x].y += w.y * f;
                }
            }
        }
        if constexpr (WPR > 1) {
            __syncthreads();
#pragma unroll
            for (int x = 0; x < kVec / 2; ++x) part[warp][lane + 32 * x] = acc[x];
            if (lane == 0) part_l[warp] = ll;
            __syncthreads();
            if (wi == 0) {
#pragma unroll
                for (int w = 1; w < WPR; ++w) {
                    ll += part_l[warp + w];
#pragma unroll
                    for (int x = 0; x < kVec / 2; ++x) {
                        const float2 v = part[warp + w][lane + 32 * x];
                        acc[x].x += v.x;
                        acc[x].y += v.y;
                    }
                }
            }
        }
        if (wi != 0 || r >= rows) continue;
        const int tok = s.q0 + (r0 + r) / kv.group, head = rec.h * kv.group + (r0 + r) % kv.group;
        bool bad = ll != ll;
#pragma unroll
        for (int x = 0; x < kVec / 2; ++x) bad |= acc[x].x != acc[x].x || acc[x].y != acc[x].y;
        if (__any_sync(~0u, bad)) {
            attend_row<T>(a, rec.b, tok, head, s.pos0 + (r0 + r) / kv.group);
            continue;
        }
        const float inv = ll == 0.f ? 0.f : 1.f / ll;
        T* dst = static_cast<T*>(a.out) + tok * a.o_ts + head * a.o_hs + 2 * lane;
#pragma unroll
        for (int x = 0; x < kVec / 2; ++x)
            if (2 * lane + 64 * x < kv.d) *reinterpret_cast<uint32_t*>(dst + 64 * x) = Elem<T>::pack(acc[x].x * inv, acc[x].y * inv);
        if (lane == 0 && a.lse) a.lse[static_cast<int64_t>(tok) * kv.hq + head] = ll == 0.f ? kNegInf : (mm + log2f(ll)) * kLn2;
    }
}

// Launched while the first kernel runs (it waits for its end by itself), one column of blocks per boundary.
template <typename T, int ROWS, int DH, int WPR>
cudaError_t launch_attend_join(const AttendArgs& a, int n_ctas, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(n_ctas - 1, WPR > 1 ? 1 : ROWS / kJoinWarps);
    cfg.blockDim = dim3(kJoinWarps * 32);
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attend_join_kernel<T, ROWS, DH, WPR>, a);
}

}  // namespace moe

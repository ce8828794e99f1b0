// The join of the pieces of row tiles that CTA boundaries cut: both attention
// engines' second kernel.
#pragma once

#include "attention_common.cuh"

namespace moe {

constexpr int kJoinWarps = 8;

// Block c stands for the boundary before CTA c + 1; the rows of a tile that several boundaries cut are dealt
// over their blocks.  A row is taken by one warp, or by eight that share its pieces where they are
// many.  The sums' order is that of the pieces' CTAs, whatever order they were finished in, so two
// runs give the same bits.
template <typename T, int ROWS, int DH>
__global__ void __launch_bounds__(kJoinWarps * 32) attend_join_kernel(const AttendArgs a) {
    wait_for_stream();
    constexpr int kVec = DH / 64;  // pairs of components per lane: lane + 32 x
    __shared__ float2 part[kJoinWarps][DH / 2];
    __shared__ float part_l[kJoinWarps];
    const int cta = blockIdx.x + 1;
    const BoundaryRec rec = a.recs[cta];
    if (!rec.cut) return;
    const KvArgs& kv = a.kv;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c0 = static_cast<int>(div_line(rec.begin, rec.per)), c1 = static_cast<int>(div_line(rec.begin + rec.n - 1, rec.per));
    const int share = c1 - c0 + 1 > 8 ? kJoinWarps : 1;  // warps per row
    const int wi = share > 1 ? warp : 0;
    const int r0 = rec.rt * ROWS, rows = min(rec.q_len * kv.group - r0, ROWS);
    auto slot_of = [&](int p) { return 2 * static_cast<int64_t>(p) + (p * rec.per >= rec.begin ? 0 : 1); };
    const int step = c1 - c0;
    for (int k = 0; cta - (c0 + 1) + k * step < rows; k += kJoinWarps / share) {
        const int r = cta - (c0 + 1) + (k + (share > 1 ? 0 : warp)) * step;
        float mm = kNegInf, ll = 0.f;
        float2 acc[kVec];
#pragma unroll
        for (int x = 0; x < kVec; ++x) acc[x] = make_float2(0.f, 0.f);
        if (r < rows) {
            for (int p = c0 + lane; p <= c1; p += 32) mm = fmaxf(mm, a.part_ml[slot_of(p) * ROWS + r].x);
            constexpr int kAhead = 4;
            for (int p0 = c0 + wi; p0 <= c1; p0 += kAhead * share) {
                float2 v[kAhead], o[kAhead][kVec];
#pragma unroll
                for (int y = 0; y < kAhead; ++y) {
                    const int p = min(p0 + y * share, c1);
                    const int64_t at = slot_of(p) * ROWS + r;
                    v[y] = a.part_ml[at];
#pragma unroll
                    for (int x = 0; x < kVec; ++x) o[y][x] = reinterpret_cast<const float2*>(a.part_o + at * DH)[lane + 32 * x];
                }
                if (p0 == c0 + wi) {
#pragma unroll
                    for (int x = 16; x; x >>= 1) mm = fmaxf(mm, __shfl_xor_sync(~0u, mm, x));
                }
                const float base = mm == kNegInf ? 0.f : mm;
#pragma unroll
                for (int y = 0; y < kAhead; ++y) {
                    if (p0 + y * share > c1) break;
                    const float f = exp2_fast(v[y].x - base);
                    ll += v[y].y * f;
#pragma unroll
                    for (int x = 0; x < kVec; ++x) {
                        acc[x].x += o[y][x].x * f;
                        acc[x].y += o[y][x].y * f;
                    }
                }
            }
        }
        if (share > 1) {  // (every warp of the block has the same row)
            __syncthreads();
#pragma unroll
            for (int x = 0; x < kVec; ++x) part[warp][lane + 32 * x] = acc[x];
            if (lane == 0) part_l[warp] = ll;
            __syncthreads();
            if (warp == 0) {
#pragma unroll
                for (int w = 1; w < kJoinWarps; ++w) {
                    ll += part_l[w];
#pragma unroll
                    for (int x = 0; x < kVec; ++x) {
                        const float2 v = part[w][lane + 32 * x];
                        acc[x].x += v.x;
                        acc[x].y += v.y;
                    }
                }
            }
        }
        if (wi != 0 || r >= rows) continue;
        int i, g;
        row_of(kv, r0 + r, i, g);
        const int tok = rec.q0 + i, head = rec.h * kv.group + g;
        bool bad = ll != ll;
#pragma unroll
        for (int x = 0; x < kVec; ++x) bad |= acc[x].x != acc[x].x || acc[x].y != acc[x].y;
        if (__any_sync(~0u, bad)) {
            attend_row<T>(a, rec.b, tok, head, rec.pos0 + i);
            continue;
        }
        const float inv = ll == 0.f ? 0.f : 1.f / ll;
        T* dst = static_cast<T*>(a.out) + tok * a.o_ts + head * a.o_hs + 2 * lane;
#pragma unroll
        for (int x = 0; x < kVec; ++x)
            if (2 * lane + 64 * x < kv.d) *reinterpret_cast<uint32_t*>(dst + 64 * x) = Elem<T>::pack(acc[x].x * inv, acc[x].y * inv);
        if (lane == 0 && a.lse) a.lse[static_cast<int64_t>(tok) * kv.hq + head] = ll == 0.f ? kNegInf : (mm + log2f(ll)) * kLn2;
    }
}

// The same for tiles of many rows, which lie as [component / 4][row][4]: a block takes 32 rows and 64
// components of a tile, a lane per row, two fours of components per warp; the rows are written through shared
// memory.  MANY: the last four pieces leave out the loads of those that are not there, else the last piece's are
// repeated.  Measured on whole calls, repeated | left out: 4 x 3 tokens of 16 / 2 heads of 256 at 16384 (about ten
// pieces a tile) 20.0 | 17.9 us, 2 x 6 15.2 | 14.1; 4096-token prompts (two or three) of heads of 128 140 | 142, of
// 256 99.1 | 101.2.
template <typename T, int ROWS, int DH, bool MANY>
__global__ void __launch_bounds__(kJoinWarps * 32) attend_join_rows_kernel(const AttendArgs a) {
    wait_for_stream();
    constexpr int kSlices = DH / 64;
    __shared__ uint32_t rows_out[32][33];  // (odd: a column of rows lies in different banks)
    __shared__ unsigned bad_rows;
    const int cta = blockIdx.x + 1;
    const BoundaryRec rec = a.recs[cta];
    if (!rec.cut) return;
    const KvArgs& kv = a.kv;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c0 = static_cast<int>(div_line(rec.begin, rec.per)), c1 = static_cast<int>(div_line(rec.begin + rec.n - 1, rec.per));
    const int r0 = rec.rt * ROWS, rows = min(rec.q_len * kv.group - r0, ROWS);
    auto slot_of = [&](int p) { return 2 * static_cast<int64_t>(p) + (p * rec.per >= rec.begin ? 0 : 1); };
    const int step = c1 - c0;  // boundaries of the tile: its parts go round them
    for (int v = (cta - (c0 + 1)) + step * blockIdx.y; v / kSlices * 32 < rows; v += step * gridDim.y) {
        const int g = v / kSlices, col = v % kSlices * 64;  // rows 32 g .., components col ..
        const int r = 32 * g + lane;
        if (threadIdx.x == 0) bad_rows = 0;
        // pieces four at a time (two or three are usual), their loads all under way at once; the sums are
        // rescaled between the fours
        float mm = kNegInf, ll = 0.f;
        float4 acc[2] = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
        auto add = [](float4& to, const float4& x, float f) {
            to.x += x.x * f;
            to.y += x.y * f;
            to.z += x.z * f;
            to.w += x.w * f;
        };
        for (int p0 = c0; p0 <= c1; p0 += 4) {
            float2 ml[4];
            float4 x[4], y[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (MANY) {
                    ml[i] = make_float2(kNegInf, 0.f);
                    if (p0 + i > c1) continue;
                }
                const int64_t slot = slot_of(min(p0 + i, c1));
                ml[i] = a.part_ml[slot * ROWS + r];
                const float4* o = reinterpret_cast<const float4*>(a.part_o + slot * ROWS * DH) + (col / 4 + 2 * warp) * ROWS + r;
                x[i] = o[0];
                y[i] = o[ROWS];
            }
            const float top = fmaxf(mm, fmaxf(fmaxf(ml[0].x, ml[1].x), fmaxf(ml[2].x, ml[3].x)));  // (the last may count twice)
            const float base = top == kNegInf ? 0.f : top, f0 = exp2_fast(mm - base);
            mm = top;
            ll *= f0;
#pragma unroll
            for (int i = 0; i < 2; ++i) acc[i] = make_float4(acc[i].x * f0, acc[i].y * f0, acc[i].z * f0, acc[i].w * f0);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (p0 + i > c1) break;
                const float f = exp2_fast(ml[i].x - base);
                ll += ml[i].y * f;
                add(acc[0], x[i], f);
                add(acc[1], y[i], f);
            }
        }
        const float inv = ll == 0.f ? 0.f : 1.f / ll;
        bool bad = ll != ll;
        __syncthreads();
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const float4 o = acc[x];
            bad |= o.x != o.x || o.y != o.y || o.z != o.z || o.w != o.w;
            rows_out[lane][4 * warp + 2 * x] = Elem<T>::pack(o.x * inv, o.y * inv);
            rows_out[lane][4 * warp + 2 * x + 1] = Elem<T>::pack(o.z * inv, o.w * inv);
        }
        const unsigned bads = __ballot_sync(~0u, bad && r < rows);
        if (lane == 0 && bads) atomicOr(&bad_rows, bads);
        if (warp == 0 && col == 0 && r < rows && a.lse) {
            int i, hg;
            row_of(kv, r0 + r, i, hg);
            a.lse[static_cast<int64_t>(rec.q0 + i) * kv.hq + rec.h * kv.group + hg] = ll == 0.f ? kNegInf : (mm + log2f(ll)) * kLn2;
        }
        __syncthreads();
        const unsigned again = bad_rows;
        for (int y = warp; y < 32 && 32 * g + y < rows; y += kJoinWarps) {
            int i, hg;
            row_of(kv, r0 + 32 * g + y, i, hg);
            const int tok = rec.q0 + i, head = rec.h * kv.group + hg;
            if (again >> y & 1) {
                attend_row<T>(a, rec.b, tok, head, rec.pos0 + i, col, col + 64);
                continue;
            }
            if (col + 2 * lane < kv.d)
                reinterpret_cast<uint32_t*>(static_cast<T*>(a.out) + tok * a.o_ts + head * a.o_hs + col)[lane] = rows_out[y][lane];
        }
        __syncthreads();
    }
}

template <typename T, int ROWS, int DH>
cudaError_t launch_attend_join(const AttendArgs& a, int n_ctas, cudaStream_t st) {
    return launch_in_stream(attend_join_kernel<T, ROWS, DH>, dim3(n_ctas - 1), kJoinWarps * 32, 0, 1, st, a);
}
// tiles: row tiles of the call at most.
template <typename T, int ROWS, int DH>
cudaError_t launch_attend_join_rows(const AttendArgs& a, int n_ctas, int64_t tiles, cudaStream_t st) {
    auto kernel = n_ctas > 4 * tiles ? attend_join_rows_kernel<T, ROWS, DH, true> : attend_join_rows_kernel<T, ROWS, DH, false>;
    return launch_in_stream(kernel, dim3(n_ctas - 1, ROWS / 32 * (DH / 64) / 2), kJoinWarps * 32, 0, 1, st, a);
}

}  // namespace moe

// Device helpers shared by the attention kernels: element types, the ragged
// batch, the deal of row tiles and key units over the grid, and the exact row.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "attention.h"
#include "common.cuh"

namespace moe {

template <typename T>
struct Elem;
template <>
struct Elem<__nv_bfloat16> {
    static __device__ __forceinline__ float2 unpack(uint32_t w) {
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    }
    static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
        uint32_t r;
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;\n" : "=r"(r) : "f"(hi), "f"(lo));
        return r;
    }
};
template <>
struct Elem<__half> {
    static __device__ __forceinline__ float2 unpack(uint32_t w) {
        return __half22float2(*reinterpret_cast<const __half2*>(&w));
    }
    static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
        uint32_t r;
        asm("cvt.rn.f16x2.f32 %0, %1, %2;\n" : "=r"(r) : "f"(hi), "f"(lo));
        return r;
    }
};

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
    return y;
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ uint64_t pair(float x, float y) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};\n" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ float2 unpair(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;\n" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// Every kernel here is launched beside the end of the one before it in the stream: it waits for that one's
// end (and with it for all before) first, and only then lets the next be launched, so that what a kernel may
// rely on when it starts is complete.
__device__ __forceinline__ void wait_for_stream() {
    asm volatile("griddepcontrol.wait;\ngriddepcontrol.launch_dependents;\n" ::: "memory");
}

// The same where the next kernel begins beside this one and does not wait for it: it relies on what was complete when this one
// began.  The wait makes that visible to this grid; the fences, here before the launch and there at its beginning
// (begin_beside), carry it on, with the launch in the place of a flag that is written and read.  That a launch orders as
// much as such a flag does is taken for granted: the instructions' description says when the next may start, and no more.
__device__ __forceinline__ void wait_and_hand_on() {
    asm volatile("griddepcontrol.wait;\nfence.acq_rel.gpu;\ngriddepcontrol.launch_dependents;\n" ::: "memory");
}
__device__ __forceinline__ void begin_beside() { asm volatile("fence.acq_rel.gpu;\ngriddepcontrol.launch_dependents;\n" ::: "memory"); }

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kNegInf = -INFINITY;

// ---------------------------------------------------------------- the ragged batch
__device__ __forceinline__ int div_by(int n, const Divisor& d) {
    return static_cast<int>((__umulhi(n, d.mul) + static_cast<uint32_t>(n)) >> d.shift);
}
// A quotient of the line's units: almost always of 32-bit numbers, which is several times shorter.
__device__ __forceinline__ long long div_line(long long n, long long d) {
    if (((n | d) >> 32) == 0) return static_cast<uint32_t>(n) / static_cast<uint32_t>(d);
    return n / d;
}
// Row r of a sequence's (token, head of the group) rows.
__device__ __forceinline__ void row_of(const KvArgs& a, int r, int& tok, int& g) {
    tok = div_by(r, a.by_group);
    g = r - tok * a.group;
}

struct SeqInfo {
    int q0;     // first token
    int q_len;
    int pos0;   // position of the first token (may be negative)
};

__device__ __forceinline__ SeqInfo seq_info(const KvArgs& a, int b) {
    SeqInfo s;
    const int e = min(max(__ldg(a.q_start + b + 1), 0), a.n_tokens);
    s.q0 = min(max(__ldg(a.q_start + b), 0), a.n_tokens);
    s.q_len = max(e - s.q0, 0);
    s.pos0 = max(__ldg(a.kv_len + b), 0) - s.q_len;
    return s;
}

// Page id of `idx` of sequence b, or -1 where there is none to read.
__device__ __forceinline__ int page_id(const KvArgs& a, int b, int idx) {
    if (idx >= a.width) return -1;
    const int id = __ldg(a.table + static_cast<int64_t>(b) * a.width + idx);
    return id >= 0 && id < a.n_pages ? id : -1;
}

// The last position that a window ending at position p leaves out, or -1: not below, so that what is taken from it stays
// in 32 bits whatever the window (p may be negative).
__device__ __forceinline__ int before_window(int window, int p) { return window > 0 && p >= window ? p - window : -1; }

// Keys [lo, hi) that rows [r0, r1) (row = token * group + head of the group) see, at least one of them.
__device__ __forceinline__ void key_range(const KvArgs& a, int window, const SeqInfo& s, int r0, int r1, int& lo, int& hi) {
    const int p0 = s.pos0 + div_by(r0, a.by_group), p1 = s.pos0 + div_by(r1 - 1, a.by_group);
    hi = min(p1, a.cap - 1) + 1;
    lo = before_window(window, p0) + 1;
    if (hi <= lo) lo = hi = 0;
}

// ---------------------------------------------------------------- the deal
// The batch's work is a line of units: sequence by sequence, row tile by row tile (ROWS rows of one
// sequence's token-major (token, head of the group) rows), key/value head by head, key unit by key
// unit (KEYS consecutive positions).  CTA c takes units [c per, (c + 1) per), so the grid's shares
// differ by one unit at most however ragged the batch is.  Pieces of a cut tile are put together by the
// join.  A tile whose rows see nothing has one unit (its rows still have to be written), and each tile
// counts `extra` units more at its end, for what a CTA spends on beginning and ending it.
struct Deal {
    int split;           // 0: a tile is one unit of the line
    int extra;
};

template <int ROWS>
__device__ __forceinline__ int row_tiles(const AttendArgs& a, const SeqInfo& s) {
    const int rows = s.q_len * a.kv.group;
    return rows < a.rows_lo || rows > a.rows_hi ? 0 : (rows + ROWS - 1) / ROWS;
}
// First key unit and number of key units of row tile rt.
template <int ROWS, int KEYS>
__device__ __forceinline__ int key_units(const AttendArgs& a, const SeqInfo& s, int rt, int& first) {
    const int r1 = min((rt + 1) * ROWS, s.q_len * a.kv.group);
    int lo, hi;
    key_range(a.kv, a.window, s, rt * ROWS, r1, lo, hi);
    first = lo / KEYS;
    return max((hi + KEYS - 1) / KEYS - first, 1);
}
// What the tile counts for in the line.
template <int ROWS, int KEYS>
__device__ __forceinline__ int tile_weight(const AttendArgs& a, const Deal& d, const SeqInfo& s, int rt) {
    if (!d.split) return 1;
    int first;
    const int n = key_units<ROWS, KEYS>(a, s, rt, first);
    return n + d.extra;
}

struct Cursor {
    long long u, end;  // the CTA's next place in the line, and its end
    long long begin;   // where it began
    int b, rt, h;      // the tile there
    int first, n;      // its first key unit and its key units
    int off, take;     // the key units before this piece, and the piece's
    int pass;          // how far the piece reaches in the line
    SeqInfo s;
    Deal d;
    __device__ __forceinline__ bool whole() const { return take == n; }
};

// The keys of the piece that begins at `off` of its tile (none where that is in the tile's extra units).
__device__ __forceinline__ void deal_take(Cursor& c) {
    if (!c.d.split) {
        c.take = c.n;
        c.pass = 1;
        return;
    }
    c.pass = static_cast<int>(min(static_cast<long long>(c.n + c.d.extra - c.off), c.end - c.u));
    c.take = max(min(c.n, c.off + c.pass) - c.off, 0);
}

// prefix[b] = the line's length before sequence b, prefix[n_seqs] all of it.  Called by the whole block.
template <int ROWS, int KEYS>
__device__ __forceinline__ void deal_prefix(const AttendArgs& a, const Deal& d, long long* prefix) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int B = a.kv.n_seqs;
    constexpr int kFew = 8;           // more tiles than this are summed by a warp
    constexpr long long kOpen = -1;
    for (int b = threadIdx.x; b < B; b += blockDim.x) {
        const SeqInfo s = seq_info(a.kv, b);
        const int nt = row_tiles<ROWS>(a, s);
        long long sum = 0;
        for (int rt = 0; rt < nt && nt <= kFew; ++rt) sum += tile_weight<ROWS, KEYS>(a, d, s, rt);
        prefix[b + 1] = nt <= kFew ? sum * a.kv.hkv : kOpen;
    }
    __syncthreads();
    for (int b = warp; b < B; b += warps) {
        if (prefix[b + 1] != kOpen) continue;
        const SeqInfo s = seq_info(a.kv, b);
        const int nt = row_tiles<ROWS>(a, s);
        long long sum = 0;
        for (int rt = lane; rt < nt; rt += 32) sum += tile_weight<ROWS, KEYS>(a, d, s, rt);
#pragma unroll
        for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
        if (lane == 0) prefix[b + 1] = sum * a.kv.hkv;
    }
    __syncthreads();
    if (warp == 0) {
        long long carry = 0;
        if (lane == 0) prefix[0] = 0;
        for (int b0 = 0; b0 < B; b0 += 32) {
            long long x = b0 + lane < B ? prefix[b0 + lane + 1] : 0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long y = __shfl_up_sync(~0u, x, o);
                if (lane >= o) x += y;
            }
            if (b0 + lane < B) prefix[b0 + lane + 1] = x + carry;
            carry += __shfl_sync(~0u, x, 31);
        }
    }
    __syncthreads();
}

// Past the current piece, to the next one that has keys.
template <int ROWS, int KEYS>
__device__ __forceinline__ void deal_next(const AttendArgs& a, Cursor& c) {
    do {
        c.u += c.pass;
        c.off = 0;
        if (c.u >= c.end) return;
        if (++c.h == a.kv.hkv) {
            c.h = 0;
            ++c.rt;
            while (c.rt >= row_tiles<ROWS>(a, c.s)) {  // ends at the sequence that holds unit u
                c.s = seq_info(a.kv, ++c.b);
                c.rt = 0;
            }
            c.n = key_units<ROWS, KEYS>(a, c.s, c.rt, c.first);
        }
        deal_take(c);
    } while (c.take == 0);
}

// Inclusive sums over a warp's lanes.
__device__ __forceinline__ long long lane_sums(long long x) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(~0u, x, o);
        if ((threadIdx.x & 31) >= o) x += y;
    }
    return x;
}

constexpr int kDealWords = 32;  // shared words of deal_begin beside one per sequence

// The share of CTA (or pair of CTAs) `me` of `all`.  Called by the whole block.  prefix: n_seqs + kDealWords
// shared words.  A share has min_per units at least.  Sets `c` in every thread, and this CTA's record of the
// tile that its share begins in.  Batches of up to 32 sequences (where the time until a CTA knows its share counts) are dealt
// by one warp, a lane per sequence: 2.2 us from the kernel's start for 8 sequences, against 3.3 with the block.
template <int ROWS, int KEYS>
__device__ void deal_begin(const AttendArgs& a, long long* prefix, int min_per, int extra, int me, int all, Cursor& c) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int B = a.kv.n_seqs;
    c.d.split = a.split;
    c.d.extra = extra;
    c.b = c.rt = c.h = c.off = c.take = c.pass = c.first = c.n = 0;
    long long total = 0, per = 1, rel = 0;
    int nt = 0;  // row tiles of the sequence that the share begins in
    auto place = [&]() {
        per = max(div_line(total + all - 1, all), static_cast<long long>(a.split ? min_per : 0));
        c.u = c.begin = min(me * per, total);
        c.end = min(c.u + per, total);
    };
    if (B <= 32) {
        if (warp == 0) {
            SeqInfo s = {0, 0, 0};
            int own = 0;
            if (lane < B) {
                s = seq_info(a.kv, lane);
                own = row_tiles<ROWS>(a, s);
            }
            auto length = [&]() {  // of this lane's sequence in the line
                constexpr int kFew = 4;  // more tiles than this are summed by the warp
                long long sum = 0;
                for (int rt = 0; rt < own && own <= kFew; ++rt) sum += tile_weight<ROWS, KEYS>(a, c.d, s, rt);
                for (unsigned many = __ballot_sync(~0u, own > kFew); many; many &= many - 1) {
                    const int src = __ffs(many) - 1, n = __shfl_sync(~0u, own, src);
                    const SeqInfo o = {__shfl_sync(~0u, s.q0, src), __shfl_sync(~0u, s.q_len, src), __shfl_sync(~0u, s.pos0, src)};
                    long long part = 0;
                    for (int rt = lane; rt < n; rt += 32) part += tile_weight<ROWS, KEYS>(a, c.d, o, rt);
#pragma unroll
                    for (int x = 16; x; x >>= 1) part += __shfl_xor_sync(~0u, part, x);
                    if (lane == src) sum = part;
                }
                return sum * a.kv.hkv;
            };
            const long long len = length(), sums = lane_sums(len);
            total = __shfl_sync(~0u, sums, 31);
            place();
            if (c.u < c.end) {
                c.b = __ffs(__ballot_sync(~0u, sums > c.u)) - 1;
                rel = c.u - __shfl_sync(~0u, sums - len, c.b);
                c.s = {__shfl_sync(~0u, s.q0, c.b), __shfl_sync(~0u, s.q_len, c.b), __shfl_sync(~0u, s.pos0, c.b)};
                nt = __shfl_sync(~0u, own, c.b);
            }
        }
    } else {
        deal_prefix<ROWS, KEYS>(a, c.d, prefix);
        total = prefix[B];
        place();
        if (warp == 0 && c.u < c.end) {
            int lo = 0, hi = B - 1;  // the sequence that holds unit u: the last b with prefix[b] <= u
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (prefix[mid] <= c.u) lo = mid;
                else hi = mid - 1;
            }
            c.b = lo;
            c.s = seq_info(a.kv, lo);
            nt = row_tiles<ROWS>(a, c.s);
            rel = c.u - prefix[lo];
        }
    }
    Cursor* shared = reinterpret_cast<Cursor*>(prefix + B + 2);
    static_assert(sizeof(Cursor) + 2 * 8 <= kDealWords * 8, "deal_begin's shared words");
    if (warp == 0) {
        int idx = 0;
        if (c.u < c.end) {
            for (int t0 = 0;; t0 += 32) {  // the sequence's tiles, 32 at a time
                const int rt = t0 + lane;
                const int n = rt < nt ? tile_weight<ROWS, KEYS>(a, c.d, c.s, rt) : 0;
                const long long x = lane_sums(static_cast<long long>(n) * a.kv.hkv);
                const unsigned past = __ballot_sync(~0u, x > rel);
                if (past || t0 + 32 >= nt) {
                    const int l = past ? __ffs(past) - 1 : 31;
                    rel -= __shfl_sync(~0u, x - static_cast<long long>(n) * a.kv.hkv, l);
                    const int weight = max(__shfl_sync(~0u, n, l), 1);
                    c.rt = min(t0 + l, nt - 1);
                    c.h = static_cast<int>(div_line(rel, weight));
                    idx = static_cast<int>(rel - static_cast<long long>(c.h) * weight);
                    break;
                }
                rel -= __shfl_sync(~0u, x, 31);
            }
            c.n = key_units<ROWS, KEYS>(a, c.s, c.rt, c.first);
            c.off = a.split ? idx : 0;
            deal_take(c);
        }
        if (lane == 0 && a.split) {
            BoundaryRec r;
            r.begin = c.u - idx;
            r.per = per;
            r.n = c.n;
            r.cut = idx > 0 && idx < r.n;
            r.rt = c.rt;
            r.h = c.h;
            r.q0 = c.s.q0;
            r.q_len = c.s.q_len;
            r.pos0 = c.s.pos0;
            r.b = c.b;
            a.recs[me] = r;
        }
        if (c.u < c.end && c.take == 0) deal_next<ROWS, KEYS>(a, c);
        if (lane == 0) *shared = c;
    }
    __syncthreads();
    c = *shared;
}

// ---------------------------------------------------------------- the exact row
// One (token, head) row over the positions it sees and no others, by one warp.  The tiled kernels
// multiply the values of a masked position by a weight of zero, which is no zero where the value is
// not finite; a row that ends with a NaN is therefore taken again here.  (A row whose NaN is its own
// comes out the same.)  Writes components [col0, col1), and lse with component 0.
template <typename T>
__device__ __noinline__ void attend_row(const AttendArgs& a, int b, int token, int head, int pos, int col0 = 0, int col1 = 256) {
    const int lane = threadIdx.x & 31;
    const bool on = lane * 8 < a.kv.d;
    const int hk = head / a.kv.group;
    float q[8] = {}, o[8] = {};
    if (on) {
        const uint4 w = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.q) + token * a.q_ts + head * a.q_hs + lane * 8);
        const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = Elem<T>::unpack(ww[i]);
            q[2 * i] = f.x;
            q[2 * i + 1] = f.y;
        }
    }
    const int hi = min(pos, a.kv.cap - 1) + 1;
    const int lo = before_window(a.window, pos) + 1;
    const float c = a.scale * kLog2e;
    float m = kNegInf, l = 0.f;
    for (int j = lo; j < hi; ++j) {
        const int at = div_by(j, a.kv.by_page), id = page_id(a.kv, b, at);
        const int64_t row = j - at * a.kv.page;
        uint4 kw = make_uint4(0, 0, 0, 0), vw = kw;
        if (on && id >= 0) {
            kw = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.kv.k) + id * a.kv.k_ps + row * a.kv.k_rs + hk * a.kv.k_hs + lane * 8);
            vw = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.kv.v) + id * a.kv.v_ps + row * a.kv.v_rs + hk * a.kv.v_hs + lane * 8);
        }
        const uint32_t k4[4] = {kw.x, kw.y, kw.z, kw.w}, v4[4] = {vw.x, vw.y, vw.z, vw.w};
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = Elem<T>::unpack(k4[i]);
            s += q[2 * i] * f.x + q[2 * i + 1] * f.y;
        }
#pragma unroll
        for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(~0u, s, x);
        s *= c;
        const float mn = fmaxf(m, s);  // a NaN score is not the maximum, but it reaches l below
        const float base = mn == kNegInf ? 0.f : mn;
        const float f = exp2f(m - base), p = exp2f(s - base);
        m = mn;
        l = l * f + p;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 g = Elem<T>::unpack(v4[i]);
            o[2 * i] = o[2 * i] * f + p * g.x;
            o[2 * i + 1] = o[2 * i + 1] * f + p * g.y;
        }
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    if (on && lane * 8 >= col0 && lane * 8 < col1) {
        uint4 w;
        w.x = Elem<T>::pack(o[0] * inv, o[1] * inv);
        w.y = Elem<T>::pack(o[2] * inv, o[3] * inv);
        w.z = Elem<T>::pack(o[4] * inv, o[5] * inv);
        w.w = Elem<T>::pack(o[6] * inv, o[7] * inv);
        *reinterpret_cast<uint4*>(static_cast<T*>(a.out) + token * a.o_ts + head * a.o_hs + lane * 8) = w;
    }
    if (lane == 0 && col0 == 0 && a.lse) a.lse[static_cast<int64_t>(token) * a.kv.hq + head] = l == 0.f ? kNegInf : (m + log2f(l)) * kLn2;
}

// Rows of the tokens that belong to no sequence: zeros, and -inf.  Called by the whole grid.
template <typename T>
__device__ void clear_stray_rows(const AttendArgs& a) {
    if (!a.lead) return;
    const int s0 = min(max(__ldg(a.kv.q_start), 0), a.kv.n_tokens);
    const int s1 = min(max(__ldg(a.kv.q_start + a.kv.n_seqs), s0), a.kv.n_tokens);
    const int stray = s0 + a.kv.n_tokens - s1;
    if (stray == 0) return;
    for (int i = blockIdx.x; i < stray; i += gridDim.x) {
        const int t = i < s0 ? i : s1 + (i - s0);
        const int chunks = a.kv.d / 8;
        for (int x = threadIdx.x; x < a.kv.hq * chunks; x += blockDim.x)
            *reinterpret_cast<uint4*>(static_cast<T*>(a.out) + t * a.o_ts + (x / chunks) * a.o_hs + (x % chunks) * 8) =
                make_uint4(0, 0, 0, 0);
        if (a.lse)
            for (int x = threadIdx.x; x < a.kv.hq; x += blockDim.x) a.lse[static_cast<int64_t>(t) * a.kv.hq + x] = kNegInf;
    }
}

// Launches `kernel` as above, in clusters of `cluster` blocks.
template <typename... Params, typename... Args>
cudaError_t launch_in_stream(void (*kernel)(Params...), dim3 grid, int block, size_t smem, int cluster, cudaStream_t st, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = cluster;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace moe

// Attention over the paged cache with the keys split over the warps of the
// whole GPU, on mma.sync: the engine of decoding batches (a few rows against a
// long cache).
//
// Per row: s_j = scale q . k_j over the positions j that the row sees; with a
// running maximum m, l = sum_j 2^(s_j log2 e - m) and o = sum_j 2^(s_j log2 e - m) v_j
// are kept in fp32 in one pass over the cache and rescaled when m grows; the
// row is o / l.  Rows of one key/value head are taken together (token-major:
// row = token * group + head of the group), 16 at a time, so the cache is read
// once for a group's heads.
//
// Bound: HBM, the K and V bytes of the visible positions.  A CTA is 8 warps
// (4 at D = 256) of their own pipelines: a warp takes 16 keys at a time, K and V by
// 16-byte cp.async into its own ring (chunks XOR-swizzled by row so that
// ldmatrix reads without bank conflicts), and keeps its own m, l, o; no
// barrier inside a piece.  At a piece's end the warps' states are joined in
// shared memory, while the copies of the CTA's next piece are on their way: a
// warp's copies run through its units of all pieces without a stop.  The pieces
// come from the deal; pieces of one row tile go to the workspace and a second
// kernel joins them in a fixed order.
#include "attend_join.cuh"
#include "attention_common.cuh"

namespace moe {
namespace {

constexpr int kKeys = 16;       // keys of a unit: one warp's step
constexpr int kMinShare = 4;    // units of a CTA at least, where there are few
// What a tile's beginning and end count for: 64 ragged decoding sequences (up to 16384 positions, 32 / 8
// heads of 128) 213.5 us, without it 220.
constexpr int kExtra = 4;

template <int DH>
struct SplitCfg {
    static constexpr int kWarps = DH == 256 ? 4 : 8;
    static constexpr int kStages = DH == 64 ? 6 : 3;
    static constexpr int kCpr = DH / 8;                    // 16-byte chunks per row
    static constexpr int kTile = kKeys * DH;               // elements of K (or V) in a stage
    static constexpr int kQBytes = kSplitRows * DH * 2;
    static constexpr int kWarpBytes = kStages * 2 * kTile * 2;
    static constexpr int kStageBytes = 2 * kTile * 2;
    static constexpr int kOffRings = 2 * kQBytes;          // (the queries of this piece and of the next)
    static constexpr int kOffMl = kOffRings + kWarps * kWarpBytes;
    static constexpr int kOffStage = kOffMl + kWarps * kSplitRows * 8;
    static constexpr int kOffPrefix = kOffStage + kWarps * 4;
    static constexpr bool kQRegs = DH <= 128;              // the queries' fragments stay in registers
    static_assert(kStageBytes >= kSplitRows * DH * 4, "a stage holds a warp's state at the join");
};

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];\n"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];\n"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
template <typename T>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma16816<__nv_bfloat16>(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma16816<__half>(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Byte offset of 16-byte chunk c of row r in a tile whose rows are CPR chunks.
template <int CPR>
__device__ __forceinline__ uint32_t chunk_at(int r, int c) {
    return static_cast<uint32_t>(r * CPR + (c ^ (r & 7))) * 16;
}

// Where a warp's keys lie: the row offsets (elements) of a unit's 16 keys, one unit ahead of its
// copies, so that the page ids are on their way while the unit before is computed.  ALIGNED: pages
// of a multiple of 16 positions, a unit lies in one page; else each key is looked up by itself.
template <bool ALIGNED>
struct Rows {
    int64_t k, v;  // ALIGNED: of the unit's first key (every lane); else of key lane % 16
    bool ok;
    int id, at;    // the next unit's page and the key's (or first key's) row in it
    __device__ __forceinline__ void fetch(const KvArgs& a, int b, int unit, int end) {
        const int key = unit * kKeys + (ALIGNED ? 0 : (threadIdx.x & 15));
        const int p = div_by(key, a.by_page);
        at = key - p * a.page;
        id = unit < end ? page_id(a, b, p) : -1;
    }
    __device__ __forceinline__ void settle(const KvArgs& a, int h) {
        ok = id >= 0;
        const int64_t i = ok ? id : 0;
        k = i * a.k_ps + static_cast<int64_t>(at) * a.k_rs + h * a.k_hs;
        v = i * a.v_ps + static_cast<int64_t>(at) * a.v_rs + h * a.v_hs;
    }
};

// A warp's way through its keys: the unit whose copies come next, in its piece.
template <bool ALIGNED>
struct Feed {
    Cursor c;
    int unit, end;     // next unit of this warp in the piece, the piece's end
    int hi;            // keys from here on no row of the tile sees
    Rows<ALIGNED> rows;
    template <int WARPS>
    __device__ __forceinline__ void enter(const AttendArgs& a, int warp) {  // the cursor's piece, or a later one
        while (c.u < c.end) {
            int lo;
            const int r0 = c.rt * kSplitRows;
            key_range(a.kv, a.window, c.s, r0, min(r0 + kSplitRows, c.s.q_len * a.kv.group), lo, hi);
            unit = c.first + c.off + warp;
            end = c.first + c.off + c.take;
            if (unit < end) {
                rows.fetch(a.kv, c.b, unit, end);
                return;
            }
            deal_next<kSplitRows, kKeys>(a, c);
        }
    }
};

template <typename T, int DH, bool ALIGNED>
__global__ void __launch_bounds__(SplitCfg<DH>::kWarps * 32, 1) attend_split_kernel(const AttendArgs a) {
    using C = SplitCfg<DH>;
    extern __shared__ __align__(1024) unsigned char smem[];
    float2* ml = reinterpret_cast<float2*>(smem + C::kOffMl);  // [warps][rows]
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const KvArgs& kv = a.kv;
    const T* kc = static_cast<const T*>(kv.k);
    const T* vc = static_cast<const T*>(kv.v);
    int* ml_stage = reinterpret_cast<int*>(smem + C::kOffStage);  // [warps]
    unsigned char* ring = smem + C::kOffRings + warp * C::kWarpBytes;
    const int chunks = kv.d / 8;

    // components past D are never copied: zero once (rows of the ring, and of the queries)
    if (kv.d < DH)
        for (int i = threadIdx.x; i < C::kOffMl / 16; i += blockDim.x) reinterpret_cast<uint4*>(smem)[i] = make_uint4(0, 0, 0, 0);

    if (a.lead) wait_for_stream();
    else wait_and_hand_on();  // the tcgen05 kernel of the same batch comes next
    // a small table is brought near while the lengths are: its entries are the next to be waited for
    if (static_cast<int64_t>(kv.n_seqs) * kv.width <= 1024)
        for (int i = threadIdx.x * 8; i < kv.n_seqs * kv.width; i += blockDim.x * 8)
            asm volatile("prefetch.global.L1 [%0];\n" ::"l"(kv.table + i));
    if (a.lead && blockIdx.x == 0 && threadIdx.x == 0) a.hdr->status = kDevOk;  // (nothing here waits)
    Cursor c;
    deal_begin<kSplitRows, kKeys>(a, reinterpret_cast<long long*>(smem + C::kOffPrefix), kMinShare, kExtra, blockIdx.x, gridDim.x, c);
    clear_stray_rows<T>(a);
    const float sc = a.scale * kLog2e;

    Feed<ALIGNED> feed;
    feed.c = c;
    feed.template enter<C::kWarps>(a, warp);
    auto issue = [&](int stage) {
        if (feed.c.u < feed.c.end) {
            Rows<ALIGNED>& rw = feed.rows;
            rw.settle(kv, feed.c.h);
            unsigned char* sk = ring + stage * C::kStageBytes;
            const int key0 = feed.unit * kKeys;
            const bool all = key0 + kKeys <= feed.hi && rw.ok;  // (ALIGNED: every key of the unit is read)
            constexpr int kRowsPer = 32 / C::kCpr;
            const int x = lane % C::kCpr, row0 = lane / C::kCpr;
            // chunk_at(i kRowsPer + row0, x), its row's low bits apart: row0 is below kRowsPer
            unsigned char* at = sk + row0 * C::kCpr * 16;
            const int xs = x ^ (row0 & 7);
            const T *kp = kc + rw.k + row0 * kv.k_rs + x * 8, *vp = vc + rw.v + row0 * kv.v_rs + x * 8;
            const int64_t k_step = kRowsPer * kv.k_rs, v_step = kRowsPer * kv.v_rs;
#pragma unroll
            for (int i = 0; i < kKeys / kRowsPer; ++i) {
                const int r = i * kRowsPer + row0;
                bool ok;
                if constexpr (ALIGNED) {
                    ok = all || (rw.ok && key0 + r < feed.hi);
                } else {
                    ok = __shfl_sync(~0u, rw.ok ? 1 : 0, r) && key0 + r < feed.hi;
                    kp = kc + __shfl_sync(~0u, rw.k, r) + x * 8;
                    vp = vc + __shfl_sync(~0u, rw.v, r) + x * 8;
                }
                if (x < chunks) {  // a key that no row sees is zeros: whatever the cache holds there stays out
                    unsigned char* to = at + i * kRowsPer * C::kCpr * 16 + ((xs ^ (i * kRowsPer & 7)) << 4);
                    cp_async16(to, kp, ok ? 16 : 0);
                    cp_async16(to + C::kTile * 2, vp, ok ? 16 : 0);
                }
                if constexpr (ALIGNED) {
                    kp += k_step;
                    vp += v_step;
                }
            }
            feed.unit += C::kWarps;
            if (feed.unit < feed.end) {
                rw.fetch(kv, feed.c.b, feed.unit, feed.end);
            } else {
                deal_next<kSplitRows, kKeys>(a, feed.c);
                feed.template enter<C::kWarps>(a, warp);
            }
        }
        cp_async_commit();
    };
    // the queries of the cursor's tile; zeros past the rows
    auto queries = [&](int buf) {
        const int r0 = c.rt * kSplitRows, rows = min(c.s.q_len * kv.group - r0, kSplitRows);
        for (int i = threadIdx.x; i < kSplitRows * chunks; i += blockDim.x) {
            const int r = i / chunks, x = i - r * chunks;
            int tok, g;
            row_of(kv, r0 + min(r, rows - 1), tok, g);
            cp_async16(smem + buf * C::kQBytes + chunk_at<C::kCpr>(r, x),
                       static_cast<const T*>(a.q) + (c.s.q0 + tok) * a.q_ts + (c.h * kv.group + g) * a.q_hs + x * 8,
                       r < rows ? 16 : 0);
        }
        cp_async_commit();
    };
#pragma unroll
    for (int s = 0; s < C::kStages - 1; ++s) issue(s);
    int stage = 0, fill = C::kStages - 1, qb = 0;
    if (c.u < c.end) queries(0);
    cp_async_wait<0>();
    __syncthreads();

    while (c.u < c.end) {
        const int r0 = c.rt * kSplitRows;
        const int rows = min(c.s.q_len * kv.group - r0, kSplitRows);
        const int unit0 = c.first + c.off, unit1 = unit0 + c.take;
        const int mat = lane >> 3, mrow = lane & 7;
        uint32_t qf[C::kQRegs ? DH / 16 : 1][4];
        const uint32_t q_addr = smem_u32(smem + qb * C::kQBytes);
        if constexpr (C::kQRegs) {
#pragma unroll
            for (int ks = 0; ks < DH / 16; ++ks) ldsm4(qf[ks], q_addr + chunk_at<C::kCpr>((mat & 1) * 8 + mrow, ks * 2 + (mat >> 1)));
        }
        // this thread's two rows: positions they see
        int p_hi[2], p_lo[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int r = (lane >> 2) + 8 * x;
            const int p = c.s.pos0 + div_by(r0 + min(r, rows - 1), kv.by_group);
            p_hi[x] = min(p, kv.cap - 1);
            p_lo[x] = before_window(a.window, p);
        }
        const int all_hi = c.s.pos0 + div_by(r0, kv.by_group);                                          // every row sees keys <= all_hi
        const int all_lo = before_window(a.window, c.s.pos0 + div_by(r0 + rows - 1, kv.by_group));  // and > all_lo

        float o[DH / 8][4];
#pragma unroll
        for (int n = 0; n < DH / 8; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
        float m[2] = {kNegInf, kNegInf}, l[2] = {0.f, 0.f};

        for (int u = unit0 + warp; u < unit1; u += C::kWarps) {
            issue(fill);
            fill = fill + 1 == C::kStages ? 0 : fill + 1;
            cp_async_wait<C::kStages - 1>();
            __syncwarp();
            const uint32_t sk = smem_u32(ring + stage * 2 * C::kTile * 2), sv = sk + C::kTile * 2;
            stage = stage + 1 == C::kStages ? 0 : stage + 1;
            float s[2][4] = {}, s2[2][4] = {};  // (two sums each: the products of one wait for one another)
#pragma unroll
            for (int ks = 0; ks < DH / 16; ++ks) {
                uint32_t kf[4];
                ldsm4(kf, sk + chunk_at<C::kCpr>((mat >> 1) * 8 + mrow, ks * 2 + (mat & 1)));
                uint32_t qv[4];
                if constexpr (C::kQRegs) {
#pragma unroll
                    for (int x = 0; x < 4; ++x) qv[x] = qf[ks][x];
                } else {
                    ldsm4(qv, q_addr + chunk_at<C::kCpr>((mat & 1) * 8 + mrow, ks * 2 + (mat >> 1)));
                }
                mma16816<T>(ks & 1 ? s2[0] : s[0], qv, kf[0], kf[1]);
                mma16816<T>(ks & 1 ? s2[1] : s[1], qv, kf[2], kf[3]);
            }
            const int key0 = u * kKeys;
            const bool masked = key0 + kKeys - 1 > min(all_hi, kv.cap - 1) || key0 <= all_lo;
            float mx[2] = {kNegInf, kNegInf};
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float v = (s[n][i] + s2[n][i]) * sc;
                    if (masked) {
                        const int key = key0 + n * 8 + (lane & 3) * 2 + (i & 1);
                        if (key > p_hi[i >> 1] || key <= p_lo[i >> 1]) v = kNegInf;
                    }
                    s[n][i] = v;
                    mx[i >> 1] = fmaxf(mx[i >> 1], v);
                }
            bool grew = false;
            float base[2], f[2];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                mx[x] = fmaxf(mx[x], __shfl_xor_sync(~0u, mx[x], 1));
                mx[x] = fmaxf(mx[x], __shfl_xor_sync(~0u, mx[x], 2));
                const float mn = fmaxf(m[x], mx[x]);
                base[x] = mn == kNegInf ? 0.f : mn;
                f[x] = exp2_fast(m[x] - base[x]);
                grew |= mn != m[x];
                m[x] = mn;
            }
            if (__any_sync(~0u, grew)) {
#pragma unroll
                for (int n = 0; n < DH / 8; ++n) {
                    o[n][0] *= f[0];
                    o[n][1] *= f[0];
                    o[n][2] *= f[1];
                    o[n][3] *= f[1];
                }
                l[0] *= f[0];
                l[1] *= f[1];
            }
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    s[n][i] = exp2_fast(s[n][i] - base[i >> 1]);
                    l[i >> 1] += s[n][i];
                }
            // the weights as the second product's operand: rounded to the element type, their sum l is not
            const uint32_t pf[4] = {Elem<T>::pack(s[0][0], s[0][1]), Elem<T>::pack(s[0][2], s[0][3]),
                                    Elem<T>::pack(s[1][0], s[1][1]), Elem<T>::pack(s[1][2], s[1][3])};
#pragma unroll
            for (int j = 0; j < DH / 16; ++j) {
                uint32_t vf[4];
                ldsm4t(vf, sv + chunk_at<C::kCpr>((mat & 1) * 8 + mrow, j * 2 + (mat >> 1)));
                mma16816<T>(o[2 * j], pf, vf[0], vf[1]);
                mma16816<T>(o[2 * j + 1], pf, vf[2], vf[3]);
            }
            __syncwarp();  // the stage is read before its next copies
        }

        // this warp's state, in the stage whose copies come next (the others' are under way)
        ml_stage[warp] = fill;
        float* so = reinterpret_cast<float*>(ring + fill * C::kStageBytes);  // [rows][DH]
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            l[x] += __shfl_xor_sync(~0u, l[x], 1);
            l[x] += __shfl_xor_sync(~0u, l[x], 2);
            const int r = (lane >> 2) + 8 * x;
            if (r < rows) {
                if ((lane & 3) == 0) ml[warp * kSplitRows + r] = make_float2(m[x], l[x]);
#pragma unroll
                for (int n = 0; n < DH / 8; ++n)
                    *reinterpret_cast<float2*>(so + r * DH + n * 8 + (lane & 3) * 2) = make_float2(o[n][2 * x], o[n][2 * x + 1]);
            }
        }
        const bool whole = c.whole();
        const int64_t slot = 2 * static_cast<int64_t>(blockIdx.x) + (c.u == c.begin ? 0 : 1);
        const int q0 = c.s.q0, pos0 = c.s.pos0, h = c.h, b = c.b;
        deal_next<kSplitRows, kKeys>(a, c);
        qb ^= 1;
        if (c.u < c.end) queries(qb);  // of the next piece
        __syncthreads();
        // the join of the warps: a warp per row
        for (int r = warp; r < rows; r += C::kWarps) {
            float mw = kNegInf, lw = 0.f;
            if (lane < C::kWarps) {
                const float2 v = ml[lane * kSplitRows + r];
                mw = v.x;
                lw = v.y;
            }
            float mm = mw;
#pragma unroll
            for (int x = C::kWarps / 2; x; x >>= 1) mm = fmaxf(mm, __shfl_xor_sync(~0u, mm, x));
            mm = __shfl_sync(~0u, mm, 0);
            const float fw = mw == kNegInf ? 0.f : exp2_fast(mw - mm);
            float ll = lw * fw;
#pragma unroll
            for (int x = C::kWarps / 2; x; x >>= 1) ll += __shfl_xor_sync(~0u, ll, x);
            ll = __shfl_sync(~0u, ll, 0);
            float acc[DH / 32] = {};
#pragma unroll
            for (int w = 0; w < C::kWarps; ++w) {
                const float fx = __shfl_sync(~0u, fw, w);
                if (fx == 0.f) continue;
                const float* p = reinterpret_cast<const float*>(smem + C::kOffRings + w * C::kWarpBytes + ml_stage[w] * C::kStageBytes) + r * DH + lane * 2;
#pragma unroll
                for (int x = 0; x < DH / 64; ++x) {
                    const float2 v = *reinterpret_cast<const float2*>(p + x * 64);
                    acc[2 * x] += v.x * fx;
                    acc[2 * x + 1] += v.y * fx;
                }
            }
            if (whole) {
                int i, g;
                row_of(kv, r0 + r, i, g);
                const int tok = q0 + i, head = h * kv.group + g;
                const float inv = ll == 0.f ? 0.f : 1.f / ll;
                bool bad = ll != ll;
#pragma unroll
                for (int x = 0; x < DH / 32; ++x) bad |= acc[x] != acc[x];
                if (__any_sync(~0u, bad)) {
                    attend_row<T>(a, b, tok, head, pos0 + i);
                    continue;
                }
                T* dst = static_cast<T*>(a.out) + tok * a.o_ts + head * a.o_hs + lane * 2;
#pragma unroll
                for (int x = 0; x < DH / 64; ++x)
                    if (x * 64 + lane * 2 < kv.d)
                        *reinterpret_cast<uint32_t*>(dst + x * 64) = Elem<T>::pack(acc[2 * x] * inv, acc[2 * x + 1] * inv);
                if (lane == 0 && a.lse) a.lse[static_cast<int64_t>(tok) * kv.hq + head] = ll == 0.f ? kNegInf : (mm + log2f(ll)) * kLn2;
            } else {
                float* dst = a.part_o + (slot * kSplitRows + r) * DH + lane * 2;
#pragma unroll
                for (int x = 0; x < DH / 64; ++x) *reinterpret_cast<float2*>(dst + x * 64) = make_float2(acc[2 * x], acc[2 * x + 1]);
                if (lane == 0) a.part_ml[slot * kSplitRows + r] = make_float2(mm, ll);
            }
        }
        cp_async_wait<0>();
        __syncthreads();
        if (kv.d < DH) {  // the state overwrote the stage's zero columns
            for (int i = lane; i < C::kStageBytes / 16; i += 32) reinterpret_cast<uint4*>(ring + fill * C::kStageBytes)[i] = make_uint4(0, 0, 0, 0);
            __syncwarp();
        }
    }
}

template <typename T, int DH, bool ALIGNED>
cudaError_t launch_t(const AttendArgs& a, int n_ctas, int max_items, cudaStream_t st) {
    using C = SplitCfg<DH>;
    const int smem = C::kOffPrefix + (a.kv.n_seqs + kDealWords) * 8;
    cudaError_t e = cudaFuncSetAttribute(attend_split_kernel<T, DH, ALIGNED>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    const int grid = a.split ? n_ctas : max(1, min(max_items, n_ctas * 8));
    return launch_in_stream(attend_split_kernel<T, DH, ALIGNED>, dim3(grid), C::kWarps * 32, smem, 1, st, a);
}

template <typename T, int DH>
cudaError_t launch_d(const AttendArgs& a, int n_ctas, int max_items, cudaStream_t st) {
    return a.kv.page % kKeys == 0 ? launch_t<T, DH, true>(a, n_ctas, max_items, st) : launch_t<T, DH, false>(a, n_ctas, max_items, st);
}

template <typename T>
cudaError_t launch_j(const AttendArgs& a, int n_ctas, cudaStream_t st) {
    switch (padded_dim(a.kv.d)) {
        case 64: return launch_attend_join<T, kSplitRows, 64>(a, n_ctas, st);
        case 128: return launch_attend_join<T, kSplitRows, 128>(a, n_ctas, st);
        default: return launch_attend_join<T, kSplitRows, 256>(a, n_ctas, st);
    }
}

template <typename T>
cudaError_t launch_e(const AttendArgs& a, int n_ctas, int max_items, cudaStream_t st) {
    switch (padded_dim(a.kv.d)) {
        case 64: return launch_d<T, 64>(a, n_ctas, max_items, st);
        case 128: return launch_d<T, 128>(a, n_ctas, max_items, st);
        default: return launch_d<T, 256>(a, n_ctas, max_items, st);
    }
}

}  // namespace

cudaError_t launch_attend_split_join(const AttendArgs& a, int dtype, int n_ctas, cudaStream_t st) {
    if (!a.split || n_ctas < 2) return cudaSuccess;
    return dtype == 0 ? launch_j<__nv_bfloat16>(a, n_ctas, st) : launch_j<__half>(a, n_ctas, st);
}

cudaError_t launch_attend_split(const AttendArgs& a, int dtype, int n_ctas, int max_items, cudaStream_t st) {
    return dtype == 0 ? launch_e<__nv_bfloat16>(a, n_ctas, max_items, st) : launch_e<__half>(a, n_ctas, max_items, st);
}

}  // namespace moe

// Attention over the paged cache on the fifth-generation tensor cores: the
// engine of chunks and prompts (many rows against the same keys).
//
// The mathematics is attend_split.cu's: one pass over the keys with a running
// reference m and sum l per row, s = scale q . k, p = 2^(s log2 e - m), o = sum p v,
// the row is o / l.  Rows are (token, head of the group) pairs of one
// key/value head, token-major, so a tile of 128 rows reads the cache once for
// all heads of the group.
//
// Bound: the tensor pipe (4 D flops per pair and head) against the 2^x of the
// special-function units and their surrounding instructions (one per pair and
// head).  Per tile of 128 rows x 128 keys: S = Q K^T (operands in shared memory, 128 fp32
// accumulator columns in tensor memory), two softmax warpgroups read S and write P back over S as
// packed 16-bit values, and O += P V takes P from tensor memory and V from shared
// memory as an MN-major operand (rows of the cache are rows of K there, no transposition).
//   D <= 128: two tiles of 128 rows per CTA share the keys' tiles; while one tile's
//     softmax runs the tensor pipe does the other's products.  (D <= 64 has columns to spare: P gets its
//     own, and S of the next keys follows as soon as S is read.)
//   D <= 256: one tile (O takes 256 of the 512 columns); S is double-buffered, so the
//     tensor pipe does the next keys' S while the softmax of this one runs; so too with D <= 128 where
//     the rows fill one tile only.
//   D > 64: CTAs work in pairs (cta_group::2): an MMA covers 256 rows, 128 of each CTA, and each CTA
//     brings half of K (64 keys) and half of V (half the components), so the bytes that
//     each SM takes from L2, and from its shared memory for an MMA, are halved.
// The reference m is raised, and O rescaled, only when a row's maximum has grown
// by more than 2^8 over it: P stays below 2^8 (exact enough in 16 bits: the rounding is relative)
// and almost every tile leaves O alone.
//
// K and V come by TMA straight from the pages (4-D map: component, row, head,
// page; boxes of as many rows as divide both page and tile), into a ring of
// slots; pages that are not there and rows past the last visible one read zeros, and
// the rows of V behind it inside a box are cleared by hand, so whatever the cache holds there
// stays out of the sums.  Work is dealt in equal shares of 128-key units; the pieces of a cut
// tile go through the workspace and the join.
//
// Warps: 0 MMA issue (one lane) and the tensor-memory allocation, 1 the K tiles, 3 the V tiles (a
// box takes its lane about 100 cycles to issue, and pages of 16 make 16 boxes a tile), 2 Q, then two
// warpgroups per row tile: softmax and output, a thread for half of a row's keys (64 of a tile's 128)
// and half of its output, so that the way from S to P is half as long; the halves exchange their
// maxima through shared memory.
// Measured: 8192-token prompt, 16 / 2 heads of 256: 332 to 340 us by the card, 1.65 PFLOP/s, 86% of the tensor pipe's
// cycles; 4096 tokens of 32 / 8 heads of 128 139 us, 0.99 PFLOP/s (softmax, P, P V and the next Q K in a chain); heads
// of 64 107 us, 0.64 PFLOP/s.  At 64 and 128 components the 96 registers a thread do not hold everything: 56 bytes of
// stack, 468 and 524 bytes of spill loads (none at 256).  Alternating S buffers for a single row tile: 32 sequences of 8 tokens at 8000
// positions 343 -> 244 us, for which that 4096-token prompt went from 142 to 146 when it came.
// Every wait is bounded; a timeout sets the status word and every role leaves, having waited (again with a limit) for
// its own copies in flight.  The softmax warps' exchange is ended by the warp that leaves (pair_exchange.h).
#include <algorithm>

#include "attend_join.cuh"
#include "attention_common.cuh"
#include "pair_exchange.h"
#include "tcgen05.cuh"

namespace moe {
namespace {

constexpr int kTcKeys = 128;  // keys of a unit

template <int DH>
struct TcCfg {
    static constexpr int CG = DH == 64 ? 1 : 2;         // CTAs that share a tile of keys
    static constexpr int NQ = DH == 256 ? 1 : 2;        // row tiles of 128 per CTA
    static constexpr int kTile = 128 * CG;              // rows of a tile over its CTAs
    static constexpr int kRows = kTile * NQ;
    static constexpr int kKKeys = kTcKeys / CG;         // a CTA's share of K: these keys, all components,
    static constexpr int kVCols = DH / CG;              // of V: all keys, these components
    static constexpr int kKBlocks = DH / 64, kVBlocks = kVCols / 64;  // in column blocks of 64
    static constexpr int kSlot = kKKeys * DH * 2;
    static constexpr int kSlots = DH == 64 ? 10 : DH == 128 ? 9 : 5;
    // Key tiles that a row tile's beginning and end count for.  A 4096-token prompt of 32 / 8 heads of 128 takes 140 us,
    // without it 224 (heads of 64 107 and 207, 16 / 2 of 256 100 and 164): the first row tiles are short,
    // so an equal share of keys holds many of them.
    static constexpr int kExtra = 3;
    static constexpr bool kOwnP = DH == 64;             // P has columns of its own, so S is free once it is read
    // K tiles ahead of V, by the row tiles that have rows
    static __device__ constexpr int look(int act) { return act == 2 && !kOwnP ? 1 : 2; }
    static constexpr int kQTile = 128 * DH * 2;
    static constexpr int kThreads = 128 + 256 * NQ;
    static constexpr int kSCol = 0, kOCol = 256;        // two S buffers of 128 columns, then O
    static constexpr int kPCol = kOwnP ? kOCol + NQ * DH : kSCol, kPStep = kOwnP ? 64 : 128;  // P, by buffer
    static constexpr int kOffQ = 0;
    static constexpr int kOffRing = kOffQ + NQ * kQTile;
    static constexpr int kOffEx = kOffRing + kSlots * kSlot;  // [NQ][2][2][128]: what the halves of a row exchange
    static constexpr int kOffBars = kOffEx + NQ * 2048;
    static constexpr int kBars = 2 * kSlots + 11 + 3 * NQ + 2;
    static constexpr int kOffMisc = kOffBars + 8 * kBars;
    static constexpr int kOffStart = kOffMisc + 16;     // the cursor at the share's beginning
    static constexpr int kSmem = kOffStart + sizeof(Cursor);
    static_assert((kOwnP ? kPCol + 2 * kPStep : kOCol + NQ * DH) <= 512, "tensor-memory columns");
    static_assert(kSmem <= 227 * 1024, "shared memory");
};

template <typename T>
struct MmaFmt;
template <>
struct MmaFmt<__nv_bfloat16> {
    static constexpr uint32_t v = 1;
};
template <>
struct MmaFmt<__half> {
    static constexpr uint32_t v = 0;
};

// kind::f16 instruction descriptor: fp32 accumulator, A and B of one type, M = m, N = n; b_mn: B is MN-major.
template <typename T>
__device__ constexpr uint32_t idesc16(int m, int n, bool b_mn) {
    return (1u << 4) | (MmaFmt<T>::v << 7) | (MmaFmt<T>::v << 10) | (b_mn ? 1u << 16 : 0u) | (static_cast<uint32_t>(n >> 3) << 17) |
           (static_cast<uint32_t>(m >> 4) << 24);
}

// The meeting of the two softmax warps of the same rows, at a named barrier.
struct WarpPairBarrier {
    int id;
    __device__ __forceinline__ void sync() { asm volatile("bar.sync %0, 64;\n" ::"r"(id) : "memory"); }
    __device__ __forceinline__ void arrive() { asm volatile("bar.arrive %0, 64;\n" ::"r"(id) : "memory"); }
};

__device__ __forceinline__ float max3(float x, float y, float z) {
    float r;
    asm("max.f32 %0, %1, %2, %3;\n" : "=f"(r) : "f"(x), "f"(y), "f"(z));
    return r;
}

// Of the rows of a softmax warp in the whole tiles from `c` on, those that ended with a NaN, taken again one by one
// (every second: the warp of the rows' other half has the others).  A row can take as long as its context is long:
// this comes after all the pieces, when no role waits for the warp.
template <typename T, int DH>
__device__ __noinline__ void retake_rows(const AttendArgs& a, Cursor c, int rank, int w, int quarter, int half) {
    using C = TcCfg<DH>;
    const KvArgs& kv = a.kv;
    const int lane = threadIdx.x & 31;
    while (c.u < c.end) {
        const int r0 = c.rt * C::kRows + C::kTile * w + 128 * rank;
        const int rows = c.whole() ? min(c.s.q_len * kv.group - r0, 32 * quarter + 32) : 0;
        for (int r = 32 * quarter + half; r < rows; r += 2) {
            int tok, hg;
            row_of(kv, r0 + r, tok, hg);
            const int head = c.h * kv.group + hg;
            bool odd = false;
            if (lane * 8 < kv.d) {
                const uint4 o = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.out) + (c.s.q0 + tok) * a.o_ts + head * a.o_hs + lane * 8);
                const uint32_t o4[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 f = Elem<T>::unpack(o4[i]);
                    odd |= f.x != f.x || f.y != f.y;
                }
            }
            if (__any_sync(~0u, odd)) attend_row<T>(a, c.b, c.s.q0 + tok, head, c.s.pos0 + tok);
        }
        deal_next<C::kRows, kTcKeys>(a, c);
    }
}

template <typename T, int DH>
__global__ void __launch_bounds__(TcCfg<DH>::kThreads, 1)
    attend_tc_kernel(const AttendArgs a, int box_rows, int q_boxes, const __grid_constant__ CUtensorMap kmap,
                     const __grid_constant__ CUtensorMap vmap, const __grid_constant__ CUtensorMap qmap) {
    using C = TcCfg<DH>;
    constexpr int CG = C::CG;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBars);
    // What the issuing CTA waits for is counted on its own barriers, by both CTAs of a pair; what it
    // tells is committed to both CTAs' copies.
    uint64_t* full = bars;                    // [slots] each CTA's loader: the slot's bytes have landed
    uint64_t* empty = full + C::kSlots;       // [slots] MMA commit: the slot is read
    // ([3]: an S buffer's uses by its own row tile, two, and those of the second buffer by a row tile that alternates)
    uint64_t* s_full = empty + C::kSlots;     // [3] MMA commit: S is there
    uint64_t* p_full = s_full + 3;            // [3] each CTA's eight softmax warps: P is there, S is read
    uint64_t* s_read = p_full + 3;            // [2] (P in its own columns) the same warps: S is read
    uint64_t* q_full = s_read + 2;            // [NQ] each CTA's Q warps: Q is in shared memory
    uint64_t* q_free = q_full + C::NQ;        // [NQ] MMA commit: the tile's last S is there
    uint64_t* o_done = q_free + C::NQ;        // [3] MMA commit: P V is added
    uint64_t* o_free = o_done + 3;            // [NQ] each CTA's eight softmax warps: the tile's O is read
    uint64_t* tail = o_free + C::NQ;          // the bytes of a V slot that is cleared by hand
    uint64_t* done = tail + 1;                // MMA commit: everything issued has finished
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
    int* abort_flag = reinterpret_cast<int*>(tmem_holder + 1);
    int* odd = abort_flag + 1;                // some row of a whole tile ended with a NaN
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const KvArgs& kv = a.kv;
    const Ctl ctl{abort_flag, a.hdr};

    if (smem_u32(smem) & 1023u) {  // (the swizzled tiles' places; the same in every CTA)
        if (tid == 0) atomicOr(&a.hdr->status, kDevTimeout);
        return;
    }
    if (tid == 0) {
        for (int i = 0; i < C::kSlots; ++i) {
            mbar_init(full + i, CG);
            mbar_init(empty + i, 1);
        }
        for (int i = 0; i < 3; ++i) {
            mbar_init(s_full + i, 1);
            mbar_init(p_full + i, 8 * CG);
            if (i < 2) mbar_init(s_read + i, 8 * CG);
            mbar_init(o_done + i, 1);
        }
        for (int i = 0; i < C::NQ; ++i) {
            mbar_init(q_full + i, CG);
            mbar_init(q_free + i, 1);
            mbar_init(o_free + i, 8 * CG);
        }
        mbar_init(tail, 1);
        mbar_init(done, 1);
        *abort_flag = *odd = 0;
        asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    }
    if (warp == 0) tmem_alloc<CG>(tmem_holder, 512);
    if (a.follows) begin_beside();  // the split kernel has waited
    else wait_for_stream();
    if (a.lead && blockIdx.x == 0 && tid == 0) a.hdr->status = kDevOk;
    const int rank = CG == 2 ? blockIdx.x & 1 : 0, me = blockIdx.x / CG;
    Cursor c;
    deal_begin<C::kRows, kTcKeys>(a, reinterpret_cast<long long*>(smem + C::kOffRing), 2, C::kExtra, me, gridDim.x / CG, c);  // (scratch: the ring)
    if (tid == 0) *reinterpret_cast<Cursor*>(smem + C::kOffStart) = c;
    clear_stray_rows<T>(a);
    tc_fence_before();
    fence_async_proxy();  // the scratch was written through the generic proxy, the ring is written by TMA
    __syncthreads();
    if constexpr (CG == 2) cluster_sync();  // the peer's barriers and tensor memory are there
    tc_fence_after();
    const uint32_t tmem = *tmem_holder;
    const uint32_t ring = smem_u32(smem + C::kOffRing);
    // Row tiles of the CTA (pair) that have rows, of the cursor's.
    auto active = [&]() { return C::NQ == 2 && c.s.q_len * kv.group - c.rt * C::kRows > C::kTile ? 2 : 1; };
    // The two S (P) buffers.  Two row tiles have one each; one alone alternates between them (except where P has columns
    // of its own), beginning each piece with the first, so that S of the next keys is ready when the softmax of these ends.
    // Barriers go by who uses a buffer (set 0 and 1: a row tile its own, 2: the first row tile the second buffer), so
    // that their phases are waited for by the warps that the next phase waits for: none can be missed, however
    // late the second row tile's warps are in the piece before.
    // uses: bit s is the parity of the times that set s has been used, the phase of its barriers.
    auto buf_of = [&](int w, int act, int j) { return act == 1 && !C::kOwnP ? j & 1 : w; };
    auto set_of = [&](int w, int act, int j) { return act == 1 && !C::kOwnP ? (j & 1) * 2 : w; };
    bool ok = true;

    if (warp < 4) {
        if constexpr (C::NQ == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 64;\n");
        if (warp == 0) {
          if (rank == 0) {
            // ------------------------------------------------------------ MMA issue
            const bool leader = elect_one();
            const uint64_t qd = sdesc(smem_u32(smem + C::kOffQ)), kd = sdesc(ring), vd = sdesc_mn(ring, kTcKeys * 128);
            int slot = 0;                     // the next ring slot of K or V,
            uint32_t phase = 0;               // and the phase of its barrier
            uint32_t uses = 0;                // of the sets, by the tiles whose P V is issued
            uint32_t items[2] = {0, 0};       // row tiles so far, by warpgroup
            auto qk = [&](int w, int buf, int set, int s) {  // S[buf] = Q[w] K^T, K in slot s
                if (leader) {
#pragma unroll
                    for (int k = 0; k < DH / 16; ++k)
                        mma_f16_ss<CG>(tmem + C::kSCol + 128 * buf, qd + ((w * C::kQTile + k / 4 * 16384 + k % 4 * 32) >> 4),
                                       kd + ((s * C::kSlot + k / 4 * (C::kKKeys * 128) + k % 4 * 32) >> 4), idesc16<T>(C::kTile, kTcKeys, false),
                                       k > 0);
                    mma_commit<CG>(s_full + set);
                }
                __syncwarp();
            };
            auto pv = [&](int w, int buf, int set, int s, bool first) {  // O[w] (+)= P[buf] V, V in slot s
                if (leader) {
#pragma unroll
                    for (int k = 0; k < kTcKeys / 16; ++k)
                        mma_f16_ta<CG>(tmem + C::kOCol + DH * w, tmem + C::kPCol + C::kPStep * buf + 8 * k, vd + ((s * C::kSlot + k * 2048) >> 4),
                                       idesc16<T>(C::kTile, DH, true), !first || k > 0);
                    mma_commit<CG>(o_done + set);
                }
                __syncwarp();
            };
            auto commit = [&](uint64_t* bar) {
                if (leader) mma_commit<CG>(bar);
                __syncwarp();
            };
            auto wait = [&](uint64_t* bar, uint32_t ph) { ok = __all_sync(~0u, ok && wait_bar(bar, ph, ctl)); };
            auto advance = [&]() {
                if (++slot == C::kSlots) slot = 0, phase ^= 1;
            };
            while (ok && c.u < c.end) {
                const int n = c.take;
                const int act = active();
                if constexpr (C::kOwnP) {
                    // slots: K0, K1, then V(j), K(j + 2); S of the next keys while the softmax of these runs
                    auto next_s = [&](int j) {
                        wait(full + slot, phase);
#pragma unroll
                        for (int w = 0; w < 2; ++w) {
                            if (w >= act) break;
                            if (j == 0) wait(q_full + w, items[w] & 1);
                            else wait(s_read + w, uses >> w & 1);
                            if (!ok) return;
                            tc_fence_after();
                            qk(w, w, w, slot);
                            if (j + 1 == n) commit(q_free + w);
                        }
                        commit(empty + slot);
                        advance();
                    };
                    next_s(0);
                    for (int j = 0; j < n && ok; ++j) {
                        if (j + 1 < n) next_s(j + 1);
                        if (ok) wait(full + slot, phase);
#pragma unroll
                        for (int w = 0; w < 2; ++w) {
                            if (w >= act || !ok) break;
                            wait(p_full + w, uses >> w & 1);
                            if (j == 0) wait(o_free + w, (items[w] & 1) ^ 1);
                            if (!ok) break;
                            tc_fence_after();
                            pv(w, w, w, slot, j == 0);
                            uses ^= 1u << w;
                        }
                        if (!ok) break;
                        commit(empty + slot);
                        advance();
                    }
                    // (the last S's reading is not waited for above: P of the same tile follows it)
                } else if (act == 2) {
                    // slots: K0, then V(j), K(j + 1)
                    wait(full + slot, phase);
#pragma unroll
                    for (int w = 0; w < 2; ++w) {
                        if (w >= act) break;
                        wait(q_full + w, items[w] & 1);
                        if (!ok) break;
                        tc_fence_after();
                        qk(w, w, w, slot);
                        if (n == 1) commit(q_free + w);
                    }
                    if (!ok) break;
                    commit(empty + slot);
                    advance();
                    for (int j = 0; j < n && ok; ++j) {
                        const int vs = slot;
                        wait(full + slot, phase);
                        advance();
                        const bool more = j + 1 < n;
                        const int ks = slot;
#pragma unroll
                        for (int w = 0; w < 2; ++w) {
                            if (w >= act) break;
                            wait(p_full + w, uses >> w & 1);
                            if (j == 0) wait(o_free + w, (items[w] & 1) ^ 1);
                            if (!ok) break;
                            tc_fence_after();
                            pv(w, w, w, vs, j == 0);
                            uses ^= 1u << w;
                            if (w == act - 1) commit(empty + vs);
                            if (more) {
                                if (w == 0) wait(full + ks, phase);
                                if (!ok) break;
                                qk(w, w, w, ks);
                                if (j + 2 == n) commit(q_free + w);
                            }
                        }
                        if (ok && more) {
                            commit(empty + ks);
                            advance();
                        }
                    }
                } else {
                    // slots: K0, K1, then V(j), K(j + 2)
                    wait(q_full, items[0] & 1);
                    auto next_s = [&](int j) {
                        wait(full + slot, phase);
                        if (!ok) return;
                        tc_fence_after();
                        qk(0, j & 1, (j & 1) * 2, slot);
                        commit(empty + slot);
                        if (j + 1 == n) commit(q_free);
                        advance();
                    };
                    for (int j = 0; j < min(n, 2) && ok; ++j) next_s(j);
                    for (int j = 0; j < n && ok; ++j) {
                        const int set = (j & 1) * 2;
                        wait(full + slot, phase);
                        wait(p_full + set, uses >> set & 1);
                        if (j == 0) wait(o_free, (items[0] & 1) ^ 1);
                        if (!ok) break;
                        tc_fence_after();
                        pv(0, j & 1, set, slot, j == 0);
                        uses ^= 1u << set;
                        commit(empty + slot);
                        advance();
                        if (j + 2 < n) next_s(j + 2);
                    }
                }
                for (int w = 0; w < act; ++w) ++items[w];
                deal_next<C::kRows, kTcKeys>(a, c);
            }
            if (leader) mma_commit_own<CG>(done);
            __syncwarp();
            drain_bar(done, 0, global_ns() + kWaitNs);
          }
        } else if (warp == 1 || warp == 3) {
            // ------------------------------------------------------------ K tiles (warp 1), V tiles (warp 3)
            int base = 0;             // ring slots taken before this piece,
            int top = 0;              // and by this warp's latest copies
            uint32_t tails = 0;
            int lo, hi;
            // Lane i brings box i of `rows` rows (at most 16 boxes) from key `key0` on: where it lies.
            auto where = [&](int key0, int boxes, int& row, int& page) {
                const int key = key0 + lane * box_rows;
                page = kv.n_pages;  // outside the map: zeros
                row = 0;
                if (lane < boxes && key < hi) {
                    const int p = div_by(key, kv.by_page), id = page_id(kv, c.b, p);
                    row = key - p * kv.page;
                    if (id >= 0) page = id;
                }
            };
            // The slot of use `use` of the ring, free.
            auto claim = [&](int use) {
                const int slot = use % C::kSlots;
                ok = __all_sync(~0u, wait_bar(empty + slot, (use / C::kSlots & 1) ^ 1, ctl));
                return slot;
            };
            auto load_k = [&](int unit, int use) {
                int row, page;
                constexpr int kKeys = C::kKKeys;
                const int boxes = kKeys / box_rows;
                where(unit * kTcKeys + rank * kKeys, boxes, row, page);
                const int slot = claim(use);
                if (!ok) return;
                top = use + 1;
                const uint32_t bar = leaders(full + slot);
                if (lane == 0) mbar_expect_tx(bar, C::kSlot);
                __syncwarp();
                if (lane < boxes)
#pragma unroll
                    for (int b = 0; b < C::kKBlocks; ++b)
                        tma_tile4d<CG>(ring + slot * C::kSlot + (b * kKeys + lane * box_rows) * 128, &kmap, b * 64, row, c.h, page, bar);
            };
            auto load_v = [&](int unit, int use) {
                int row, page;
                const int boxes = kTcKeys / box_rows;
                where(unit * kTcKeys, boxes, row, page);
                const int slot = claim(use);
                if (!ok) return;
                top = use + 1;
                const int last = hi - unit * kTcKeys;  // rows that some row of the tile sees
                const bool cut = last > 0 && last < kTcKeys && last % box_rows != 0;
                const uint32_t there = leaders(full + slot), bar = cut ? own_bar(tail) : there;
                if (lane == 0) mbar_expect_tx(bar, C::kSlot);
                __syncwarp();
                if (lane < boxes)
#pragma unroll
                    for (int b = 0; b < C::kVBlocks; ++b)
                        tma_tile4d<CG>(ring + slot * C::kSlot + (b * kTcKeys + lane * box_rows) * 128, &vmap, rank * C::kVCols + b * 64, row, c.h,
                                       page, bar);
                if (cut) {  // the box's rows behind the last visible one
                    ok = __all_sync(~0u, wait_bar(tail, tails & 1, ctl));
                    if (!ok) return;
                    ++tails;
                    const int end = (last + box_rows - 1) / box_rows * box_rows;
                    const int per = (end - last) * 8;
                    for (int x = lane; x < per * C::kVBlocks; x += 32) {
                        const int b = x / per, y = x - b * per;
                        *reinterpret_cast<uint4*>(smem + C::kOffRing + slot * C::kSlot + (b * kTcKeys + last) * 128 + y * 16) =
                            make_uint4(0, 0, 0, 0);
                    }
                    fence_async_proxy();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(there);
                }
            };
            while (ok && c.u < c.end) {
                const int n = c.take;
                const int r0 = c.rt * C::kRows;
                key_range(kv, a.window, c.s, r0, min(r0 + C::kRows, c.s.q_len * kv.group), lo, hi);
                const int unit0 = c.first + c.off;
                const int look = C::look(active());  // (in the ring, K is so many tiles ahead of V)
                for (int j = 0; j < n && ok; ++j) {
                    if (warp == 1) load_k(unit0 + j, base + j + max(j - look + 1, 0));
                    else load_v(unit0 + j, base + j + min(j + look, n));
                }
                base += 2 * n;
                deal_next<C::kRows, kTcKeys>(a, c);
            }
            // Nothing is on its way to this CTA's memory when it leaves: every slot's last use has landed and been
            // read (or, after a timeout, the limit has passed), those of a piece that was given up among them.
            // (Both CTAs' copies count on the first one's barriers, and a pair leaves together.)
            top = max(top, base);
            const uint64_t end = global_ns() + kWaitNs;
            for (int u = max(top - C::kSlots, 0); u < top; ++u) {
                if (rank == 0) drain_bar(full + u % C::kSlots, (u / C::kSlots) & 1, end);
                drain_bar(empty + u % C::kSlots, (u / C::kSlots) & 1, end);
            }
        } else {
            // ------------------------------------------------------------ Q
            uint32_t items[2] = {0, 0};
            constexpr int kCpr = DH / 8, kPer = 32 / kCpr;  // chunks per row, rows per warp step
            const int x = lane % kCpr;
            while (ok && c.u < c.end) {
                const int all = c.s.q_len * kv.group - c.rt * C::kRows;
#pragma unroll 1
                for (int w = 0; w < C::NQ; ++w) {
                    if (all <= C::kTile * w || !ok) break;
                    uint8_t* sq = smem + C::kOffQ + w * C::kQTile;
                    const int r0 = c.rt * C::kRows + C::kTile * w + 128 * rank;
                    const int rows = min(c.s.q_len * kv.group - r0, 128);
                    ok = __all_sync(~0u, wait_bar(q_free + w, (items[w] & 1) ^ 1, ctl));
                    if (!ok) break;
                    ++items[w];
                    if (q_boxes) {  // (heads of a group, tokens): the tile's rows in order, as boxes of 64 components
                        if (lane == 0) {
                            const uint32_t bar = leaders(q_full + w);
                            mbar_expect_tx(bar, C::kQTile);
#pragma unroll
                            for (int b = 0; b < DH / 64; ++b)
                                tma_tile3d<CG>(smem_u32(sq) + b * 16384, &qmap, b * 64, c.h * kv.group,
                                               c.s.q0 + div_by(r0, kv.by_group), bar);
                        }
                        __syncwarp();
                        continue;
                    }
                    // where the rows begin: each lane finds its rows' places once, then passes them round
#pragma unroll 1
                    for (int g = 0; g < 128; g += 32) {
                        int tok, hg;
                        row_of(kv, r0 + max(min(g + lane, rows - 1), 0), tok, hg);
                        const int64_t at = static_cast<int64_t>(c.s.q0 + tok) * a.q_ts + (c.h * kv.group + hg) * a.q_hs;
#pragma unroll 8
                        for (int i = 0; i < 32; i += kPer) {
                            const int64_t from = __shfl_sync(~0u, at, i + lane / kCpr);
                            const int r = g + i + lane / kCpr;
                            const bool in = r < rows && x * 8 < kv.d;
                            cp_async16(sq + (x / 8) * 16384 + r * 128 + (((x & 7) ^ (r & 7)) << 4),
                                       static_cast<const T*>(a.q) + (in ? from + x * 8 : 0), in ? 16 : 0);
                        }
                    }
                    cp_async_commit();
                    cp_async_wait<0>();
                    fence_async_proxy();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(leaders(q_full + w));
                }
                deal_next<C::kRows, kTcKeys>(a, c);
            }
            for (int w = 0; w < C::NQ; ++w)
                if (items[w]) drain_bar(q_free + w, (items[w] - 1) & 1, global_ns() + kWaitNs);  // (its arrival, too, has come)
        }
    } else {
        // ---------------------------------------------------------------- softmax, half a row per thread
        if constexpr (C::NQ == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 104;\n");
        const int w = (warp - 4) / 8;               // the row tile
        const int half = ((warp - 4) / 4) & 1;      // keys 64 half .. of a tile, columns DH / 2 half .. of O
        const int row = tid & 127;                  // tile row = tensor-memory lane
        const uint32_t lane_base = static_cast<uint32_t>(32 * (warp & 3)) << 16;
        const uint32_t o_col = tmem + lane_base + C::kOCol + DH * w + DH / 2 * half;
        PairExchange<WarpPairBarrier> other{reinterpret_cast<uint32_t*>(smem + C::kOffEx) + 512 * w + row, 128, half, 0, {1 + 4 * w + (warp & 3)}};
        const float sc = a.scale * kLog2e;
        uint32_t uses = 0;                          // of the sets, before this tile
        // The other half's value in x's place; false: it has left, and so does this one.
        auto exchange = [&](float& x) { return ok = __all_sync(~0u, other.swap(x)); };
        while (ok && c.u < c.end) {
            const int n = c.take;
            const int r0 = c.rt * C::kRows + C::kTile * w + 128 * rank;
            const int rows = min(c.s.q_len * kv.group - r0, 128);  // of this CTA's part of the row tile (may be none)
            const int act = active();
            if (w >= act) {
                deal_next<C::kRows, kTcKeys>(a, c);
                continue;
            }
            const bool mine = row < rows;
            const bool live = (row & ~31) < rows;   // some row of the warp is one
            const int r_in = r0 + max(min(row, rows - 1), 0);
            int tok_i, hg;
            row_of(kv, r_in, tok_i, hg);
            const int pos = c.s.pos0 + tok_i;
            const int p_hi = min(pos, kv.cap - 1);
            const int p_lo = before_window(a.window, pos);
            float m = kNegInf;                       // the reference, in units of S
            uint64_t l2 = pair(0.f, 0.f);
            // (P V of two tiles can be under way when an alternating row tile has stored the second P: a barrier each)
            auto added = [&](int j) {  // P V of tile j, the last one counted in `uses`
                const int set = set_of(w, act, j);
                ok = __all_sync(~0u, wait_bar(o_done + set, (uses >> set & 1) ^ 1, ctl));
                return ok;
            };
            for (int j = 0; j < n; ++j) {
                const int buf = buf_of(w, act, j), set = set_of(w, act, j);
                ok = __all_sync(~0u, wait_bar(s_full + set, uses >> set & 1, ctl));
                if (!ok) break;
                if (live) {
                    tc_fence_after();
                    uint32_t v[64];
                    const uint32_t s_col = tmem + lane_base + C::kSCol + 128 * buf;
                    tmem_ld32(s_col + 64 * half, v);
                    tmem_ld32(s_col + 64 * half + 32, v + 32);
                    tmem_ld_wait();
                    tmem_tie<32>(v);
                    tmem_tie<32>(v + 32);
                    if constexpr (C::kOwnP) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(leaders(s_read + buf));
                    }
                    const int key0 = (c.first + c.off + j) * kTcKeys + 64 * half;
                    const int rel_hi = p_hi - key0, rel_lo = p_lo - key0;
                    if (__any_sync(~0u, rel_hi < 63)) {
#pragma unroll
                        for (int i = 0; i < 64; ++i)
                            if (i > rel_hi) v[i] = __float_as_uint(kNegInf);
                    }
                    if (__any_sync(~0u, rel_lo >= 0)) {
#pragma unroll
                        for (int i = 0; i < 64; ++i)
                            if (i <= rel_lo) v[i] = __float_as_uint(kNegInf);
                    }
                    float mx[4];
#pragma unroll
                    for (int x = 0; x < 4; ++x) mx[x] = max3(__uint_as_float(v[x]), __uint_as_float(v[x + 4]), __uint_as_float(v[x + 8]));
#pragma unroll
                    for (int i = 12; i < 60; i += 8)
#pragma unroll
                        for (int x = 0; x < 4; ++x) mx[x] = max3(mx[x], __uint_as_float(v[i + x]), __uint_as_float(v[i + 4 + x]));
#pragma unroll
                    for (int x = 0; x < 4; ++x) mx[x] = fmaxf(mx[x], __uint_as_float(v[60 + x]));
                    float top = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]);
                    float top2 = top;
                    const bool there = other.swap(top2);  // (S of both halves is read: P may be stored over it)
                    top = fmaxf(top, top2);
                    // (with m = -inf, as at the piece's beginning, the difference is inf, or NaN if the row has seen nothing yet)
                    const bool grew = (top - m) * sc > 8.f;
                    if (__any_sync(~0u, grew || !there)) {  // (one vote: whether the other has left is looked at where it is rare)
                        if (!(ok = __all_sync(~0u, there))) break;
                        float f = 1.f;
                        if (grew) {
                            f = m == kNegInf ? 0.f : exp2_fast((m - top) * sc);
                            m = top;
                        }
                        if (j > 0) {
                            // O is rescaled between the products: the one before has to be there
                            if (!added(j - 1)) break;
                            tc_fence_after();
                            const uint64_t f2 = pair(f, f);
                            l2 = mul2(l2, f2);
#pragma unroll 1
                            for (int i = 0; i < DH / 2; i += 16) {
                                uint32_t o[16];
                                tmem_ld16(o_col + i, o);
                                tmem_ld_wait();
                                tmem_tie<16>(o);
#pragma unroll
                                for (int x = 0; x < 16; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * f);
                                tmem_st16(o_col + i, o);
                            }
                        }
                    }
                    if constexpr (C::kOwnP) {  // the product before has read its P
                        if (j > 0 && !added(j - 1)) break;
                        tc_fence_after();
                    }
                    const float base = m == kNegInf ? 0.f : m * sc;
                    const uint64_t sc2 = pair(sc, sc), nb2 = pair(-base, -base);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t pk[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const int e = 32 * h + 2 * i;
                            const float2 x = unpair(fma2(pair(__uint_as_float(v[e]), __uint_as_float(v[e + 1])), sc2, nb2));
                            const float p0 = exp2_fast(x.x), p1 = exp2_fast(x.y);
                            l2 = add2(l2, pair(p0, p1));
                            pk[i] = Elem<T>::pack(p0, p1);  // the product's operand: 16 bits; the sum l is of the fp32 values
                        }
                        tmem_st16(tmem + lane_base + C::kPCol + C::kPStep * buf + 32 * half + 16 * h, pk);
                    }
                    tmem_st_wait();
                    tc_fence_before();
                } else if constexpr (C::kOwnP) {
                    if (lane == 0) mbar_arrive(leaders(s_read + buf));
                    // (S may be two tiles ahead of P: not to count for this tile's P before the last one's is complete)
                    if (j > 0 && !added(j - 1)) break;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(leaders(p_full + set));
                uses ^= 1u << set;
            }
            if (!ok || !added(n - 1)) break;
            // ------------------------------------------------------------ the tile's output
            tc_fence_after();
            const bool whole = c.whole();
            const int tok = c.s.q0 + tok_i, head = c.h * kv.group + hg;
            bool bad = false;
            const int part = 2 * me + (c.u == c.begin ? 0 : 1), r_tile = C::kTile * w + 128 * rank + row;
            if (live) {
                const float2 lp = unpair(l2);
                float l = lp.x + lp.y, l_other = l;
                if (!exchange(l_other)) break;
                l += l_other;
                bad = l != l;
                const float inv = l == 0.f ? 0.f : 1.f / l;
                if (whole) {
                    // 32 columns (four 16-byte chunks) at a time, transposed over four lanes: a store instruction then
                    // writes 64-byte pieces of 8 rows instead of 16-byte pieces of 32.
                    const int64_t at = tok * a.o_ts + head * a.o_hs;
                    T* dst[4];
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        dst[x] = static_cast<T*>(a.out) + __shfl_sync(~0u, at, (lane & ~3) + x) + DH / 2 * half + (lane & 3) * 8;
                    uint64_t t2 = pair(0.f, 0.f);  // 0 times every value: NaN where one is not finite
                    const uint64_t inv2 = pair(inv, inv), zero2 = pair(0.f, 0.f);
                    uint32_t o[2][16];
                    tmem_ld16(o_col, o[0]);
#pragma unroll
                    for (int i = 0; i < DH / 2; i += 32) {
                        uint32_t u[4][4];
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            tmem_ld_wait();
                            tmem_tie<16>(o[y]);
                            if (i + 16 * y + 16 < DH / 2) tmem_ld16(o_col + i + 16 * y + 16, o[y ^ 1]);
#pragma unroll
                            for (int x = 0; x < 8; ++x) {
                                const uint64_t v = pair(__uint_as_float(o[y][2 * x]), __uint_as_float(o[y][2 * x + 1]));
                                t2 = fma2(v, zero2, t2);
                                const float2 f = unpair(mul2(v, inv2));
                                u[2 * y + x / 4][x % 4] = Elem<T>::pack(f.x, f.y);
                            }
                        }
#pragma unroll
                        for (int b = 1; b <= 2; b *= 2)
#pragma unroll
                            for (int x = 0; x < 4; ++x) {
                                if (x & b) continue;
#pragma unroll
                                for (int y = 0; y < 4; ++y) {
                                    const uint32_t got = __shfl_xor_sync(~0u, lane & b ? u[x][y] : u[x | b][y], b);
                                    if (lane & b) u[x][y] = got;
                                    else u[x | b][y] = got;
                                }
                            }
                        if (DH / 2 * half + i + (lane & 3) * 8 < kv.d)
#pragma unroll
                            for (int x = 0; x < 4; ++x)
                                if ((row & ~3) + x < rows) *reinterpret_cast<uint4*>(dst[x] + i) = make_uint4(u[x][0], u[x][1], u[x][2], u[x][3]);
                    }
                    const float2 t = unpair(t2);
                    bad |= t.x != t.x || t.y != t.y;
                } else {
                    // a piece: rows side by side ([component / 4][row][4]), so that a warp's stores are contiguous
                    float* dst = a.part_o + (static_cast<int64_t>(part) * C::kRows * DH) + (DH / 8 * half * C::kRows + r_tile) * 4;
                    uint32_t o[2][16];
                    tmem_ld16(o_col, o[0]);
#pragma unroll
                    for (int i = 0; i < DH / 2; i += 16) {
                        const int y = i / 16 & 1;
                        tmem_ld_wait();
                        tmem_tie<16>(o[y]);
                        if (i + 16 < DH / 2) tmem_ld16(o_col + i + 16, o[y ^ 1]);
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            *reinterpret_cast<uint4*>(dst + (i / 4 + x) * C::kRows * 4) = make_uint4(o[y][4 * x], o[y][4 * x + 1], o[y][4 * x + 2], o[y][4 * x + 3]);
                    }
                }
                if (mine && half == 0) {
                    if (!whole) a.part_ml[part * C::kRows + r_tile] = make_float2(m == kNegInf ? kNegInf : m * sc, l);
                    else if (a.lse) a.lse[static_cast<int64_t>(tok) * kv.hq + head] = l == 0.f ? kNegInf : (m * sc + log2f(l)) * kLn2;
                }
                tc_fence_before();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(leaders(o_free + w));
            if (mine && bad && whole) *odd = 1;
            deal_next<C::kRows, kTcKeys>(a, c);
        }
        float end = 0.f;
        if (!ok) {
            other.leave();
        } else if (exchange(end)) {  // (both halves of the rows are stored, and what they set in `odd`)
            if (*odd) retake_rows<T, DH>(a, *reinterpret_cast<const Cursor*>(smem + C::kOffStart), rank, w, warp & 3, half);
        }
    }

    tc_fence_before();
    __syncthreads();
    if constexpr (CG == 2) cluster_sync();  // the peer has read this CTA's shared and tensor memory
    // (started beside the kernel before it: not to be complete before that is, for what waits for this one)
    if (a.follows && tid == 0) asm volatile("griddepcontrol.wait;\n" ::: "memory");
    if (warp == 0) {
        tc_fence_after();
        tmem_free<CG>(tmem, 512);
    }
}

// The queries [tokens][heads][D] as a 3-D map (component, head, token), boxes of 64 components x the heads of
// a group x as many tokens as make 128 rows.
cudaError_t make_qmap(const AttendArgs& a, int dtype, CUtensorMap* map) {
    Encode encode = nullptr;
    if (cudaError_t e = get_encode(&encode); e != cudaSuccess) return e;
    const KvArgs& kv = a.kv;
    const cuuint32_t elem[3] = {1, 1, 1};
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(kv.d), static_cast<cuuint64_t>(kv.hq), static_cast<cuuint64_t>(kv.n_tokens)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(kv.hq > 1 ? 2 * a.q_hs : 16), static_cast<cuuint64_t>(kv.n_tokens > 1 ? 2 * a.q_ts : 16)};
    const cuuint32_t boxes[3] = {64, static_cast<cuuint32_t>(kv.group), static_cast<cuuint32_t>(128 / kv.group)};
    const CUresult r = encode(map, dtype == 0 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void*>(a.q), dims,
                              strides, boxes, elem, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// The cache [pages][page_size][heads][D] as a 4-D map (component, row, head, page), boxes of 64 components x
// `box` rows in 128-byte-swizzled rows.  Anything outside reads zeros: components past D, the page past the last.
cudaError_t make_map(const KvArgs& kv, const void* base, int64_t ps, int64_t rs, int64_t hs, int dtype, int box, CUtensorMap* map) {
    Encode encode = nullptr;
    if (cudaError_t e = get_encode(&encode); e != cudaSuccess) return e;
    const cuuint32_t elem[4] = {1, 1, 1, 1};
    const cuuint64_t dims[4] = {static_cast<cuuint64_t>(kv.d), static_cast<cuuint64_t>(kv.page), static_cast<cuuint64_t>(kv.hkv),
                                static_cast<cuuint64_t>(kv.n_pages)};
    auto bytes = [](int64_t s, int64_t n) { return static_cast<cuuint64_t>(n > 1 ? 2 * s : 16); };  // (a size of one has no stride)
    const cuuint64_t strides[3] = {bytes(rs, kv.page), bytes(hs, kv.hkv), bytes(ps, kv.n_pages)};
    const cuuint32_t boxes[4] = {64, static_cast<cuuint32_t>(box), 1, 1};
    const CUresult r = encode(map, dtype == 0 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, const_cast<void*>(base), dims,
                              strides, boxes, elem, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <typename T, int DH>
cudaError_t launch_t(const AttendArgs& a, int dtype, int n_ctas, cudaStream_t st) {
    using C = TcCfg<DH>;
    const int box = std::min(tc_box_rows(a.kv.page), C::kKKeys);
    CUtensorMap kmap, vmap;
    if (cudaError_t e = make_map(a.kv, a.kv.k, a.kv.k_ps, a.kv.k_rs, a.kv.k_hs, dtype, box, &kmap); e != cudaSuccess) return e;
    if (cudaError_t e = make_map(a.kv, a.kv.v, a.kv.v_ps, a.kv.v_rs, a.kv.v_hs, dtype, box, &vmap); e != cudaSuccess) return e;
    // Queries by TMA where the heads of a group divide a tile (then a tile begins with a token) and the strides fit a
    // map; else row by row.
    const int64_t most = int64_t(1) << 39;
    const bool q_boxes = 128 % a.kv.group == 0 && (a.kv.hq == 1 || (a.q_hs > 0 && a.q_hs < most)) && (a.kv.n_tokens == 1 || (a.q_ts > 0 && a.q_ts < most));
    CUtensorMap qmap = kmap;
    if (q_boxes)
        if (cudaError_t e = make_qmap(a, dtype, &qmap); e != cudaSuccess) return e;
    cudaError_t e = cudaFuncSetAttribute(attend_tc_kernel<T, DH>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    const int groups = n_ctas / C::CG;
    return launch_in_stream(attend_tc_kernel<T, DH>, dim3(groups * C::CG), C::kThreads, C::kSmem, C::CG, st, a, box, q_boxes ? 1 : 0, kmap, vmap, qmap);
}

template <typename T, int DH>
cudaError_t launch_j(const AttendArgs& a, int64_t rows, int n_ctas, cudaStream_t st) {
    constexpr int kRows = TcCfg<DH>::kRows;
    const int groups = n_ctas / TcCfg<DH>::CG;
    const int64_t tiles = a.kv.n_seqs * ((rows + kRows - 1) / kRows) * a.kv.hkv;
    return groups < 2 ? cudaSuccess : launch_attend_join_rows<T, kRows, DH>(a, groups, tiles, st);
}

template <typename T>
cudaError_t launch_e(const AttendArgs& a, int dtype, int n_ctas, cudaStream_t st) {
    switch (padded_dim(a.kv.d)) {
        case 64: return launch_t<T, 64>(a, dtype, n_ctas, st);
        case 128: return launch_t<T, 128>(a, dtype, n_ctas, st);
        default: return launch_t<T, 256>(a, dtype, n_ctas, st);
    }
}

}  // namespace

int tc_box_rows(int page) { return std::min(page & -page, kTcKeys); }
int tc_part_rows(int d, int n_ctas) {
    switch (padded_dim(d)) {
        case 64: return 2 * (n_ctas / TcCfg<64>::CG) * TcCfg<64>::kRows;
        case 128: return 2 * (n_ctas / TcCfg<128>::CG) * TcCfg<128>::kRows;
        default: return 2 * (n_ctas / TcCfg<256>::CG) * TcCfg<256>::kRows;
    }
}

cudaError_t launch_attend_tc_join(const AttendArgs& a, int dtype, int64_t rows, int n_ctas, cudaStream_t st) {
    const bool bf = dtype == 0;
    switch (padded_dim(a.kv.d)) {
        case 64: return bf ? launch_j<__nv_bfloat16, 64>(a, rows, n_ctas, st) : launch_j<__half, 64>(a, rows, n_ctas, st);
        case 128: return bf ? launch_j<__nv_bfloat16, 128>(a, rows, n_ctas, st) : launch_j<__half, 128>(a, rows, n_ctas, st);
        default: return bf ? launch_j<__nv_bfloat16, 256>(a, rows, n_ctas, st) : launch_j<__half, 256>(a, rows, n_ctas, st);
    }
}

cudaError_t launch_attend_tc(const AttendArgs& a, int dtype, int n_ctas, cudaStream_t st) {
    return dtype == 0 ? launch_e<__nv_bfloat16>(a, dtype, n_ctas, st) : launch_e<__half>(a, dtype, n_ctas, st);
}

}  // namespace moe

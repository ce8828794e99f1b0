// Latent attention on the fifth-generation tensor cores: every head of a layer
// reads the same cache row, as its key with all components and as its value
// with the first Dc.
//
// The mathematics, per (token, head) row: one pass over the keys with a running
// reference m and sum l, s_j = scale q . x_j, p_j = 2^(s_j log2 e - m),
// o = sum p_j x_j[0 .. Dc), the row is o / l.
//
// Bound: HBM while the rows are few (a row of the cache, 2 (Dc + R) bytes, does 2 (2 Dc + R) flops per head: the ridge is at
// about 130 heads), the tensor pipe beyond.  A CTA takes a tile of ROWS = 16, 32 or 64 (token, head) rows, token-major,
// against units of 32 keys, which come by TMA straight from the pages and are read from shared memory by both
// products, so a CTA brings a cache row once:
//   S = Q X^T       64 rows (of which ROWS count) x 32 keys, A = Q and B = X both along the components; fp32 in tensor
//                   memory, four buffers, so that S is computed ahead of the softmax
//   O^T += X^T P^T  turned over: 128 components of the latent part x ROWS rows, four times, A = X along the keys' other
//                   direction (no transposition is needed), B = P.  The accumulator takes 4 ROWS columns of tensor memory,
//                   where O of 128 rows x 512 components alone would fill all of it.
// A softmax thread has the matrix-fragment places of S (two rows, 8 values), four lanes and two warps a row.  P goes to
// shared memory in 16 bits.  The reference m is raised, and O rescaled, only when a row's maximum has grown by more than 2^8 over it.
// In fp16 the weights are 2^7 times as large (m is 7 less in base 2): at most 2^15, which the type holds, and what it rounds away
// begins at 2^-32 of the largest one, not at 2^-25.
//
// The keys come eight rows at a time with all their components, 9 KB that lie side by side in the cache, so that what DRAM opens
// is read at once (boxes of 64 components x 64 rows stream at 3.3 TB/s, these at 5.6).  In shared memory such a group is
// [block of 64 components][row], a swizzle atom each, so a product finds its next eight keys a group further, its next 64
// components a KB further.  The ring has 128 keys (160 with few rows).
// Pages that are not there and rows past the last visible one read zeros, and rows behind it inside a group are
// cleared by hand.  Work is dealt in equal shares of units; the pieces of a cut tile go through the workspace and the join.
//
// Warps: 0 the products S and the tensor-memory allocation, 3 the products O, each issued by one lane, so that neither waits
// for what the other needs; 1 the keys, 2 the queries, 4 to 11 softmax and output, a warp for half of the keys of 16 rows.
// Every wait is bounded; a timeout sets the status word and every role leaves, having waited (again with a limit) for
// its own copies in flight.  The softmax warps meet at a barrier once per tile, whatever became of their waits, and leave
// together.
//
// Measured, bf16, 512 + 64 components, device time with the join: one sequence of 131071 positions, 32 heads 38.1 us (4.0 TB/s;
// 22 by its bytes), 64 ragged ones up to 16384 of 16, 32, 64, 128 heads 65, 69, 84, 140 us (5.3, 5.0, 4.2, 2.5 TB/s; 51 to 52 by
// their bytes; from 65 heads on two CTAs read the same keys, from DRAM 1.7 times), 509 tokens of 32 heads at 8000 positions beside eight single ones 367 us
// (0.78 PFLOP/s; 145 by its operations).  The products fill the chunk's time: S takes 36 steps of about 30 cycles for 32 keys, O 8 of
// 52.  Why these steps are longer than the pipe's rate says is not measured: half of its rows are idle in S, and both operands come from
// shared memory anew in each step, 3 and 6 KB, which at 128 bytes a cycle are 24 and 48 cycles.
#include <algorithm>

#include "latent_common.cuh"
#include "tcgen05.cuh"

namespace moe {
namespace {

constexpr int kKeys = 32;  // of a unit: what a wait of the products is for
// Keys that a tile's beginning and end count for in the deal: four sequences' 48 rows and one tile of 131071 keys take the same with 128 to 768.
constexpr int kExtra = 128;
constexpr int kJoinWarps = 8;
// What m is less than the row's reference, in base 2.
template <typename T>
constexpr float kLift = 0.f;
template <>
constexpr float kLift<__half> = 7.f;

// ROWS rows of a CTA.
template <int ROWS>
struct LatCfg {
    static constexpr int kBlocks = (kMaxLatent + kMaxLatentRot) / 64;
    static constexpr int kUnits = ROWS == 64 ? 4 : 5;            // of the ring
    static constexpr int kS = 4;                                 // buffers of S: units that S may be ahead
    static constexpr int kPs = 2;                                // buffers of P, side by side in rows of 128 bytes
    static constexpr int kQBlock = ROWS * 128;                   // bytes: ROWS queries of 64 components
    static constexpr int kQ = kBlocks * kQBlock;
    static constexpr int kP = ROWS * 128;
    static constexpr int kRing = kUnits * kKeys * kBlocks * 128;
    static constexpr int kThreads = 384;
    static constexpr int kOCol = 0, kSCol = 4 * ROWS, kCols = 512;
    static constexpr int kOffQ = 0;
    // (S is of 64 rows of Q: where ROWS is less, the MMA reads what lies behind them, at most 6 KB behind Q's end, into
    // rows of S that are never looked at)
    static constexpr int kOffP = kQ;
    static constexpr int kOffRing = kOffP + kP;
    static constexpr int kOffBars = kOffRing + kRing;
    static constexpr int kBars = 2 * kUnits + 2 * kS + 2 * kPs + 6;
    static constexpr int kOffAt = (kOffBars + 8 * kBars + 15) & ~15;   // [ROWS] where an output row begins
    static constexpr int kOffFactor = kOffAt + 8 * ROWS;               // [ROWS] what O's rows are multiplied by
    static constexpr int kOffEx = kOffFactor + 4 * ROWS;               // [2][ROWS] what the halves of a row tell one another
    static constexpr int kOffMisc = kOffEx + 8 * ROWS;
    static constexpr int kOffStart = kOffMisc + 16;                    // the cursor at the share's beginning
    static constexpr int kSmem = kOffStart + sizeof(Cursor);
    static_assert(kSCol + kS * kKeys <= kCols, "tensor-memory columns");
    static_assert(kSmem <= 227 * 1024, "shared memory");
};

// 16 lanes x 16 columns of 32 bits, as the accumulator fragments of 16 x 8 matrices (no wait).
__device__ __forceinline__ void tmem_ld_frag(uint32_t taddr, uint32_t* v) {
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
                 : "r"(taddr));
}

// Barrier 1 of the 256 softmax threads: plain, or with the OR of a predicate.
__device__ __forceinline__ void softmax_sync() {
    __syncwarp();
    asm volatile("bar.sync 1, 256;\n" ::: "memory");
}
__device__ __forceinline__ bool softmax_any(bool x) {
    uint32_t r;
    __syncwarp();
    asm volatile("{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n bar.red.or.pred q, 1, 256, p;\n selp.u32 %0, 1, 0, q;\n}\n"
                 : "=r"(r) : "r"(static_cast<uint32_t>(x)) : "memory");
    return r != 0;
}

// A place in a ring of N, and the phase of its barrier.
template <int N>
struct Place {
    int slot = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next() {
        if (++slot == N) slot = 0, phase ^= 1;
    }
};

// Shared-memory matrix descriptor, 128-byte swizzle: 8-row groups `group` bytes apart; across (an operand that is read across its
// rows): the next 64 values `across` bytes on.
__device__ __forceinline__ uint64_t sdesc_groups(uint32_t saddr, uint32_t group, uint32_t across = 16) {
    return static_cast<uint64_t>((saddr >> 4) & 0x3FFF) | static_cast<uint64_t>(across >> 4) << 16 | static_cast<uint64_t>(group >> 4) << 32 |
           static_cast<uint64_t>(1) << 46 | static_cast<uint64_t>(2) << 61;
}

// Arrivals on the CTA's own barriers.
__device__ __forceinline__ void arrive_own(uint64_t* bar) { asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];\n" ::"r"(smem_u32(bar)) : "memory"); }
__device__ __forceinline__ void arrive_expect(uint64_t* bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n" ::"r"(smem_u32(bar)), "r"(bytes) : "memory");
}
// Bytes to come, without an arrival.
__device__ __forceinline__ void expect(uint64_t* bar, uint32_t bytes) {
    asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;\n" ::"r"(smem_u32(bar)), "r"(bytes) : "memory");
}

// What is read once is the first to leave L2, where the pieces' sums have to stay.
__device__ __forceinline__ uint64_t l2_policy(bool once) {
    uint64_t first, normal;
    asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;\n" : "=l"(first));
    asm("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;\n" : "=l"(normal));
    return once ? first : normal;
}

// Eight rows of the cache, all their 64-component blocks, [block][row] -> shared memory; counted on `bar`.  WIDE: a box
// has all blocks (rows of whole blocks), else one box each.
__device__ __forceinline__ void load_rows(uint32_t dst, const CUtensorMap* map, bool wide, int blocks, int row, int page, uint32_t bar, uint64_t policy) {
    if (wide) {
        asm volatile(
            "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, {%2, %3, %4, %5}], [%6], "
            "%7;\n" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(row), "r"(0), "r"(page), "r"(bar), "l"(policy) : "memory");
        return;
    }
    for (int b = 0; b < blocks; ++b) tma_tile3d<1>(dst + b * 1024, map, 64 * b, row, page, bar);
}

// The rows of the CTA's whole tiles that ended with a NaN, taken again one by one by the softmax warps (0.85 us a key and more).
template <typename T, int ROWS>
__device__ __noinline__ void retake_rows(const LatentArgs& a, Cursor c, int warp) {
    const int lane = threadIdx.x & 31;
    while (c.u < c.end) {
        const int r0 = c.rt * ROWS;
        const int rows = c.whole() ? min(c.s.q_len * a.kv.group - r0, ROWS) : 0;
        for (int r = warp; r < rows; r += 8) {
            int tok, head;
            row_of(a.kv, r0 + r, tok, head);
            bool odd = false;
            for (int e = lane * 8; e < a.kv.d; e += 256) {
                const uint4 o = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.out) + (c.s.q0 + tok) * a.o_ts + head * a.o_hs + e);
                const uint32_t o4[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 f = Elem<T>::unpack(o4[i]);
                    odd |= f.x != f.x || f.y != f.y;
                }
            }
            if (__any_sync(~0u, odd)) latent_row<T>(a, c.b, c.s.q0 + tok, head, c.s.pos0 + tok);
        }
        deal_next<ROWS, kKeys>(a, c);
    }
}

template <typename T, int ROWS>
__global__ void __launch_bounds__(LatCfg<ROWS>::kThreads, 1)
    attend_latent_kernel(const __grid_constant__ LatentArgs a, int wide, int q_rows, const __grid_constant__ CUtensorMap map, const __grid_constant__ CUtensorMap qmap) {
    using C = LatCfg<ROWS>;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint64_t* empty = reinterpret_cast<uint64_t*>(smem + C::kOffBars);  // [units of the ring] MMA commit: the unit is read
    uint64_t* full = empty + C::kUnits;      // [units of the ring] the unit's bytes have landed
    uint64_t* s_full = full + C::kUnits;     // [kS] MMA commit: S is there
    uint64_t* s_free = s_full + C::kS;       // [kS] the softmax warps: S is read
    uint64_t* p_full = s_free + C::kS;       // [kPs] the softmax warps: P is there, O rescaled
    uint64_t* o_done = p_full + C::kPs;      // [kPs] MMA commit: the unit's O is added, P is read
    uint64_t* o_free = o_done + C::kPs;      // the softmax warps: the piece's O is read
    uint64_t* q_full = o_free + 1;           // the queries are there
    uint64_t* q_free = q_full + 1;           // MMA commit: the piece's last S is there
    uint64_t* cut_in = q_free + 1;           // the bytes of eight rows that are cleared by hand
    uint64_t* done = cut_in + 1;             // [2] MMA commit: everything that S's, O's warp issued has finished
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
    int* abort_flag = reinterpret_cast<int*>(tmem_holder + 1);
    int* odd = abort_flag + 1;               // some row of a whole tile ended with a NaN
    int64_t* row_at = reinterpret_cast<int64_t*>(smem + C::kOffAt);
    float* factor = reinterpret_cast<float*>(smem + C::kOffFactor);
    float* ex = reinterpret_cast<float*>(smem + C::kOffEx);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const KvArgs& kv = a.kv;
    const Ctl ctl{abort_flag, a.hdr};

    if (smem_u32(smem) & 1023u) {  // (the swizzled tiles' places; the same in every CTA)
        if (tid == 0) atomicOr(&a.hdr->status, kDevTimeout);
        return;
    }
    if (tid == 0) {
        for (int i = 0; i < C::kUnits; ++i) {
            mbar_init(empty + i, 1);
            mbar_init(full + i, 1);
        }
        for (int i = 0; i < C::kS; ++i) {
            mbar_init(s_full + i, 1);
            mbar_init(s_free + i, 8);
        }
        for (int i = 0; i < C::kPs; ++i) {
            mbar_init(p_full + i, 8);
            mbar_init(o_done + i, 1);
        }
        mbar_init(o_free, 8);
        mbar_init(q_full, 1);
        mbar_init(q_free, 1);
        mbar_init(cut_in, 1);
        mbar_init(done, 1);
        mbar_init(done + 1, 1);
        *abort_flag = *odd = 0;
        asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    }
    __syncwarp();
    if (warp == 0) tmem_alloc<1>(tmem_holder, C::kCols);
    wait_for_stream();
    if (blockIdx.x == 0 && tid == 0) a.hdr->status = kDevOk;
    Cursor c;
    deal_begin<ROWS, kKeys>(a, reinterpret_cast<long long*>(smem + C::kOffRing), 1, kExtra / kKeys, blockIdx.x, gridDim.x, c);  // (scratch: the ring)
    if (tid == 0) *reinterpret_cast<Cursor*>(smem + C::kOffStart) = c;
    clear_stray_rows<T>(a);  // (kv.d is what the outputs have)
    tc_fence_before();
    fence_async_proxy();  // the scratch was written through the generic proxy, the ring is written by TMA
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(~0u, *tmem_holder, 0);
    const int blocks = (a.dk + 63) / 64;         // of a row of the cache, 64 components each
    const int parts = (kv.d + 127) / 128;        // of the latent part: 128 components each, the last may reach behind it
    const uint32_t group = blocks * 1024, unit = kKeys / 8 * group;  // bytes of eight rows, of a unit
    bool ok = true;
    // (the lanes leave the loop one by one; what follows may be an instruction of the whole warp, as the accesses to tensor memory are)
    auto wait = [&](uint64_t* bar, uint32_t phase) {
        ok = __all_sync(~0u, ok && wait_bar(bar, phase, ctl));
        __syncwarp();
        return ok;
    };

    if (warp == 0) {
        // ---------------------------------------------------------------- S = Q X^T
        const bool leader = elect_one();
        const uint64_t qd = sdesc(smem_u32(smem + C::kOffQ)), kd = sdesc_groups(smem_u32(smem + C::kOffRing), group);
        Place<C::kUnits> in;
        Place<C::kS> s;
        uint32_t items = 0;                  // pieces so far
        while (ok && c.u < c.end) {
            const int n = c.take;
            if (!wait(q_full, items & 1)) break;
            for (int j = 0; j < n; ++j) {
                if (!wait(s_free + s.slot, s.phase ^ 1) || !wait(full + in.slot, in.phase)) break;
                tc_fence_after();
                if (leader) {
                    const uint32_t s_col = tmem + C::kSCol + kKeys * s.slot;
                    uint64_t q = qd, k = kd + ((in.slot * unit) >> 4);
                    for (int x = 0; x < blocks; ++x, q += C::kQBlock >> 4, k += 1024 >> 4) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) mma_f16_ss<1>(s_col, q + 2 * i, k + 2 * i, idesc16<T>(64, kKeys, false), x > 0 || i > 0);
                    }
                    mma_commit<1>(s_full + s.slot);
                    if (j + 1 == n) mma_commit<1>(q_free);
                }
                __syncwarp();
                in.next();
                s.next();
            }
            ++items;
            deal_next<ROWS, kKeys>(a, c);
        }
        if (leader) mma_commit<1>(done);
        __syncwarp();
        drain_bar(done, 0, global_ns() + kWaitNs);
    } else if (warp == 3) {
        // ---------------------------------------------------------------- O^T += X^T P^T
        const bool leader = elect_one();
        const uint64_t vd = sdesc_groups(smem_u32(smem + C::kOffRing), group, 1024), pd = sdesc(smem_u32(smem + C::kOffP));
        Place<C::kUnits> in;
        Place<C::kPs> p;
        uint32_t items = 0;
        while (ok && c.u < c.end) {
            const int n = c.take;
            for (int j = 0; j < n; ++j) {
                if (!wait(p_full + p.slot, p.phase) || (j == 0 && !wait(o_free, (items & 1) ^ 1))) break;
                tc_fence_after();
                if (leader) {
                    uint64_t v = vd + ((in.slot * unit) >> 4);
#pragma unroll
                    for (int k = 0; k < kKeys / 16; ++k, v += 2 * group >> 4) {  // 16 keys, 128 components at a time
                        for (int x = 0; x < parts; ++x)
                            mma_f16_ss<1>(tmem + C::kOCol + ROWS * x, v + (x * 2048 >> 4), pd + ((p.slot * 64 + k * 32) >> 4), idesc16<T>(128, ROWS, false, true),
                                          j > 0 || k > 0);
                    }
                    mma_commit<1>(empty + in.slot);
                    mma_commit<1>(o_done + p.slot);
                }
                __syncwarp();
                in.next();
                p.next();
            }
            ++items;
            deal_next<ROWS, kKeys>(a, c);
        }
        if (leader) mma_commit<1>(done + 1);
        __syncwarp();
        drain_bar(done + 1, 0, global_ns() + kWaitNs);
    } else if (warp == 1) {
        // ---------------------------------------------------------------- the keys: lane i has rows 8 i .. of a unit
        Place<C::kUnits> in;
        uint32_t uses = 0, cuts = 0;         // units begun so far, those cut
        const uint32_t ring = smem_u32(smem + C::kOffRing);
        while (ok && c.u < c.end) {
            int lo, hi;
            const int r0 = c.rt * ROWS;
            key_range(kv, 0, c.s, r0, min(r0 + ROWS, c.s.q_len * kv.group), lo, hi);
            const uint64_t policy = l2_policy(c.s.q_len * kv.group <= ROWS);
            for (int j = 0; j < c.take && ok; ++j) {
                const int key0 = (c.first + c.off + j) * kKeys, key = key0 + 8 * lane;
                const int p = div_by(max(key, 0), kv.by_page), row = key - p * kv.page;
                const bool seen = lane < kKeys / 8 && key < hi && p < kv.width;
                // (looked at when the slot is free)
                const int id = seen ? __ldg(kv.table + static_cast<int64_t>(c.b) * kv.width + p) : -1;
                const int last = hi - key0;       // rows that some row of the tile sees
                // eight rows of which some are seen: those behind are cleared before the products may read them
                const int cut = last > 0 && last < kKeys && last % 8 != 0 ? last / 8 : -1;
                uint64_t* there = full + in.slot;
                const uint32_t dst = ring + in.slot * unit + lane * group;
                ++uses;
                if (wait(empty + in.slot, in.phase ^ 1)) {
                    if (lane == 0) {
                        if (cut < 0) {
                            arrive_expect(there, unit);
                        } else {
                            expect(there, unit - group);
                            arrive_expect(cut_in, group);
                        }
                    }
                    __syncwarp();
                    if (lane < kKeys / 8) {       // outside the map: zeros
                        const int page = static_cast<unsigned>(id) < static_cast<unsigned>(kv.n_pages) ? id : kv.n_pages, y = seen ? row : 0;
                        load_rows(dst, &map, wide, blocks, y, page, smem_u32(lane == cut ? cut_in : there), policy);
                    }
                }
                __syncwarp();
                if (ok && cut >= 0) {
                    const bool got = __all_sync(~0u, wait_bar(cut_in, cuts & 1, ctl));
                    if (!got) drain_bar(cut_in, cuts & 1, global_ns() + kWaitNs);
                    ++cuts;
                    ok = got;
                    if (!ok) break;
                    const int first = last % 8, per = (8 - first) * 8;
                    uint8_t* at = smem + C::kOffRing + in.slot * unit + cut * group + first * 128;
                    for (int x = lane; x < per * blocks; x += 32) *reinterpret_cast<uint4*>(at + x / per * 1024 + x % per * 16) = make_uint4(0, 0, 0, 0);
                    fence_async_proxy();
                    __syncwarp();
                    if (lane == 0) arrive_own(there);
                }
                in.next();
            }
            deal_next<ROWS, kKeys>(a, c);
        }
        // Nothing is on its way to this CTA's memory when it leaves: the ring's last units have landed and been read (or, after
        // a timeout, the limit has passed).
        const uint64_t end = global_ns() + kWaitNs;
        for (uint32_t u = uses > C::kUnits ? uses - C::kUnits : 0; u < uses; ++u) {
            drain_bar(full + u % C::kUnits, u / C::kUnits & 1, end);
            drain_bar(empty + u % C::kUnits, u / C::kUnits & 1, end);
        }
    } else if (warp == 2) {
        // ---------------------------------------------------------------- the queries
        uint32_t items = 0;
        while (ok && c.u < c.end) {
            if (!wait(q_free, (items & 1) ^ 1)) break;
            ++items;
            const int r0 = c.rt * ROWS, rows = min(c.s.q_len * kv.group - r0, ROWS);
            if (q_rows) {  // a box of ROWS rows for each block; rows past the sequence's are whatever follows
                if (lane == 0) {
                    int tok, head;
                    row_of(kv, r0, tok, head);
                    arrive_expect(q_full, blocks * C::kQBlock);
                    const int y = q_rows == 1 ? (c.s.q0 + tok) * kv.group + head : head, z = q_rows == 1 ? 0 : c.s.q0 + tok;
                    for (int x = 0; x < blocks; ++x) tma_tile3d<1>(smem_u32(smem + C::kOffQ) + x * C::kQBlock, &qmap, 64 * x, y, z, own_bar(q_full));
                }
                __syncwarp();
                deal_next<ROWS, kKeys>(a, c);
                continue;
            }
            // where the rows begin: each lane finds its rows' places once, then passes them round
            for (int g = 0; g < ROWS; g += 32) {
                int tok, head;
                row_of(kv, r0 + max(min(g + lane, rows - 1), 0), tok, head);
                const int64_t at = static_cast<int64_t>(c.s.q0 + tok) * a.q_ts + head * a.q_hs;
#pragma unroll 1
                for (int i = 0; i < min(ROWS - g, 32); i += 4) {  // 8 lanes a row, the blocks one after another
                    const int64_t from = __shfl_sync(~0u, at, i + lane / 8);
                    const int r = g + i + lane / 8, x = lane & 7;
                    uint8_t* dst = smem + C::kOffQ + r * 128 + ((x ^ (r & 7)) << 4);
#pragma unroll 3
                    for (int y = 0; y < blocks; ++y) {
                        const bool in = r < rows && y * 64 + x * 8 < a.dk;
                        cp_async16(dst + y * C::kQBlock, static_cast<const T*>(a.q) + (in ? from + y * 64 + x * 8 : 0), in ? 16 : 0);
                    }
                }
            }
            cp_async_commit();
            cp_async_wait<0>();
            fence_async_proxy();
            __syncwarp();
            if (lane == 0) arrive_own(q_full);
            deal_next<ROWS, kKeys>(a, c);
        }
        if (items) {  // (its arrival, too, has come; after a timeout the queries may still be on their way)
            drain_bar(q_full, (items - 1) & 1, global_ns() + kWaitNs);
            drain_bar(q_free, (items - 1) & 1, global_ns() + kWaitNs);
        }
    } else {
        // ---------------------------------------------------------------- softmax and output
        const int w = warp & 3;                   // S: rows 16 w ..; O^T: components 32 w .. of each 128
        const int half = warp / 4 - 1;            // S: keys kKeys / 2 half ..; O^T: every second 128 components
        constexpr int kN = kKeys / 4;              // values of S of a thread
        const uint32_t lane_base = static_cast<uint32_t>(32 * w) << 16;
        const float sc = a.scale * kLog2e;
        Place<C::kS> sb;
        Place<C::kPs> pb, before;                 // P's place, and that of the unit before
        while (ok && c.u < c.end) {
            const int n = c.take;
            const int r0 = c.rt * ROWS, rows = min(c.s.q_len * kv.group - r0, ROWS);
            const bool live = 16 * w < rows;
            int pos[2];                           // of this thread's rows: 16 w + lane / 4, and 8 on
#pragma unroll
            for (int x = 0; x < 2; ++x)
                pos[x] = min(c.s.pos0 + div_by(r0 + max(min(16 * w + lane / 4 + 8 * x, rows - 1), 0), kv.by_group), kv.cap - 1);
            const int all = min(c.s.pos0 + div_by(r0 + max(min(16 * w, rows - 1), 0), kv.by_group), kv.cap - 1);  // every row of the warp sees keys <= all
            if (tid - 128 < rows) {
                int tok, head;
                row_of(kv, r0 + tid - 128, tok, head);
                row_at[tid - 128] = (c.s.q0 + tok) * a.o_ts + head * a.o_hs;
            }
            float m[2] = {kNegInf, kNegInf};      // the references, in units of S
            float l[2] = {0.f, 0.f};              // this thread's part of the sums
            for (int j = 0; j < n; ++j) {
                wait(s_full + sb.slot, sb.phase);
                uint32_t v[kN];
                float top[2] = {kNegInf, kNegInf};
                bool grew = false;
                if (ok && live) {
                    tc_fence_after();
                    tmem_ld_frag(tmem + lane_base + C::kSCol + kKeys * sb.slot + kKeys / 2 * half, v);
                    tmem_ld_wait();
                    tmem_tie<kN>(v);
                    tc_fence_before();
                }
                __syncwarp();
                if (ok && lane == 0) arrive_own(s_free + sb.slot);
                sb.next();
                if (ok && live) {
                    const int key0 = (c.first + c.off + j) * kKeys + kKeys / 2 * half;
                    if (key0 + kKeys / 2 - 1 > all) {
#pragma unroll
                        for (int i = 0; i < kN; ++i)
                            if (key0 + 8 * (i / 4) + 2 * (lane & 3) + (i & 1) > pos[i >> 1 & 1]) v[i] = __float_as_uint(kNegInf);
                    }
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        float even = __uint_as_float(v[2 * x]), uneven = __uint_as_float(v[2 * x + 1]);
#pragma unroll
                        for (int i = 4; i < kN; i += 4) even = fmaxf(even, __uint_as_float(v[i + 2 * x])), uneven = fmaxf(uneven, __uint_as_float(v[i + 2 * x + 1]));
                        top[x] = fmaxf(even, uneven);
                        top[x] = fmaxf(top[x], __shfl_xor_sync(~0u, top[x], 1));
                        top[x] = fmaxf(top[x], __shfl_xor_sync(~0u, top[x], 2));
                        grew |= (top[x] - m[x]) * sc > 8.f;  // (m = -inf: inf, or NaN if the row has seen nothing yet)
                    }
                }
                if (softmax_any(grew || !ok)) {  // (of either half of a row: the same for both)
                    if (live && (lane & 3) == 0) {
                        ex[ROWS * half + 16 * w + lane / 4] = top[0];
                        ex[ROWS * half + 16 * w + lane / 4 + 8] = top[1];
                    }
                    ok = !softmax_any(!ok);
                    if (!ok) break;
                    if (live) {
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            top[x] = fmaxf(top[x], ex[ROWS * (half ^ 1) + 16 * w + lane / 4 + 8 * x]);
                            float f = 1.f;
                            if ((top[x] - m[x]) * sc > 8.f) {
                                f = m[x] == kNegInf ? 0.f : exp2_fast((m[x] - top[x]) * sc);
                                m[x] = top[x];
                            }
                            l[x] *= f;
                            if ((lane & 3) == 0 && half == 0) factor[16 * w + lane / 4 + 8 * x] = f;
                        }
                    }
                    if (j > 0) {  // O is rescaled between the products: the one before has to be there
                        softmax_sync();
                        if (wait(o_done + before.slot, before.phase)) {
                            tc_fence_after();
#pragma unroll 1
                            for (int x = 16 * half; x < parts * ROWS; x += 32) {
                                uint32_t o[16];
                                tmem_ld16(tmem + lane_base + C::kOCol + x, o);
                                tmem_ld_wait();
                                tmem_tie<16>(o);
#pragma unroll
                                for (int y = 0; y < 16; ++y)
                                    if (x % ROWS + y < rows) o[y] = __float_as_uint(__uint_as_float(o[y]) * factor[x % ROWS + y]);
                                tmem_st16(tmem + lane_base + C::kOCol + x, o);
                            }
                            tmem_st_wait();
                        }
                    }
                }
                // what P's place held before is read (of a piece's first units it is known: the piece before ended with a wait for its last product)
                if (j >= C::kPs) wait(o_done + pb.slot, pb.phase ^ 1);
                if (ok && live) {
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const float base = m[x] == kNegInf ? 0.f : m[x] * sc - kLift<T>;
                        const int r = 16 * w + lane / 4 + 8 * x;
                        uint8_t* at = smem + C::kOffP + r * 128 + (lane & 3) * 4;
#pragma unroll
                        for (int i = 0; i < kKeys / 16; ++i) {
                            const float p0 = exp2_fast(fmaf(__uint_as_float(v[4 * i + 2 * x]), sc, -base));
                            const float p1 = exp2_fast(fmaf(__uint_as_float(v[4 * i + 2 * x + 1]), sc, -base));
                            l[x] += p0 + p1;
                            // the product's operand: 16 bits; the sum l is of the fp32 values
                            *reinterpret_cast<uint32_t*>(at + (((4 * pb.slot + kKeys / 16 * half + i) ^ (r & 7)) << 4)) = Elem<T>::pack(p0, p1);
                        }
                    }
                    fence_async_proxy();
                }
                tc_fence_before();
                __syncwarp();
                if (ok && lane == 0) arrive_own(p_full + pb.slot);
                before = pb;
                pb.next();
            }
            if (ok) wait(o_done + before.slot, before.phase);
            if (softmax_any(!ok)) {
                ok = false;
                break;
            }
            // ------------------------------------------------------------ the tile's output
            tc_fence_after();
            const bool whole = c.whole();
            const int64_t part0 = (2 * static_cast<int64_t>(blockIdx.x) + (c.u == c.begin ? 0 : 1)) * ROWS;  // its first row among the pieces'
            if (live) {
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    l[x] += __shfl_xor_sync(~0u, l[x], 1);
                    l[x] += __shfl_xor_sync(~0u, l[x], 2);
                    if (half == 1 && (lane & 3) == 0) ex[ROWS + 16 * w + lane / 4 + 8 * x] = l[x];
                }
            }
            softmax_sync();
            if (live && half == 0 && (lane & 3) == 0) {
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const int r = 16 * w + lane / 4 + 8 * x;
                    if (r >= rows) continue;
                    const float sum = l[x] + ex[ROWS + r];
                    factor[r] = sum == 0.f ? 0.f : 1.f / sum;
                    if (sum != sum) *odd = 1;
                    if (!whole) {
                        a.part_ml[part0 + r] = make_float2(m[x] == kNegInf ? kNegInf : m[x] * sc - kLift<T>, sum);
                    } else if (a.lse) {
                        int tok, head;
                        row_of(kv, r0 + r, tok, head);
                        a.lse[static_cast<int64_t>(c.s.q0 + tok) * kv.hq + head] = sum == 0.f ? kNegInf : (m[x] * sc - kLift<T> + log2f(sum)) * kLn2;
                    }
                }
            }
            softmax_sync();
            bool bad = false;
            for (int x = half; x < parts; x += 2) {
                const int e = 128 * x + 32 * w + lane;    // this thread's component
                float* dst = a.part_o + part0 * (128 * parts) + e;
                if (!whole) {
                    // (rows past the tile's are written, too, and never read)
                    constexpr int kR = ROWS < 32 ? ROWS : 32;
#pragma unroll 1
                    for (int y = 0; y < rows; y += kR) {
                        uint32_t o[kR];
                        __syncwarp();
                        if constexpr (kR == 32) tmem_ld32(tmem + lane_base + C::kOCol + ROWS * x + y, o);
                        else tmem_ld16(tmem + lane_base + C::kOCol + ROWS * x + y, o);
                        tmem_ld_wait();
                        tmem_tie<kR>(o);
#pragma unroll
                        for (int r = 0; r < kR; ++r, dst += 128 * parts) *dst = __uint_as_float(o[r]);
                    }
                    continue;
                }
#pragma unroll 1
                for (int y = 0; y < rows; y += 16) {
                    uint32_t o[16];
                    __syncwarp();                     // (the lanes store different rows)
                    tmem_ld16(tmem + lane_base + C::kOCol + ROWS * x + y, o);
                    tmem_ld_wait();
                    tmem_tie<16>(o);
#pragma unroll
                    for (int r = 0; r < 16; r += 2) {
                        // two rows: the even lane of a pair writes both lanes' components of the first, the odd lane of the second
                        const float2 f = *reinterpret_cast<const float2*>(factor + y + r);
                        const float f0 = __uint_as_float(o[r]) * f.x, f1 = __uint_as_float(o[r + 1]) * f.y;
                        bad |= e < kv.d && ((f0 != f0 && y + r < rows) || (f1 != f1 && y + r + 1 < rows));
                        const float got = __shfl_xor_sync(~0u, lane & 1 ? f0 : f1, 1);
                        const int rr = y + r + (lane & 1);
                        if (rr < rows && (e & ~1) < kv.d)
                            *reinterpret_cast<uint32_t*>(static_cast<T*>(a.out) + row_at[rr] + (e & ~1)) =
                                lane & 1 ? Elem<T>::pack(got, f1) : Elem<T>::pack(f0, got);
                    }
                }
            }
            tc_fence_before();
            if (bad) *odd = 1;
            softmax_sync();                           // (`factor` and `row_at` are read)
            if (lane == 0) arrive_own(o_free);
            deal_next<ROWS, kKeys>(a, c);
        }
        if (ok && *odd) retake_rows<T, ROWS>(a, *reinterpret_cast<const Cursor*>(smem + C::kOffStart), warp - 4);
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_free<1>(tmem, C::kCols);
    }
}

// ---------------------------------------------------------------- the join
// The pieces of a cut tile: CTAs c0 to c1 have one each.
template <int ROWS>
struct CutTile {
    BoundaryRec rec;
    int c0, c1, rows;
    __device__ __forceinline__ CutTile(const LatentArgs& a, const BoundaryRec& r) : rec(r) {
        c0 = static_cast<int>(div_line(r.begin, r.per));
        c1 = static_cast<int>(div_line(r.begin + r.n - 1, r.per));
        rows = min(r.q_len * a.kv.group - r.rt * ROWS, ROWS);
    }
    // Row r of CTA p's piece among the pieces' rows.
    __device__ __forceinline__ int64_t at(int p, int r) const { return (2 * static_cast<int64_t>(p) + (p * rec.per >= rec.begin ? 0 : 1)) * ROWS + r; }
};

__device__ __forceinline__ void add_scaled(float4& to, const float4& x, float f) {
    to.x += x.x * f;
    to.y += x.y * f;
    to.z += x.z * f;
    to.w += x.w * f;
}

// Whether four components of a row from `col + 4 lane` on have a NaN (what lies behind the latent part may be anything).
__device__ __forceinline__ bool odd_four(const LatentArgs& a, const float4& o, int col) {
    return col + 4 * (threadIdx.x & 31) < a.kv.d && (o.x != o.x || o.y != o.y || o.z != o.z || o.w != o.w);
}

// Writes 128 components of a row from `col` on, a warp four a lane, and with component 0 the row's lse.
template <typename T, int ROWS>
__device__ __forceinline__ void join_store(const LatentArgs& a, const CutTile<ROWS>& t, int r, const float4& o, int col, float m, float l) {
    const KvArgs& kv = a.kv;
    const int lane = threadIdx.x & 31;
    int i, head;
    row_of(kv, t.rec.rt * ROWS + r, i, head);
    const int tok = t.rec.q0 + i;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    if (col + 4 * lane < kv.d)
        *reinterpret_cast<uint2*>(static_cast<T*>(a.out) + tok * a.o_ts + head * a.o_hs + col + 4 * lane) =
            make_uint2(Elem<T>::pack(o.x * inv, o.y * inv), Elem<T>::pack(o.z * inv, o.w * inv));
    if (lane == 0 && col == 0 && a.lse) a.lse[static_cast<int64_t>(tok) * kv.hq + head] = l == 0.f ? kNegInf : (m + log2f(l)) * kLn2;
}

// Components [col0, col1) of a row that has a NaN, taken again.
template <typename T, int ROWS>
__device__ __forceinline__ void join_retake(const LatentArgs& a, const CutTile<ROWS>& t, int r, int col0, int col1) {
    int i, head;
    row_of(a.kv, t.rec.rt * ROWS + r, i, head);
    latent_row<T>(a, t.rec.b, t.rec.q0 + i, head, t.rec.pos0 + i, col0, col1);
}

// A row by a warp, its pieces' loads two at a time.
template <typename T, int ROWS>
__device__ __forceinline__ void join_few(const LatentArgs& a, const CutTile<ROWS>& t, int r, int parts) {
    constexpr int kVec = kMaxLatent / 128;  // fours of components of a lane
    const int lane = threadIdx.x & 31;
    float mm = kNegInf, ll = 0.f;
    float4 acc[kVec];
#pragma unroll
    for (int x = 0; x < kVec; ++x) acc[x] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int p = t.c0; p <= t.c1; p += 2) {
        const bool two = p < t.c1;
        const int64_t at0 = t.at(p, r), at1 = t.at(min(p + 1, t.c1), r);
        float4 o0[kVec], o1[kVec];
#pragma unroll
        for (int x = 0; x < kVec; ++x) {
            o0[x] = o1[x] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (x < parts) o0[x] = reinterpret_cast<const float4*>(a.part_o + at0 * (128 * parts) + 128 * x)[lane];
            if (x < parts && two) o1[x] = reinterpret_cast<const float4*>(a.part_o + at1 * (128 * parts) + 128 * x)[lane];
        }
        const float2 v0 = a.part_ml[at0], v1 = two ? a.part_ml[at1] : make_float2(kNegInf, 0.f);
        const float top = fmaxf(mm, fmaxf(v0.x, v1.x)), base = top == kNegInf ? 0.f : top;
        const float f = exp2_fast(mm - base), f0 = exp2_fast(v0.x - base), f1 = exp2_fast(v1.x - base);
        mm = top;
        ll = ll * f + v0.y * f0 + v1.y * f1;
#pragma unroll
        for (int x = 0; x < kVec; ++x) {
            acc[x] = make_float4(acc[x].x * f, acc[x].y * f, acc[x].z * f, acc[x].w * f);
            add_scaled(acc[x], o0[x], f0);
            if (two) add_scaled(acc[x], o1[x], f1);
        }
    }
    bool odd = ll != ll;
#pragma unroll
    for (int x = 0; x < kVec; ++x) odd |= x < parts && odd_four(a, acc[x], 128 * x);
    if (__any_sync(~0u, odd)) {  // (once, however many of its components: it is a walk over all keys)
        join_retake<T, ROWS>(a, t, r, 0, kMaxLatent);
        return;
    }
#pragma unroll
    for (int x = 0; x < kVec; ++x)
        if (x < parts) join_store<T, ROWS>(a, t, r, acc[x], 128 * x, mm, ll);
}

// 128 components of a row by the block, eight of the pieces' loads at a time in a warp.  part, part_ml: of the block.
template <typename T, int ROWS>
__device__ __forceinline__ void join_many(const LatentArgs& a, const CutTile<ROWS>& t, int r, int col, int parts, float4 (*part)[32], float2* part_ml) {
    constexpr int kNext = 8;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float mm = kNegInf, ll = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int p0 = t.c0 + warp; p0 <= t.c1; p0 += kNext * kJoinWarps) {
        float2 v[kNext];
        float4 o[kNext];
#pragma unroll
        for (int y = 0; y < kNext; ++y) {
            const int p = p0 + y * kJoinWarps;
            v[y] = make_float2(kNegInf, 0.f);
            o[y] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (p > t.c1) continue;
            v[y] = a.part_ml[t.at(p, r)];
            o[y] = reinterpret_cast<const float4*>(a.part_o + t.at(p, r) * (128 * parts) + col)[lane];
        }
        float top = mm;
#pragma unroll
        for (int y = 0; y < kNext; ++y) top = fmaxf(top, v[y].x);
        const float base = top == kNegInf ? 0.f : top, f = exp2_fast(mm - base);
        mm = top;
        ll *= f;
        acc = make_float4(acc.x * f, acc.y * f, acc.z * f, acc.w * f);
#pragma unroll
        for (int y = 0; y < kNext; ++y) {
            const float g = exp2_fast(v[y].x - base);
            ll += v[y].y * g;
            if (p0 + y * kJoinWarps <= t.c1) add_scaled(acc, o[y], g);
        }
    }
    __syncthreads();
    if (lane == 0) part_ml[warp] = make_float2(mm, ll);
    part[warp][lane] = acc;
    __syncthreads();
    if (warp != 0) return;
    float top = kNegInf, sum = 0.f;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) top = fmaxf(top, part_ml[w].x);
    const float base = top == kNegInf ? 0.f : top;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) {
        const float f = exp2_fast(part_ml[w].x - base);
        sum += part_ml[w].y * f;
        add_scaled(o, part[w][lane], f);
    }
    if (__any_sync(~0u, sum != sum || odd_four(a, o, col))) join_retake<T, ROWS>(a, t, r, col, col + 128);
    else join_store<T, ROWS>(a, t, r, o, col, top, sum);
}

// The join of the pieces of the cut tiles.  Block (i, y) stands for the boundary before CTA i + 1; the items of a tile, eight rows, a
// warp each, or where the pieces are many, 128 components of one row, are dealt over the blocks of the boundaries that cut it.  (One line of
// all items for all blocks, found by sums over the boundaries, takes 2 us more.)  The sums' order goes by the pieces' CTAs alone, so two
// runs give the same bits.
constexpr int kManyPieces = 9;
constexpr int kJoinTurns = 8;  // blocks of a boundary: 4 and 16 take 1 us more on four sequences' 48 rows
template <typename T, int ROWS>
__global__ void __launch_bounds__(kJoinWarps * 32, 3) latent_join_kernel(const __grid_constant__ LatentArgs a) {
    wait_for_stream();
    __shared__ float4 part[kJoinWarps][32];
    __shared__ float2 part_ml[kJoinWarps];
    const int warp = threadIdx.x >> 5, parts = (a.kv.d + 127) / 128;
    const BoundaryRec rec = a.recs[blockIdx.x + 1];
    if (!rec.cut) return;
    const CutTile<ROWS> t(a, rec);
    const int step = t.c1 - t.c0, first = blockIdx.x - t.c0 + step * blockIdx.y;
    if (step + 1 >= kManyPieces) {
        for (int k = first; k < t.rows * parts; k += step * kJoinTurns) join_many<T, ROWS>(a, t, k / parts, k % parts * 128, parts, part, part_ml);
    } else {
        for (int k = first; k * kJoinWarps < t.rows; k += step * kJoinTurns)
            if (k * kJoinWarps + warp < t.rows) join_few<T, ROWS>(a, t, k * kJoinWarps + warp, parts);
    }
}

// The cache [pages][page_size][Dc + R], eight rows at a time in 128-byte-swizzled rows of 64 components.  Rows of whole blocks of
// 64: a 4-D map (component, row, block, page), a box has the rows' every block; else a 3-D map (component, row, page) and a box a
// block, which leaves out what lies behind a row's end.  The page past the last reads zeros.
cudaError_t make_map(const LatentArgs& a, int dtype, bool wide, CUtensorMap* map) {
    Encode encode = nullptr;
    if (cudaError_t e = get_encode(&encode); e != cudaSuccess) return e;
    const KvArgs& kv = a.kv;
    const cuuint64_t row = 2 * kv.k_rs, page = kv.n_pages > 1 ? 2 * kv.k_ps : 16, n_rows = kv.page, n_pages = kv.n_pages, blocks = a.dk / 64;
    const cuuint32_t elem[4] = {1, 1, 1, 1};
    const cuuint64_t dims4[4] = {64, n_rows, blocks, n_pages}, strides4[3] = {row, 128, page};
    const cuuint32_t boxes4[4] = {64, 8, static_cast<cuuint32_t>(blocks), 1};
    const cuuint64_t dims3[3] = {static_cast<cuuint64_t>(a.dk), n_rows, n_pages}, strides3[2] = {row, page};
    const cuuint32_t boxes3[3] = {64, 8, 1};
    const CUresult r = encode(map, dtype == 0 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, wide ? 4 : 3, kv.k, wide ? dims4 : dims3,
                              wide ? strides4 : strides3, wide ? boxes4 : boxes3, elem, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// The queries as a 3-D map (component, head, token), boxes of 64 components x `rows` (token, head) rows: by rows of uniform
// stride where there is one (returns 1: second coordinate token * heads + head), else where whole heads of a token or whole
// tokens make a tile (returns 2).  0: no map.
template <int ROWS>
int make_qmap(const LatentArgs& a, int dtype, CUtensorMap* map, cudaError_t* err) {
    const KvArgs& kv = a.kv;
    const int64_t most = int64_t(1) << 39;
    const bool heads = kv.hq > 1, tokens = kv.n_tokens > 1;
    if ((heads && (a.q_hs <= 0 || a.q_hs >= most)) || (tokens && (a.q_ts <= 0 || a.q_ts >= most))) return 0;
    const bool uniform = !heads || !tokens || a.q_ts == a.q_hs * kv.hq;
    const int bh = std::min(kv.hq, ROWS);
    if (!uniform && (ROWS % bh != 0 || kv.hq % bh != 0)) return 0;
    Encode encode = nullptr;
    if ((*err = get_encode(&encode)) != cudaSuccess) return 0;
    const int64_t step = 2 * (heads ? a.q_hs : tokens ? a.q_ts : 8);
    const cuuint32_t elem[3] = {1, 1, 1};
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(a.dk), static_cast<cuuint64_t>(uniform ? int64_t(kv.hq) * kv.n_tokens : kv.hq),
                                static_cast<cuuint64_t>(uniform ? 1 : kv.n_tokens)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(step), static_cast<cuuint64_t>(uniform ? 16 : 2 * a.q_ts)};
    const cuuint32_t boxes[3] = {64, static_cast<cuuint32_t>(uniform ? ROWS : bh), static_cast<cuuint32_t>(uniform ? 1 : ROWS / bh)};
    const CUresult r = encode(map, dtype == 0 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void*>(a.q), dims,
                              strides, boxes, elem, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    *err = r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
    return uniform ? 1 : 2;
}

// Up to so many positions a row tile stays with one CTA: the pieces' way through memory and the second kernel cost more than
// the keys' streaming by one.  Few tiles: one sequence of 16 heads, whole | split, 100 positions 9.6 | 10.5 us, 200 11.9 | 11.0.  Tiles
// for half of the GPU and more: 64 sequences of 128 heads at 500 30.6 us, split 39; 32 of 16 heads (a fifth of the GPU) split
// 16.3, whole 19.5.
constexpr int64_t kWholeKeys = 128, kWholeKeysMany = 1024;

template <typename T, int ROWS>
cudaError_t launch_r(LatentArgs a, int dtype, int64_t rows, int n_ctas, cudaStream_t st) {
    using C = LatCfg<ROWS>;
    const bool wide = a.dk % 64 == 0;
    CUtensorMap map;
    if (cudaError_t e = make_map(a, dtype, wide, &map); e != cudaSuccess) return e;
    CUtensorMap qmap = map;
    cudaError_t e = cudaSuccess;
    const int q_rows = make_qmap<ROWS>(a, dtype, &qmap, &e);
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(attend_latent_kernel<T, ROWS>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    const bool many = 2 * a.kv.n_seqs * ((rows + ROWS - 1) / ROWS) >= n_ctas;
    a.split = n_ctas > 1 && a.max_keys > (many ? kWholeKeysMany : kWholeKeys);
    e = launch_in_stream(attend_latent_kernel<T, ROWS>, dim3(n_ctas), C::kThreads, C::kSmem, 1, st, a, wide ? 1 : 0, q_rows, map, qmap);
    if (e != cudaSuccess || !a.split) return e;
    return launch_in_stream(latent_join_kernel<T, ROWS>, dim3(n_ctas - 1, kJoinTurns), kJoinWarps * 32, 0, 1, st, a);
}

// The fewest rows of a CTA that hold a token's, up to 64 (what is computed for rows that do not count costs time; more rows leave no
// room for the keys).  us, 64 ragged sequences | one of 131071:
//   16 heads   ROWS 16 65.2 | 37.4, 32 66.7 | 37.9;  units of 64 keys 69.6 | 40.1
//   32 heads   ROWS 32 69.1 | 38.4, 64 73.2 | 40.7;  units of 64 keys 73.4 | 41.4
//   64 heads   units of 32 keys 84.3 | 44.3, of 64 84.9 | 44.0
//   128 heads  units of 32 keys 141.0 | 65.9, of 64 143.5 | 66.4
// and a chunk of 509 tokens of 32 heads: units of 32 keys 372, of 64 390.
template <typename T>
cudaError_t launch_t(const LatentArgs& a, int dtype, int64_t rows, int n_ctas, cudaStream_t st) {
    if (rows <= 16) return launch_r<T, 16>(a, dtype, rows, n_ctas, st);
    if (rows <= 32) return launch_r<T, 32>(a, dtype, rows, n_ctas, st);
    return launch_r<T, 64>(a, dtype, rows, n_ctas, st);
}

}  // namespace

int latent_part_rows(int n_ctas) { return 2 * n_ctas * 64; }

cudaError_t launch_latent(const LatentArgs& a, int dtype, int64_t rows, int n_ctas, cudaStream_t st) {
    return dtype == 0 ? launch_t<__nv_bfloat16>(a, dtype, rows, n_ctas, st) : launch_t<__half>(a, dtype, rows, n_ctas, st);
}

}  // namespace moe

// C ABI of the attention operators: argument checks, workspace carving, engine
// choice and launches.  Host code only.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <initializer_list>

#include "attention.h"
#include "kernels.h"
#include "moe_w4a8.h"
#include "moe_w4a8_attention.h"

#define MOE_API extern "C" __attribute__((visibility("default")))

namespace {

constexpr int64_t kMaxSeqs = 2048;
constexpr int64_t kMaxHeads = 1024;
constexpr int64_t kMaxHeadDim = 256;
constexpr int64_t kI32 = (int64_t(1) << 31) - 1;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Sizes and strides of a batch (no pointers).
int check_sizes(const moe_kv_batch_t* b) {
    if (!b) return MOE_ERR_INVALID_ARG;
    for (int64_t v : {b->n_seqs, b->n_q_heads, b->n_kv_heads, b->head_dim, b->page_size, b->n_pages, b->table_width,
                      b->max_q_len, b->max_kv_len})
        if (v < 1) return MOE_ERR_INVALID_ARG;
    if (b->n_q_heads % b->n_kv_heads != 0 || b->head_dim % 8 != 0 || (b->dtype != MOE_DTYPE_BF16 && b->dtype != MOE_DTYPE_FP16))
        return MOE_ERR_INVALID_ARG;
    for (int64_t v : {b->k_page_stride, b->k_row_stride, b->k_head_stride, b->v_page_stride, b->v_row_stride, b->v_head_stride})
        if (v < 0 || v % 8 != 0) return MOE_ERR_INVALID_ARG;
    if (b->head_dim > kMaxHeadDim || b->n_q_heads > kMaxHeads || b->n_seqs > kMaxSeqs || b->page_size > kI32 ||
        b->n_pages > kI32 || b->table_width > kI32)
        return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

int check_batch(const moe_kv_batch_t* b, int64_t n_tokens) {
    if (int rc = check_sizes(b)) return rc;
    if (n_tokens < 0) return MOE_ERR_INVALID_ARG;
    for (const void* p : {static_cast<const void*>(b->k_cache), static_cast<const void*>(b->v_cache)})
        if (!p || !aligned16(p)) return MOE_ERR_INVALID_ARG;
    for (const int32_t* p : {b->block_table, b->q_start, b->kv_len})
        if (!p || !aligned4(p)) return MOE_ERR_INVALID_ARG;
    if (n_tokens > kI32 / b->n_q_heads) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

// One [T][heads][D] array.
int check_rows(const void* p, int64_t token_stride, int64_t head_stride) {
    return p && aligned16(p) && token_stride >= 0 && head_stride >= 0 && token_stride % 8 == 0 && head_stride % 8 == 0
               ? MOE_OK
               : MOE_ERR_INVALID_ARG;
}

moe::KvArgs kv_args(const moe_kv_batch_t* b, int64_t n_tokens) {
    moe::KvArgs a{};
    a.k = b->k_cache;
    a.v = b->v_cache;
    a.k_ps = b->k_page_stride;
    a.k_rs = b->k_row_stride;
    a.k_hs = b->k_head_stride;
    a.v_ps = b->v_page_stride;
    a.v_rs = b->v_row_stride;
    a.v_hs = b->v_head_stride;
    a.table = b->block_table;
    a.q_start = b->q_start;
    a.kv_len = b->kv_len;
    a.n_tokens = static_cast<int>(n_tokens);
    a.n_seqs = static_cast<int>(b->n_seqs);
    a.hq = static_cast<int>(b->n_q_heads);
    a.hkv = static_cast<int>(b->n_kv_heads);
    a.group = a.hq / a.hkv;
    a.d = static_cast<int>(b->head_dim);
    a.page = static_cast<int>(b->page_size);
    a.n_pages = static_cast<int>(b->n_pages);
    a.width = static_cast<int>(b->table_width);
    const __int128 cap = static_cast<__int128>(b->table_width) * b->page_size;
    a.cap = static_cast<int>(cap < kI32 - 512 ? cap : kI32 - 512);  // a last tile's end stays in range
    a.by_page = moe::make_divisor(a.page);
    a.by_group = moe::make_divisor(a.group);
    return a;
}

// Workspace of attend: the status word, then for each engine (both may run for one batch) boundary records and
// the pieces' sums and accumulators.
struct AttendLayout {
    int n_ctas;
    size_t hdr, recs[2], ml[2], o[2], total;
};

AttendLayout attend_layout(const moe_kv_batch_t* b) {
    AttendLayout L{};
    L.n_ctas = moe::num_sms();
    const int d = static_cast<int>(b->head_dim);
    size_t at = 0;
    auto take = [&](size_t bytes) { size_t here = at; at = (at + bytes + 255) & ~size_t(255); return here; };
    L.hdr = take(sizeof(moe::Header));
    for (int e = 0; e < 2; ++e) {
        const size_t rows = e == 0 ? 2 * L.n_ctas * moe::kSplitRows : moe::tc_part_rows(d, L.n_ctas);
        L.recs[e] = take(sizeof(moe::BoundaryRec) * L.n_ctas);
        L.ml[e] = take(sizeof(float2) * rows);
        L.o[e] = take(sizeof(float) * rows * moe::padded_dim(d));
    }
    L.total = at;
    return L;
}

// The tcgen05 engine takes batches whose rows fill more than one 16-row tile of the split engine, from pages that
// TMA boxes of whole 8-row groups divide.  Two of those tiles go to the split engine too where the caches' visible part is
// small (it reads it once for each): 4 sequences of 5 tokens (20 rows) at 500 positions of 8 heads of 128, 8 MB,
// 12.5 us against 19.5; 4 of 3 tokens (24 rows) at 6000 positions of 2 heads of 256, 49 MB, 35 us against 25.
constexpr int64_t kSmallCache = 16 << 20;

bool use_tc(const moe_kv_batch_t* b, int64_t rows) {
    if (rows <= moe::kSplitRows || moe::tc_box_rows(static_cast<int>(b->page_size)) < 8) return false;
    const int64_t keys = std::min<int64_t>(b->max_kv_len, kI32) * std::min<int64_t>(b->n_seqs, kMaxSeqs);
    if (rows <= 2 * moe::kSplitRows && keys <= kSmallCache / (4 * b->n_kv_heads * b->head_dim)) return false;
    for (int64_t s : {b->k_page_stride, b->k_row_stride, b->k_head_stride, b->v_page_stride, b->v_row_stride, b->v_head_stride})
        if (s == 0 || s >= int64_t(1) << 39) return false;  // what a tensor map can hold
    return true;
}

// Up to this many positions a row tile stays with one CTA: the pieces' way through memory and the second
// kernel cost more than the keys' streaming by one CTA.  32 / 8 heads of 128, whole | split: one sequence of 100
// positions 5.9 | 9.3 us, 760 11.3 | 8.9, 1500 17.1 | 9.6; eight sequences of 760 11.9 | 13.6, of 1000 15.8 | 15.8.
// (One sequence would gain from a lower bound, eight from a higher one.)
constexpr int64_t kWholeKeys = 768;

#define MOE_ATTEND(call)                                                         \
    do {                                                                         \
        if (int rc = moe::cuda_status((call), "paged_attention")) return rc;     \
    } while (0)

}  // namespace

MOE_API int moe_w4a8_kv_append(const moe_kv_batch_t* batch, const moe_head_prep_t* prep, int64_t n_tokens, const void* q,
                               int64_t q_token_stride, int64_t q_head_stride, const void* k, int64_t k_token_stride,
                               int64_t k_head_stride, const void* v, int64_t v_token_stride, int64_t v_head_stride, void* q_out,
                               int64_t q_out_token_stride, int64_t q_out_head_stride, void* stream) {
    if (int rc = check_batch(batch, n_tokens)) return rc;
    if (!prep || prep->rot_dim < 0 || prep->rot_dim % 2 != 0 || prep->rot_dim > batch->head_dim || !(prep->eps >= 0.f) ||
        !std::isfinite(prep->eps) || !std::isfinite(prep->weight_offset))
        return MOE_ERR_INVALID_ARG;
    if (prep->rot_dim > 0 && (!prep->cos_sin || !aligned16(prep->cos_sin) || prep->table_rows < 1)) return MOE_ERR_INVALID_ARG;
    for (const float* w : {prep->q_weight, prep->k_weight})
        if (w && !aligned16(w)) return MOE_ERR_INVALID_ARG;
    if (prep->positions && !aligned4(prep->positions)) return MOE_ERR_INVALID_ARG;
    if (n_tokens == 0) return MOE_OK;
    for (int rc : {check_rows(q, q_token_stride, q_head_stride), check_rows(k, k_token_stride, k_head_stride),
                   check_rows(v, v_token_stride, v_head_stride), check_rows(q_out, q_out_token_stride, q_out_head_stride)})
        if (rc) return rc;
    moe::AppendArgs a{};
    a.kv = kv_args(batch, n_tokens);
    a.q = q;
    a.k = k;
    a.v = v;
    a.q_out = q_out;
    a.q_ts = q_token_stride;
    a.q_hs = q_head_stride;
    a.k_ts = k_token_stride;
    a.k_hs = k_head_stride;
    a.v_ts = v_token_stride;
    a.v_hs = v_head_stride;
    a.o_ts = q_out_token_stride;
    a.o_hs = q_out_head_stride;
    a.cos_sin = prep->cos_sin;
    a.q_weight = prep->q_weight;
    a.k_weight = prep->k_weight;
    a.positions = prep->positions;
    a.table_rows = prep->table_rows;
    a.rot = static_cast<int>(prep->rot_dim);
    a.interleaved = prep->interleaved != 0;
    a.eps = prep->eps;
    a.weight_offset = prep->weight_offset;
    a.inv_d = 1.f / static_cast<float>(a.kv.d);
    return moe::cuda_status(moe::launch_kv_append(a, static_cast<int>(batch->dtype), static_cast<cudaStream_t>(stream)), "kv_append");
}

MOE_API size_t moe_w4a8_paged_attention_workspace_size(const moe_kv_batch_t* batch) {
    return check_sizes(batch) == MOE_OK ? attend_layout(batch).total : 0;
}

MOE_API int moe_w4a8_paged_attention(const moe_kv_batch_t* batch, int64_t n_tokens, const void* q, int64_t q_token_stride,
                                     int64_t q_head_stride, void* out, int64_t out_token_stride, int64_t out_head_stride, float* lse,
                                     float scale, int64_t window, void* workspace, size_t workspace_bytes, void* stream) {
    if (int rc = check_batch(batch, n_tokens)) return rc;
    if (!(scale > 0.f) || !std::isfinite(scale) || window < 0 || (lse && !aligned4(lse))) return MOE_ERR_INVALID_ARG;
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return MOE_ERR_INVALID_ARG;
    const AttendLayout L = attend_layout(batch);
    if (workspace_bytes < L.total) return MOE_ERR_WORKSPACE_TOO_SMALL;
    if (n_tokens == 0) return MOE_OK;
    for (int rc : {check_rows(q, q_token_stride, q_head_stride), check_rows(out, out_token_stride, out_head_stride)})
        if (rc) return rc;
    moe::AttendArgs a{};
    a.kv = kv_args(batch, n_tokens);
    a.q = q;
    a.out = out;
    a.lse = lse;
    a.q_ts = q_token_stride;
    a.q_hs = q_head_stride;
    a.o_ts = out_token_stride;
    a.o_hs = out_head_stride;
    a.scale = scale;
    a.window = window >= kI32 ? 0 : static_cast<int>(window);  // (no position is as far from another)
    char* ws = static_cast<char*>(workspace);
    a.hdr = moe::ws_at<moe::Header>(workspace, L.hdr);
    a.lead = 1;
    a.rows_hi = static_cast<int>(kI32);
    auto pieces = [&](int e) {
        a.recs = reinterpret_cast<moe::BoundaryRec*>(ws + L.recs[e]);
        a.part_ml = reinterpret_cast<float2*>(ws + L.ml[e]);
        a.part_o = reinterpret_cast<float*>(ws + L.o[e]);
    };
    const int dtype = static_cast<int>(batch->dtype);
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int64_t max_q = std::min(batch->max_q_len, n_tokens);
    const int64_t rows = max_q * a.kv.group;
    if (!use_tc(batch, rows)) {
        const int64_t tiles = (rows + moe::kSplitRows - 1) / moe::kSplitRows;
        const int64_t items = std::min<int64_t>(batch->n_seqs * tiles * a.kv.hkv, int64_t(1) << 30);
        const int64_t keys = std::min<int64_t>(std::min(batch->max_kv_len, a.window > 0 ? a.window + tiles * moe::kSplitRows : kI32), a.kv.cap);
        a.split = keys > kWholeKeys;
        pieces(0);
        MOE_ATTEND(moe::launch_attend_split(a, dtype, L.n_ctas, static_cast<int>(items), st));
        MOE_ATTEND(moe::launch_attend_split_join(a, dtype, L.n_ctas, st));
        return MOE_OK;
    }
    // Sequences of few rows among longer ones (decoding requests beside a chunk) go to the split engine: a tile of
    // 256 or 512 rows that they fill by a few streams their keys at less than half its rate: a chunk among
    // decoding requests 132 us (131 now), all on the tcgen05 engine 172.
    a.split = 1;
    moe::AttendArgs few = a;
    const bool mixed = a.kv.group <= moe::kSplitRows && n_tokens <= (batch->n_seqs - 1) * max_q + moe::kSplitRows / a.kv.group;  // (there may be some)
    if (mixed) {
        pieces(0);
        few = a;
        few.rows_hi = moe::kSplitRows;
        few.lead = 0;
        MOE_ATTEND(moe::launch_attend_split(few, dtype, L.n_ctas, 0, st));
        a.rows_lo = moe::kSplitRows + 1;
        a.follows = 1;
    }
    pieces(1);
    MOE_ATTEND(moe::launch_attend_tc(a, dtype, L.n_ctas, st));
    if (mixed) MOE_ATTEND(moe::launch_attend_split_join(few, dtype, L.n_ctas, st));
    MOE_ATTEND(moe::launch_attend_tc_join(a, dtype, rows, L.n_ctas, st));
    return MOE_OK;
}

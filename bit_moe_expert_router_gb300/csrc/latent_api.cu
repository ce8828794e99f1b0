// C ABI of latent attention: argument checks, workspace carving and launches.
// Host code only.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <initializer_list>

#include "kernels.h"
#include "latent.h"
#include "moe_w4a8.h"
#include "moe_w4a8_latent.h"

#define MOE_API extern "C" __attribute__((visibility("default")))

namespace {

constexpr int64_t kMaxSeqs = 2048;
constexpr int64_t kMaxHeads = 1024;
constexpr int64_t kI32 = (int64_t(1) << 31) - 1;
constexpr int64_t kMaxStride = int64_t(1) << 39;  // what a tensor map can hold

bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Sizes and strides of a batch (no pointers).
int check_sizes(const moe_latent_batch_t* b) {
    if (!b) return MOE_ERR_INVALID_ARG;
    for (int64_t v : {b->n_seqs, b->n_heads, b->latent_dim, b->page_size, b->n_pages, b->table_width, b->max_q_len, b->max_kv_len})
        if (v < 1) return MOE_ERR_INVALID_ARG;
    if (b->latent_dim % 8 != 0 || b->rot_dim < 0 || b->rot_dim % 8 != 0 || (b->dtype != MOE_DTYPE_BF16 && b->dtype != MOE_DTYPE_FP16))
        return MOE_ERR_INVALID_ARG;
    for (int64_t v : {b->page_stride, b->row_stride})
        if (v < 0 || v % 8 != 0) return MOE_ERR_INVALID_ARG;
    if (b->latent_dim > moe::kMaxLatent || b->rot_dim > moe::kMaxLatentRot) return MOE_ERR_UNSUPPORTED;
    if (b->row_stride < b->latent_dim + b->rot_dim) return MOE_ERR_INVALID_ARG;
    if (b->n_heads > kMaxHeads || b->n_seqs > kMaxSeqs || b->page_size % 8 != 0 || b->page_size > kI32 || b->n_pages > kI32 ||
        b->table_width > kI32 || b->page_stride >= kMaxStride || b->row_stride >= kMaxStride)
        return MOE_ERR_UNSUPPORTED;
    if (b->n_pages > 1 && b->page_stride == 0) return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}

int check_batch(const moe_latent_batch_t* b, int64_t n_tokens) {
    if (int rc = check_sizes(b)) return rc;
    if (n_tokens < 0) return MOE_ERR_INVALID_ARG;
    if (!b->cache || !aligned(b->cache, 16)) return MOE_ERR_INVALID_ARG;
    for (const int32_t* p : {b->block_table, b->q_start, b->kv_len})
        if (!p || !aligned(p, 4)) return MOE_ERR_INVALID_ARG;
    if (n_tokens > (kI32 - 512) / b->n_heads) return MOE_ERR_UNSUPPORTED;  // (a last row tile's end stays in range)
    return MOE_OK;
}

// A token array: its strides.
int check_rows(const void* p, std::initializer_list<int64_t> strides) {
    if (!p || !aligned(p, 16)) return MOE_ERR_INVALID_ARG;
    for (int64_t s : strides)
        if (s < 0 || s % 8 != 0) return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}

moe::KvArgs kv_args(const moe_latent_batch_t* b, int64_t n_tokens) {
    moe::KvArgs a{};
    a.k = a.v = b->cache;
    a.k_ps = a.v_ps = b->page_stride;
    a.k_rs = a.v_rs = b->row_stride;
    a.table = b->block_table;
    a.q_start = b->q_start;
    a.kv_len = b->kv_len;
    a.n_tokens = static_cast<int>(n_tokens);
    a.n_seqs = static_cast<int>(b->n_seqs);
    a.hq = a.group = static_cast<int>(b->n_heads);
    a.hkv = 1;
    a.d = static_cast<int>(b->latent_dim);
    a.page = static_cast<int>(b->page_size);
    a.n_pages = static_cast<int>(b->n_pages);
    a.width = static_cast<int>(b->table_width);
    const __int128 cap = static_cast<__int128>(b->table_width) * b->page_size;
    a.cap = static_cast<int>(cap < kI32 - 512 ? cap : kI32 - 512);  // a last tile's end stays in range
    a.by_page = moe::make_divisor(a.page);
    a.by_group = moe::make_divisor(a.group);
    return a;
}

// Workspace of attend: the status word, boundary records, the pieces' sums and accumulators.
struct LatentLayout {
    int n_ctas;
    size_t hdr, recs, ml, o, total;
};

LatentLayout latent_layout(const moe_latent_batch_t* b) {
    LatentLayout L{};
    L.n_ctas = moe::num_sms();
    size_t at = 0;
    auto take = [&](size_t bytes) { size_t here = at; at = (at + bytes + 255) & ~size_t(255); return here; };
    const size_t rows = moe::latent_part_rows(L.n_ctas);
    L.hdr = take(sizeof(moe::Header));
    L.recs = take(sizeof(moe::BoundaryRec) * L.n_ctas);
    L.ml = take(sizeof(float2) * rows);
    L.o = take(sizeof(float) * rows * ((b->latent_dim + 127) / 128 * 128));
    L.total = at;
    return L;
}

}  // namespace

MOE_API int moe_w4a8_latent_append(const moe_latent_batch_t* batch, const moe_head_prep_t* prep, int64_t n_tokens, const void* latent,
                                   int64_t latent_token_stride, const void* k_rot, int64_t k_rot_token_stride, const void* q_rot,
                                   int64_t q_rot_token_stride, int64_t q_rot_head_stride, void* q_rot_out, int64_t q_rot_out_token_stride,
                                   int64_t q_rot_out_head_stride, void* stream) {
    if (int rc = check_batch(batch, n_tokens)) return rc;
    if (!prep || prep->rot_dim != batch->rot_dim || prep->q_weight || !(prep->eps >= 0.f) || !std::isfinite(prep->eps) ||
        !std::isfinite(prep->weight_offset))
        return MOE_ERR_INVALID_ARG;
    if (prep->rot_dim > 0 && (!prep->cos_sin || !aligned(prep->cos_sin, 16) || prep->table_rows < 1)) return MOE_ERR_INVALID_ARG;
    if (prep->k_weight && !aligned(prep->k_weight, 16)) return MOE_ERR_INVALID_ARG;
    if (prep->positions && !aligned(prep->positions, 4)) return MOE_ERR_INVALID_ARG;
    if (n_tokens == 0) return MOE_OK;
    if (int rc = check_rows(latent, {latent_token_stride})) return rc;
    if (prep->rot_dim > 0)
        for (int rc : {check_rows(k_rot, {k_rot_token_stride}), check_rows(q_rot, {q_rot_token_stride, q_rot_head_stride}),
                       check_rows(q_rot_out, {q_rot_out_token_stride, q_rot_out_head_stride})})
            if (rc) return rc;
    moe::LatentAppendArgs a{};
    a.kv = kv_args(batch, n_tokens);
    a.latent = latent;
    a.k_rot = k_rot;
    a.q_rot = q_rot;
    a.q_out = q_rot_out;
    a.c_ts = latent_token_stride;
    a.k_ts = k_rot_token_stride;
    a.q_ts = q_rot_token_stride;
    a.q_hs = q_rot_head_stride;
    a.o_ts = q_rot_out_token_stride;
    a.o_hs = q_rot_out_head_stride;
    a.cos_sin = prep->cos_sin;
    a.weight = prep->k_weight;
    a.positions = prep->positions;
    a.table_rows = prep->table_rows;
    a.rot = static_cast<int>(prep->rot_dim);
    a.interleaved = prep->interleaved != 0;
    a.eps = prep->eps;
    a.weight_offset = prep->weight_offset;
    a.inv_d = 1.f / static_cast<float>(a.kv.d);
    return moe::cuda_status(moe::launch_latent_append(a, static_cast<int>(batch->dtype), static_cast<cudaStream_t>(stream)), "latent_append");
}

MOE_API size_t moe_w4a8_latent_attention_workspace_size(const moe_latent_batch_t* batch) {
    return check_sizes(batch) == MOE_OK ? latent_layout(batch).total : 0;
}

MOE_API int moe_w4a8_latent_attention(const moe_latent_batch_t* batch, int64_t n_tokens, const void* q, int64_t q_token_stride,
                                      int64_t q_head_stride, void* out, int64_t out_token_stride, int64_t out_head_stride, float* lse,
                                      float scale, void* workspace, size_t workspace_bytes, void* stream) {
    if (int rc = check_batch(batch, n_tokens)) return rc;
    if (!(scale > 0.f) || !std::isfinite(scale) || (lse && !aligned(lse, 4))) return MOE_ERR_INVALID_ARG;
    if (!workspace || !aligned(workspace, 256)) return MOE_ERR_INVALID_ARG;
    const LatentLayout L = latent_layout(batch);
    if (workspace_bytes < L.total) return MOE_ERR_WORKSPACE_TOO_SMALL;
    if (n_tokens == 0) return MOE_OK;
    for (int rc : {check_rows(q, {q_token_stride, q_head_stride}), check_rows(out, {out_token_stride, out_head_stride})})
        if (rc) return rc;
    moe::LatentArgs a{};
    a.kv = kv_args(batch, n_tokens);
    a.dk = static_cast<int>(batch->latent_dim + batch->rot_dim);
    a.q = q;
    a.out = out;
    a.lse = lse;
    a.q_ts = q_token_stride;
    a.q_hs = q_head_stride;
    a.o_ts = out_token_stride;
    a.o_hs = out_head_stride;
    a.scale = scale;
    a.lead = 1;
    a.rows_hi = static_cast<int>(kI32);
    char* ws = static_cast<char*>(workspace);
    a.hdr = moe::ws_at<moe::Header>(workspace, L.hdr);
    a.recs = reinterpret_cast<moe::BoundaryRec*>(ws + L.recs);
    a.part_ml = reinterpret_cast<float2*>(ws + L.ml);
    a.part_o = reinterpret_cast<float*>(ws + L.o);
    a.max_keys = std::min<int64_t>(batch->max_kv_len, a.kv.cap);
    const int64_t rows = std::min(batch->max_q_len, n_tokens) * a.kv.group;
    return moe::cuda_status(moe::launch_latent(a, static_cast<int>(batch->dtype), rows, L.n_ctas, static_cast<cudaStream_t>(stream)),
                            "latent_attention");
}

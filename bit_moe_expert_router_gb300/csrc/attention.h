// Internal arguments and launchers of the attention operators (host side; the
// C ABI in attention_api.cu validates everything before calling these).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace moe {

struct Header;

// Division of 0 <= n < 2^31 by a fixed 1 <= d < 2^31 by multiplication: with s = ceil(log2 d) and
// m = floor(2^32 (2^s - d) / d) + 1, n / d = (n + high word of n m) >> s.
struct Divisor {
    uint32_t mul, shift;
};
inline Divisor make_divisor(int d) {
    uint32_t s = 0;
    while ((int64_t(1) << s) < d) ++s;
    return {static_cast<uint32_t>(((((uint64_t(1) << s) - d) << 32) / d) + 1), s};
}

// A paged cache and its ragged batch, as the kernels take it.
struct KvArgs {
    void* k;
    void* v;
    int64_t k_ps, k_rs, k_hs;  // page, row and head strides, elements
    int64_t v_ps, v_rs, v_hs;
    const int32_t* table;      // [n_seqs][width]
    const int32_t* q_start;    // [n_seqs + 1]
    const int32_t* kv_len;     // [n_seqs]
    int n_tokens, n_seqs, hq, hkv, group, d, page, n_pages, width;
    int cap;                   // positions a row of the table can hold
    Divisor by_page, by_group;
};

struct AppendArgs {
    KvArgs kv;
    const void *q, *k, *v;
    void* q_out;
    int64_t q_ts, q_hs, k_ts, k_hs, v_ts, v_hs, o_ts, o_hs;
    const float* cos_sin;
    const float* q_weight;
    const float* k_weight;
    const int32_t* positions;
    int64_t table_rows;
    int rot, interleaved;
    float eps, weight_offset, inv_d;
};

struct AttendArgs {
    KvArgs kv;
    const void* q;
    void* out;
    float* lse;                // [n_tokens][hq] or null
    int64_t q_ts, q_hs, o_ts, o_hs;
    float scale;
    int window;                // 0: none
    int split;                 // pieces of a row tile may go to several CTAs
    int rows_lo, rows_hi;      // the sequences of so many rows per key/value head are this kernel's
    int lead;                  // of two kernels for one batch: this one clears the status and the stray rows
    int follows;               // launched beside the kernel before it
    Header* hdr;               // workspace: the status word
    struct BoundaryRec* recs;  // workspace: one per CTA
    float* part_o;             // [2 * CTAs][tile rows][padded D]
    float2* part_ml;           // [2 * CTAs][tile rows]: running maximum (base 2), sum
};

// What the join knows of the row tile that CTA c's share begins in: written by CTA c.
struct BoundaryRec {
    long long begin;   // where the tile begins in the line of units,
    long long per;     // units of the line per CTA,
    int n;             // and the tile's
    int cut;           // 1 if the tile began before CTA c
    int rt, h;         // row tile and key/value head
    int q0, q_len, pos0, b;  // the sequence: first token, tokens, first token's position, number
};

cudaError_t launch_kv_append(const AppendArgs& a, int dtype, cudaStream_t st);

// Head sizes are padded to one of three.
inline int padded_dim(int d) { return d <= 64 ? 64 : d <= 128 ? 128 : 256; }

// Attention on mma.sync with the keys split over the warps of the GPU.
constexpr int kSplitRows = 16;
cudaError_t launch_attend_split(const AttendArgs& a, int dtype, int n_ctas, int max_items, cudaStream_t st);
cudaError_t launch_attend_split_join(const AttendArgs& a, int dtype, int n_ctas, cudaStream_t st);

// Attention on tcgen05; pages of a multiple of 8 positions.
int tc_box_rows(int page);  // rows of a page that one TMA box takes
int tc_part_rows(int d, int n_ctas);  // rows of all pieces
cudaError_t launch_attend_tc(const AttendArgs& a, int dtype, int n_ctas, cudaStream_t st);
// rows: of a sequence per key/value head, at most
cudaError_t launch_attend_tc_join(const AttendArgs& a, int dtype, int64_t rows, int n_ctas, cudaStream_t st);

}  // namespace moe

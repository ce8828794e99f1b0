// Internal arguments and launchers of latent attention (host side; the C ABI
// in latent_api.cu validates everything before calling these).
#pragma once

#include "attention.h"

namespace moe {

// A latent batch goes as one with a single key/value head: kv.k is the cache, kv.d the latent part of its rows (what
// the outputs have), kv.group = kv.hq the heads.
struct LatentArgs : AttendArgs {
    int dk;            // components of a row, and of a query
    int64_t max_keys;  // of a sequence, by the caller's bound
};

struct LatentAppendArgs {
    KvArgs kv;
    const void *latent, *k_rot, *q_rot;
    void* q_out;
    int64_t c_ts, k_ts, q_ts, q_hs, o_ts, o_hs;
    const float* cos_sin;
    const float* weight;
    const int32_t* positions;
    int64_t table_rows;
    int rot, interleaved;
    float eps, weight_offset, inv_d;
};

constexpr int kMaxLatent = 512, kMaxLatentRot = 64;

cudaError_t launch_latent_append(const LatentAppendArgs& a, int dtype, cudaStream_t st);

// rows: of a sequence, by the caller's bound.  The rows of a tile and whether it is cut go by the bounds.
int latent_part_rows(int n_ctas);  // rows of all pieces, whatever the tile
cudaError_t launch_latent(const LatentArgs& a, int dtype, int64_t rows, int n_ctas, cudaStream_t st);

}  // namespace moe

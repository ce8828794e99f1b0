// Latent attention, a warp for each (token, head) row: the keys one after
// another with a running maximum and sum.
#include "latent_common.cuh"

namespace moe {
namespace {

template <typename T>
__global__ void __launch_bounds__(128) attend_latent_kernel(const LatentArgs a) {
    wait_for_stream();
    if (blockIdx.x == 0 && threadIdx.x == 0) a.hdr->status = kDevOk;  // (nothing here waits)
    const int64_t row = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
    if (row >= static_cast<int64_t>(a.kv.n_tokens) * a.kv.hq) return;
    const int t = static_cast<int>(row / a.kv.hq), head = static_cast<int>(row % a.kv.hq);
    const int b = find_seq(a.kv, t);
    int pos = -1;
    if (b >= 0) {
        const SeqInfo s = seq_info(a.kv, b);
        pos = s.pos0 + t - s.q0;
    }
    latent_row<T>(a, max(b, 0), t, head, pos);
}

}  // namespace

int latent_part_rows(int n_ctas) { return 2 * n_ctas * 64; }

cudaError_t launch_latent(const LatentArgs& a, int dtype, int64_t, int, cudaStream_t st) {
    const dim3 grid(static_cast<unsigned>((static_cast<int64_t>(a.kv.n_tokens) * a.kv.hq + 3) / 4));
    return dtype == 0 ? launch_in_stream(attend_latent_kernel<__nv_bfloat16>, grid, 128, 0, 1, st, a)
                      : launch_in_stream(attend_latent_kernel<__half>, grid, 128, 0, 1, st, a);
}

}  // namespace moe

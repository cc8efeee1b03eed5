// K6 without a pool: q and k normed and rotated into tensors of their own.
#include "append_kernel.cuh"

namespace pva {

cudaError_t launch_norm_rope(const ForwardParams& p, const RopeParams& rp, int head_dim, cudaStream_t s) {
    if (p.total_tokens <= 0 || rp_rows<kFlat>(p, rp) == 0) return cudaSuccess;
    if (head_dim == 128) return rp.norm ? launch_kv<128, kFlat, true>(p, rp, s) : launch_kv<128, kFlat, false>(p, rp, s);
    if (head_dim == 64) return rp.norm ? launch_kv<64, kFlat, true>(p, rp, s) : launch_kv<64, kFlat, false>(p, rp, s);
    return cudaErrorInvalidValue;
}

}  // namespace pva

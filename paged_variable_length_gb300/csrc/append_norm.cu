// K6: the launches of the append kernel with the norm of q and k.
#include "append_kernel.cuh"

namespace pva {

cudaError_t launch_append_norm(const ForwardParams& p, const RopeParams& rp, int head_dim, int kv_dtype, cudaStream_t s) {
    if (head_dim == 128) return launch_d<128, true>(p, rp, kv_dtype, s);
    if (head_dim == 64) return launch_d<64, true>(p, rp, kv_dtype, s);
    return cudaErrorInvalidValue;
}

}  // namespace pva

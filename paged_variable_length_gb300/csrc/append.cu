// K6: the launches of the append kernel without a norm, and the MXFP4 pool's read-back.
#include "append_kernel.cuh"

namespace pva {
namespace {

// The batch's new tokens' rows of an MXFP4 pool as bf16 (exact), to k / v [T, Hkv, D].  A lane
// turns 4 bytes of codes into 8 elements, a warp takes kLoadSteps such steps of a token's K and V
// rows.  Bound: HBM (the bf16 rows written).
constexpr int kLoadSteps = 8;

template <int D>
__global__ void __launch_bounds__(kThreads) load_kernel(const ForwardParams p, uint16_t* k, uint16_t* v, int row_bytes) {
    PlanHeader* hdr = reinterpret_cast<PlanHeader*>(p.ws + p.lay.header);
    dev::grid_dep_wait();
    dev::grid_dep_launch();
    const uint32_t errors = hdr->error_bits;
    constexpr int D8 = D / 8;
    const int Hkv = p.num_kv_heads, lanes = Hkv * D8;  // lanes' worth of a row
    const int64_t t = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    if (t >= p.total_tokens) return;
    const int lane = threadIdx.x & 31, l0 = blockIdx.y * (32 * kLoadSteps) + lane;
    const int req = token_request(p, t);
    if (errors & kErrFatal) return;
    const int64_t slot = token_slot(p, t, req, p.slots == nullptr ? token_index(p, 0, t, req) : 0, &hdr->error_bits,
                                    lane == 0);
    if (slot < 0) return;
    uint32_t w[kLoadSteps], e[kLoadSteps];
#pragma unroll
    for (int i = 0; i < kLoadSteps; ++i) {
        const int l = l0 + 32 * i;
        w[i] = e[i] = 0;
        if (l < 2 * lanes) {
            const bool is_v = l >= lanes;
            const int x = is_v ? l - lanes : l, h = x / D8, at = (x - h * D8) * 8;
            const uint8_t* row = reinterpret_cast<const uint8_t*>(is_v ? p.v_pool : p.k_pool) + slot * row_bytes;
            w[i] = *reinterpret_cast<const uint32_t*>(row + mx::codes_at(h, Hkv, D) + at / 2);
            e[i] = row[mx::scales_at(h, Hkv, D) + at / mx::kBlock];
        }
    }
#pragma unroll
    for (int i = 0; i < kLoadSteps; ++i) {
        const int l = l0 + 32 * i;
        if (l >= 2 * lanes) break;
        const bool is_v = l >= lanes;
        const float f = mx::scale_f32(e[i]);
        auto two = [&](uint32_t f16x2) {
            const __half2 hv = *reinterpret_cast<__half2*>(&f16x2);
            return dev::pack_bf16x2(__low2float(hv) * f, __high2float(hv) * f);
        };
        *reinterpret_cast<uint4*>((is_v ? v : k) + (t * lanes + (is_v ? l - lanes : l)) * 8) =
            make_uint4(two(mx::e2m1x2_to_f16x2<0>(w[i])), two(mx::e2m1x2_to_f16x2<1>(w[i])),
                       two(mx::e2m1x2_to_f16x2<2>(w[i])), two(mx::e2m1x2_to_f16x2<3>(w[i])));
    }
}

}  // namespace

cudaError_t launch_append(const ForwardParams& p, const RopeParams& rp, int head_dim, int kv_dtype, cudaStream_t s) {
    if (p.total_tokens <= 0) return cudaSuccess;
    if (rp.norm) return launch_append_norm(p, rp, head_dim, kv_dtype, s);
    if (head_dim == 128) return launch_d<128, false>(p, rp, kv_dtype, s);
    if (head_dim == 64) return launch_d<64, false>(p, rp, kv_dtype, s);
    return cudaErrorInvalidValue;
}

cudaError_t launch_load_mx(const ForwardParams& p, void* k, void* v, int head_dim, cudaStream_t s) {
    if (p.total_tokens <= 0) return cudaSuccess;
    const dim3 grid = token_grid(p, cdiv(2 * p.num_kv_heads * head_dim / 8, 32 * kLoadSteps));
    auto go = [&](auto kernel) {
        return launch_programmatic(kernel, grid, (unsigned)kThreads, 0, s, p, static_cast<uint16_t*>(k),
                                   static_cast<uint16_t*>(v), mx::row_bytes(p.num_kv_heads, head_dim));
    };
    if (head_dim == 128) return go(load_kernel<128>);
    if (head_dim == 64) return go(load_kernel<64>);
    return cudaErrorInvalidValue;
}

}  // namespace pva

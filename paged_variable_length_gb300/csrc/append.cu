// K6: appending this step's keys and values to the paged pool with the rotary position
// rotation applied on the way, and the MXFP4 pool's store and read-back.
//
// For token t at position p and pair i < rot/2, with c = cos_sin[p][i], s = cos_sin[p][rot/2+i]:
//   y1 = x1 c - x2 s,  y2 = x2 c + x1 s
// where (x1, x2) is (x[i], x[i + rot/2]) (half-split) or (x[2i], x[2i + 1]) (interleaved);
// head dims from rot on pass unchanged.  Products and sums are fp32, each rounded by itself (no
// contraction: the result does not depend on how the compiler pairs them), and the result is
// rounded once, into what holds it: bf16 for q and a bf16 pool, E4M3 of y / k_scale[h], or a
// block's E2M1 codes.
//
// Bound: HBM at many tokens (each activation is read once, each result written once), latency
// at few.  A lane holds 16 consecutive elements of a head (two 16-byte loads), D/16 lanes a
// head row, so that a row of a pool of any type leaves as one vector store a lane and an MXFP4
// block is two neighbouring lanes.  The other element of a half-split pair lies rot/2 away, in
// another lane of the same row: it comes by shuffle, not by a second read.  A warp keeps its
// token's cos and sin in registers across its head rows.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "device_utils.cuh"
#include "mxfp4.cuh"
#include "pva_internal.h"

namespace pva {
namespace {

constexpr int kThreads = 128;

// Slot of new token t (the caller's mapping, or derived from the page table), -1 when it is
// not stored; reports a bad page id or slot and stores nothing then.
__device__ __forceinline__ int64_t token_slot(const ForwardParams& p, int64_t t, uint32_t* err, bool report) {
    int64_t slot;
    if (p.slots != nullptr) {
        slot = p.slots[t];
    } else {
        const int i = p.tok_req[t];
        const int c0 = p.cu[i], n = p.cu[i + 1] - c0, L = p.seqlens[i];
        const int pos = L - n + (int)(t - c0);
        const int64_t page = p.page_table[(int64_t)i * p.ld + (pos >> p.page_shift)];
        if (page < 0 || page >= p.num_pages) {
            if (report) dev::set_error(err, kErrPage);
            return -1;
        }
        slot = (page << p.page_shift) + (pos & (p.page_size - 1));
    }
    if (slot < -1 || slot >= p.num_slots) {
        if (report) dev::set_error(err, kErrSlot);
        return -1;
    }
    return slot;
}

// Position of new token t in its request.
__device__ __forceinline__ int token_position(const ForwardParams& p, const RopeParams& rp, int64_t t) {
    if (rp.positions != nullptr) return rp.positions[t];
    int i;
    if (p.tok_req != nullptr) {
        i = p.tok_req[t];
    } else {  // the plan keeps no request per token with a caller's slot mapping: search cu
        int lo = 0, hi = rp.batch - 1;  // the last request whose first token is <= t
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (p.cu[mid] <= t) lo = mid;
            else hi = mid - 1;
        }
        i = lo;
    }
    const int c0 = p.cu[i];
    return p.seqlens[i] - (p.cu[i + 1] - c0) + (int)(t - c0);
}

// One MXFP4 block half: the lane's 16 elements of head h (lane pair (j even, j odd) = a block).
__device__ __forceinline__ void store_mx(uint8_t* row, const float (&y)[16], int h, int e0, int Hkv, int D, bool write) {
    uint32_t amax = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) amax = max(amax, __float_as_uint(y[i]) & 0x7FFFFFFFu);
    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    const uint32_t e = mx::scale_byte(amax);
    const float f = mx::inv_scale_f32(e);
    uint32_t w[2] = {0, 0};
    if (e != (uint32_t)mx::kScaleNan) {
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i >> 2] |= mx::f32x2_to_e2m1x2(y[2 * i] * f, y[2 * i + 1] * f) << (8 * (i & 3));
    }
    if (!write) return;
    *reinterpret_cast<uint2*>(row + mx::codes_at(h, Hkv, D) + e0 / 2) = make_uint2(w[0], w[1]);
    if ((e0 & 16) == 0) row[mx::scales_at(h, Hkv, D) + e0 / mx::kBlock] = (uint8_t)e;
}

__device__ __forceinline__ void unpack16(const int4& a, const int4& b, float (&x)[16]) {
    const uint32_t w[8] = {(uint32_t)a.x, (uint32_t)a.y, (uint32_t)a.z, (uint32_t)a.w,
                           (uint32_t)b.x, (uint32_t)b.y, (uint32_t)b.z, (uint32_t)b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

__device__ __forceinline__ void store_bf16(uint16_t* dst, const float (&y)[16]) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = dev::pack_bf16x2(y[2 * i], y[2 * i + 1]);
    reinterpret_cast<uint4*>(dst)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    reinterpret_cast<uint4*>(dst)[1] = make_uint4(w[4], w[5], w[6], w[7]);
}

// KV: PVA_KV_BF16, PVA_KV_E4M3 or PVA_KV_MXFP4.  R: head-row steps a warp takes (each 512
// elements); a warp serves one token.
template <int D, int KV, int R>
__global__ void __launch_bounds__(kThreads) append_kernel(const ForwardParams p, const RopeParams rp) {
    constexpr int LR = D / 16;   // lanes of a head row
    constexpr int RW = 32 / LR;  // head rows of a step
    PlanHeader* hdr = reinterpret_cast<PlanHeader*>(p.ws + p.lay.header);
    // the kernel before this one (the plan, the previous layer's last) finishes first; the
    // attention kernels that follow set up behind it (as behind the store kernel)
    dev::grid_dep_wait();
    dev::grid_dep_launch();
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        hdr->pad[0] = 0;  // decode kernel work counter
        hdr->pad[1] = 0;  // prefill kernel work counter
    }
    if (hdr->error_bits & kErrFatal) return;
    const int lane = threadIdx.x & 31, j = lane % LR, sub = lane / LR;
    const int Hq = rp.q != nullptr ? p.num_qo_heads : 0, Hkv = p.num_kv_heads;
    const int rows = Hq + 2 * Hkv;
    const int jobs = (rows + R * RW - 1) / (R * RW);  // warps a token takes
    const int64_t job = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const int64_t t = job / jobs;
    if (t >= p.total_tokens) return;
    const int row0 = (int)(job - t * jobs) * (R * RW);

    // the warp's rows: all loads first
    int4 a[R], b[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int row = row0 + r * RW + sub;
        a[r] = b[r] = make_int4(0, 0, 0, 0);
        if (row < rows) {
            const uint16_t* src = row < Hq ? rp.q + t * rp.ld_q + row * D
                                  : row < Hq + Hkv ? p.k + t * rp.ld_k + (row - Hq) * D
                                                   : p.v + t * rp.ld_v + (row - Hq - Hkv) * D;
            const int4* s4 = reinterpret_cast<const int4*>(src + j * 16);
            a[r] = s4[0];
            b[r] = s4[1];
        }
    }
    // cos and sin of the lane's elements; element e of the lane is head dim 16j + e
    const int rot = rp.rot_dim;
    float c[16], s[16];
    if (rot > 0) {
        const int pos = token_position(p, rp, t);
        if (pos < 0 || pos >= rp.max_positions) {
            if (lane == 0) dev::set_error(&hdr->error_bits, kErrPosition);
            return;  // (every warp of the token: nothing of it is written)
        }
        const float* cs = rp.cos_sin + (int64_t)pos * rot;
        if (16 * j < rot && row0 < Hq + Hkv) {
            if (rp.interleaved) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float4 cc = __ldg(reinterpret_cast<const float4*>(cs + 8 * j) + i);
                    const float4 ss = __ldg(reinterpret_cast<const float4*>(cs + rot / 2 + 8 * j) + i);
                    const float cv[4] = {cc.x, cc.y, cc.z, cc.w}, sv[4] = {ss.x, ss.y, ss.z, ss.w};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        c[8 * i + 2 * k] = c[8 * i + 2 * k + 1] = cv[k];
                        s[8 * i + 2 * k] = -sv[k];
                        s[8 * i + 2 * k + 1] = sv[k];
                    }
                }
            } else {
#pragma unroll
                for (int h = 0; h < 2; ++h) {  // the lane's two 8-element chunks
                    const int ch = 2 * j + h, half = rot / 16;
                    const bool lower = ch < half;
                    const float* cc = cs + 8 * (lower ? ch : ch - half);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float4 cv = __ldg(reinterpret_cast<const float4*>(cc) + i);
                        const float4 sv = __ldg(reinterpret_cast<const float4*>(cc + rot / 2) + i);
                        c[8 * h + 4 * i] = cv.x, c[8 * h + 4 * i + 1] = cv.y, c[8 * h + 4 * i + 2] = cv.z,
                                      c[8 * h + 4 * i + 3] = cv.w;
                        s[8 * h + 4 * i] = lower ? -sv.x : sv.x;
                        s[8 * h + 4 * i + 1] = lower ? -sv.y : sv.y;
                        s[8 * h + 4 * i + 2] = lower ? -sv.z : sv.z;
                        s[8 * h + 4 * i + 3] = lower ? -sv.w : sv.w;
                    }
                }
            }
        }
    }
    const int64_t slot = row0 + R * RW > Hq ? token_slot(p, t, &hdr->error_bits, lane == 0) : -1;

#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int row = row0 + r * RW + sub;
        float x[16];
        if (rot > 0 && !rp.interleaved) {
            // the pair's other element: chunk ch +- rot/16 of the same row
            const int half = rot / 16;
            uint32_t w[8] = {(uint32_t)a[r].x, (uint32_t)a[r].y, (uint32_t)a[r].z, (uint32_t)a[r].w,
                             (uint32_t)b[r].x, (uint32_t)b[r].y, (uint32_t)b[r].z, (uint32_t)b[r].w};
            uint32_t o[8];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int ch = 2 * j + h;
                const int other = ch < half ? ch + half : ch < 2 * half ? ch - half : ch;
                const int from = sub * LR + other / 2;
#pragma unroll
                for (int i = 0; i < 4; ++i)  // an odd distance swaps the lane's chunks
                    o[4 * h + i] = __shfl_sync(0xffffffffu, (half & 1) ? w[4 * (h ^ 1) + i] : w[4 * h + i], from);
            }
            unpack16(a[r], b[r], x);
            if (row < Hq + Hkv) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (16 * j + 8 * h >= rot) continue;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float o0 = __uint_as_float(o[4 * h + i] << 16);
                        const float o1 = __uint_as_float(o[4 * h + i] & 0xFFFF0000u);
                        const int e = 8 * h + 2 * i;
                        x[e] = __fadd_rn(__fmul_rn(x[e], c[e]), __fmul_rn(o0, s[e]));
                        x[e + 1] = __fadd_rn(__fmul_rn(x[e + 1], c[e + 1]), __fmul_rn(o1, s[e + 1]));
                    }
                }
            }
        } else {
            unpack16(a[r], b[r], x);
            if (rot > 0 && row < Hq + Hkv && 16 * j < rot) {
#pragma unroll
                for (int e = 0; e < 16; e += 2) {
                    const float x0 = x[e], x1 = x[e + 1];
                    x[e] = __fadd_rn(__fmul_rn(x0, c[e]), __fmul_rn(x1, s[e]));
                    x[e + 1] = __fadd_rn(__fmul_rn(x1, c[e + 1]), __fmul_rn(x0, s[e + 1]));
                }
            }
        }
        if (row < Hq) store_bf16(rp.q_out + (t * Hq + row) * D + j * 16, x);
        const bool is_v = row >= Hq + Hkv;
        const int h = is_v ? row - Hq - Hkv : row - Hq;
        const bool kv = row >= Hq && row < rows && slot >= 0;
        if constexpr (KV == PVA_KV_MXFP4) {  // the block's maximum is a shuffle: every lane takes part
            uint8_t* pool = reinterpret_cast<uint8_t*>(is_v ? p.v_pool : p.k_pool);
            store_mx(pool + slot * rp.row_bytes, x, h, j * 16, Hkv, D, kv);
        } else if (kv) {
            const int64_t at = (slot * Hkv + h) * D + j * 16;
            if constexpr (KV == PVA_KV_BF16) {
                store_bf16((is_v ? p.v_pool : p.k_pool) + at, x);
            } else {
                const float sc = (is_v ? p.v_scale : p.k_scale)[h];
                uint32_t w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    w[i] = dev::f32x2_to_e4m3x2(__fdiv_rn(x[4 * i], sc), __fdiv_rn(x[4 * i + 1], sc)) |
                           (dev::f32x2_to_e4m3x2(__fdiv_rn(x[4 * i + 2], sc), __fdiv_rn(x[4 * i + 3], sc)) << 16);
                *reinterpret_cast<uint4*>(reinterpret_cast<uint8_t*>(is_v ? p.v_pool : p.k_pool) + at) =
                    make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
    }
}

// The batch's new tokens' rows of an MXFP4 pool as bf16 (exact), to k / v [T, Hkv, D].  A lane
// turns 8 bytes of codes and their scale into 16 elements.
__global__ void __launch_bounds__(kThreads) load_kernel(const ForwardParams p, uint16_t* k, uint16_t* v, int D,
                                                        int row_bytes) {
    PlanHeader* hdr = reinterpret_cast<PlanHeader*>(p.ws + p.lay.header);
    dev::grid_dep_wait();
    dev::grid_dep_launch();
    if (hdr->error_bits & kErrFatal) return;
    const int Hkv = p.num_kv_heads, lanes = Hkv * D / 16, D16 = D / 16;
    const int64_t n = 2 * (int64_t)p.total_tokens * lanes;
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (i >= n) return;
    const int64_t job = i / lanes;  // (token, K | V)
    const int l = (int)(i - job * lanes), h = l / D16, e0 = (l - h * D16) * 16;
    const int64_t t = job >> 1;
    const bool is_v = job & 1;
    const int64_t slot = token_slot(p, t, &hdr->error_bits, l == 0 && !is_v);
    if (slot < 0) return;
    const uint8_t* row = reinterpret_cast<const uint8_t*>(is_v ? p.v_pool : p.k_pool) + slot * row_bytes;
    const uint2 w = *reinterpret_cast<const uint2*>(row + mx::codes_at(h, Hkv, D) + e0 / 2);
    const float f = mx::scale_f32(row[mx::scales_at(h, Hkv, D) + e0 / mx::kBlock]);
    uint32_t o[8];
    auto two = [&](uint32_t f16x2) {
        const __half2 hv = *reinterpret_cast<__half2*>(&f16x2);
        return dev::pack_bf16x2(__low2float(hv) * f, __high2float(hv) * f);
    };
    o[0] = two(mx::e2m1x2_to_f16x2<0>(w.x)), o[1] = two(mx::e2m1x2_to_f16x2<1>(w.x));
    o[2] = two(mx::e2m1x2_to_f16x2<2>(w.x)), o[3] = two(mx::e2m1x2_to_f16x2<3>(w.x));
    o[4] = two(mx::e2m1x2_to_f16x2<0>(w.y)), o[5] = two(mx::e2m1x2_to_f16x2<1>(w.y));
    o[6] = two(mx::e2m1x2_to_f16x2<2>(w.y)), o[7] = two(mx::e2m1x2_to_f16x2<3>(w.y));
    uint4* dst = reinterpret_cast<uint4*>((is_v ? v : k) + (t * Hkv + h) * D + e0);
    dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
    dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
}

template <int D, int KV>
cudaError_t launch_kv(const ForwardParams& p, const RopeParams& rp, cudaStream_t s) {
    constexpr int R = 2;
    constexpr int RW = 32 / (D / 16);
    const int rows = (rp.q != nullptr ? p.num_qo_heads : 0) + 2 * p.num_kv_heads;
    const int64_t warps = (int64_t)p.total_tokens * ((rows + R * RW - 1) / (R * RW));
    const int64_t blocks = cdiv(warps, kThreads / 32);
    return launch_programmatic(append_kernel<D, KV, R>, (unsigned)blocks, (unsigned)kThreads, 0, s, p, rp);
}

template <int D>
cudaError_t launch_d(const ForwardParams& p, const RopeParams& rp, int kv_dtype, cudaStream_t s) {
    switch (kv_dtype) {
        case PVA_KV_BF16: return launch_kv<D, PVA_KV_BF16>(p, rp, s);
        case PVA_KV_E4M3: return launch_kv<D, PVA_KV_E4M3>(p, rp, s);
        case PVA_KV_MXFP4: return launch_kv<D, PVA_KV_MXFP4>(p, rp, s);
    }
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_append(const ForwardParams& p, const RopeParams& rp, int head_dim, int kv_dtype, cudaStream_t s) {
    if (p.total_tokens <= 0) return cudaSuccess;
    if (head_dim == 128) return launch_d<128>(p, rp, kv_dtype, s);
    if (head_dim == 64) return launch_d<64>(p, rp, kv_dtype, s);
    return cudaErrorInvalidValue;
}

cudaError_t launch_load_mx(const ForwardParams& p, void* k, void* v, int head_dim, cudaStream_t s) {
    if (p.total_tokens <= 0) return cudaSuccess;
    const int64_t lanes = 2 * (int64_t)p.total_tokens * p.num_kv_heads * head_dim / 16;
    return launch_programmatic(load_kernel, (unsigned)cdiv(lanes, kThreads), (unsigned)kThreads, 0, s, p,
                               static_cast<uint16_t*>(k), static_cast<uint16_t*>(v), head_dim,
                               mx::row_bytes(p.num_kv_heads, head_dim));
}

}  // namespace pva

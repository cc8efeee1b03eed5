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
// at few.  A lane holds 16 elements of a head (two 16-byte loads), D/16 lanes a head row; a warp
// keeps its token's cosines and sines in registers across its head rows.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "device_utils.cuh"
#include "mxfp4.cuh"
#include "pva_internal.h"

namespace pva {
namespace {

constexpr int kThreads = 128;

// Request of new token t as the plan recorded it (with a caller's slot mapping it did not: -1).
// Loaded before the error word has been looked at, so it is not followed until then.
__device__ __forceinline__ int token_request(const ForwardParams& p, int64_t t) {
    return p.tok_req != nullptr ? p.tok_req[t] : -1;
}

// Slot of new token t of request i (the caller's mapping, or derived from the page table at
// position pos of the request), -1 when it is not stored; reports a bad page id or slot and
// stores nothing then.
__device__ __forceinline__ int64_t token_slot(const ForwardParams& p, int64_t t, int i, int pos, uint32_t* err,
                                              bool report) {
    int64_t slot;
    if (p.slots != nullptr) {
        slot = p.slots[t];
    } else {
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

// Index of new token t in its request i; i < 0: the request is the last whose first token is <= t.
__device__ __forceinline__ int token_index(const ForwardParams& p, int batch, int64_t t, int i) {
    if (i < 0) {
        int lo = 0, hi = batch - 1;
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

// A lane holds the 8-element chunks j and j + D/16 of a head row, so that every access of a warp
// is whole 128-byte lines (16 consecutive elements a lane left each store half sectors: 50 us
// against 30 for the 4-bit append of 9 k tokens).  How the elements pair:
//   kNone   no rotation;
//   kSplit  half-split pairs over the whole head: a lane has both elements of its 8 pairs;
//   kInter  interleaved pairs: 4 in each chunk;
//   kPart   half-split pairs over part of the head: a pair's other element lies rot/2 away, in
//           another lane of the row, and comes by shuffle;
//   kLow    the same where rot <= D/2: only the lane's first chunk turns, half the cosines, sines
//           and shuffles (the 4-bit append and read-back of 9 k tokens, rot = D/2: 46.5 us, 54.5 as kPart).
constexpr int kNone = 0, kSplit = 1, kInter = 2, kPart = 3, kLow = 4;

// x c + z s, every product and the sum rounded by itself.  (As packed pairs the assembler contracts
// a product and the sum into one rounding, explicit roundings or not.)
__device__ __forceinline__ float turn(float x, float c, float z, float s) {
    return __fadd_rn(__fmul_rn(x, c), __fmul_rn(z, s));
}

__device__ __forceinline__ void unpack8(const int4& a, float (&x)[16], int at) {
    const uint32_t w[4] = {(uint32_t)a.x, (uint32_t)a.y, (uint32_t)a.z, (uint32_t)a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[at + 2 * i] = __uint_as_float(w[i] << 16);
        x[at + 2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

// The row's elements as they leave: e0 / e1 are the head dims of the lane's two chunks.
__device__ __forceinline__ void store_bf16(uint16_t* row, const float (&y)[16], int e0, int e1) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = dev::pack_bf16x2(y[2 * i], y[2 * i + 1]);
    *reinterpret_cast<uint4*>(row + e0) = make_uint4(w[0], w[1], w[2], w[3]);
    *reinterpret_cast<uint4*>(row + e1) = make_uint4(w[4], w[5], w[6], w[7]);
}

__device__ __forceinline__ void store_e4m3(uint8_t* row, const float (&y)[16], int e0, int e1, float sc) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = dev::f32x2_to_e4m3x2(__fdiv_rn(y[4 * i], sc), __fdiv_rn(y[4 * i + 1], sc)) |
               (dev::f32x2_to_e4m3x2(__fdiv_rn(y[4 * i + 2], sc), __fdiv_rn(y[4 * i + 3], sc)) << 16);
    *reinterpret_cast<uint2*>(row + e0) = make_uint2(w[0], w[1]);
    *reinterpret_cast<uint2*>(row + e1) = make_uint2(w[2], w[3]);
}

// The larger of two, NaN if either is one.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// MXFP4: a block is the same chunk of four neighbouring lanes.  Every lane of the warp takes part;
// `write` says whose row is stored.
__device__ __forceinline__ void store_mx(uint8_t* row, const float (&y)[16], int h, int e0, int e1, int Hkv, int D,
                                         bool write) {
    uint32_t m[2];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        float a = fabsf(y[8 * c]);
#pragma unroll
        for (int i = 1; i < 8; ++i) a = max_nan(a, fabsf(y[8 * c + i]));
        m[c] = __float_as_uint(a);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        m[i] = max(m[i], __shfl_xor_sync(0xffffffffu, m[i], 1));
        m[i] = max(m[i], __shfl_xor_sync(0xffffffffu, m[i], 2));
    }
    if (!write) return;
    uint8_t* codes = row + mx::codes_at(h, Hkv, D);
    uint8_t* scales = row + mx::scales_at(h, Hkv, D);
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        const uint32_t e = mx::scale_byte(m[c]);
        uint32_t w = mx::f32x8_to_e2m1x8(y + 8 * c, mx::inv_scale_f32(e));
        if (e == (uint32_t)mx::kScaleNan) w = 0;
        const int at = c ? e1 : e0;
        *reinterpret_cast<uint32_t*>(codes + at / 2) = w;
        if (at % mx::kBlock == 0) scales[at / mx::kBlock] = (uint8_t)e;
    }
}

// KV: PVA_KV_BF16, PVA_KV_E4M3 or PVA_KV_MXFP4.  R: row steps a warp takes (each 512 elements);
// a warp serves one token.  (kPart alone needs its registers bounded: five blocks an SM, 52.8 us for
// the append and read-back above with rot = 3/4 D, against 56.0 unbounded and 58.6 at six; 0 leaves
// the others unbounded, a bound of 1 cost the bf16 append 5 us.)
template <int D, int KV, int MODE, int R>
__global__ void __launch_bounds__(kThreads, MODE == kPart ? 5 : 0) append_kernel(const ForwardParams p, const RopeParams rp) {
    constexpr int LR = D / 16;   // lanes of a head row
    constexpr int RW = 32 / LR;  // head rows of a step
    PlanHeader* hdr = reinterpret_cast<PlanHeader*>(p.ws + p.lay.header);
    // the kernel before this one (the plan, the previous layer's last) finishes first; the
    // attention kernels that follow set up behind it (as behind the store kernel)
    dev::grid_dep_wait();
    dev::grid_dep_launch();
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) {
        hdr->pad[0] = 0;  // decode kernel work counter
        hdr->pad[1] = 0;  // prefill kernel work counter
    }
    const uint32_t errors = hdr->error_bits;
    const int lane = threadIdx.x & 31, j = lane % LR, sub = lane / LR;
    const int Hq = rp.q != nullptr ? p.num_qo_heads : 0, Hkv = p.num_kv_heads;
    const int rows = Hq + 2 * Hkv;
    const int64_t t = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    if (t >= p.total_tokens) return;
    const int row0 = blockIdx.y * (R * RW);
    const int e0 = 8 * j, e1 = 8 * (j + LR);

    // the warp's rows: all loads first, the token's request and the error word beside them
    const int req = token_request(p, t);
    int4 a[R], b[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int row = row0 + r * RW + sub;
        a[r] = b[r] = make_int4(0, 0, 0, 0);
        if (row < rows) {
            const uint16_t* src = row < Hq ? rp.q + t * rp.ld_q + row * D
                                  : row < Hq + Hkv ? p.k + t * rp.ld_k + (row - Hq) * D
                                                   : p.v + t * rp.ld_v + (row - Hq - Hkv) * D;
            a[r] = *reinterpret_cast<const int4*>(src + e0);
            b[r] = *reinterpret_cast<const int4*>(src + e1);
        }
    }
    if (errors & kErrFatal) return;
    const int index = MODE != kNone || p.slots == nullptr ? token_index(p, rp.batch, t, req) : 0;
    const int64_t slot = row0 + R * RW > Hq ? token_slot(p, t, req, index, &hdr->error_bits, lane == 0) : -1;
    // cosines and sines: of the lane's 8 pairs (kInter: 4 of each chunk), or of its elements that may
    // turn (kPart: 16, kLow: the first 8)
    constexpr int NC = MODE == kPart ? 16 : 8;
    const int rot = rp.rot_dim, half = rot / 16;  // half: chunks between the elements of a kPart or kLow pair
    float c[NC], s[NC];
    if constexpr (MODE != kNone) {
        const int pos = rp.positions != nullptr ? rp.positions[t] : index;
        if (pos < 0 || pos >= rp.max_positions) {
            if (lane == 0) dev::set_error(&hdr->error_bits, kErrPosition);
            return;  // (every warp of the token: nothing of it is written)
        }
        const float* cs = rp.cos_sin + (int64_t)pos * rot;
        auto take = [&](int at, int pair) {  // four pairs' values
            const float4 cv = __ldg(reinterpret_cast<const float4*>(cs + pair));
            const float4 sv = __ldg(reinterpret_cast<const float4*>(cs + rot / 2 + pair));
            c[at] = cv.x, c[at + 1] = cv.y, c[at + 2] = cv.z, c[at + 3] = cv.w;
            s[at] = sv.x, s[at + 1] = sv.y, s[at + 2] = sv.z, s[at + 3] = sv.w;
        };
        if (row0 < Hq + Hkv) {
            if constexpr (MODE == kSplit) {
                take(0, 8 * j);
                take(4, 8 * j + 4);
            } else {
#pragma unroll
                for (int h = 0; h < (MODE == kLow ? 1 : 2); ++h) {
                    const int ch = j + h * LR;
                    if (8 * ch >= rot) continue;
                    if constexpr (MODE == kInter) {
                        take(4 * h, 4 * ch);
                    } else {
                        take(8 * h, 8 * (ch < half ? ch : ch - half));
                        take(8 * h + 4, 8 * (ch < half ? ch : ch - half) + 4);
                        if (ch < half) {  // the first element of a pair takes -sin
#pragma unroll
                            for (int i = 0; i < 8; ++i) s[8 * h + i] = -s[8 * h + i];
                        }
                    }
                }
            }
        }
    }

#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int row = row0 + r * RW + sub;
        const bool turned = row < Hq + Hkv;
        float x[16];
        unpack8(a[r], x, 0);
        unpack8(b[r], x, 8);
        if constexpr (MODE == kSplit) {
            if (turned) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float u = x[i], w = x[8 + i];
                    x[i] = turn(u, c[i], w, -s[i]);
                    x[8 + i] = turn(w, c[i], u, s[i]);
                }
            }
        } else if constexpr (MODE == kInter) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (!turned || (i < 4 ? e0 : e1) >= rot) continue;
                const float u = x[2 * i], w = x[2 * i + 1];
                x[2 * i] = turn(u, c[i], w, -s[i]);
                x[2 * i + 1] = turn(w, c[i], u, s[i]);
            }
        } else if constexpr (MODE == kPart || MODE == kLow) {
#pragma unroll
            for (int h = 0; h < (MODE == kLow ? 1 : 2); ++h) {
                const int ch = j + h * LR;
                const int other = ch < half ? ch + half : ch < 2 * half ? ch - half : ch;  // the pair's chunk
                const uint32_t wa[4] = {(uint32_t)a[r].x, (uint32_t)a[r].y, (uint32_t)a[r].z, (uint32_t)a[r].w};
                const uint32_t wb[4] = {(uint32_t)b[r].x, (uint32_t)b[r].y, (uint32_t)b[r].z, (uint32_t)b[r].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t oa = __shfl_sync(0xffffffffu, wa[i], sub * LR + other % LR);
                    const uint32_t ob = MODE == kPart ? __shfl_sync(0xffffffffu, wb[i], sub * LR + other % LR) : 0;
                    const uint32_t o = MODE == kLow || other < LR ? oa : ob;
                    const int e = 8 * h + 2 * i;
                    if (turned && 8 * ch < rot) {
                        x[e] = turn(x[e], c[e], __uint_as_float(o << 16), s[e]);
                        x[e + 1] = turn(x[e + 1], c[e + 1], __uint_as_float(o & 0xFFFF0000u), s[e + 1]);
                    }
                }
            }
        }
        if (row < Hq) store_bf16(rp.q_out + (t * Hq + row) * D, x, e0, e1);
        const bool is_v = row >= Hq + Hkv;
        const int h = is_v ? row - Hq - Hkv : row - Hq;
        const bool kv = row >= Hq && row < rows && slot >= 0;
        uint8_t* pool = reinterpret_cast<uint8_t*>(is_v ? p.v_pool : p.k_pool);
        if constexpr (KV == PVA_KV_MXFP4) {
            if (row0 + (r + 1) * RW > Hq) store_mx(pool + slot * rp.row_bytes, x, h, e0, e1, Hkv, D, kv);
        } else if (kv) {
            if constexpr (KV == PVA_KV_BF16)
                store_bf16(reinterpret_cast<uint16_t*>(pool) + (slot * Hkv + h) * D, x, e0, e1);
            else
                store_e4m3(pool + (slot * Hkv + h) * D, x, e0, e1, (is_v ? p.v_scale : p.k_scale)[h]);
        }
    }
}

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

// Head rows of a token that the append moves.
int rp_rows(const ForwardParams& p, const RopeParams& rp) {
    return (rp.q != nullptr ? p.num_qo_heads : 0) + 2 * p.num_kv_heads;
}

// x: groups of tokens, a warp each; y: parts of a token's rows.
dim3 token_grid(const ForwardParams& p, int64_t parts) {
    return dim3((unsigned)cdiv(p.total_tokens, kThreads / 32), (unsigned)parts);
}

template <int D, int KV, int MODE, int R>
cudaError_t launch_r(const ForwardParams& p, const RopeParams& rp, cudaStream_t s) {
    const dim3 grid = token_grid(p, cdiv(rp_rows(p, rp), R * 32 / (D / 16)));
    return launch_programmatic(append_kernel<D, KV, MODE, R>, grid, (unsigned)kThreads, 0, s, p, rp);
}

template <int D, int KV, int MODE>
cudaError_t launch_mode(const ForwardParams& p, const RopeParams& rp, cudaStream_t s) {
    // four steps a warp (2 KiB of loads in flight each) carry HBM's rate (16.6 k tokens, bf16: 65.3 us in a
    // graph, against 74.2 at one, 68.9 at two and 67.8 at six); one step a warp has the shortest chain of
    // instructions for batches that do not fill the SMs with warps at four (one token: 4.8 us, 6.2 at four)
    const int64_t warps = (int64_t)p.total_tokens * cdiv(rp_rows(p, rp), 4 * 32 / (D / 16));
    return warps < rp.sm_count * 8 ? launch_r<D, KV, MODE, 1>(p, rp, s) : launch_r<D, KV, MODE, 4>(p, rp, s);
}

template <int D, int KV>
cudaError_t launch_kv(const ForwardParams& p, const RopeParams& rp, cudaStream_t s) {
    if (rp.rot_dim == 0) return launch_mode<D, KV, kNone>(p, rp, s);
    if (rp.interleaved) return launch_mode<D, KV, kInter>(p, rp, s);
    if (rp.rot_dim == D) return launch_mode<D, KV, kSplit>(p, rp, s);
    return 2 * rp.rot_dim <= D ? launch_mode<D, KV, kLow>(p, rp, s) : launch_mode<D, KV, kPart>(p, rp, s);
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

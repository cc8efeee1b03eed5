// K11: linear attention of requests with many new tokens, in chunks of 128 on the 5th-generation tensor
// cores.  For a chunk with c_i the sum of the log decays up to token i and S the state before it:
//   o_i = scale (e^{c_i} q_i^T S + sum_{j <= i} e^{c_i - c_j} (q_i . k_j) v_j)
//   S'  = e^{c_end} S + sum_j (e^{c_end - c_j} k_j) v_j^T
// Four products of 128 rows: Q K^T, P V and Q S for each q head, (w K)^T V once for its kv head.
//
// A work unit is a segment of a request and a kv head; its chunks run one after another, with the state
// in the registers of a warpgroup (fp32, a row of S a thread) and every product's accumulator in TMEM:
//   warps 0-3    P: a row of Q K^T a thread, times 2^(c_i - c_j) below the diagonal, to bf16 in TMEM (the
//                A operand of P V); then the row of O: scale (e^{c_i} (Q S) + P V), to bf16 in HBM.  The two
//                accumulators stay apart because e^{c_i} would otherwise be rounded into q or S a second time;
//   warps 4-7    S <- e^{c_end} S + (w K)^T V, and its bf16 copy in shared memory for the next chunk's Q S;
//   warps 8-11   w K, as three bf16 parts that together hold all 24 bits of the fp32 product (so that the
//                fp32 state keeps its own), 16 tokens at a time; also zero the rows of V behind the request's
//                last token, and note whether V holds an infinity or a NaN;
//   warp 12      issues the MMAs; warp 13 loads K, warp 14 V and Q (TMA, 128-byte swizzle); warp 15
//                sums the decays (in 64 bits: differences of far sums keep their bits).
// Roundings to bf16: P and the copy of S, each half a step of the term it scales; out.
//
// Weight 0 times an infinity or a NaN of V behind the diagonal would reach the chunk's earlier tokens, so a
// chunk with one takes P V row by row on the CUDA cores, over the keys that each row sees.
//
// States pass: only w K, V and the state update; the segments' own states and decays go to the workspace,
// and the main pass starts a segment from those before it.
//
// Every wait is bounded; a timeout sets PVA_DEVERR_TIMEOUT and the CTA winds down (outstanding copies
// and MMAs waited for, TMEM freed) without trapping.
#include <cuda.h>  // CUtensorMap and the tensor-map encoder's types (resolved through the runtime)
#include <cuda_runtime.h>

#include <atomic>
#include <cstring>
#include <mutex>

#include "device_utils.cuh"
#include "linear.h"
#include "tc_utils.cuh"

namespace pva {
namespace {

constexpr int kThreads = 512;
constexpr int kMmaWarp = 12, kLoadK = 13, kLoadQV = 14, kDecayWarp = 15;
// Registers a thread: launched with 128, the state's warpgroup rises to what the others give away
// (128 + 208 + 96 + 80 = 4 x 128, so the increase never waits for registers that are not there).
constexpr int kRegsLaunch = 128, kRegsState = 208, kRegsScale = 96, kRegsCtrl = 80;
static_assert(kRegsLaunch + kRegsState + kRegsScale + kRegsCtrl == 4 * kRegsLaunch, "register split must balance");
constexpr int kRegion = kChunk * 128;  // 128 rows of 128 bytes (64 bf16 columns), swizzled
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColP = 0, kColQS = 128, kColPV = 256, kColState = 384;  // TMEM columns
constexpr int kPart = 16;                 // tokens of a staged part of w K
constexpr int kParts = kChunk / kPart;
constexpr int kPartRegion = kPart * 128;  // 16 rows of 128 bytes

template <int D>
struct SmemMap {
    static constexpr int kHalves = D / 64;
    static constexpr int kTile = kRegion * kHalves;
    static constexpr int kStateRegion = D * 128;
    static constexpr int kSplit = kPartRegion * kHalves;  // one of the three bf16 parts of 16 tokens
    static constexpr int kQ = 0;                          // two stages
    static constexpr int kK = kQ + 2 * kTile;             // one
    static constexpr int kV = kK + kTile;                 // two
    static constexpr int kS = kV + 2 * kTile;             // bf16 copy of the state
    static constexpr int kW = kS + kStateRegion * kHalves;  // two stages of w K
    // (D 64: the 128-row A operand of the state's product reaches one region past the part it is of;
    // what lies there ends in TMEM lanes that nobody reads)
    static constexpr int kBytes = kW + 2 * 3 * kSplit + (D == 64 ? kPartRegion : 0);
};

struct Bars {
    uint64_t q_full[2], q_empty[2], k_full, k_empty, v_full[2], v_empty[2], v_ok[2];
    uint64_t p_full, p_ready, o_ready, o_free;
    uint64_t w_full[2], w_empty[2], ds_full, ds_free, s_full, s_empty;
    uint64_t dec_full[2], dec_empty[2], drain;
    alignas(16) float c[2][kChunk];  // sums of the log decays up to each token of the chunk, in log2 units
    float w[2][kChunk];  // 2^(c_end - c_j); 0 behind the last token
    float end[2];        // 2^c_end
    int32_t v_bad[2][4];
    uint32_t tmem_base;
    int32_t abort_flag;
    uint64_t wait_limit;
};

// Work waits: of a converged warp (voted, so that it leaves together or not at all), and of one thread.
__device__ __forceinline__ bool give_up(Bars* b, uint32_t* err) {
    b->abort_flag = 1;
    dev::set_error(err, kErrTimeout);
    return false;
}
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, Bars* b, uint32_t* err) {
    if (__all_sync(0xffffffffu, dev::mbar_wait(bar, parity, b->wait_limit))) return true;
    if ((threadIdx.x & 31) == 0) give_up(b, err);
    __syncwarp();
    return false;
}
__device__ __forceinline__ bool wait_one(uint64_t* bar, uint32_t parity, Bars* b, uint32_t* err) {
    return dev::mbar_wait(bar, parity, b->wait_limit) || give_up(b, err);
}

__device__ __forceinline__ void arrive_warp(uint64_t* bar) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) dev::mbar_arrive(bar);
}

// The k-th unit of this CTA, or -1: rows of gridDim.x units, every other one backwards (units come most
// tokens first).
__device__ __forceinline__ int unit_at(int k, int n_units) {
    const int g = gridDim.x, u = k * g + ((k & 1) ? g - 1 - (int)blockIdx.x : (int)blockIdx.x);
    return u < n_units ? u : -1;
}
__device__ __forceinline__ int chunks_of(int ntok) { return (ntok + kChunk - 1) / kChunk; }

// Whether a pair of bf16 holds an infinity or a NaN.
__device__ __forceinline__ uint32_t odd_pair(uint32_t w) {
    return ((w & 0x7F80u) == 0x7F80u) | ((w & 0x7F800000u) == 0x7F800000u);
}

template <int D, bool STATES>
__global__ void __launch_bounds__(kThreads, 1)
    linear_chunk_kernel(const LinParams p, const __grid_constant__ CUtensorMap q_map,
                        const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map) {
    using L = SmemMap<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ Bars bars;
    Bars* b = &bars;
    // the plan, the activations and the states may come from the kernel before this one
    dev::grid_dep_wait();
    dev::grid_dep_launch();
    PlanHeader* hdr = reinterpret_cast<PlanHeader*>(p.ws + p.lay.header);
    uint32_t* err = &hdr->error_bits;
    const int Hkv = p.num_kv_heads, G = STATES ? 0 : p.group;
    const int n_units = (STATES ? hdr->n_casc_tiles : hdr->n_pre_tiles) * Hkv;
    if ((hdr->error_bits & kErrFatal) || (int)blockIdx.x >= n_units) return;
    const LinItem* items = reinterpret_cast<const LinItem*>(p.ws + (STATES ? p.lay.pre_items : p.lay.items));
    float* seg_state = reinterpret_cast<float*>(p.ws + p.lay.seg_state);
    float* seg_decay = reinterpret_cast<float*>(p.ws + p.lay.seg_decay);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < 2; ++s) {
            dev::mbar_init(&b->q_full[s], 1);
            dev::mbar_init(&b->q_empty[s], 1);
            dev::mbar_init(&b->v_full[s], 1);
            dev::mbar_init(&b->v_empty[s], 1);
            dev::mbar_init(&b->v_ok[s], 4);
            dev::mbar_init(&b->w_full[s], 4);
            dev::mbar_init(&b->w_empty[s], 1);
            dev::mbar_init(&b->dec_full[s], 1);
            dev::mbar_init(&b->dec_empty[s], STATES ? 8 : 12);
        }
        dev::mbar_init(&b->k_full, 1);
        dev::mbar_init(&b->k_empty, 5);
        dev::mbar_init(&b->p_full, 1);
        dev::mbar_init(&b->p_ready, 4);
        dev::mbar_init(&b->o_ready, 1);
        dev::mbar_init(&b->o_free, 4);
        dev::mbar_init(&b->ds_full, 1);
        dev::mbar_init(&b->ds_free, 4);
        dev::mbar_init(&b->s_full, 4);
        dev::mbar_init(&b->s_empty, 1);
        dev::mbar_init(&b->drain, 1);
        b->abort_flag = 0;
        b->wait_limit = dev::wait_limit(hdr->wait_override);
        dev::fence_barrier_init();
    }
    if (warp == kMmaWarp) {
        tc::tmem_alloc(&b->tmem_base, kTmemCols);
        tc::tmem_relinquish();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = b->tmem_base;

    if (warp >= 12) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsCtrl));
        if (warp == kMmaWarp) {
            // ========================================================== MMA issuer (the whole warp, one lane elected)
            const uint32_t id_qk = tc::idesc_bf16_f32(128, 128, 0, 0), id_v = tc::idesc_bf16_f32(128, D, 0, 1);
            const uint32_t id_kv = tc::idesc_bf16_f32(128, D, 1, 1);
            constexpr uint32_t kDescHi = tc::smem_desc_hi(1024, tc::kSwizzle128B);
            const uint32_t q_lo = tc::smem_desc_lo(dev::smem_u32(smem + L::kQ), 16);
            const uint32_t k_lo = tc::smem_desc_lo(dev::smem_u32(smem + L::kK), 16);
            const uint32_t v_lo = tc::smem_desc_lo(dev::smem_u32(smem + L::kV), kRegion);
            const uint32_t s_lo = tc::smem_desc_lo(dev::smem_u32(smem + L::kS), L::kStateRegion);
            const uint32_t w_lo = tc::smem_desc_lo(dev::smem_u32(smem + L::kW), kPartRegion);
            auto wait = [&](uint64_t* bar, uint32_t parity) { return wait_warp(bar, parity, b, err); };
            uint32_t n = 0, h = 0;  // chunks and q heads so far
            // the state's product of chunk n: 16 tokens at a time, three parts of w K each
            auto state_product = [&]() -> bool {
                const int st = n & 1;
                if (!wait(&b->v_ok[st], (n >> 1) & 1) || (n > 0 && !wait(&b->ds_free, (n - 1) & 1))) return false;
                for (int s = 0; s < kParts; ++s) {
                    const uint32_t i = n * kParts + s;
                    if (!wait(&b->w_full[i & 1], (i >> 1) & 1)) return false;
                    tc::fence_after_sync();
                    const uint32_t b0 = v_lo + ((st * L::kTile + s * kPartRegion) >> 4);
#pragma unroll
                    for (int x = 0; x < 3; ++x)
                        tc::mma_ss_warp(tmem + kColState, w_lo + (((i & 1) * 3 + x) * L::kSplit >> 4), b0, kDescHi, id_kv,
                                        s > 0 || x > 0 ? 1u : 0u);
                    tc::mma_commit_warp(&b->w_empty[i & 1]);
                }
                tc::mma_commit_warp(&b->ds_full);
                return true;
            };
            bool ok = true;
            for (int k = 0, u; ok && (u = unit_at(k, n_units)) >= 0; ++k) {
                const int nch = chunks_of(items[u / Hkv].ntok);
                for (int c = 0; ok && c < nch; ++c, ++n) {
                    const int st = n & 1;
                    if constexpr (STATES) {
                        ok = state_product();
                        tc::mma_commit_warp(&b->k_empty);
                        tc::mma_commit_warp(&b->v_empty[st]);
                        continue;
                    }
                    if (!(ok = wait(&b->k_full, n & 1))) break;
                    for (int g = 0; g < G; ++g, ++h) {
                        const int qs = h & 1;
                        if (!(ok = wait(&b->q_full[qs], (h >> 1) & 1))) break;
                        tc::fence_after_sync();
                        const uint32_t q0 = q_lo + (qs * L::kTile >> 4);
                        // Q K^T (the P of the head before was read by its P V, issued before this)
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk) {
                            const uint32_t off = (uint32_t)((kk >> 2) * kRegion + (kk & 3) * 32) >> 4;
                            tc::mma_ss_warp(tmem + kColP, q0 + off, k_lo + off, kDescHi, id_qk, kk > 0 ? 1u : 0u);
                        }
                        tc::mma_commit_warp(&b->p_full);
                        if (g == G - 1) tc::mma_commit_warp(&b->k_empty);
                        if (g == 0 && !(ok = state_product() && wait(&b->s_full, n & 1))) break;
                        if (h > 0 && !(ok = wait(&b->o_free, (h - 1) & 1))) break;
                        tc::fence_after_sync();
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk) {
                            const uint32_t off = (uint32_t)((kk >> 2) * kRegion + (kk & 3) * 32) >> 4;
                            tc::mma_ss_warp(tmem + kColQS, q0 + off, s_lo + (kk * 2048 >> 4), kDescHi, id_v, kk > 0 ? 1u : 0u);
                        }
                        if (!(ok = wait(&b->p_ready, h & 1))) break;
                        tc::fence_after_sync();
                        const bool bad = (b->v_bad[st][0] | b->v_bad[st][1] | b->v_bad[st][2] | b->v_bad[st][3]) != 0;
                        if (!bad) {
                            const uint32_t b0 = v_lo + (st * L::kTile >> 4);
#pragma unroll
                            for (int kk = 0; kk < kChunk / 16; ++kk)
                                tc::mma_ts_warp(tmem + kColPV, tmem + kColP + kk * 8, b0 + (kk * 2048 >> 4), kDescHi, id_v,
                                                kk > 0 ? 1u : 0u);
                        }
                        tc::mma_commit_warp(&b->o_ready);
                        tc::mma_commit_warp(&b->q_empty[qs]);
                        if (g == G - 1) {
                            tc::mma_commit_warp(&b->v_empty[st]);
                            tc::mma_commit_warp(&b->s_empty);
                        }
                    }
                }
            }
            // every MMA issued must complete before TMEM is released
            tc::mma_commit_warp(&b->drain);
            (void)dev::mbar_wait(&b->drain, 0);
            __syncwarp();
        } else if (warp == kLoadK && lane == 0) {
            uint32_t n = 0;
            bool ok = true;
            for (int k = 0, u; ok && (u = unit_at(k, n_units)) >= 0; ++k) {
                const LinItem it = items[u / Hkv];
                const int kvh = u % Hkv;
                for (int c = 0; c < chunks_of(it.ntok); ++c, ++n) {
                    if (!(ok = wait_one(&b->k_empty, (n & 1) ^ 1, b, err)) || b->abort_flag) {
                        ok = false;
                        break;
                    }
                    dev::mbar_arrive_expect_tx(&b->k_full, L::kTile);
#pragma unroll
                    for (int x = 0; x < L::kHalves; ++x)
                        tc::tma_load_3d(smem + L::kK + x * kRegion, &k_map, 64 * x, kvh, it.tok0 + c * kChunk, &b->k_full);
                }
            }
            if (n > 0) (void)dev::mbar_wait(&b->k_full, (n - 1) & 1);  // its copies land before the CTA leaves
        } else if (warp == kLoadQV && lane == 0) {
            uint32_t n = 0, h = 0;
            bool ok = true;
            for (int k = 0, u; ok && (u = unit_at(k, n_units)) >= 0; ++k) {
                const LinItem it = items[u / Hkv];
                const int kvh = u % Hkv;
                for (int c = 0; ok && c < chunks_of(it.ntok); ++c) {
                    if (!(ok = wait_one(&b->v_empty[n & 1], ((n >> 1) & 1) ^ 1, b, err)) || b->abort_flag) {
                        ok = false;
                        break;
                    }
                    dev::mbar_arrive_expect_tx(&b->v_full[n & 1], L::kTile);
#pragma unroll
                    for (int x = 0; x < L::kHalves; ++x)
                        tc::tma_load_3d(smem + L::kV + (n & 1) * L::kTile + x * kRegion, &v_map, 64 * x, kvh,
                                        it.tok0 + c * kChunk, &b->v_full[n & 1]);
                    ++n;
                    for (int g = 0; g < G; ++g, ++h) {
                        if (!(ok = wait_one(&b->q_empty[h & 1], ((h >> 1) & 1) ^ 1, b, err)) || b->abort_flag) {
                            ok = false;
                            break;
                        }
                        dev::mbar_arrive_expect_tx(&b->q_full[h & 1], L::kTile);
#pragma unroll
                        for (int x = 0; x < L::kHalves; ++x)
                            tc::tma_load_3d(smem + L::kQ + (h & 1) * L::kTile + x * kRegion, &q_map, 64 * x, kvh * G + g,
                                            it.tok0 + c * kChunk, &b->q_full[h & 1]);
                    }
                }
            }
            for (uint32_t s = 0; s < 2; ++s) {  // the last copies into either stage
                if (n > s) (void)dev::mbar_wait(&b->v_full[(n - 1 - s) & 1], ((n - 1 - s) >> 1) & 1);
                if (h > s) (void)dev::mbar_wait(&b->q_full[(h - 1 - s) & 1], ((h - 1 - s) >> 1) & 1);
            }
        } else if (warp == kDecayWarp) {
            // ========================================================== sums of the log decays, four tokens a lane
            uint32_t n = 0;
            bool ok = true;
            for (int k = 0, u; ok && (u = unit_at(k, n_units)) >= 0; ++k) {
                const LinItem it = items[u / Hkv];
                const int kvh = u % Hkv, nch = chunks_of(it.ntok);
                double total = 0.0;  // of the unit
                for (int c = 0; ok && c < nch; ++c, ++n) {
                    double sum[4], x = 0.0;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int t = c * kChunk + 4 * lane + i;
                        if (t < it.ntok) {
                            const float g = p.log_decay[(p.ld_decay ? (int64_t)(it.tok0 + t) * p.ld_decay : 0) + kvh];
                            x += (double)(g < kLeastLogDecay ? kLeastLogDecay : g) * 1.4426950408889634074;
                        }
                        sum[i] = x;
                    }
#pragma unroll
                    for (int d = 1; d < 32; d *= 2) {
                        const double y = __shfl_up_sync(0xffffffffu, x, d);
                        if (lane >= d) x += y;
                    }
                    const double before = x - sum[3], end = __shfl_sync(0xffffffffu, x, 31);
                    const int st = n & 1;
                    if (!(ok = wait_warp(&b->dec_empty[st], ((n >> 1) & 1) ^ 1, b, err))) break;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const double ci = before + sum[i];
                        b->c[st][4 * lane + i] = (float)ci;
                        b->w[st][4 * lane + i] = c * kChunk + 4 * lane + i < it.ntok ? exp2f((float)(end - ci)) : 0.f;
                    }
                    if (lane == 0) b->end[st] = exp2f((float)end);
                    arrive_warp(&b->dec_full[st]);
                    total += end;
                }
                if (STATES && ok && lane == 0) seg_decay[(int64_t)(it.base + it.seg + 1) * Hkv + kvh] = exp2f((float)total);
            }
        }
    } else if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsScale));
        // ============================================================== w K in three bf16 parts; a look at V
        const int tid = threadIdx.x - 256, wq = warp - 8;
        const int r = tid >> 3, cc = tid & 7;  // token of a part, 16-byte chunk of its row
        uint32_t n = 0;
        bool ok = true;
        for (int k = 0, u; ok && (u = unit_at(k, n_units)) >= 0; ++k) {
            const int ntok = items[u / Hkv].ntok;
            for (int c = 0; ok && c < chunks_of(ntok); ++c, ++n) {
                const int st = n & 1, nval = min(kChunk, ntok - c * kChunk);
                uint8_t* V = smem + L::kV + st * L::kTile;
                if (!(ok = wait_warp(&b->v_full[st], (n >> 1) & 1, b, err))) break;
                {   // row tid of V
                    uint32_t odd = 0;
#pragma unroll
                    for (int x = 0; x < D / 8; ++x) {
                        uint4* at = reinterpret_cast<uint4*>(V + (x >> 3) * kRegion + tid * 128 + (((x ^ tid) & 7) << 4));
                        if (tid < nval) {
                            const uint4 y = *at;
                            odd |= odd_pair(y.x) | odd_pair(y.y) | odd_pair(y.z) | odd_pair(y.w);
                        } else {
                            *at = make_uint4(0, 0, 0, 0);
                        }
                    }
                    const int any = __any_sync(0xffffffffu, odd != 0);
                    if (lane == 0) b->v_bad[st][wq] = any;
                    if (nval < kChunk) tc::fence_proxy_async_smem();
                    arrive_warp(&b->v_ok[st]);
                }
                if (!(ok = wait_warp(&b->k_full, n & 1, b, err) && wait_warp(&b->dec_full[st], (n >> 1) & 1, b, err))) break;
                const uint8_t* K = smem + L::kK;
                for (int s = 0; s < kParts; ++s) {
                    const uint32_t i = n * kParts + s;
                    const int row = s * kPart + r;
                    const float w = b->w[st][row];
                    uint4 part[L::kHalves][3];
#pragma unroll
                    for (int x = 0; x < L::kHalves; ++x) {
                        const uint4 y = *reinterpret_cast<const uint4*>(K + x * kRegion + row * 128 + (((cc ^ row) & 7) << 4));
                        const uint32_t e[4] = {y.x, y.y, y.z, y.w};
                        uint32_t hi[4], mid[4], lo[4];
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            float f[2] = {__uint_as_float(e[q] << 16) * w, __uint_as_float(e[q] & 0xFFFF0000u) * w};
                            float m[2], l[2];
#pragma unroll
                            for (int z = 0; z < 2; ++z) {
                                if (row >= nval) f[z] = 0.f;  // (whatever lies there times 0)
                                // the upper 8 bits, the next 8 and the rest: each difference is exact; an
                                // infinity keeps nothing behind its first part
                                const float top = __uint_as_float(__float_as_uint(f[z]) & 0xFFFF0000u);
                                m[z] = fabsf(f[z]) == INFINITY ? 0.f : f[z] - top;
                                l[z] = m[z] - __uint_as_float(__float_as_uint(m[z]) & 0xFFFF0000u);
                            }
                            hi[q] = dev::prmt(__float_as_uint(f[0]), __float_as_uint(f[1]), 0x7632);
                            mid[q] = dev::prmt(__float_as_uint(m[0]), __float_as_uint(m[1]), 0x7632);
                            lo[q] = dev::pack_bf16x2(l[0], l[1]);
                        }
                        part[x][0] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                        part[x][1] = make_uint4(mid[0], mid[1], mid[2], mid[3]);
                        part[x][2] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                    }
                    if (!(ok = wait_warp(&b->w_empty[i & 1], ((i >> 1) & 1) ^ 1, b, err))) break;
                    uint8_t* W = smem + L::kW + (i & 1) * 3 * L::kSplit;
#pragma unroll
                    for (int x = 0; x < L::kHalves; ++x)
#pragma unroll
                        for (int q = 0; q < 3; ++q)
                            *reinterpret_cast<uint4*>(W + q * L::kSplit + x * kPartRegion + r * 128 + (((cc ^ r) & 7) << 4)) =
                                part[x][q];
                    tc::fence_proxy_async_smem();
                    arrive_warp(&b->w_full[i & 1]);
                }
                if (!ok) break;
                arrive_warp(&b->k_empty);
                arrive_warp(&b->dec_empty[st]);
            }
        }
    } else if (warp >= 4) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsState));
        // ============================================================== the state, a row a thread
        const int row = threadIdx.x - 128;
        const bool live = row < D;
        const uint32_t t_ds = tmem + kColState + ((uint32_t)((warp & 3) * 32) << 16);
        uint32_t n = 0;
        bool ok = true;
        const int64_t per_head = (int64_t)D * D;
        for (int k = 0, u; ok && (u = unit_at(k, n_units)) >= 0; ++k) {
            const LinItem it = items[u / Hkv];
            const int kvh = u % Hkv, nch = chunks_of(it.ntok);
            float S[D / 32][32];
#pragma unroll
            for (int x = 0; x < D; ++x) S[x >> 5][x & 31] = 0.f;
            auto segment_state = [&](int i) { return seg_state + ((int64_t)(it.base + i) * Hkv + kvh) * per_head + row * D; };
            auto add = [&](const float* src, float f) {  // S <- f S + src
#pragma unroll
                for (int x = 0; x < D; x += 4) {
                    const float4 y = *reinterpret_cast<const float4*>(src + x);
                    S[x >> 5][x & 31] = fmaf(f, S[x >> 5][x & 31], y.x);
                    S[x >> 5][(x & 31) + 1] = fmaf(f, S[x >> 5][(x & 31) + 1], y.y);
                    S[x >> 5][(x & 31) + 2] = fmaf(f, S[x >> 5][(x & 31) + 2], y.z);
                    S[x >> 5][(x & 31) + 3] = fmaf(f, S[x >> 5][(x & 31) + 3], y.w);
                }
            };
            auto put = [&](float* dst) {
#pragma unroll
                for (int x = 0; x < D; x += 4)
                    *reinterpret_cast<float4*>(dst + x) = make_float4(S[x >> 5][x & 31], S[x >> 5][(x & 31) + 1],
                                                                      S[x >> 5][(x & 31) + 2], S[x >> 5][(x & 31) + 3]);
            };
            // The start.  Of a request in segments the states pass leaves a copy of the first one's start (in
            // the main pass the last segment may write the slot before the first has read it), and the end of
            // the first segment from there, of the others from zero.
            if (live) {
                if (it.seg == 0) {
                    if (it.in >= 0)
                        add(STATES || it.nseg == 1 ? p.states + ((int64_t)it.in * Hkv + kvh) * per_head + row * D
                                                   : segment_state(0), 0.f);
                    if (STATES) put(segment_state(0));
                } else if (!STATES) {
                    add(segment_state(1), 0.f);
#pragma unroll 1
                    for (int i = 2; i <= it.seg; ++i) add(segment_state(i), seg_decay[(int64_t)(it.base + i) * Hkv + kvh]);
                }
            }
            for (int c = 0; ok && c < nch; ++c, ++n) {
                const int st = n & 1;
                if constexpr (!STATES) {
                    if (n > 0 && !(ok = wait_warp(&b->s_empty, (n - 1) & 1, b, err))) break;
                    if (live) {
#pragma unroll
                        for (int x = 0; x < D; x += 8) {
                            const float* y = &S[x >> 5][x & 31];
                            const uint32_t at = dev::smem_u32(smem + L::kS) + (x >> 6) * L::kStateRegion + row * 128 +
                                                ((((x >> 3) ^ row) & 7) << 4);
                            dev::st_shared_v4(at, dev::pack_bf16x2(y[0], y[1]), dev::pack_bf16x2(y[2], y[3]),
                                              dev::pack_bf16x2(y[4], y[5]), dev::pack_bf16x2(y[6], y[7]));
                        }
                    }
                    tc::fence_proxy_async_smem();
                    arrive_warp(&b->s_full);
                }
                if (!(ok = wait_warp(&b->dec_full[st], (n >> 1) & 1, b, err))) break;
                const float end = b->end[st];
                arrive_warp(&b->dec_empty[st]);
                if (!(ok = wait_warp(&b->ds_full, n & 1, b, err))) break;
                tc::fence_after_sync();
#pragma unroll
                for (int x = 0; x < D / 32; ++x) {
                    float d[32];
                    tc::tmem_ld32_async(t_ds + 32 * x, d);
                    tc::tmem_wait_ld_regs(d);
#pragma unroll
                    for (int i = 0; i < 32; ++i) S[x][i] = fmaf(end, S[x][i], d[i]);
                }
                tc::fence_before_sync();
                arrive_warp(&b->ds_free);
            }
            if (ok && live) {
                if (STATES) put(segment_state(it.seg + 1));
                else if (it.out >= 0 && it.seg == it.nseg - 1) put(p.states + ((int64_t)it.out * Hkv + kvh) * per_head + row * D);
            }
        }
    } else if constexpr (!STATES) {
        // ============================================================== P and O, a row a thread
        const int row = threadIdx.x;
        const uint32_t lane_base = (uint32_t)(warp * 32) << 16;
        const uint32_t t_p = tmem + kColP + lane_base, t_qs = tmem + kColQS + lane_base, t_pv = tmem + kColPV + lane_base;
        uint32_t n = 0, h = 0;
        bool ok = true;
        for (int k = 0, u; ok && (u = unit_at(k, n_units)) >= 0; ++k) {
            const LinItem it = items[u / Hkv];
            const int kvh = u % Hkv;
            for (int c = 0; ok && c < chunks_of(it.ntok); ++c, ++n) {
                const int st = n & 1, nval = min(kChunk, it.ntok - c * kChunk);
                if (!(ok = wait_warp(&b->dec_full[st], (n >> 1) & 1, b, err) && wait_warp(&b->v_ok[st], (n >> 1) & 1, b, err)))
                    break;
                const bool bad = (b->v_bad[st][0] | b->v_bad[st][1] | b->v_bad[st][2] | b->v_bad[st][3]) != 0;
                const float ci = b->c[st][row], ei = dev::fast_exp2(ci) * p.scale;
                for (int g = 0; g < G; ++g, ++h) {
                    if (!(ok = wait_warp(&b->p_full, h & 1, b, err))) break;
                    tc::fence_after_sync();
                    // 32 keys at a time; those past the warp's own rows have no weight.  (The packed weights of
                    // block x lie in columns 16 x .. of the scores, which are read by then.)
#pragma unroll
                    for (int x = 0; x < kChunk / 32; ++x) {
                        uint32_t pk[16];
                        if (x <= warp) {
                            float s[32];
                            tc::tmem_ld32_async(t_p + 32 * x, s);
                            tc::tmem_wait_ld_regs(s);
#pragma unroll
                            for (int i = 0; i < 32; i += 4) {
                                const float4 cj = *reinterpret_cast<const float4*>(&b->c[st][32 * x + i]);
                                s[i] *= dev::fast_exp2(ci - cj.x);
                                s[i + 1] *= dev::fast_exp2(ci - cj.y);
                                s[i + 2] *= dev::fast_exp2(ci - cj.z);
                                s[i + 3] *= dev::fast_exp2(ci - cj.w);
                            }
                            if (x == warp) {  // the diagonal (whatever the hidden ones hold)
#pragma unroll
                                for (int i = 1; i < 32; ++i) s[i] = i <= lane ? s[i] : 0.f;
                            }
#pragma unroll
                            for (int i = 0; i < 16; ++i) pk[i] = dev::pack_bf16x2(s[2 * i], s[2 * i + 1]);
                        } else {
#pragma unroll
                            for (int i = 0; i < 16; ++i) pk[i] = 0;
                        }
                        tc::tmem_st16u(t_p + 16 * x, pk);
                    }
                    tc::tmem_wait_st();
                    if (bad) {  // P V over the keys that the row sees, from the same bf16 weights
                        const uint8_t* V = smem + L::kV + st * L::kTile;
#pragma unroll 1
                        for (int x = 0; x < D / 32; ++x) {
                            float o[32];
#pragma unroll
                            for (int i = 0; i < 32; ++i) o[i] = 0.f;
#pragma unroll 1
                            for (int j0 = 0; j0 < kChunk; j0 += 64) {
                                if (j0 > 32 * warp + 31) break;
                                float pw[32];  // 64 weights
                                tc::tmem_ld32_async(t_p + j0 / 2, pw);
                                tc::tmem_wait_ld_regs(pw);
#pragma unroll
                                for (int j = 0; j < 64; ++j) {
                                    const uint32_t w2 = __float_as_uint(pw[j >> 1]);
                                    const float wj = __uint_as_float((j & 1) ? w2 & 0xFFFF0000u : w2 << 16);
                                    const int vr = j0 + j;
                                    if (vr > row) continue;
#pragma unroll
                                    for (int e = 0; e < 4; ++e) {
                                        const uint4 y = *reinterpret_cast<const uint4*>(
                                            V + (x >> 1) * kRegion + vr * 128 + ((((x & 1) * 4 + e) ^ (vr & 7)) << 4));
                                        const uint32_t vw[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                                        for (int i = 0; i < 4; ++i) {
                                            o[8 * e + 2 * i] = fmaf(wj, __uint_as_float(vw[i] << 16), o[8 * e + 2 * i]);
                                            o[8 * e + 2 * i + 1] =
                                                fmaf(wj, __uint_as_float(vw[i] & 0xFFFF0000u), o[8 * e + 2 * i + 1]);
                                        }
                                    }
                                }
                            }
                            __syncwarp();
                            tc::tmem_st32(t_pv + 32 * x, o);
                        }
                        tc::tmem_wait_st();
                    }
                    tc::fence_before_sync();
                    arrive_warp(&b->p_ready);
                    // O
                    if (!(ok = wait_warp(&b->o_ready, h & 1, b, err))) break;
                    tc::fence_after_sync();
                    uint16_t* dst = p.out + ((int64_t)(it.tok0 + c * kChunk + row) * p.num_qo_heads + kvh * G + g) * D;
#pragma unroll
                    for (int x = 0; x < D / 32; ++x) {
                        float a[32], o[32];
                        tc::tmem_ld32_async(t_qs + 32 * x, a);
                        tc::tmem_ld32_async(t_pv + 32 * x, o);
                        tc::tmem_wait_ld_regs(a);
                        tc::tmem_wait_ld_regs(o);
                        if (x == D / 32 - 1) {
                            tc::fence_before_sync();
                            arrive_warp(&b->o_free);
                        }
                        if (row < nval) {
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                uint32_t w[4];
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    const int z = 8 * e + 2 * i;
                                    w[i] = dev::pack_bf16x2(fmaf(ei, a[z], p.scale * o[z]), fmaf(ei, a[z + 1], p.scale * o[z + 1]));
                                }
                                *reinterpret_cast<uint4*>(dst + 32 * x + 8 * e) = make_uint4(w[0], w[1], w[2], w[3]);
                            }
                        }
                        __syncwarp();
                    }
                }
                if (ok) arrive_warp(&b->dec_empty[st]);
            }
        }
    }
    __syncwarp();
    tc::fence_before_sync();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, kTmemCols);
    }
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn tensor_map_encoder() {
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q{};
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(f);
    });
    return fn;
}

// [T, heads, D] with ld elements between tokens; a box is 64 columns of one head for 128 tokens.
bool encode(CUtensorMap* m, const uint16_t* x, int64_t tokens, int heads, int D, int64_t ld) {
    const EncodeTiledFn enc = tensor_map_encoder();
    if (enc == nullptr) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)tokens};
    const cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)ld * 2};
    const cuuint32_t box[3] = {64, 1, (cuuint32_t)kChunk};
    const cuuint32_t elem_strides[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint16_t*>(x), dims, strides, box, elem_strides,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool STATES>
cudaError_t launch(const LinParams& p, int ctas, cudaStream_t s) {
    auto kernel = linear_chunk_kernel<D, STATES>;
    const size_t smem = SmemMap<D>::kBytes + 1024;
    static_assert(SmemMap<D>::kBytes + 1024 + sizeof(Bars) <= 227 * 1024, "shared memory per block");
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    // The register split assumes that the launch allocates exactly kRegsLaunch registers a thread: with
    // fewer, the state warpgroup's increase could not be satisfied.  Refuse to launch rather than risk that.
    static std::atomic<int> launch_regs{-1};
    if (launch_regs.load(std::memory_order_relaxed) < 0) {
        cudaFuncAttributes attr{};
        e = cudaFuncGetAttributes(&attr, kernel);
        if (e != cudaSuccess) return e;
        launch_regs.store(attr.numRegs, std::memory_order_relaxed);
    }
    if (launch_regs.load(std::memory_order_relaxed) != kRegsLaunch) return cudaErrorInvalidConfiguration;
    CUtensorMap q, k, v;
    if (!encode(&q, p.q, p.total_tokens, p.num_qo_heads, D, p.ld_q) ||
        !encode(&k, p.k, p.total_tokens, p.num_kv_heads, D, p.ld_k) ||
        !encode(&v, p.v, p.total_tokens, p.num_kv_heads, D, p.ld_v))
        return cudaErrorInvalidValue;
    return launch_programmatic(kernel, dim3((unsigned)ctas), (unsigned)kThreads, smem, s, p, q, k, v);
}

}  // namespace

cudaError_t launch_linear_chunks(const LinParams& p, int head_dim, bool states, int ctas, cudaStream_t s) {
    if (ctas <= 0) return cudaSuccess;
    if (head_dim == 128) return states ? launch<128, true>(p, ctas, s) : launch<128, false>(p, ctas, s);
    if (head_dim == 64) return states ? launch<64, true>(p, ctas, s) : launch<64, false>(p, ctas, s);
    return cudaErrorInvalidValue;
}

}  // namespace pva

// K11: linear attention of requests with many new tokens, in chunks of 128 on the 5th-generation tensor
// cores.  For a chunk with c_i the sum of the log decays up to token i and S the state before it:
//   o_i = scale e^{c_i + r} (q_i^T (e^{-r} S) + sum_{j <= i} (q_i . k_j) e^{-c_j - r} v_j)      for any r
//   S'  = e^{c_end} S + sum_j (e^{c_end - c_j} k_j) v_j^T
// Four products of 128 rows: Q K^T, Q S and P V for each q head, (w K)^T V once for its kv head.
//
// A work unit is a segment of a request, a kv head and some of its q heads; its chunks run one after
// another, with the state in the registers of a warpgroup (fp32, a row of S a thread) and every product's
// accumulator in TMEM (two of Q K^T, so that the next head's runs while this one's weights are made):
//   warps 0-3    P: a row of Q K^T a thread, times e^{-c_j - r} up to the diagonal, to bf16 in TMEM (the A
//                operand of P V, which adds to Q S);
//   warps 4-7    S <- e^{c_end} S + (w K)^T V, and e^{-r} S as bf16 in shared memory for the next chunk's Q S;
//   warps 8-11   w K, as three bf16 parts that together hold all 24 bits of the fp32 product (so that the
//                fp32 state keeps its own), 16 tokens at a time; also zero the rows of V behind the request's
//                last token, and note whether V holds an infinity or a NaN;
//   warps 12-15  the rows of O, times scale e^{c_i + r}, to bf16 in HBM (in the states pass w K too);
//   warp 16      issues the MMAs of the outputs, warp 17 the state's; warp 18 loads Q, K and V (TMA, 128-byte
//                swizzle); warp 19 sums the decays (in 64 bits; the state's weights are formed of
//                differences of those, the outputs' of the sums rounded to fp32).
// Roundings to bf16: P and the copy of S, each half a step of the term it scales; out.  (8 prompts of normal values: out
// is 2.35e-3 of its norm off, which is what the plain form makes with those two roundings, and 1.66e-3 with the last
// alone.)  The sums' roundings move an output's weights by 2^-23 ln 2 of the chunk's sum (log2): 2e-5 at 2^8, 1.7e-3 at the
// 20 000 that 128 tokens can come to.
//
// r (a whole number of powers of two) is 0, or halfway in a chunk whose sums go further than 2^60, so that weights stay
// within 2^+-60: up to sums of 2^120 (0.65 a token).  In chunks beyond that ("deep") row i's weights are
// e^{c_i - r_i - c_j} with r_i = c_i held to +-40 (log2), its part of Q S is scaled by e^{c_i - r_i} in TMEM before
// P V adds to it, and O takes e^{r_i}.  A chunk with a token that drops the state (a log decay of -inf) is deep too: its
// sums start anew there, and to the tokens from it on the keys before it and S are hidden, whatever they hold.  (With an r of
// 0 alone a prompt of 16 k tokens, 8 kv heads, takes 117 us for 112.)
// Weight 0 times an infinity or a NaN of V behind the diagonal would reach the chunk's
// earlier tokens, so a chunk with one takes P V row by row on the CUDA cores, over the keys that each row sees.
//
// States pass: only w K, V and the state update; the segments' own states and decays go to the workspace, where
// the scan (K12) makes of them the states that the main pass starts its segments from.
//
// Measured: 8 prompts of 0.5-3.7 k tokens, 32 heads of 128, 168 us (561 MB, 3.3 TB/s; tensor pipe 33 % of active
// cycles), 16 k tokens of 32/8 heads 112 us with the states pass (26) and the scan (8).  Bound: the roles' hand-offs, some
// 200 cycles each, a dozen in a row a chunk, and the fetching of instructions.  (O in warps of their own: when they came in,
// the prompts went from 170 us, with the warps of P writing it, to 165, the 16 k tokens from 122 to 110.)
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

constexpr int kThreads = 640;
constexpr int kMmaWarp = 16, kStateMmaWarp = 17, kLoadWarp = 18, kDecayWarp = 19;
// Registers a thread: launched with 96, the state's warpgroup rises to what the others give away
// (72 + 184 + 64 + 80 + 80 = 5 x 96, so the increase never waits for registers that are not there).
constexpr int kRegsLaunch = 96, kRegsP = 72, kRegsState = 184, kRegsScale = 64, kRegsO = 80, kRegsCtrl = 80;
static_assert(kRegsP + kRegsState + kRegsScale + kRegsO + kRegsCtrl == 5 * kRegsLaunch && kRegsScale <= kRegsO,
              "register split must balance");
constexpr int kRegion = kChunk * 128;  // 128 rows of 128 bytes (64 bf16 columns), swizzled
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColP = 0, kColO = 256, kColState = 384;  // TMEM columns (two buffers of Q K^T)
constexpr float kReach = 60.f;            // largest power (log2) that enters the weights of a chunk with one r
constexpr float kDeep = 40.f;             // the same of one with an r for each row
constexpr int kDrops = 2;                 // in the place of "deep"
constexpr int kPart = 16;                 // tokens of a staged part of w K
constexpr int kParts = kChunk / kPart;
constexpr int kPartRegion = kPart * 128;  // 16 rows of 128 bytes

template <int D, bool STATES>
struct SmemMap {
    static constexpr int kHalves = D / 64;
    static constexpr int kTile = kRegion * kHalves;
    static constexpr int kStateRegion = D * 128;
    static constexpr int kSplit = kPartRegion * kHalves;  // one of the three bf16 parts of 16 tokens
    // K lies in halves of 64 tokens, each let go by itself: with one tile the load of the next first half (some
    // 3000 cycles) runs behind the weighting of this second one
    static constexpr int kHalvesK = STATES || D == 64 ? 4 : 2;
    // staged parts of w K, as many as there is room for: a part takes two warps some 2000 cycles, its MMAs 200
    static constexpr int kStagesW = D == 64 ? 8 : STATES ? 4 : 2;
    static constexpr int kQ = 0;                                    // two stages
    static constexpr int kK = kQ + (STATES ? 0 : 2 * kTile);
    static constexpr int kV = kK + kHalvesK / 2 * kTile;            // two stages
    static constexpr int kS = kV + 2 * kTile;                       // bf16 copy of the state (and its way to memory)
    static constexpr int kW = kS + kStateRegion * kHalves;
    // (D 64: the 128-row A operand of the state's product reaches one region past the part it is of;
    // what lies there ends in TMEM lanes that nobody reads)
    static constexpr int kBytes = kW + kStagesW * 3 * kSplit + (D == 64 ? kPartRegion : 0);
};

struct Bars {
    uint64_t q_full[2], q_empty[2], k_full[4], k_empty[4], v_full[2], v_empty[2], v_ok[2];
    uint64_t p_full[2], p_ready[2], qs_full[2], o_ready, o_free;
    uint64_t w_full[kParts], w_empty[kParts], ds_full, ds_free, s_full, s_empty;
    uint64_t dec_full[2], dec_empty[2], drain[2];
    alignas(16) float c[2][kChunk];  // sums of the log decays up to each token of the chunk, in log2 units
    alignas(16) float f[2][kChunk];  // 2^(-c_j - r)
    float w[2][kChunk];              // 2^(c_end - c_j); -0 (the key counts as 0) behind the last token and of what is dropped
    float end[2], r[2], down[2];     // 2^c_end (-1: the state is dropped); r (log2); 2^-r
    int32_t deep[2];                 // no r will do; kDrops: a token drops the state
    int32_t last[2];                 // (kDrops) the last token that does
    alignas(4) int8_t first[2][kChunk];  // (kDrops) the same up to each token, -1: none; what lies before it is hidden from it
    alignas(16) int32_t v_bad[2][8];
    uint32_t tmem_base;
    int32_t abort_flag;
    uint64_t wait_limit;
};

// The kernel is 20 warps in half a dozen roles, each going through its own code once a chunk: much of what keeps it
// from running is the fetching of instructions (at 126 KB of code a weighted part of 16 keys took 3000 cycles,
// at 97 KB 2100, alone 600).  So the code is kept short: loops rolled where they can be, one site for what a role does twice,
// no inlined handling of waits that ran out.

// Waits for a phase, at most limit ns (0: a look), asleep for up to kNap ns at a time (without that the warps that wait
// look some sixty times a chunk each, and take more than half of all issue slots).
constexpr uint32_t kNap = 20000;
__device__ __forceinline__ bool phase_done(uint64_t* bar, uint32_t parity, uint64_t limit) {
    if (dev::mbar_test_wait(bar, parity)) return true;
    if (limit == 0) return false;
    const uint64_t t0 = dev::globaltimer();
    do {
        uint32_t done;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2, %3;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(done)
            : "r"(dev::smem_u32(bar)), "r"(parity), "r"(kNap)
            : "memory");
        if (done) return true;
    } while (dev::globaltimer() - t0 <= limit);
    return false;
}

// Work waits: of a converged warp (voted, so that it leaves together or not at all), and of one thread.  A role
// whose wait ran out leaves its loops and then calls give_up.
struct Waits {
    uint64_t limit;
    __device__ __forceinline__ bool warp(uint64_t* bar, uint32_t parity) const {
        return __all_sync(0xffffffffu, phase_done(bar, parity, limit));
    }
    __device__ __forceinline__ bool one(uint64_t* bar, uint32_t parity) const { return phase_done(bar, parity, limit); }
};

// Whether a phase has completed, without waiting: for a converged warp.
__device__ __forceinline__ bool seen_warp(uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, dev::mbar_test_wait(bar, parity));
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

// A unit's segment, kv head and q heads g0 .. g1 - 1 of that head's group.
struct Unit {
    LinItem it;
    int kvh, g0, g1;
};
template <bool STATES>
__device__ __forceinline__ Unit unit_of(const LinItem* items, int u, const LinParams& p, unsigned parts) {
    const unsigned head = (unsigned)u / parts, part = (unsigned)u - head * parts;
    const unsigned item = head / (unsigned)p.num_kv_heads;
    Unit x;
    x.it = items[item];
    x.kvh = (int)(head - item * p.num_kv_heads);
    x.g0 = STATES ? 0 : (int)((unsigned)p.group * part / parts);
    x.g1 = STATES ? 0 : (int)((unsigned)p.group * (part + 1) / parts);
    return x;
}
__device__ __forceinline__ bool v_is_bad(const Bars* b, int st) {
    const int4 x = *reinterpret_cast<const int4*>(&b->v_bad[st][0]), y = *reinterpret_cast<const int4*>(&b->v_bad[st][4]);
    return (x.x | x.y | x.z | x.w | y.x | y.y | y.z | y.w) != 0;
}
__device__ __forceinline__ int chunks_of(int ntok) { return (ntok + kChunk - 1) / kChunk; }

// acc + 0 x, for pairs of bf16: stays 0 unless x is an infinity or a NaN.
__device__ __forceinline__ uint32_t note_odd(uint32_t acc, uint32_t x) {
    uint32_t r;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(x), "r"(0u), "r"(acc));
    return r;
}
__device__ __forceinline__ bool is_odd(uint32_t acc) { return (acc & 0x7FFF7FFFu) != 0; }

__device__ __forceinline__ float lo_f32(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f32(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// (a0, a1) * (b0, b1), one packed instruction.
__device__ __forceinline__ void fmul2(float& d0, float& d1, float a0, float a1, float b0, float b1) {
    asm("{\n\t.reg .b64 ra, rb, rd;\n\t"
        "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
        "mul.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
        : "=f"(d0), "=f"(d1)
        : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}
// What truncation to bf16 leaves of a pair (exact): f - (upper 16 bits of f).
__device__ __forceinline__ void rest2(float& m0, float& m1, float f0, float f1) {
    dev::ffma2(m0, m1, hi_f32(__float_as_uint(f0)), hi_f32(__float_as_uint(f1)), -1.f, -1.f, f0, f1);
}

// D[tmem] = A B for 128 rows and D columns of A (K-major tile): by a converged warp, one lane elected.  B advances by
// the same steps of 16 (K-major, `bk`) or by 16 rows.
template <int D>
__device__ __noinline__ void products(uint32_t d, uint32_t a, uint32_t b, bool bk, uint32_t idesc) {
    constexpr uint32_t kDescHi = tc::smem_desc_hi(1024, tc::kSwizzle128B);
#pragma unroll 1
    for (int half = 0; half < D / 64; ++half) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            tc::mma_ss_warp(d, a + (32 * i >> 4), b + ((bk ? 32 : 2048) * i >> 4), kDescHi, idesc, i > 0 ? 1u : (uint32_t)half);
        a += kRegion >> 4;
        b += (bk ? kRegion : 4 * 2048) >> 4;
    }
}

// A chunk with an infinity or a NaN in V, or with deep sums: this warp's rows of O (Q S so far) times `part`,
// plus (bad) the product of their weights with V over the keys each row sees.  Rarely called, so kept small.
template <int D>
__device__ __noinline__ void finish_rows(uint32_t t_o, uint32_t t_p, const uint8_t* V, int row, float part, bool bad) {
    const int last = row | 31;  // of the warp's rows
#pragma unroll 1
    for (int x = 0; x < D / 32; ++x) {
        float o[32];
        tc::tmem_ld32_async(t_o + 32 * x, o);
        tc::tmem_wait_ld_regs(o);
#pragma unroll
        for (int i = 0; i < 32; ++i) o[i] *= part;
#pragma unroll 1
        for (int j = 0; bad && j <= last; ++j) {
            const uint32_t w2 = tc::tmem_ld1(t_p + j / 2);
            const float w = (j & 1) ? hi_f32(w2) : lo_f32(w2);
            if (j <= row) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint4 y = *reinterpret_cast<const uint4*>(V + (x >> 1) * kRegion + j * 128 +
                                                                    ((((x & 1) * 4 + e) ^ (j & 7)) << 4));
                    const uint32_t v[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        o[8 * e + 2 * i] = fmaf(w, lo_f32(v[i]), o[8 * e + 2 * i]);
                        o[8 * e + 2 * i + 1] = fmaf(w, hi_f32(v[i]), o[8 * e + 2 * i + 1]);
                    }
                }
            }
            __syncwarp();
        }
        tc::tmem_st32(t_o + 32 * x, o);
    }
    tc::tmem_wait_st();
}

// What a token that drops the state needs lies in functions of its own, out of the roles' way: on the same box the 8
// prompts take 167 us and 12 chunks of D 64 32.5, without any of it 165 and 31.1, with all of it in the roles' loops
// 173 and 34.7.

// The decay warp's part of a chunk with such tokens (or with NaN decays): the sums start anew at each.  g: the first
// token's log decay, of ntok; returns whether there are any.  (In line behind that warp's own: as a call it cost the
// prompts another 3 us.)
__device__ __forceinline__ bool sums_with_drops(Bars* b, int st, const float* g, int64_t ld, int ntok) {
    const int lane = threadIdx.x & 31;
    double sum[4], y = 0.0;
    int first[4], f = -1;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float x = 4 * lane + i < ntok ? g[(4 * lane + i) * ld] : 0.f;
        const bool drop = x <= kDropLogDecay;
        y = drop ? 0.0 : y + (double)x * 1.4426950408889634074;
        if (drop) f = 4 * lane + i;
        sum[i] = y, first[i] = f;
    }
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const double z = __shfl_up_sync(0xffffffffu, y, d);
        const int before = __shfl_up_sync(0xffffffffu, f, d);
        if (lane >= d && f < 0) y += z, f = before;
    }
    const double up = __shfl_up_sync(0xffffffffu, y, 1), end = __shfl_sync(0xffffffffu, y, 31);
    const int up_first = __shfl_up_sync(0xffffffffu, f, 1), last = __shfl_sync(0xffffffffu, f, 31);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (lane > 0 && first[i] < 0) sum[i] += up, first[i] = up_first;
        const int t = 4 * lane + i;
        b->c[st][t] = (float)sum[i];
        b->w[st][t] = t >= last && t < ntok ? dev::fast_exp2((float)(end - sum[i])) : -0.f;
        b->first[st][t] = (int8_t)first[i];
    }
    if (lane == 0) {
        b->end[st] = last >= 0 ? -1.f : dev::fast_exp2((float)end);
        b->deep[st] = last >= 0 ? kDrops : 1;
        b->last[st] = last;
        b->r[st] = 0.f;
        b->down[st] = 1.f;
    }
    return last >= 0;
}

// An infinity or a NaN in this warp's 16 rows of V (`odd`: in the lane's part of one): where a later token drops the state
// the row becomes 0, since its weight of 0 would not keep it from the state.
template <int D>
__device__ __noinline__ bool hide_odd_rows(Bars* b, uint8_t* V, int row, bool odd, int st, uint32_t parity) {
    if (!__all_sync(0xffffffffu, phase_done(&b->dec_full[st], parity, b->wait_limit))) return false;
    if (b->deep[st] != kDrops) return true;
    if (odd && row < b->last[st]) {
#pragma unroll 1
        for (int ch = (threadIdx.x & 1) * (D / 16), e = ch + D / 16; ch < e; ++ch)
            *reinterpret_cast<uint4*>(V + (ch >> 3) * kRegion + row * 128 + (((ch ^ row) & 7) << 4)) = make_uint4(0, 0, 0, 0);
    }
    tc::fence_proxy_async_smem();
    return true;
}

// finish_rows for a chunk with tokens that drop the state: this row's weights of the keys before `first` become 0, and
// so does its part of Q S where there is one; and (an infinity or a NaN in V) the product with V over the keys up to
// `last`, -1: the tensor cores add it.  V comes from memory: in shared memory odd rows may be 0.
template <int D>
__device__ __noinline__ void drop_rows(uint32_t t_o, uint32_t t_p, const uint16_t* V, int64_t ld_v, int row, int last, int first,
                                       float part) {
#pragma unroll 1
    for (int x = 0; x <= row >> 5; ++x) {
        float w[16];
        uint32_t y[16];
        tc::tmem_ld16_async(t_p + 16 * x, w);
        tc::tmem_wait_ld16_regs(w);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int j = 32 * x + 2 * i;
            y[i] = __float_as_uint(w[i]) & (j >= first ? 0xFFFFFFFFu : j + 1 >= first ? 0xFFFF0000u : 0u);
        }
        tc::tmem_st16u(t_p + 16 * x, y);
    }
    tc::tmem_wait_st();
#pragma unroll 1
    for (int x = 0; x < D / 16; ++x) {  // (16 columns at a time: with 32 it needs more registers than its warps have)
        float o[16];
        uint32_t y16[16];
        tc::tmem_ld16_async(t_o + 16 * x, o);
        tc::tmem_wait_ld16_regs(o);
#pragma unroll
        for (int i = 0; i < 16; ++i) o[i] = first < 0 ? o[i] * part : 0.f;
#pragma unroll 1
        for (int j = 0; j <= last; ++j) {
            const uint32_t w2 = tc::tmem_ld1(t_p + j / 2);
            const float w = (j & 1) ? hi_f32(w2) : lo_f32(w2);
            if (j <= row && j >= first) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const uint4 y = __ldg(reinterpret_cast<const uint4*>(V + j * ld_v + 16 * x + 8 * e));
                    const uint32_t v[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        o[8 * e + 2 * i] = fmaf(w, lo_f32(v[i]), o[8 * e + 2 * i]);
                        o[8 * e + 2 * i + 1] = fmaf(w, hi_f32(v[i]), o[8 * e + 2 * i + 1]);
                    }
                }
            }
            __syncwarp();
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) y16[i] = __float_as_uint(o[i]);
        tc::tmem_st16u(t_o + 16 * x, y16);
    }
    tc::tmem_wait_st();
}

template <int D, bool STATES>
__global__ void __launch_bounds__(kThreads, 1)
    linear_chunk_kernel(const LinParams p, const __grid_constant__ CUtensorMap q_map,
                        const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map) {
    using L = SmemMap<D, STATES>;
    constexpr uint32_t KH = L::kHalvesK, KS = KH / 2;
    constexpr int kScaleWarps = STATES ? 8 : 4;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ Bars bars;
    Bars* b = &bars;
    // the plan, the activations and the states may come from the kernel before this one
    dev::grid_dep_wait();
    dev::grid_dep_launch();
    PlanHeader* hdr = reinterpret_cast<PlanHeader*>(p.ws + p.lay.header);
    uint32_t* err = &hdr->error_bits;
    const int Hkv = p.num_kv_heads;
    const unsigned parts = STATES ? 1 : hdr->n_casc_units;  // CTAs that share a kv head's q heads
    const int n_units = (STATES ? hdr->n_casc_tiles : hdr->n_pre_tiles) * Hkv * (int)parts;
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
            dev::mbar_init(&b->v_empty[s], STATES ? 1 : 2);
            dev::mbar_init(&b->v_ok[s], kScaleWarps);
            dev::mbar_init(&b->p_full[s], 1);
            dev::mbar_init(&b->p_ready[s], 4);
            dev::mbar_init(&b->qs_full[s], 1);
            dev::mbar_init(&b->dec_full[s], 1);
            dev::mbar_init(&b->dec_empty[s], STATES ? 12 : 16);
        }
        for (uint32_t s = 0; s < KH; ++s) {
            dev::mbar_init(&b->k_full[s], 1);
            dev::mbar_init(&b->k_empty[s], STATES ? 8 : 9);
        }
        for (int s = 0; s < kParts; ++s) {
            dev::mbar_init(&b->w_full[s], 2);
            dev::mbar_init(&b->w_empty[s], 1);
        }
        dev::mbar_init(&b->o_ready, 1);
        dev::mbar_init(&b->o_free, 4);
        dev::mbar_init(&b->ds_full, 1);
        dev::mbar_init(&b->ds_free, 4);
        dev::mbar_init(&b->s_full, 4);
        dev::mbar_init(&b->s_empty, 1);
        dev::mbar_init(&b->drain[0], 1);
        dev::mbar_init(&b->drain[1], 1);
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
    const Waits wait{b->wait_limit};
    bool ok = true;  // none of this warp's waits ran out

    if (warp >= 16) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsCtrl));
        constexpr uint32_t kDescHi = tc::smem_desc_hi(1024, tc::kSwizzle128B);
        const uint32_t v_lo = tc::smem_desc_lo(dev::smem_u32(smem + L::kV), kRegion);
        if (warp == kMmaWarp) {
            // ========================================================== MMAs of the outputs (one lane elected)
            if constexpr (!STATES) {
                const uint32_t id_qk = tc::idesc_bf16_f32(128, 128, 0, 0), id_v = tc::idesc_bf16_f32(128, D, 0, 1);
                const uint32_t q_lo = tc::smem_desc_lo(dev::smem_u32(smem + L::kQ), 16);
                const uint32_t k_lo = tc::smem_desc_lo(dev::smem_u32(smem + L::kK), 16);
                const uint32_t s_lo = tc::smem_desc_lo(dev::smem_u32(smem + L::kS), L::kStateRegion);
                uint32_t n = 0, h = 0;  // chunks and q heads so far
                // Q K^T runs one head ahead: its own place in the sequence of heads
                // (the unit after the one at hand is looked up while that one runs)
                int q_left = 0, q_heads = 0, qg = 0;  // chunks left of its unit, the unit's heads, head
                uint32_t qn = 0, qh = 0;
                bool more = false;
                int next_left = 0, next_heads = 0;
                auto inputs_seen = [&] {
                    // (both halves of K: copies need not land in the order in which they were begun)
                    return seen_warp(&b->q_full[qh & 1], (qh >> 1) & 1) &&
                           (qg > 0 || (seen_warp(&b->k_full[2 * (qn % KS) + 1], (qn / KS) & 1) &&
                                       seen_warp(&b->k_full[2 * (qn % KS)], (qn / KS) & 1)));
                };
                // (the weights that lay in this buffer were read by the P V of two heads before, issued already)
                auto inputs_there = [&] {
                    return (qg > 0 || (wait.warp(&b->k_full[2 * (qn % KS)], (qn / KS) & 1) &&
                                       wait.warp(&b->k_full[2 * (qn % KS) + 1], (qn / KS) & 1))) &&
                           wait.warp(&b->q_full[qh & 1], (qh >> 1) & 1);
                };
                auto issue_qk = [&] {
                    tc::fence_after_sync();
                    const uint32_t q0 = q_lo + ((qh & 1) * L::kTile >> 4), k0 = k_lo + (qn % KS * L::kTile >> 4);
                    products<D>(tmem + kColP + 128 * (qh & 1), q0, k0, true, id_qk);
                    tc::mma_commit_warp(&b->p_full[qh & 1]);
                    ++qh;
                    if (++qg == q_heads) {
                        tc::mma_commit_warp(&b->k_empty[2 * (qn % KS)]);
                        tc::mma_commit_warp(&b->k_empty[2 * (qn % KS) + 1]);
                        qg = 0;
                        ++qn;
                        if (--q_left == 0) {
                            q_left = next_left, q_heads = next_heads;
                            more = next_left > 0;
                        }
                    }
                };
                for (int k = 0, u; ok && (u = unit_at(k, n_units)) >= 0; ++k) {
                    int nch = next_left, G = next_heads;
                    next_left = next_heads = 0;
                    for (int i = k == 0 ? 0 : 1; i < 2; ++i) {  // (at first this one as well)
                        const int v = unit_at(k + i, n_units);
                        if (v < 0) break;
                        const Unit x = unit_of<STATES>(items, v, p, parts);
                        next_left = chunks_of(x.it.ntok), next_heads = x.g1 - x.g0;
                        if (i == 0) nch = q_left = next_left, G = q_heads = next_heads, more = true, next_left = 0;
                    }
                    for (int c = 0; ok && c < nch; ++c, ++n) {
                        const int st = n & 1;
                        for (int g = 0; ok && g < G; ++g, ++h) {
                            // What a head takes: its scores (issued during the head before, if their operands were there by
                            // then), Q S, P V.  Steps 0: scores, if not issued yet; 1: Q S; 2: the next head's scores if P is
                            // not there yet and their operands are; 3: P V; 4: the next head's scores if their operands are there.
#pragma unroll 1
                            for (int step = 0; ok && step < 5; ++step) {
                                if (step == 1) {
                                    ok = (g > 0 || wait.warp(&b->s_full, n & 1)) && (h == 0 || wait.warp(&b->o_free, (h - 1) & 1));
                                    if (!ok) break;
                                    tc::fence_after_sync();
                                    products<D>(tmem + kColO, q_lo + ((h & 1) * L::kTile >> 4), s_lo, false, id_v);
                                    tc::mma_commit_warp(&b->qs_full[h & 1]);
                                    tc::mma_commit_warp(&b->q_empty[h & 1]);
                                    if (g == G - 1) tc::mma_commit_warp(&b->s_empty);
                                } else if (step == 3) {
                                    if (!(ok = wait.warp(&b->p_ready[h & 1], (h >> 1) & 1))) break;
                                    tc::fence_after_sync();
                                    if (!v_is_bad(b, st)) {
                                        const uint32_t b0 = v_lo + (st * L::kTile >> 4);
#pragma unroll 4
                                        for (int kk = 0; kk < kChunk / 16; ++kk)
                                            tc::mma_ts_warp(tmem + kColO, tmem + kColP + 128 * (h & 1) + kk * 8,
                                                            b0 + (kk * 2048 >> 4), kDescHi, id_v, 1u);
                                    }
                                    tc::mma_commit_warp(&b->o_ready);
                                    if (g == G - 1) tc::mma_commit_warp(&b->v_empty[st]);
                                } else if (more && qh == h + (step > 0) &&
                                           (step != 2 || !seen_warp(&b->p_ready[h & 1], (h >> 1) & 1)) &&
                                           (step == 0 || inputs_seen())) {
                                    if (step == 0) ok = inputs_there();
                                    if (ok) issue_qk();
                                }
                            }
                        }
                    }
                }
            }
            // every MMA issued must complete before TMEM is released
            tc::mma_commit_warp(&b->drain[0]);
            (void)dev::mbar_wait(&b->drain[0], 0);
            __syncwarp();
        } else if (warp == kStateMmaWarp) {
            // ========================================================== MMAs of the state: 16 tokens at a time, three
            // parts of w K each
            const uint32_t id_kv = tc::idesc_bf16_f32(128, D, 1, 1);
            const uint32_t w_lo = tc::smem_desc_lo(dev::smem_u32(smem + L::kW), kPartRegion);
            uint32_t n = 0;
            for (int k = 0, u; ok && (u = unit_at(k, n_units)) >= 0; ++k) {
                const int nch = chunks_of(unit_of<STATES>(items, u, p, parts).it.ntok);
                for (int c = 0; ok && c < nch; ++c, ++n) {
                    const int st = n & 1;
                    if (!(ok = wait.warp(&b->v_ok[st], (n >> 1) & 1) && (n == 0 || wait.warp(&b->ds_free, (n - 1) & 1)))) break;
                    uint32_t b0 = v_lo + (st * L::kTile >> 4);
#pragma unroll 1
                    for (int s = 0; s < kParts; ++s, b0 += kPartRegion >> 4) {
                        if (!(ok = wait.warp(&b->w_full[s], n & 1))) break;
                        tc::fence_after_sync();
                        const uint32_t a0 = w_lo + ((s % L::kStagesW) * (3 * L::kSplit) >> 4);
#pragma unroll
                        for (int x = 0; x < 3; ++x)
                            tc::mma_ss_warp(tmem + kColState, a0 + (x * L::kSplit >> 4), b0, kDescHi, id_kv, x > 0 ? 1u : (uint32_t)s);
                        tc::mma_commit_warp(&b->w_empty[s]);
                    }
                    if (!ok) break;
                    tc::mma_commit_warp(&b->ds_full);
                    tc::mma_commit_warp(&b->v_empty[st]);
                }
            }
            tc::mma_commit_warp(&b->drain[1]);
            (void)dev::mbar_wait(&b->drain[1], 0);
            __syncwarp();
        } else if (warp == kLoadWarp && lane == 0) {
            // ========================================================== loads: of a chunk V, its first Q, K (as two
            // halves), its other Q
            uint32_t n = 0, h = 0, kh = 0;  // loads begun: V, Q, halves of K
            auto load = [&](uint64_t* empty, uint64_t* full, uint32_t turn, uint8_t* at, const CUtensorMap* map, int head, int t0,
                            uint32_t bytes) -> bool {
                if (!wait.one(empty, (turn & 1) ^ 1) || b->abort_flag) return ok = false;
                dev::mbar_arrive_expect_tx(full, bytes);
#pragma unroll
                for (int i = 0; i < L::kHalves; ++i) tc::tma_load_3d(at + i * kRegion, map, 64 * i, head, t0, full);
                return true;
            };
            for (int k = 0, u; ok && (u = unit_at(k, n_units)) >= 0; ++k) {
                const Unit x = unit_of<STATES>(items, u, p, parts);
                for (int c = 0; ok && c < chunks_of(x.it.ntok); ++c) {
                    const int t0 = x.it.tok0 + c * kChunk, heads = x.g1 - x.g0;
#pragma unroll 1
                    for (int i = 0; ok && i < heads + 3; ++i) {  // (0: V, 1: Q 0, 2 and 3: K, 4 ..: Q 1 ..)
                        const int j = STATES && i > 0 ? i + 1 : i;
                        if (j == 0) {
                            n += load(&b->v_empty[n & 1], &b->v_full[n & 1], n >> 1, smem + L::kV + (n & 1) * L::kTile, &v_map, x.kvh,
                                      t0, L::kTile);
                        } else if (j == 2 || j == 3) {
                            kh += load(&b->k_empty[kh % KH], &b->k_full[kh % KH], kh / KH,
                                       smem + L::kK + (kh % KH / 2) * L::kTile + (kh & 1) * (kRegion / 2), &k_map, x.kvh,
                                       t0 + 64 * (j - 2), L::kTile / 2);
                        } else if (j < heads + 3) {
                            h += load(&b->q_empty[h & 1], &b->q_full[h & 1], h >> 1, smem + L::kQ + (h & 1) * L::kTile, &q_map,
                                      x.kvh * p.group + x.g0 + (j == 1 ? 0 : j - 3), t0, L::kTile);
                        }
                    }
                }
            }
            // the last copies into every stage land before the CTA leaves
            for (uint32_t s = 0; s < 4; ++s) {
                if (s < 2 && n > s) (void)dev::mbar_wait(&b->v_full[(n - 1 - s) & 1], ((n - 1 - s) >> 1) & 1);
                if (s < 2 && h > s) (void)dev::mbar_wait(&b->q_full[(h - 1 - s) & 1], ((h - 1 - s) >> 1) & 1);
                if (s < KH && kh > s) (void)dev::mbar_wait(&b->k_full[(kh - 1 - s) % KH], ((kh - 1 - s) / KH) & 1);
            }
        } else if (warp == kDecayWarp) {
            // ========================================================== sums of the log decays, four tokens a lane
            uint32_t n = 0;
            for (int k = 0, u; ok && (u = unit_at(k, n_units)) >= 0; ++k) {
                const Unit x = unit_of<STATES>(items, u, p, parts);
                const int nch = chunks_of(x.it.ntok);
                double total = 0.0;  // of the unit
                bool dropped = false;
                float g4[4];
                auto load = [&](int c) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int t = c * kChunk + 4 * lane + i;
                        g4[i] = t < x.it.ntok ? p.log_decay[(p.ld_decay ? (int64_t)(x.it.tok0 + t) * p.ld_decay : 0) + x.kvh] : 0.f;
                    }
                };
                load(0);
                for (int c = 0; ok && c < nch; ++c, ++n) {
                    double sum[4], y = 0.0;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        y += (double)(g4[i] <= kDropLogDecay ? -INFINITY : g4[i]) * 1.4426950408889634074;
                        sum[i] = y;
                    }
                    if (c + 1 < nch) load(c + 1);
#pragma unroll
                    for (int d = 1; d < 32; d *= 2) {
                        const double z = __shfl_up_sync(0xffffffffu, y, d);
                        if (lane >= d) y += z;
                    }
                    const double up = __shfl_up_sync(0xffffffffu, y, 1), before = lane > 0 ? up : 0.0;
                    const double end = __shfl_sync(0xffffffffu, y, 31);
                    const int st = n & 1;
                    if (!(ok = wait.warp(&b->dec_empty[st], ((n >> 1) & 1) ^ 1))) break;
                    float cf[4], least = INFINITY, most = -INFINITY;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        cf[i] = (float)(before + sum[i]);
                        least = fminf(least, cf[i]), most = fmaxf(most, cf[i]);
                        if (cf[i] != cf[i]) most = INFINITY;  // (a NaN)
                    }
#pragma unroll
                    for (int d = 1; d < 32; d *= 2) {
                        least = fminf(least, __shfl_xor_sync(0xffffffffu, least, d));
                        most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, d));
                    }
                    const float r = least >= -kReach && most <= kReach ? 0.f : rintf(-0.5f * (least + most));
                    const bool deep = !(fabsf(r) <= kReach && -least - r <= kReach && -most - r >= -kReach);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        b->c[st][4 * lane + i] = cf[i];
                        b->f[st][4 * lane + i] = dev::fast_exp2(-cf[i] - r);
                        b->w[st][4 * lane + i] =
                            c * kChunk + 4 * lane + i < x.it.ntok ? dev::fast_exp2((float)(end - (before + sum[i]))) : -0.f;
                    }
                    if (lane == 0) {
                        b->end[st] = dev::fast_exp2((float)end);
                        b->deep[st] = deep;
                        b->r[st] = deep ? 0.f : r;
                        b->down[st] = deep ? 1.f : dev::fast_exp2(-r);
                    }
                    if (__builtin_expect(!(least > -INFINITY && most < INFINITY), 0)) {  // (what lies there by now is written again)
                        const float* g = p.log_decay + (p.ld_decay ? (int64_t)(x.it.tok0 + c * kChunk) * p.ld_decay : 0) + x.kvh;
                        dropped |= sums_with_drops(b, st, g, p.ld_decay, x.it.ntok - c * kChunk);
                    }
                    arrive_warp(&b->dec_full[st]);
                    total += end;
                }
                if (STATES && ok && lane == 0)
                    seg_decay[(int64_t)(x.it.base + x.it.seg + 1) * Hkv + x.kvh] = dropped ? -1.f : exp2f((float)total);
            }
        }
    } else if (!STATES && warp >= 12) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsO));
        if constexpr (!STATES) {
        // ============================================================== O to memory, a row a thread
        const int row = threadIdx.x - 384, first = row & ~3;
        const uint32_t t_o = tmem + kColO + ((uint32_t)((warp & 3) * 32) << 16);
        const int64_t step = (int64_t)p.num_qo_heads * D;
        uint32_t n = 0, h = 0;
        for (int k = 0, u; ok && (u = unit_at(k, n_units)) >= 0; ++k) {
            const Unit un = unit_of<STATES>(items, u, p, parts);
            for (int tok = un.it.tok0, left = un.it.ntok; ok && left > 0; ++n, tok += kChunk, left -= kChunk) {
                const int st = n & 1;
                if (!(ok = wait.warp(&b->dec_full[st], (n >> 1) & 1))) break;
                const float ci = b->c[st][row];
                const float factor = p.scale * dev::fast_exp2(b->deep[st] != 0 ? fminf(fmaxf(ci, -kDeep), kDeep) : ci + b->r[st]);
                arrive_warp(&b->dec_empty[st]);
                // (four lanes turn 4 x 4 chunks of 16 bytes among them, so that a row's 64 bytes go out together: by each
                // thread's own row, 16 bytes at a time, it took 3800 cycles)
                uint16_t* dst = p.out + ((int64_t)(tok + first) * p.num_qo_heads + un.kvh * p.group + un.g0) * D + 8 * (lane & 3);
                for (int g = un.g0; g < un.g1; ++g, ++h, dst += D) {
                    if (!(ok = wait.warp(&b->o_ready, h & 1))) break;
                    tc::fence_after_sync();
#pragma unroll 1
                    for (int x = 0; x < D / 32; ++x) {
                        float o[32];
                        tc::tmem_ld32_async(t_o + 32 * x, o);
                        tc::tmem_wait_ld_regs(o);
                        if (x == D / 32 - 1) {
                            tc::fence_before_sync();
                            arrive_warp(&b->o_free);
                        }
                        uint32_t w[4][4];
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            float y0, y1;
                            fmul2(y0, y1, o[2 * i], o[2 * i + 1], factor, factor);
                            w[i >> 2][i & 3] = dev::pack_bf16x2(y0, y1);
                        }
#pragma unroll
                        for (int m = 1; m <= 2; m *= 2) {
                            const bool up = (lane & m) != 0;
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                if (e & m) continue;
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? w[e][i] : w[e | m][i], m);
                                    if (up) w[e][i] = got;
                                    else w[e | m][i] = got;
                                }
                            }
                        }
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (first + e < left)
                                *reinterpret_cast<uint4*>(dst + e * step + 32 * x) = make_uint4(w[e][0], w[e][1], w[e][2], w[e][3]);
                        __syncwarp();
                    }
                }
            }
        }
        }
    } else if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsScale));
        // ============================================================== w K in three bf16 parts; a look at V
        // Two warps make a part of 16 tokens: pair i the parts i, i + kScaleWarps / 2 and so on.
        const int wq = warp - 8, pair = wq >> 1;
        const int r0 = (wq & 1) * 8 + (lane >> 3), cc = lane & 7;  // first token of a part's, 16-byte chunk of its row
        uint32_t n = 0;
        for (int k = 0, u; ok && (u = unit_at(k, n_units)) >= 0; ++k) {
            const int ntok = unit_of<STATES>(items, u, p, parts).it.ntok;
            for (int c = 0; ok && c < chunks_of(ntok); ++c, ++n) {
                const int st = n & 1, nval = min(kChunk, ntok - c * kChunk);
                uint8_t* V = smem + L::kV + st * L::kTile;
                if (!(ok = wait.warp(&b->v_full[st], (n >> 1) & 1))) break;
#pragma unroll 1
                for (int x0 = wq; x0 < 8; x0 += kScaleWarps) {  // half a row of V a lane (D 64: a quarter of one in either half)
                    const int row = x0 * 16 + (lane >> 1);
                    constexpr int kEach = D / 16;
                    uint4* at[kEach];
#pragma unroll
                    for (int x = 0; x < kEach; ++x) {
                        const int ch = (lane & 1) * kEach + x;
                        at[x] = reinterpret_cast<uint4*>(V + (ch >> 3) * kRegion + row * 128 + (((ch ^ row) & 7) << 4));
                    }
                    uint32_t odd = 0;
                    if (row < nval) {
                        uint4 y[kEach];
#pragma unroll
                        for (int x = 0; x < kEach; ++x) y[x] = *at[x];
#pragma unroll
                        for (int x = 0; x < kEach; ++x)
                            odd = note_odd(note_odd(note_odd(note_odd(odd, y[x].x), y[x].y), y[x].z), y[x].w);
                    } else {
#pragma unroll
                        for (int x = 0; x < kEach; ++x) *at[x] = make_uint4(0, 0, 0, 0);
                    }
                    const int any = __any_sync(0xffffffffu, is_odd(odd));
                    if (lane == 0) b->v_bad[st][x0] = any;
                    if (__builtin_expect(any, 0) && !(ok = hide_odd_rows<D>(b, V, row, is_odd(odd), st, (n >> 1) & 1))) break;
                }
                if (!ok) break;
                if (nval < kChunk) tc::fence_proxy_async_smem();
                arrive_warp(&b->v_ok[st]);
                if (!(ok = wait.warp(&b->dec_full[st], (n >> 1) & 1))) break;
                const uint8_t* K = smem + L::kK + (n % KS) * L::kTile;
#pragma unroll 1
                for (int s = pair; s < kParts; s += kScaleWarps / 2) {
                    const uint32_t half = 2 * (n % KS) + (s >= 4);
                    if (!(ok = wait.warp(&b->k_full[half], (n / KS) & 1))) break;
                    const int held = (int)(n * kParts + s) - L::kStagesW;  // the part that its stage held
                    uint8_t* W = smem + L::kW + (s % L::kStagesW) * 3 * L::kSplit;
#pragma unroll
                    for (int z = 0; z < 2 * L::kHalves; ++z) {  // two tokens, their row's halves
                        const int x = z % L::kHalves, r = r0 + 4 * (z / L::kHalves), row = s * kPart + r;
                        const float w = b->w[st][row];
                        uint4 y = *reinterpret_cast<const uint4*>(K + x * kRegion + row * 128 + (((cc ^ row) & 7) << 4));
                        if (__float_as_int(w) < 0) y = make_uint4(0, 0, 0, 0);  // (whatever lies there times 0)
                        const uint32_t e[4] = {y.x, y.y, y.z, y.w};
                        uint32_t hi[4], mid[4], lo[4];
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            // the upper 8 bits, the next 8 and the rest: each difference is exact (of an infinity it is
                            // a NaN)
                            float f0, f1, m0, m1, l0, l1;
                            fmul2(f0, f1, lo_f32(e[q]), hi_f32(e[q]), w, w);
                            rest2(m0, m1, f0, f1);
                            rest2(l0, l1, m0, m1);
                            hi[q] = dev::prmt(__float_as_uint(f0), __float_as_uint(f1), 0x7632);
                            mid[q] = dev::prmt(__float_as_uint(m0), __float_as_uint(m1), 0x7632);
                            lo[q] = dev::pack_bf16x2(l0, l1);
                        }
                        if (z == 0 && held >= 0 && !(ok = wait.warp(&b->w_empty[held % kParts], (held / kParts) & 1))) break;
                        uint8_t* at = W + x * kPartRegion + r * 128 + (((cc ^ r) & 7) << 4);
                        *reinterpret_cast<uint4*>(at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                        *reinterpret_cast<uint4*>(at + L::kSplit) = make_uint4(mid[0], mid[1], mid[2], mid[3]);
                        *reinterpret_cast<uint4*>(at + 2 * L::kSplit) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                    }
                    if (!ok) break;
                    tc::fence_proxy_async_smem();
                    arrive_warp(&b->w_full[s]);
                    if ((threadIdx.x & 31) == 0) dev::mbar_arrive(&b->k_empty[half]);
                }
                if (!ok) break;
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
        const int64_t per_head = (int64_t)D * D;
        for (int k = 0, u; ok && (u = unit_at(k, n_units)) >= 0; ++k) {
            const Unit un = unit_of<STATES>(items, u, p, parts);
            const LinItem& it = un.it;
            const int nch = chunks_of(it.ntok);
            float S[D / 32][32];
#pragma unroll
            for (int x = 0; x < D; ++x) S[x >> 5][x & 31] = 0.f;
            // a state slot of this warp's rows, to or from S: through shared memory, so that whole rows are read
            // and written together (by each thread's own row a state took 4000 cycles)
            auto move = [&](float* rows, bool in) {
                constexpr int kCols = D / 2, kPer = kCols / 4;  // columns at a time, 16-byte chunks of those
                // (in the warp's own rows of the bf16 copy: 4 KiB in each of its regions)
                auto at = [&](int chunk) {
                    return reinterpret_cast<float4*>(smem + L::kS + (chunk >> 8) * L::kStateRegion + (warp & 3) * 4096 + (chunk & 255) * 16);
                };
                rows += (int64_t)(warp & 3) * 32 * D;
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    auto own = [&](int q) { return at(lane * kPer + (q ^ (lane & 7))); };
                    auto all = [&] {
                        // (every load in flight before the first is used)
                        float4 y[kPer];
#pragma unroll
                        for (int i = 0; i < kPer; ++i) {
                            const int r = (i * 32 + lane) / kPer, q = (i * 32 + lane) % kPer;
                            y[i] = in ? *reinterpret_cast<const float4*>(rows + r * D + half * kCols + 4 * q) : *at(r * kPer + (q ^ (r & 7)));
                        }
#pragma unroll
                        for (int i = 0; i < kPer; ++i) {
                            const int r = (i * 32 + lane) / kPer, q = (i * 32 + lane) % kPer;
                            if (in) *at(r * kPer + (q ^ (r & 7))) = y[i];
                            else *reinterpret_cast<float4*>(rows + r * D + half * kCols + 4 * q) = y[i];
                        }
                        __syncwarp();
                    };
                    if (in) all();
#pragma unroll
                    for (int q = 0; q < kPer; ++q) {
                        float* x = &S[(half * kCols + 4 * q) >> 5][(half * kCols + 4 * q) & 31];
                        if (in) {
                            const float4 y = *own(q);
                            x[0] = y.x, x[1] = y.y, x[2] = y.z, x[3] = y.w;
                        } else {
                            *own(q) = make_float4(x[0], x[1], x[2], x[3]);
                        }
                    }
                    __syncwarp();
                    if (!in) all();
                }
            };
            auto slot = [&](int i) { return p.states + ((int64_t)i * Hkv + un.kvh) * per_head; };
            // states in the workspace: four columns of a row, then those of the next row
            auto segment_state = [&](int i) {
                return reinterpret_cast<float4*>(seg_state + ((int64_t)(it.base + i) * Hkv + un.kvh) * per_head) + row;
            };
            // The start.  Where other CTAs work on the same request and kv head it is a copy that the kernel before
            // has made: the one that ends with the request's last token may write the slot before the others have
            // read it.  The states pass leaves the first segment's end from there, the others' from zero, and the scan
            // makes the request's state of each.
            if (n > 0 && !STATES && !(ok = wait.warp(&b->s_empty, (n - 1) & 1))) break;
            if (live && (it.seg == 0 ? it.in >= 0 : !STATES)) {
                if (it.base < 0) {
                    move(slot(it.in), true);
                } else {
                    const float4* src = segment_state(it.seg);
#pragma unroll
                    for (int x = 0; x < D; x += 4) {
                        const float4 y = src[x / 4 * D];
                        float* z = &S[x >> 5][x & 31];
                        z[0] = y.x, z[1] = y.y, z[2] = y.z, z[3] = y.w;
                    }
                }
            }
            for (int c = 0; ok && c < nch; ++c, ++n) {
                const int st = n & 1;
                if (!(ok = wait.warp(&b->dec_full[st], (n >> 1) & 1))) break;
                const float end = b->end[st], down = b->down[st];
                arrive_warp(&b->dec_empty[st]);
                if constexpr (!STATES) {
                    if (c > 0 && !(ok = wait.warp(&b->s_empty, (n - 1) & 1))) break;
                    if (live) {
#pragma unroll
                        for (int x = 0; x < D; x += 8) {
                            uint32_t w[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                float y0, y1;
                                fmul2(y0, y1, S[x >> 5][(x & 31) + 2 * i], S[x >> 5][(x & 31) + 2 * i + 1], down, down);
                                w[i] = dev::pack_bf16x2(y0, y1);
                            }
                            dev::st_shared_v4(dev::smem_u32(smem + L::kS) + (x >> 6) * L::kStateRegion + row * 128 +
                                                  ((((x >> 3) ^ row) & 7) << 4), w[0], w[1], w[2], w[3]);
                        }
                    }
                    tc::fence_proxy_async_smem();
                    arrive_warp(&b->s_full);
                }
                if (__builtin_expect(end < 0.f, 0)) {  // (dropped)
#pragma unroll
                    for (int x = 0; x < D; ++x) S[x >> 5][x & 31] = 0.f;
                }
                if (!(ok = wait.warp(&b->ds_full, n & 1))) break;
                tc::fence_after_sync();
#pragma unroll
                for (int x = 0; x < D / 16; ++x) {
                    float d[16];
                    tc::tmem_ld16_async(t_ds + 16 * x, d);
                    tc::tmem_wait_ld16_regs(d);
#pragma unroll
                    for (int i = 0; i < 16; i += 2) {
                        float &s0 = S[x >> 1][(x & 1) * 16 + i], &s1 = S[x >> 1][(x & 1) * 16 + i + 1];
                        dev::ffma2(s0, s1, end, end, s0, s1, d[i], d[i + 1]);
                    }
                }
                tc::fence_before_sync();
                arrive_warp(&b->ds_free);
            }
            if (!ok || !live) continue;
            if constexpr (STATES) {
                float4* dst = segment_state(it.seg + 1);
#pragma unroll
                for (int x = 0; x < D; x += 4) {
                    const float* z = &S[x >> 5][x & 31];
                    dst[x / 4 * D] = make_float4(z[0], z[1], z[2], z[3]);
                }
            } else if (it.out >= 0 && it.seg == it.nseg - 1 && un.g0 == 0) {
                if (!(ok = wait.warp(&b->s_empty, (n - 1) & 1))) break;
                move(slot(it.out), false);
            }
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsP));  // (in the states pass too: the split counts on it)
        if constexpr (!STATES) {
        // ============================================================== P, a row a thread
        const int row = threadIdx.x;
        const uint32_t lane_base = (uint32_t)(warp * 32) << 16;
        uint32_t n = 0, h = 0;
        for (int k = 0, u; ok && (u = unit_at(k, n_units)) >= 0; ++k) {
            const Unit un = unit_of<STATES>(items, u, p, parts);
            const int nch = chunks_of(un.it.ntok);
            for (int c = 0; ok && c < nch; ++c, ++n) {
                const int st = n & 1;
                if (!(ok = wait.warp(&b->dec_full[st], (n >> 1) & 1) && wait.warp(&b->v_ok[st], (n >> 1) & 1))) break;
                const bool bad = v_is_bad(b, st), deep = b->deep[st] != 0, drops = b->deep[st] == kDrops;
                const float ci = b->c[st][row], up = deep ? ci - fminf(fmaxf(ci, -kDeep), kDeep) : 0.f;
                const float* other = deep ? b->c[st] : b->f[st];
                for (int g = un.g0; g < un.g1; ++g, ++h) {
                    const uint32_t t_p = tmem + kColP + 128 * (h & 1) + lane_base;
                    if (!(ok = wait.warp(&b->p_full[h & 1], (h >> 1) & 1))) break;
                    tc::fence_after_sync();
                    // 32 keys at a time; those past the warp's own rows have no weight.  (The packed weights of
                    // block x lie in columns 16 x .. of the scores, which are read by then.)
#pragma unroll 1
                    for (int x = 0; x < kChunk / 32; ++x) {
                        uint32_t pk[16];
                        if (x <= warp) {
                            float s[32];
                            tc::tmem_ld32_async(t_p + 32 * x, s);
                            tc::tmem_wait_ld_regs(s);
                            if (deep) {
#pragma unroll
                                for (int i = 0; i < 32; i += 4) {
                                    const float4 cj = *reinterpret_cast<const float4*>(other + 32 * x + i);
                                    fmul2(s[i], s[i + 1], s[i], s[i + 1], dev::fast_exp2(up - cj.x), dev::fast_exp2(up - cj.y));
                                    fmul2(s[i + 2], s[i + 3], s[i + 2], s[i + 3], dev::fast_exp2(up - cj.z), dev::fast_exp2(up - cj.w));
                                }
                            } else {
#pragma unroll
                                for (int i = 0; i < 32; i += 4) {
                                    const float4 f = *reinterpret_cast<const float4*>(other + 32 * x + i);
                                    fmul2(s[i], s[i + 1], s[i], s[i + 1], f.x, f.y);
                                    fmul2(s[i + 2], s[i + 3], s[i + 2], s[i + 3], f.z, f.w);
                                }
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
                    if (bad || (deep && (drops || __any_sync(0xffffffffu, up != 0.f)))) {
                        // (two barriers: of the heads in between nobody waits for it)
                        if (!(ok = wait.warp(&b->qs_full[h & 1], (h >> 1) & 1))) break;
                        tc::fence_after_sync();
                        if (drops)
                            drop_rows<D>(tmem + kColO + lane_base, t_p, p.v + (un.it.tok0 + c * (int64_t)kChunk) * p.ld_v + un.kvh * D, p.ld_v,
                                         row, bad ? min(row | 31, un.it.ntok - c * kChunk - 1) : -1, b->first[st][row], dev::fast_exp2(up));
                        else
                            finish_rows<D>(tmem + kColO + lane_base, t_p, smem + L::kV + st * L::kTile, row,
                                           deep ? dev::fast_exp2(up) : 1.f, bad);
                    }
                    tc::fence_before_sync();
                    arrive_warp(&b->p_ready[h & 1]);
                }
                if (ok) arrive_warp(&b->dec_empty[st]);
            }
        }
        }
    }
    if (!ok) {
        b->abort_flag = 1;
        dev::set_error(err, kErrTimeout);
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

// [T, heads, D] with ld elements between tokens; a box is 64 columns of one head for so many tokens.
bool encode(CUtensorMap* m, const uint16_t* x, int64_t tokens, int heads, int D, int64_t ld, int rows) {
    const EncodeTiledFn enc = tensor_map_encoder();
    if (enc == nullptr) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)tokens};
    const cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)ld * 2};
    const cuuint32_t box[3] = {64, 1, (cuuint32_t)rows};
    const cuuint32_t elem_strides[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint16_t*>(x), dims, strides, box, elem_strides,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool STATES>
cudaError_t launch(const LinParams& p, int ctas, cudaStream_t s) {
    auto kernel = linear_chunk_kernel<D, STATES>;
    const size_t smem = SmemMap<D, STATES>::kBytes + 1024;
    static_assert(SmemMap<D, STATES>::kBytes + 1024 + sizeof(Bars) <= 227 * 1024, "shared memory per block");
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
    if (!encode(&q, p.q, p.total_tokens, p.num_qo_heads, D, p.ld_q, kChunk) ||
        !encode(&k, p.k, p.total_tokens, p.num_kv_heads, D, p.ld_k, kChunk / 2) ||
        !encode(&v, p.v, p.total_tokens, p.num_kv_heads, D, p.ld_v, kChunk))
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

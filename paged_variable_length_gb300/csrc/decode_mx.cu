// K7: decode / small-row attention streaming an MXFP4 pool (layout: mxfp4.cuh).
//
// For every q head h of kv head g: S = scale q K^T over the request's keys, the bottom-right
// causal mask, softmax, O = P V, with K and V elements code * 2^(e - 127), block by block.  The
// plan, the split of long key ranges over CTAs and their join by log-sum-exp (merge kernel) are
// those of the other pool types (decode.cu).
//
// What bounds it: a key of one kv head is D + D/16 bytes for K and V together, a quarter of a
// bf16 pool's, so at HBM's rate an SM has to take in about four times as many elements a clock
// (some 40) and the conversion of codes, not HBM, is what the inner loop is arranged around:
//   * the MMAs take the keys as their 16 rows and the query rows as their 8 columns
//     (S^T = K Q^T, O^T = V^T P^T), so that up to 8 query rows (G = 4 and one token use 4 of
//     them) cost one n8 tile, half of what they would as the 16 rows;
//   * codes become f16 pairs with one exact conversion per pair.  K's block scales are applied
//     to the fp32 partial sums, block by block (4 per 32 elements of a key) rather than to the
//     elements; V's, which belong to the contraction's index, to the f16 pairs (exact: every
//     code * scale the store writes is an f16 value);
//   * the head dimension may be summed in any order and the output dims may sit in any tile
//     row, so a lane's K fragments are 4 consecutive bytes of a block (as ldmatrix gives them)
//     and its V rows D/16 consecutive bytes of a key; two keys' V nibbles are interleaved with
//     a bit select, so that one conversion gives the pair of keys the MMA wants;
//   * P^T comes from S^T's accumulators by an 8x8 transpose in registers (movmatrix).
// Each query row enters as f16 after a multiplication by the power of two that brings its
// largest element to [1, 2) (undone in the softmax scale), so that its range is bf16's (elements
// below 2^-14 of the row's largest lose their lowest bits); P is
// rounded to f16 (2^-11 of a weight, below the output's bf16 rounding; kPShift), sums are fp32.
// Every wait is bounded, as in decode.cu.
#include <cuda_runtime.h>

#include <atomic>
#include <type_traits>

#include "device_utils.cuh"
#include "mxfp4.cuh"
#include "pva_internal.h"

namespace pva {
namespace {

// Keys per ring stage, and the keys a consumer warp takes at a time (the wider row tile, and 16
// consumer warps, have registers for fewer scores).
constexpr __host__ __device__ int mx_stage_keys(int NQ) { return NQ == 1 ? 64 : 32; }
constexpr __host__ __device__ int mx_part_keys(int D, int NQ) { return D == 128 && NQ == 1 ? 64 : 32; }
constexpr float kLn2 = 0.69314718055994530942f;
// P enters its f16 operand as 2^7 times the weight relative to a reference that the row's maximum
// may outgrow by 2^8: the largest stays below f16's maximum, and weights down to 2^-21 of the
// reference keep all of f16's bits.
constexpr float kPShift = 7.f, kSlack = 8.f;

__device__ __forceinline__ uint32_t movmatrix_t(uint32_t x) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

// D = A B (m16n8k16, f16 in, fp32 out).
__device__ __forceinline__ void mma_f16_zero(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%10,%10,%10,%10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

// C += A B.  (Neither is volatile: the compiler may place loads and conversions between them.)
__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// (a & m) | (b & ~m)
__device__ __forceinline__ uint32_t bitsel(uint32_t a, uint32_t b, uint32_t m) {
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xE4;" : "=r"(r) : "r"(a), "r"(b), "r"(m));
    return r;
}

// Bounded wait on a barrier that lets the hardware suspend the warp (up to 100 us at a time) until
// the phase completes: 16 warps polling without the hint issued a third of the kernel's
// instructions.  The lanes' results are voted, so that the warp leaves together or not at all.
__device__ __forceinline__ bool wait_suspended(uint64_t* bar, uint32_t parity, uint64_t limit, uint32_t* err) {
    bool ok;
    if (limit == 0) {
        ok = dev::mbar_test_wait(bar, parity);
    } else {
        auto attempt = [&] {
            uint32_t done;
            asm volatile(
                "{\n\t.reg .pred p;\n\t"
                "mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2, %3;\n\t"
                "selp.u32 %0, 1, 0, p;\n\t}"
                : "=r"(done)
                : "r"(dev::smem_u32(bar)), "r"(parity), "r"(100000u)
                : "memory");
            return done != 0;
        };
        ok = attempt();
        if (!ok) {
            const uint64_t t0 = dev::globaltimer();
            do ok = attempt();
            while (!ok && dev::globaltimer() - t0 <= limit);
        }
    }
    if (__all_sync(0xffffffffu, ok)) return true;
    if ((threadIdx.x & 31) == 0) dev::set_error(err, kErrTimeout);
    __syncwarp();
    return false;
}

// What the producers say of a stage: the unit it belongs to (its keys k .. min(k + stage, k1) - 1
// are staged), its number in it (index), and the query rows of the unit after it (0 tokens: not
// known yet, or none).
struct MxStage {
    int32_t k, k1, tok0, ntok;
    int32_t qpos0, nparts, slot, hb;  // slot: the unit's partial slot
    int32_t index, flags, next_tok0, next_ntok;
    int32_t next_hb, pad0, pad1, pad2;
};

constexpr int kFirst = 1, kLast = 2, kEnd = 4;  // MxStage::flags

template <int I>
struct IntTag {
    static constexpr int value = I;
};

// The ring's barriers, and those by which a head's warps hand their results to its first.
constexpr int kMaxStages = 16;
constexpr int kSmemLimit = 220 * 1024;
struct MxSmem {
    uint64_t full[kMaxStages], empty[kMaxStages];
    uint64_t xfull[kDecHeadBlock], xempty[kDecHeadBlock];
    MxStage info[kMaxStages];
};

// Launch shape: heads of a CTA (hb), consumer warps a head (kw), ring stages; bytes of a staged row
// (the pool's row, or a block of its head groups).
struct MxShape {
    int hb, kw, stages, stride;
    int exch;  // byte offset of the exchange area
    int producers;  // producer warps: 1, or 4 that share a stage's rows (small copies)
};

// Bytes of a staged row of hb heads.
constexpr __host__ __device__ int mx_stride(int hb, int D) { return (hb * (D / 2 + D / mx::kBlock) + 15) / 16 * 16; }

// Warps of the one CTA an SM holds: consumers, and a warpgroup of producers, from which registers
// move to the consumers.
template <int D, int NQ>
struct MxWarps {
    static constexpr bool kMany = D == 64 && NQ == 1;  // the only tile small enough for 16 consumers
    static constexpr int kConsumers = kMany ? 16 : 8;
    static constexpr int kProducers = 4;
    static constexpr int kThreads = 32 * (kConsumers + kProducers);
    static constexpr int kRegsLaunch = kMany ? 96 : 168;
    static constexpr int kRegsConsumer = kMany ? 104 : 208;
    static constexpr int kRegsProducer = kMany ? 64 : 88;
    static_assert(kConsumers * kRegsConsumer + kProducers * kRegsProducer == (kConsumers + kProducers) * kRegsLaunch,
                  "register split must balance");
};

// D: head dim.  NQ: n8 tiles of query rows (rows of the batch's decode groups <= 8 NQ).  HBT: heads
// of the CTA, 0: not known at compile time.  (A known row size makes the fragment addresses of a
// stage one register and constants; computed, they were a quarter of the loop's instructions.)
// MULTI: decode groups may hold several tokens, which see different keys (without: 47.8 us for 64 decodes,
// 48.9 with).
template <int D, int NQ, int HBT, bool MULTI>
__global__ void __launch_bounds__(MxWarps<D, NQ>::kThreads, 1) decode_mx_kernel(const ForwardParams p, const MxShape sp) {
    using MW = MxWarps<D, NQ>;
    const bool shared_copies = sp.producers > 1;
    constexpr int kKeys = mx_stage_keys(NQ), kHalf = kKeys / 2;
    constexpr int kPart = mx_part_keys(D, NQ), kMT = kPart / 16;
    constexpr int NB = D / mx::kBlock;  // blocks of a head
    // whether a unit's query rows are requested while the unit before is worked on (with two tiles
    // of rows the registers are short: 50.9 us with, 48.7 without for 64 requests, 64/4 heads)
    constexpr bool kQAhead = NQ == 1;
    constexpr int OT = D / 16;          // m16 tiles of the output dims
    constexpr int VW = D / 64;          // words of a lane's run of V codes (D/8 dims)
    extern __shared__ __align__(128) uint8_t smem[];
    MxSmem* sh = reinterpret_cast<MxSmem*>(smem);
    uint8_t* ring = smem + ((sizeof(MxSmem) + 127) / 128) * 128;
    PlanHeader* hdr = reinterpret_cast<PlanHeader*>(p.ws + p.lay.header);
    uint32_t* err = &hdr->error_bits;
    const uint64_t wlim = dev::wait_limit(hdr->wait_override);

    const int Hkv = p.num_kv_heads, G = p.group, Hq = p.num_qo_heads;
    const int HB = HBT ? HBT : sp.hb, KW = sp.kw, stages = sp.stages, stride = HBT ? mx_stride(HBT, D) : sp.stride;
    const int n_hb = Hkv / HB, consumers = HB * KW;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int stage_bytes = 2 * kKeys * stride;
    dev::grid_dep_launch();
    // grid order and waits: as in decode.cu (wait_late: after a tensor-core kernel with units)
    const int n_units = hdr->n_dec_units * n_hb;
    const bool wait_late = p.dec_wait_late && hdr->n_pre_tiles > 0;
    if ((hdr->error_bits & kErrFatal) || n_units == 0) {
        dev::grid_dep_wait();
        return;
    }
    const DecUnit* units = reinterpret_cast<const DecUnit*>(p.ws + p.lay.dec_units);
    const DecGroup* dgroups = reinterpret_cast<const DecGroup*>(p.ws + p.lay.dec_groups);
    // this CTA's share of the key line (balanced split), or a queue of units (share 0)
    const int share = hdr->dec_share;
    const int n_groups = hdr->n_dec_groups;
    const int line_lo = (int)blockIdx.x * share, line_hi = line_lo + share;
    auto piece = [&](int g, const DecGroup& dg, DecUnit& du) -> bool {
        const int ext = dg.kv_end - dg.tail0;
        const int a = max(dg.g0, line_lo), e = min(dg.g0 + ext, line_hi);
        if (a >= e) return false;
        du.group = g;
        du.k0 = dg.tail0 + (a - dg.g0);
        du.k1 = dg.tail0 + (e - dg.g0);
        du.split = a == dg.g0 ? 0 : (int)blockIdx.x - dg.g0 / share;
        du.req = dg.req;
        du.tok0 = dg.tok0;
        du.ntok = dg.ntok;
        du.qpos0 = dg.qpos0;
        du.nsplit = dg.nsplit;
        du.pbase = dg.pbase;
        du.nparts = dg.nparts;
        du.pad1 = 0;
        return true;
    };
    // several producer warps walk the units alike, so a queue's units then go round the CTAs in
    // turn (they are listed longest first) instead of through the counter
    const bool static_first = shared_copies || !wait_late || share > 0;
    DecUnit du_first{};
    bool have_first = false;
    int g_first = -1;
    constexpr int kPL = kKeys / 32;       // keys of a stage a producer lane looks up: lane, lane + 32
    int32_t page_first_raw[kPL] = {};
    if (static_first) {  // (the consumers too: their first query rows)
        if (share > 0) {
            int g = reinterpret_cast<const int32_t*>(p.ws + p.lay.dec_first)[blockIdx.x];
            if (g < n_groups) {
                have_first = piece(g, dgroups[g], du_first);
                if (!have_first && ++g < n_groups) have_first = piece(g, dgroups[g], du_first);
            }
            g_first = g;
        } else if ((int)blockIdx.x < n_units) {
            du_first = units[blockIdx.x / n_hb];
            have_first = true;
        }
#pragma unroll
        for (int h = 0; h < kPL; ++h) {
            const int key = du_first.k0 + lane + 32 * h;
            if (warp >= MW::kConsumers && have_first && key < du_first.k1)
                page_first_raw[h] = p.page_table[(int64_t)du_first.req * p.ld + (key >> p.page_shift)];
        }
    }
    if (threadIdx.x == 0) {
        for (int s = 0; s < stages; ++s) {
            dev::mbar_init(&sh->full[s], sp.producers);
            dev::mbar_init(&sh->empty[s], consumers);
        }
        for (int h = 0; h < kDecHeadBlock; ++h) {
            dev::mbar_init(&sh->xfull[h], KW > 1 ? KW - 1 : 1);
            dev::mbar_init(&sh->xempty[h], 1);
        }
        dev::fence_barrier_init();
    }
    __syncthreads();
    if (!wait_late) dev::grid_dep_wait();

    int32_t* sched = &hdr->pad[0];
    const int sched_base = static_first ? (int)gridDim.x : 0;

    if (warp >= MW::kConsumers) {
        // ================================================================ producers
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(MW::kRegsProducer));
        const int pwarp = warp - MW::kConsumers;
        if (pwarp >= sp.producers) return;
        // the warp's rows of a stage: all of both pools, or (of four warps) a half of one pool
        const int row_lo = shared_copies ? (pwarp >> 1) * kHalf : 0, row_hi = shared_copies ? row_lo + kHalf : kKeys;
        const int r = lane;
        int stage = 0;
        uint32_t phase = 0;
        const uint64_t policy = dev::policy_evict_first();
        const int ps_mask = p.page_size - 1;
        uint32_t armed = 0, armed_par = 0;
        // page ids of the keys k + lane (, k + lane + 32) below k1 (0 past it)
        auto pages_of = [&](int32_t (&pg)[kPL], const int32_t* prow, int k, int k1) {
#pragma unroll
            for (int h = 0; h < kPL; ++h) pg[h] = k + r + 32 * h < k1 ? prow[(k + r + 32 * h) >> p.page_shift] : 0;
        };
        // a bad page id is flagged and read as page 0, which keeps the transaction count
        auto checked = [&](int32_t page) -> int64_t {
            if (page >= 0 && page < p.num_pages) return page;
            dev::set_error(err, kErrPage);
            return 0;
        };
        int u;
        DecUnit du{};
        int32_t pg[kPL];  // page ids of the coming stage's keys
#pragma unroll
        for (int h = 0; h < kPL; ++h) pg[h] = page_first_raw[h];
        int g_cur = g_first;
        if (static_first) {
            u = have_first ? (share > 0 ? 0 : (int)blockIdx.x) : n_units;
            if (u < n_units) du = du_first;
        } else {
            u = __shfl_sync(0xffffffffu, lane == 0 ? atomicAdd(sched, 1) : 0, 0);
            if (u < n_units) {
                du = units[u / n_hb];
                pages_of(pg, p.page_table + (int64_t)du.req * p.ld, du.k0, du.k1);
            }
        }
        while (true) {
            if (!wait_suspended(&sh->empty[stage], phase ^ 1, wlim, err)) break;
            if (u >= n_units) {
                if (lane == 0) {
                    if (pwarp == 0) sh->info[stage].flags = kEnd;
                    dev::mbar_arrive(&sh->full[stage]);
                }
                armed &= ~(1u << stage);
                break;
            }
            const int hb = u % n_hb;
            const int32_t* prow = p.page_table + (int64_t)du.req * p.ld;
            if (pwarp == 0) {
                const char* qbase = reinterpret_cast<const char*>(p.q + (int64_t)du.tok0 * Hq * D);
                const int qbytes = du.ntok * Hq * D * 2;
                for (int off = lane * 128; off < qbytes; off += 32 * 128)
                    asm volatile("prefetch.global.L2 [%0];" ::"l"(qbase + off));
            }
            const int nst = (du.k1 - du.k0 + kKeys - 1) / kKeys;
            int ticket = 0, u_next = n_units, g_next = g_cur;
            DecUnit du_next{};
            for (int si_ = 0; si_ < nst; ++si_) {
                const int k = du.k0 + si_ * kKeys;
                // the next unit: ticket, then its record, then its first page ids (see decode.cu)
                if (!shared_copies && share == 0 && si_ == max(nst - 4, 0) && lane == 0) ticket = sched_base + atomicAdd(sched, 1);
                if (si_ == max(nst - 2, 0)) {
                    if (share > 0) {
                        const int gn = g_cur + 1;
                        if (gn < n_groups && piece(gn, dgroups[gn], du_next)) {
                            u_next = 0;
                            g_next = gn;
                        }
                    } else {
                        u_next = shared_copies ? u + (int)gridDim.x : __shfl_sync(0xffffffffu, ticket, 0);
                        if (u_next < n_units) du_next = units[u_next / n_hb];
                    }
                }
                int32_t cur[kPL];
#pragma unroll
                for (int h = 0; h < kPL; ++h) cur[h] = pg[h];
                if (si_ < nst - 1) pages_of(pg, prow, k + kKeys, du.k1);
                else if (u_next < n_units) pages_of(pg, p.page_table + (int64_t)du_next.req * p.ld, du_next.k0, du_next.k1);
                if (si_ != 0 && !wait_suspended(&sh->empty[stage], phase ^ 1, wlim, err)) goto producer_done;
                const int nk = min(kKeys, du.k1 - k);
                if (lane == 0 && pwarp == 0) {
                    MxStage& si = sh->info[stage];
                    si.k = k;
                    si.k1 = du.k1;
                    si.tok0 = du.tok0;
                    si.ntok = du.ntok;
                    si.qpos0 = du.qpos0;
                    si.nparts = du.nparts;
                    si.slot = du.pbase + du.split;
                    si.hb = hb;
                    si.index = si_;
                    si.flags = (si_ == 0 ? kFirst : 0) | (si_ == nst - 1 ? kLast : 0);
                    si.next_tok0 = du_next.tok0;
                    si.next_ntok = u_next < n_units ? du_next.ntok : 0;
                    si.next_hb = u_next % n_hb;
                }
                const int rows = max(min(nk, row_hi) - row_lo, 0);  // this warp's, in each of its pools
                if (lane == 0) dev::mbar_arrive_expect_tx(&sh->full[stage], (uint32_t)((shared_copies ? 1 : 2) * rows * stride));
                armed |= 1u << stage;
                armed_par = (armed_par & ~(1u << stage)) | (phase << stage);
                __syncwarp();
#pragma unroll
                for (int h = 0; h < kPL; ++h) {
                    // with every head in the CTA the rows of one page are contiguous in the pool and in
                    // the stage, and the lane of a page's first row copies them all
                    const int row = r + 32 * h, in_page = (k + row) & ps_mask;
                    if (row < row_lo || row >= row_lo + rows || (n_hb == 1 && row != row_lo && in_page != 0)) continue;
                    const int64_t src = ((checked(cur[h]) << p.page_shift) + in_page) * p.mx_row_bytes + (int64_t)hb * stride;
                    const uint32_t bytes = (uint32_t)((n_hb == 1 ? min(p.page_size - in_page, row_lo + rows - row) : 1) * stride);
                    uint8_t* dst = ring + stage * stage_bytes + row * stride;
                    if (!shared_copies || (pwarp & 1) == 0)
                        dev::bulk_g2s_hint(dst, reinterpret_cast<const uint8_t*>(p.k_pool) + src, bytes, &sh->full[stage], policy);
                    if (!shared_copies || (pwarp & 1) == 1)
                        dev::bulk_g2s_hint(dst + kKeys * stride, reinterpret_cast<const uint8_t*>(p.v_pool) + src, bytes,
                                           &sh->full[stage], policy);
                }
                if (++stage == stages) {
                    stage = 0;
                    phase ^= 1;
                }
            }
            u = u_next;
            du = du_next;
            g_cur = g_next;
        }
    producer_done:
        // every copy issued must land before the CTA may exit.  (Where another producer gave up, a stage's
        // phase cannot complete: one such wait is long enough for all copies.)
        for (int s = 0; s < stages; ++s)
            if ((armed & (1u << s)) && !dev::mbar_wait(&sh->full[s], (armed_par >> s) & 1u)) break;
        if (wait_late) dev::grid_dep_wait();
        return;
    }

    // ==================================================================== consumers
    // A head's KW warps take a unit's stages in turn, each with its own running maximum, sum and
    // output; at the unit's end the others hand theirs to the first, which joins them.  (Computing
    // the next stage's scores among the products P V of the current one holds two of the ring's few
    // stages and measured no better: 53 us either way for 64 decodes, 67 against 54 for 16 heads of
    // D 64.)
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(MW::kRegsConsumer));
    if (warp >= consumers) return;
    const int gl = warp % HB;  // kv head within the CTA's
    const int kw = warp / HB;
    const int gq = lane >> 2;  // MMA row group: a key of S^T, a run of dims of O^T, a query row of Q / P
    const int cq = lane & 3;   // MMA column pair
    const int group_bytes = min(HB, 8) * (D / 2 + NB);
    const int code_at = (gl >> 3) * group_bytes + (gl & 7) * (D / 2);  // of the head in a staged row
    const int scale_at = (gl >> 3) * group_bytes + min(HB, 8) * (D / 2) + (gl & 7) * NB;
    uint4 qraw[NQ][NB];        // the coming unit's query rows as they lie in q
    uint32_t qb[NQ][NB][4];    // query rows: per block two k-steps of B fragments
    float s[kMT][NQ][4];       // scores of the warp's stage (in units of the row's scale sl), 16 keys a tile
    float o[OT][NQ][4];
    float m[NQ][2], l[NQ][2], sl[NQ][2];
    int lim[NQ][2];
    int stage = 0;             // the stage looked at; its phase
    uint32_t phase = 0, xphase = 0;

    // B fragments of query row 8n + gq: block b, k-step t, columns (2cq, 2cq+1 | +8, +9) <- dims
    // 32b + 8cq + 4t + (0, 1 | 2, 3), the order the K fragments come in
    auto load_q = [&](int tok0, int ntok, int hb) {
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
            const int r = 8 * n + gq;
            const uint16_t* src = p.q + ((int64_t)(tok0 + r / G) * Hq + (hb * HB + gl) * G + r % G) * D + 8 * cq;
#pragma unroll
            for (int b = 0; b < NB; ++b)
                qraw[n][b] = r < ntok * G ? *reinterpret_cast<const uint4*>(src + 32 * b) : make_uint4(0, 0, 0, 0);
        }
    };
    bool have_q = have_first;  // qraw holds the coming unit's rows
    if (have_first) load_q(du_first.tok0, du_first.ntok, share > 0 ? 0 : (int)blockIdx.x % n_hb);

    auto advance = [&] {
        if (++stage == stages) {
            stage = 0;
            phase ^= 1;
        }
    };
    auto release = [&](int st) {
        __syncwarp();
        if (lane == 0) dev::mbar_arrive(&sh->empty[st]);
    };
    // S^T = K Q^T of a stage's part (kPart keys from key `at` on)
    auto scores = [&](int st, int at) {
        const uint8_t* Ks = ring + st * stage_bytes + at * stride;
        // codes: [block][keys 0-7 | 8-15]; all loads first where there are registers for them
        constexpr bool kAhead = NQ == 1 && !MW::kMany;
        uint32_t kc[kAhead ? kMT : 1][NB][2];
        auto load_k = [&](int mt, uint32_t (&c)[NB][2]) {
            const uint32_t ka = dev::smem_u32(Ks) + (mt * 16 + (lane & 15)) * stride + code_at + (lane >> 4) * 16;
#pragma unroll
            for (int b = 0; b < NB; b += 2)
                dev::ldsm_x4(ka + b * 16, c[b][0], c[b][1], c[b + 1][0], c[b + 1][1]);
        };
        if constexpr (kAhead) {
#pragma unroll
            for (int mt = 0; mt < kMT; ++mt) load_k(mt, kc[mt]);
        }
#pragma unroll
        for (int mt = 0; mt < kMT; ++mt) {
            if constexpr (!kAhead) load_k(mt, kc[0]);
            const uint8_t* kr = Ks + (mt * 16 + gq) * stride + scale_at;
            float f0[NB], f1[NB];  // scales of keys gq, gq + 8
            mx::scales_f32<NB>(kr, f0);
            mx::scales_f32<NB>(kr + 8 * stride, f1);
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                const uint32_t(&w)[2] = kc[kAhead ? mt : 0][b];
                const uint32_t a0[4] = {mx::e2m1x2_to_f16x2<0>(w[0]), mx::e2m1x2_to_f16x2<0>(w[1]),
                                        mx::e2m1x2_to_f16x2<1>(w[0]), mx::e2m1x2_to_f16x2<1>(w[1])};
                const uint32_t a1[4] = {mx::e2m1x2_to_f16x2<2>(w[0]), mx::e2m1x2_to_f16x2<2>(w[1]),
                                        mx::e2m1x2_to_f16x2<3>(w[0]), mx::e2m1x2_to_f16x2<3>(w[1])};
#pragma unroll
                for (int n = 0; n < NQ; ++n) {
                    float c[4];
                    mma_f16_zero(c, a0, qb[n][b][0], qb[n][b][1]);
                    mma_f16(c, a1, qb[n][b][2], qb[n][b][3]);
                    float(&x)[4] = s[mt][n];
                    if (b == 0) {
                        x[0] = c[0] * f0[b], x[1] = c[1] * f0[b], x[2] = c[2] * f1[b], x[3] = c[3] * f1[b];
                    } else {
                        x[0] += c[0] * f0[b], x[1] += c[1] * f0[b], x[2] += c[2] * f1[b], x[3] += c[3] * f1[b];
                    }
                }
            }
        }
    };

    // Rows of several tokens see different keys, and a hidden key's weight 0 times a NaN block of V would
    // reach them all.  So in a part with the diagonal (n keys from key k, of stage st from `at` on) the NaN
    // blocks of the head become zeros in the stage, and the rows that see the first of a block's (every row
    // from its token on) take their NaN now: a sum that is one stays one.
    auto hide_nan = [&](int st, int at, int k, int n) {
        using Word = std::conditional_t<NB == 4, uint32_t, uint16_t>;  // a key's scale bytes
        uint8_t* e = ring + st * stage_bytes + (kKeys + at) * stride + scale_at;
        bool any = false;
        for (int x = lane; x < n; x += 32) any |= __vcmpeq4(*reinterpret_cast<Word*>(e + x * stride), 0xFFFFFFFFu) != 0;
        if (!__any_sync(0xffffffffu, any)) return;
        const uint8_t* mine = e + gq * (D / 8) / mx::kBlock;  // of the lane's dims
        int first = 0;
        while (first < n && mine[first * stride] != mx::kScaleNan) ++first;
#pragma unroll
        for (int nq = 0; nq < NQ; ++nq) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if (first == n || k + first > lim[nq][i]) continue;
#pragma unroll
                for (int t = 0; t < OT; ++t) o[t][nq][i] = o[t][nq][2 + i] = __int_as_float(0x7FFFFFFF);
            }
        }
        __syncwarp();  // every lane has looked
        for (int x = lane; x < n; x += 32) {
            Word* w = reinterpret_cast<Word*>(e + x * stride);
            *w &= (Word)~__vcmpeq4(*w, 0xFFFFFFFFu);
        }
        // (these stores come before the copy that fills the stage again)
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
    };

    while (true) {
        // the unit's first stage
        if (!wait_suspended(&sh->full[stage], phase, wlim, err)) return;
        MxStage si = sh->info[stage];
        if (si.flags & kEnd) break;
        const int rows = si.ntok * G;
        const int g = si.hb * HB + gl;
        bool last = (si.flags & kLast) != 0;  // no stage of the unit lies past `stage`
        // the warp's first stage of the unit
        for (int i = 0; i < kw && !last; ++i) {
            release(stage);
            advance();
            if (!wait_suspended(&sh->full[stage], phase, wlim, err)) return;
            si = sh->info[stage];
            last = (si.flags & kLast) != 0;
        }
        int cur = stage;
        const bool mine = si.index == kw;  // (else the unit has fewer stages than the head warps)
        if (mine) {
            if (!have_q) load_q(si.tok0, si.ntok, si.hb);
            have_q = false;
#pragma unroll
            for (int n = 0; n < NQ; ++n) {
                uint32_t amax = 0;
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    const uint32_t ww[4] = {qraw[n][b].x, qraw[n][b].y, qraw[n][b].z, qraw[n][b].w};
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        amax = max(amax, max((ww[i] << 16) & 0x7FFFFFFFu, ww[i] & 0x7FFF0000u));
                }
                amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
                amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
                const int ex = min(max((int)(amax >> 23), 1), 253);
                const float f = __uint_as_float((uint32_t)(254 - ex) << 23);
                const float qs = __uint_as_float((uint32_t)ex << 23);
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    const uint32_t ww[4] = {qraw[n][b].x, qraw[n][b].y, qraw[n][b].z, qraw[n][b].w};
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        qb[n][b][i] = dev::pack_f16x2(__uint_as_float(ww[i] << 16) * f,
                                                      __uint_as_float(ww[i] & 0xFFFF0000u) * f);
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int c = 2 * cq + i;  // score columns of the lane: query rows 8n + c
                    sl[n][i] = p.scale_log2 * __shfl_sync(0xffffffffu, qs, 4 * c);
                    m[n][i] = -INFINITY;
                    l[n][i] = 0.f;
                    lim[n][i] = 8 * n + c < rows ? si.qpos0 + (8 * n + c) / G : -1;
                }
#pragma unroll
                for (int t = 0; t < OT; ++t) o[t][n][0] = o[t][n][1] = o[t][n][2] = o[t][n][3] = 0.f;
            }
        }
        int at = 0;  // the warp's part of the stage
        while (mine) {
            const int k = si.k + at, k1 = si.k1;
            scores(cur, at);
            // a part that crosses the range's end or the first token's diagonal
            if (k + kPart > si.k1 || k + kPart - 1 > si.qpos0) {
#pragma unroll
                for (int n = 0; n < NQ; ++n) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int end = min(lim[n][e & 1], si.k1 - 1) - k - gq - 8 * (e >> 1);
#pragma unroll
                        for (int mt = 0; mt < kMT; ++mt)
                            if (mt * 16 > end) s[mt][n][e] = -INFINITY;
                    }
                }
                if (MULTI && si.ntok > 1) hide_nan(cur, at, k, min(kPart, k1 - k));
            }

            // ---- online softmax: P^T as f16, transposed to the next product's operand
            uint32_t pb[kMT][NQ][2];
#pragma unroll
            for (int n = 0; n < NQ; ++n) {
                // the reference m moves only when the row's maximum outgrows it by more than 2^kSlack (its
                // first stage: always): the weights stay below 2^kSlack, and o and l are rescaled rarely
                float mx[2];
                bool grows = false;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    mx[i] = fmaxf(s[0][n][i], s[0][n][2 + i]);
#pragma unroll
                    for (int mt = 1; mt < kMT; ++mt) mx[i] = dev::fmax3(mx[i], s[mt][n][i], s[mt][n][2 + i]);
                }
#pragma unroll
                for (int d = 4; d <= 16; d *= 2) {
                    mx[0] = fmaxf(mx[0], __shfl_xor_sync(0xffffffffu, mx[0], d));
                    mx[1] = fmaxf(mx[1], __shfl_xor_sync(0xffffffffu, mx[1], d));
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    mx[i] *= sl[n][i];  // (sl > 0)
                    grows |= mx[i] > m[n][i] + kSlack;
                }
                if (__any_sync(0xffffffffu, grows)) {
                    float al[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float mn = mx[i] > m[n][i] + kSlack ? mx[i] : m[n][i];
                        al[i] = mn == -INFINITY ? 1.f : dev::fast_exp2(m[n][i] - mn);
                        m[n][i] = mn;
                        l[n][i] *= al[i];
                    }
#pragma unroll
                    for (int t = 0; t < OT; ++t) {
                        o[t][n][0] *= al[0], o[t][n][1] *= al[1];
                        o[t][n][2] *= al[0], o[t][n][3] *= al[1];
                    }
                }
                float mu[2], sum[2] = {0.f, 0.f};
#pragma unroll
                for (int i = 0; i < 2; ++i) mu[i] = kPShift - (m[n][i] == -INFINITY ? 0.f : m[n][i]);
#pragma unroll
                for (int mt = 0; mt < kMT; ++mt) {
#pragma unroll
                    for (int h = 0; h < 4; h += 2) {
                        float e0, e1;
                        dev::ffma2(e0, e1, s[mt][n][h], s[mt][n][h + 1], sl[n][0], sl[n][1], mu[0], mu[1]);
                        e0 = dev::fast_exp2(e0);
                        e1 = dev::fast_exp2(e1);
                        dev::fadd2(sum[0], sum[1], e0, e1);
                        // (key gq, rows 2cq, 2cq+1) -> (row gq, keys 2cq, 2cq+1)
                        pb[mt][n][h / 2] = movmatrix_t(dev::pack_f16x2(e0, e1));
                    }
                }
                l[n][0] += sum[0];
                l[n][1] += sum[1];
            }

            if (kQAhead && last) {  // request the next unit's query rows
                have_q = si.next_ntok > 0;
                if (have_q) load_q(si.next_tok0, si.next_ntok, si.next_hb);
            }

            // ---- O^T += V^T P^T: the lane's keys 2cq, 2cq+1 | 2cq+8, 2cq+9, dims gq*D/8 .. +D/8-1
            const uint8_t* Vs = ring + cur * stage_bytes + (kKeys + at) * stride;
#pragma unroll
            for (int mt = 0; mt < kMT; ++mt) {
                uint32_t vw[4][VW], ve[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint8_t* vr = Vs + (mt * 16 + 2 * cq + (i & 1) + (i >> 1) * 8) * stride;
                    if constexpr (VW == 2) {
                        const uint2 w = *reinterpret_cast<const uint2*>(vr + code_at + gq * (D / 16));
                        vw[i][0] = w.x, vw[i][1] = w.y;
                    } else {
                        vw[i][0] = *reinterpret_cast<const uint32_t*>(vr + code_at + gq * (D / 16));
                    }
                    ve[i] = vr[scale_at + gq * (D / 8) / mx::kBlock];
                }
                if (k + kPart > k1) {
                    // a row past the range's end holds what an earlier stage left: scale 0 (its P is 0)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (k + mt * 16 + 2 * cq + (i & 1) + (i >> 1) * 8 >= k1) ve[i] = 0;
                }
                const uint32_t f01 = dev::pack_f16x2(mx::scale_f32(ve[0]), mx::scale_f32(ve[1]));
                const uint32_t f89 = dev::pack_f16x2(mx::scale_f32(ve[2]), mx::scale_f32(ve[3]));
#pragma unroll
                for (int w = 0; w < VW; ++w) {
                    // bytes (dim 2i: x, dim 2i + 1: y) holding two keys' codes
                    const uint32_t x01 = bitsel(vw[0][w], vw[1][w] * 16u, 0x0F0F0F0Fu);
                    const uint32_t y01 = bitsel(vw[0][w] >> 4, vw[1][w], 0x0F0F0F0Fu);
                    const uint32_t x89 = bitsel(vw[2][w], vw[3][w] * 16u, 0x0F0F0F0Fu);
                    const uint32_t y89 = bitsel(vw[2][w] >> 4, vw[3][w], 0x0F0F0F0Fu);
                    auto tile = [&](auto byte) {
                        constexpr int B = decltype(byte)::value;
                        const uint32_t a[4] = {
                            mx::mul_f16x2(mx::e2m1x2_to_f16x2<B>(x01), f01), mx::mul_f16x2(mx::e2m1x2_to_f16x2<B>(y01), f01),
                            mx::mul_f16x2(mx::e2m1x2_to_f16x2<B>(x89), f89), mx::mul_f16x2(mx::e2m1x2_to_f16x2<B>(y89), f89)};
#pragma unroll
                        for (int n = 0; n < NQ; ++n) mma_f16(o[4 * w + B][n], a, pb[mt][n][0], pb[mt][n][1]);
                    };
                    tile(IntTag<0>{});
                    tile(IntTag<1>{});
                    tile(IntTag<2>{});
                    tile(IntTag<3>{});
                }
            }
            // ---- the warp's next part: of this stage, or of its next stage of the unit
            if (kPart < kKeys && at + kPart < kKeys && k + kPart < k1) {
                at += kPart;
                continue;
            }
            at = 0;
            bool more = !last;
            for (int i = 0; i < KW && more; ++i) {
                release(stage);  // (the first is the warp's own, the others other warps')
                advance();
                if (!wait_suspended(&sh->full[stage], phase, wlim, err)) return;
                si = sh->info[stage];
                last = (si.flags & kLast) != 0;
                if (i < KW - 1) more = !last;
            }
            if (!more) break;
            cur = stage;
        }
        release(stage);  // the unit's last
        advance();
        const int parts = min(KW, si.index + 1);  // warps that had a stage of the unit
        if (!kQAhead) {
            have_q = false;  // (a warp without a stage of the unit still holds its rows)
        } else if (!have_q || !mine) {
            have_q = si.next_ntok > 0;
            if (have_q) load_q(si.next_tok0, si.next_ntok, si.next_hb);
        }

        // ================================================================ the head's warps' join
        if (KW > 1) {
            constexpr int kVals = OT * 4 * NQ + 4 * NQ;
            auto area = [&](int w) {
                return reinterpret_cast<float*>(smem + sp.exch) + ((int64_t)(w - 1) * HB + gl) * (kVals * 32) + lane;
            };
            if (kw > 0) {
                // the area is free once the first warp has taken the unit before
                if (!wait_suspended(&sh->xempty[gl], xphase ^ 1, wlim, err)) return;
                if (kw < parts) {
                    float* x = area(kw);
#pragma unroll
                    for (int n = 0; n < NQ; ++n) {
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            x[(4 * n + i) * 32] = m[n][i];
                            x[(4 * n + 2 + i) * 32] = l[n][i];
                        }
#pragma unroll
                        for (int t = 0; t < OT; ++t)
#pragma unroll
                            for (int e = 0; e < 4; ++e) x[(4 * NQ + (n * OT + t) * 4 + e) * 32] = o[t][n][e];
                    }
                }
                __syncwarp();
                if (lane == 0) dev::mbar_arrive(&sh->xfull[gl]);
                xphase ^= 1;
                continue;
            }
            if (!wait_suspended(&sh->xfull[gl], xphase, wlim, err)) return;
            for (int w = 1; w < parts; ++w) {
                const float* x = area(w);
#pragma unroll
                for (int n = 0; n < NQ; ++n) {
                    float a0[2], a1[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float mo = x[(4 * n + i) * 32], lo = x[(4 * n + 2 + i) * 32];
                        const float mn = fmaxf(m[n][i], mo), mu = mn == -INFINITY ? 0.f : mn;
                        a0[i] = dev::fast_exp2(m[n][i] - mu);
                        a1[i] = dev::fast_exp2(mo - mu);
                        m[n][i] = mn;
                        l[n][i] = l[n][i] * a0[i] + lo * a1[i];
                    }
#pragma unroll
                    for (int t = 0; t < OT; ++t)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            o[t][n][e] = o[t][n][e] * a0[e & 1] + x[(4 * NQ + (n * OT + t) * 4 + e) * 32] * a1[e & 1];
                }
            }
            __syncwarp();
            if (lane == 0) dev::mbar_arrive(&sh->xempty[gl]);
            xphase ^= 1;
        }

        // ================================================================ unit epilogue
        // dim gq*D/8 + 2t (+1) of query row 8n + 2cq + i: o[t][n][i] (o[t][n][2 + i])
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float lt = l[n][i];
                lt += __shfl_xor_sync(0xffffffffu, lt, 4);
                lt += __shfl_xor_sync(0xffffffffu, lt, 8);
                lt += __shfl_xor_sync(0xffffffffu, lt, 16);
                const int r = 8 * n + 2 * cq + i;
                if (r >= rows) continue;
                const float inv = lt > 0.f ? 1.f / lt : lt;  // (a NaN stays one)
                const float lse = lt > 0.f ? m[n][i] + (__log2f(lt) - kPShift) : (lt == 0.f ? -INFINITY : lt);  // log2 domain
                if (si.nparts == 1) {
                    const int64_t orow = (int64_t)(si.tok0 + r / G) * Hq + g * G + r % G;
                    uint4* d4 = reinterpret_cast<uint4*>(p.out + orow * D + gq * (D / 8));
#pragma unroll
                    for (int t = 0; t < OT; t += 4)
                        d4[t / 4] = make_uint4(dev::pack_bf16x2(o[t][n][i] * inv, o[t][n][2 + i] * inv),
                                               dev::pack_bf16x2(o[t + 1][n][i] * inv, o[t + 1][n][2 + i] * inv),
                                               dev::pack_bf16x2(o[t + 2][n][i] * inv, o[t + 2][n][2 + i] * inv),
                                               dev::pack_bf16x2(o[t + 3][n][i] * inv, o[t + 3][n][2 + i] * inv));
                    if (p.lse != nullptr && gq == 0) p.lse[orow] = lse * kLn2;
                } else {
                    // split group: fp32 partial (normalised O, log2 LSE) for the merge kernel
                    const int64_t slot = (int64_t)si.slot * p.lay.rows_per_slot;
                    const int prow = (r / G) * Hq + g * G + r % G;
                    float4* d4 = reinterpret_cast<float4*>(reinterpret_cast<float*>(p.ws + p.lay.partial_o) +
                                                           (slot + prow) * D + gq * (D / 8));
#pragma unroll
                    for (int t = 0; t < OT; t += 2)
                        d4[t / 2] = make_float4(o[t][n][i] * inv, o[t][n][2 + i] * inv, o[t + 1][n][i] * inv,
                                                o[t + 1][n][2 + i] * inv);
                    if (gq == 0) reinterpret_cast<float*>(p.ws + p.lay.partial_lse)[slot + prow] = lse;
                }
            }
        }
    }
}

// K8: log-sum-exp join of a group's partials (and of the prefix-pass partials of shared-prefix
// members), as merge_kernel in decode.cu, for many parts over few rows: a long request alone is
// cut into as many parts as there are decode CTAs, and one warp per row read them one after
// another (128 parts of 32 rows: 28 us; here 5).  kW warps share a row, each joins every kW-th
// part with loads of several parts in flight, and the row's warps are joined through shared
// memory, in a fixed order.  kW follows the plan's parts per group: 1 up to 4 (the rows of many
// groups fill the SMs by themselves), 4 up to 16, else 16.  Layer calls in a graph with 1 / 4 / 16:
// 64 decodes (3 parts) 50.5 / 56.2 / 73.4 us, 61 decodes of 16 / 1 heads 39.1 / 41.0 / 51.0, 5 long
// requests (30 parts) 56.9 / 53.1 / 53.3, 1 x 16 k keys (147 parts) 36.0 / 22.4 / 18.8; near the second
// limit four would do (8 decodes, 19 parts: 23.6 / 21.2 / 24.1).
constexpr int kJoinWarps = 16;

template <int D>
__global__ void __launch_bounds__(32 * kJoinWarps) join_kernel(const ForwardParams p) {
    constexpr int C = D / 32;  // output columns per lane
    __shared__ float s_acc[kJoinWarps][D];
    __shared__ float2 s_ml[kJoinWarps];
    dev::grid_dep_launch();
    PlanHeader* hdr = reinterpret_cast<PlanHeader*>(p.ws + p.lay.header);
    const int n_groups = hdr->n_dec_groups, n_parts = hdr->n_partial_slots;
    if ((hdr->error_bits & kErrFatal) || n_groups == 0 || n_parts == 0) {
        dev::grid_dep_wait();
        return;
    }
    const DecGroup* groups = reinterpret_cast<const DecGroup*>(p.ws + p.lay.dec_groups);
    const float* plse = reinterpret_cast<const float*>(p.ws + p.lay.partial_lse);
    const float* pout = reinterpret_cast<const float*>(p.ws + p.lay.partial_o);
    const int rps = p.lay.rows_per_slot, Hq = p.num_qo_heads;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int kw = n_parts <= 4 * n_groups ? 1 : n_parts <= 16 * n_groups ? 4 : 16;
    const int rows_cta = kJoinWarps / kw, wi = warp % kw;  // rows a CTA joins at a time; the warp's place in its row
    const int chunks = (min(rps, max(hdr->max_group_tokens, 1) * Hq) + rows_cta - 1) / rows_cta;
    const int n_items = n_groups * chunks;
    DecGroup dg_next{};
    if ((int)blockIdx.x < n_items) dg_next = groups[blockIdx.x % n_groups];
    dev::grid_dep_wait();
    for (int it = blockIdx.x; it < n_items; it += gridDim.x) {
        const DecGroup dg = dg_next;
        if (it + (int)gridDim.x < n_items) dg_next = groups[(it + gridDim.x) % n_groups];
        const int np = dg.nparts;
        const int row = (it / n_groups) * rows_cta + warp / kw;
        const bool live = np > 1 && row < dg.ntok * Hq;
        float m = -INFINITY, l = 0.f, acc[C];
#pragma unroll
        for (int c = 0; c < C; ++c) acc[c] = 0.f;
        if (live) {
            const float* plb = plse + (int64_t)dg.pbase * rps + row;
            const float* pob = pout + ((int64_t)dg.pbase * rps + row) * D + lane * C;
            // parts wi, wi + kw, ...: 32 a round, lane s holding the s-th one's LSE
            for (int s0 = wi; s0 < np; s0 += 32 * kw) {
                const int mine = s0 + lane * kw;
                const float ls = mine < np ? __ldcg(plb + (int64_t)mine * rps) : -INFINITY;
                const int cnt = min(32, (np - s0 + kw - 1) / kw);
                float mr = ls;
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) mr = fmaxf(mr, __shfl_xor_sync(0xffffffffu, mr, o));
                const float mn = fmaxf(m, mr), mu = mn == -INFINITY ? 0.f : mn;
                const float al = dev::fast_exp2(m - mu);
                const float w = mine < np ? dev::fast_exp2(ls - mu) : 0.f;
                float ws = w;
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) ws += __shfl_xor_sync(0xffffffffu, ws, o);
                m = mn;
                l = l * al + ws;
#pragma unroll
                for (int c = 0; c < C; ++c) acc[c] *= al;
                const float* src = pob + (int64_t)s0 * rps * D;
                const int64_t step = (int64_t)kw * rps * D;
#pragma unroll 1
                for (int k0 = 0; k0 < cnt; k0 += 4) {
                    float v[4][C];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float* sp = src + (k0 + k) * step;
#pragma unroll
                        for (int c = 0; c < C; ++c) v[k][c] = 0.f;
                        if (k0 + k < cnt) {
                            if constexpr (C == 4) {
                                const float4 x = __ldcg(reinterpret_cast<const float4*>(sp));
                                v[k][0] = x.x, v[k][1] = x.y, v[k][2] = x.z, v[k][3] = x.w;
                            } else {
                                const float2 x = __ldcg(reinterpret_cast<const float2*>(sp));
                                v[k][0] = x.x, v[k][1] = x.y;
                            }
                        }
                    }
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float wk = __shfl_sync(0xffffffffu, w, (k0 + k) & 31);
                        if (k0 + k < cnt) {
#pragma unroll
                            for (int c = 0; c < C; ++c) acc[c] += wk * v[k][c];
                        }
                    }
                }
            }
        }
        if (kw > 1) {  // the row's other warps, in order
            __syncthreads();
            if (lane == 0) s_ml[warp] = make_float2(m, l);
#pragma unroll
            for (int c = 0; c < C; ++c) s_acc[warp][lane * C + c] = acc[c];
            __syncthreads();
            if (wi != 0 || !live) continue;
            float mx = m;
            for (int w = 1; w < kw; ++w) mx = fmaxf(mx, s_ml[warp + w].x);
            const float mu = mx == -INFINITY ? 0.f : mx;
            const float a0 = dev::fast_exp2(m - mu);
            l *= a0;
#pragma unroll
            for (int c = 0; c < C; ++c) acc[c] *= a0;
            for (int w = 1; w < kw; ++w) {
                const float2 ml = s_ml[warp + w];
                const float a = dev::fast_exp2(ml.x - mu);
                l += ml.y * a;
#pragma unroll
                for (int c = 0; c < C; ++c) acc[c] += a * s_acc[warp + w][lane * C + c];
            }
            m = mu;
        }
        if (!live) continue;
        const float inv = l > 0.f ? 1.f / l : l;  // (a NaN stays one)
        const int64_t orow = (int64_t)(dg.tok0 + row / Hq) * Hq + row % Hq;
        uint32_t* dst = reinterpret_cast<uint32_t*>(p.out + orow * D + lane * C);
#pragma unroll
        for (int c = 0; c < C; c += 2) dst[c / 2] = dev::pack_bf16x2(acc[c] * inv, acc[c + 1] * inv);
        if (p.lse != nullptr && lane == 0)
            p.lse[orow] = l > 0.f ? (m + __log2f(l)) * kLn2 : (l == 0.f ? -INFINITY : l);
    }
}

template <int D, int NQ, int HBT, bool MULTI>
cudaError_t launch_h(const ForwardParams& p, int producers, int ctas, cudaStream_t s) {
    const int Hkv = p.num_kv_heads;
    MxShape sp{};
    sp.hb = decode_mx_heads(Hkv, D, 8 * NQ);
    sp.kw = MxWarps<D, NQ>::kConsumers / sp.hb;
    sp.kw = sp.kw < 8 ? sp.kw : 8;
    sp.stride = mx_stride(sp.hb, D);  // (of a block of heads, or of all: then the pool's row)
    sp.producers = producers;
    const int head = (int)((sizeof(MxSmem) + 127) / 128 * 128);
    const int stage_bytes = 2 * mx_stage_keys(NQ) * sp.stride;
    int exch = 0;
    for (;; --sp.kw) {
        exch = (sp.kw - 1) * sp.hb * (D / 4 + 4) * NQ * 128;
        sp.stages = (kSmemLimit - 1024 - head - exch) / stage_bytes;
        sp.stages = sp.stages > kMaxStages ? kMaxStages : sp.stages;
        // a warp holds a stage while it waits for its next one, kw stages on
        if (sp.kw == 1 || sp.kw <= sp.stages - 2) break;
    }
    if (sp.stages < 2) return cudaErrorInvalidConfiguration;
    sp.exch = head + sp.stages * stage_bytes;
    const size_t smem = (size_t)sp.exch + exch;
    // the register split inside the kernel assumes the launch allocates exactly kRegsLaunch a thread
    static std::atomic<int> launch_regs{-1};
    if (launch_regs.load(std::memory_order_relaxed) < 0) {
        cudaFuncAttributes attr{};
        const cudaError_t ea = cudaFuncGetAttributes(&attr, decode_mx_kernel<D, NQ, HBT, MULTI>);
        if (ea != cudaSuccess) return ea;
        launch_regs.store(attr.numRegs, std::memory_order_relaxed);
    }
    if (launch_regs.load(std::memory_order_relaxed) != MxWarps<D, NQ>::kRegsLaunch) return cudaErrorInvalidConfiguration;
    // (the bound, not this call's size: another thread may be launching another head layout of the kernel)
    const cudaError_t e = cudaFuncSetAttribute(decode_mx_kernel<D, NQ, HBT, MULTI>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit);
    if (e != cudaSuccess) return e;
    return launch_programmatic(decode_mx_kernel<D, NQ, HBT, MULTI>, (unsigned)ctas, (unsigned)MxWarps<D, NQ>::kThreads, smem, s, p, sp);
}

template <int D, bool MULTI>
cudaError_t launch_dec(const ForwardParams& p, int ctas, cudaStream_t s) {
    const int hb = decode_mx_heads(p.num_kv_heads, D, p.dec_rows);
    // One warp issues a bulk copy in about 70 cycles whatever its size, so copies of one or a few
    // rows (small pages, or a block of the heads) are shared by four: 40 requests of up to 4000
    // one-slot pages, 16 heads of D 64: 42 us a layer call, against 54 with 16-byte async copies by
    // four warps.
    const int run = hb < p.num_kv_heads ? mx_stride(hb, D) : p.page_size * p.mx_row_bytes;
    const int producers = run < 2048 ? 4 : 1;
    if (p.dec_rows > 8)
        return hb == 8 ? launch_h<D, 2, 8, MULTI>(p, producers, ctas, s) : launch_h<D, 2, 0, MULTI>(p, producers, ctas, s);
    switch (hb) {
        case 1: return launch_h<D, 1, 1, MULTI>(p, producers, ctas, s);
        case 2: return launch_h<D, 1, 2, MULTI>(p, producers, ctas, s);
        case 4: return launch_h<D, 1, 4, MULTI>(p, producers, ctas, s);
        case 8: return launch_h<D, 1, 8, MULTI>(p, producers, ctas, s);
    }
    if constexpr (D == 64)
        if (hb == 16) return launch_h<D, 1, 16, MULTI>(p, producers, ctas, s);
    return launch_h<D, 1, 0, MULTI>(p, producers, ctas, s);
}

}  // namespace

// kv heads a decode CTA serves: all of them, or a block of them when its warps are fewer.
int decode_mx_heads(int num_kv_heads, int head_dim, int rows) {
    if (num_kv_heads <= kDecHeadBlock) return num_kv_heads;
    return rows <= 8 && head_dim == 64 && num_kv_heads % 16 == 0 ? 16 : kDecHeadBlock;
}

cudaError_t launch_join_mx(const ForwardParams& p, int head_dim, int ctas, cudaStream_t s) {
    if (head_dim == 128) return launch_programmatic(join_kernel<128>, (unsigned)ctas, 32u * kJoinWarps, 0, s, p);
    if (head_dim == 64) return launch_programmatic(join_kernel<64>, (unsigned)ctas, 32u * kJoinWarps, 0, s, p);
    return cudaErrorInvalidValue;
}

cudaError_t launch_decode_mx(const ForwardParams& p, int head_dim, int ctas, cudaStream_t s) {
    const bool multi = p.dec_rows > p.group;
    if (head_dim == 128) return multi ? launch_dec<128, true>(p, ctas, s) : launch_dec<128, false>(p, ctas, s);
    if (head_dim == 64) return multi ? launch_dec<64, true>(p, ctas, s) : launch_dec<64, false>(p, ctas, s);
    return cudaErrorInvalidValue;
}

}  // namespace pva

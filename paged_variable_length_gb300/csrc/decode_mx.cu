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
// largest element to [1, 2) (undone in the softmax scale), so that its range is bf16's; P is
// rounded to f16 (2^-11 of a weight, below the output's bf16 rounding; kPShift), sums are fp32.
// Every wait is bounded, as in decode.cu.
#include <cuda_runtime.h>

#include "decode_common.cuh"
#include "device_utils.cuh"
#include "mxfp4.cuh"
#include "pva_internal.h"

namespace pva {
namespace {

constexpr int kKeys = 64;  // keys per ring stage
constexpr int kMT = kKeys / 16;
constexpr float kLn2 = 0.69314718055994530942f;
// P enters its f16 operand as 2^15 times the weight: the largest weight (1) stays below f16's
// maximum, and weights down to 2^-29 of it keep all of f16's bits.
constexpr float kPShift = 15.f;

__device__ __forceinline__ uint32_t movmatrix_t(uint32_t x) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

// D = A B (m16n8k16, f16 in, fp32 out).
__device__ __forceinline__ void mma_f16_zero(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%10,%10,%10,%10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

// (a & m) | (b & ~m)
__device__ __forceinline__ uint32_t bitsel(uint32_t a, uint32_t b, uint32_t m) {
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xE4;" : "=r"(r) : "r"(a), "r"(b), "r"(m));
    return r;
}

// Barriers of the CTA beyond the ring's: a head's warps hand their partial results to its first.
struct MxSmem {
    DecSmemHead ring;
    uint64_t xfull[kDecHeadBlock], xempty[kDecHeadBlock];
};

// Launch shape: heads of a CTA (hb), consumer warps a head (kw), producer warps (pw), ring stages.
struct MxShape {
    int hb, kw, pw, stages, stride;
    int exch;  // byte offset of the exchange area
};

// Consumer warps of a CTA, one CTA an SM: the wider head and the wider row tile have registers for
// eight.
constexpr __host__ __device__ int mx_consumers(int D, int NQ) { return D == 64 && NQ == 1 ? 16 : 8; }

// D: head dim.  NQ: n8 tiles of query rows (rows of the batch's decode groups <= 8 NQ).  CP: the
// producers copy rows with 16-byte async copies (small pages) instead of one bulk copy a page run.
template <int D, int NQ, bool CP>
__global__ void __launch_bounds__(32 * (mx_consumers(D, NQ) + 2), 1) decode_mx_kernel(const ForwardParams p, const MxShape sp) {
    constexpr int NB = D / mx::kBlock;  // blocks of a head
    constexpr int OT = D / 16;          // m16 tiles of the output dims
    constexpr int VW = D / 64;          // words of a lane's run of V codes (D/8 dims)
    extern __shared__ __align__(128) uint8_t smem[];
    MxSmem* xs = reinterpret_cast<MxSmem*>(smem);
    DecSmemHead* sh = &xs->ring;
    uint8_t* ring = smem + ((sizeof(MxSmem) + 127) / 128) * 128;
    PlanHeader* hdr = reinterpret_cast<PlanHeader*>(p.ws + p.lay.header);
    uint32_t* err = &hdr->error_bits;
    const uint64_t wlim = dev::wait_limit(hdr->wait_override);

    const int Hkv = p.num_kv_heads, G = p.group, Hq = p.num_qo_heads;
    const int HB = sp.hb, KW = sp.kw, stages = sp.stages, stride = sp.stride;
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
    // CP: several producer warps walk the units alike, so a queue's units go round the CTAs in
    // turn (they are listed longest first) instead of through the counter
    const bool static_first = CP || !wait_late || share > 0;
    DecUnit du_first{};
    bool have_first = false;
    int g_first = -1;
    int32_t page_first_raw[2] = {0, 0};  // of the stage's keys lane, lane + 32
    if (static_first && warp >= consumers) {
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
        for (int h = 0; h < 2; ++h) {
            const int key = du_first.k0 + lane + 32 * h;
            if (have_first && key < du_first.k1)
                page_first_raw[h] = p.page_table[(int64_t)du_first.req * p.ld + (key >> p.page_shift)];
        }
    }
    if (threadIdx.x == 0) {
        for (int s = 0; s < stages; ++s) {
            dev::mbar_init(&sh->full[s], CP ? 32 * sp.pw + 1 : 1);
            dev::mbar_init(&sh->empty[s], consumers);
        }
        for (int h = 0; h < kDecHeadBlock; ++h) {
            dev::mbar_init(&xs->xfull[h], KW > 1 ? KW - 1 : 1);
            dev::mbar_init(&xs->xempty[h], 1);
        }
        sh->abort_flag = 0;
        dev::fence_barrier_init();
    }
    __syncthreads();
    if (!wait_late) dev::grid_dep_wait();

    int32_t* sched = &hdr->pad[0];
    const int sched_base = static_first ? (int)gridDim.x : 0;

    if (warp >= consumers) {
        // ================================================================ producers
        const int pwarp = warp - consumers;  // CP: 0 copies K rows, 1 V rows
        const int r = lane;
        int stage = 0;
        uint32_t phase = 0;
        const uint64_t policy = dev::policy_evict_first();
        const int ps_mask = p.page_size - 1;
        uint32_t armed = 0, armed_par = 0;
        // page ids of the keys k + lane, k + lane + 32 below k1 (0 past it)
        auto pages_of = [&](int32_t (&pg)[2], const int32_t* prow, int k, int k1) {
#pragma unroll
            for (int h = 0; h < 2; ++h) pg[h] = k + r + 32 * h < k1 ? prow[(k + r + 32 * h) >> p.page_shift] : 0;
        };
        // a bad page id is flagged and read as page 0, which keeps the transaction count
        auto checked = [&](int32_t page) -> int64_t {
            if (page >= 0 && page < p.num_pages) return page;
            dev::set_error(err, kErrPage);
            return 0;
        };
        // CP: this thread's copies into the stage complete its arrival
        auto arrive_copies = [&](int st) {
            asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(dev::smem_u32(&sh->full[st])) : "memory");
        };
        const int nch = stride / 16, ch_q = 32 / nch, ch_r = 32 % nch;  // CP: 16-byte chunks of a row
        int u;
        DecUnit du{};
        int32_t pg[2] = {page_first_raw[0], page_first_raw[1]};  // page ids of the coming stage's keys
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
            if (!warp_wait(&sh->empty[stage], phase ^ 1, wlim, sh, err)) break;
            if (u >= n_units) {
                if (lane == 0 && pwarp == 0) {
                    sh->info[stage].flags = kEnd;
                    dev::mbar_arrive(&sh->full[stage]);
                }
                if constexpr (CP) arrive_copies(stage);
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
                if (!CP && share == 0 && si_ == max(nst - 4, 0) && lane == 0) ticket = sched_base + atomicAdd(sched, 1);
                if (si_ == max(nst - 2, 0)) {
                    if (share > 0) {
                        const int gn = g_cur + 1;
                        if (gn < n_groups && piece(gn, dgroups[gn], du_next)) {
                            u_next = 0;
                            g_next = gn;
                        }
                    } else {
                        u_next = CP ? u + (int)gridDim.x : __shfl_sync(0xffffffffu, ticket, 0);
                        if (u_next < n_units) du_next = units[u_next / n_hb];
                    }
                }
                const int32_t cur[2] = {pg[0], pg[1]};
                if (si_ < nst - 1) pages_of(pg, prow, k + kKeys, du.k1);
                else if (u_next < n_units) pages_of(pg, p.page_table + (int64_t)du_next.req * p.ld, du_next.k0, du_next.k1);
                if (si_ != 0 && !warp_wait(&sh->empty[stage], phase ^ 1, wlim, sh, err)) goto producer_done;
                const int nk = min(kKeys, du.k1 - k);
                if (lane == 0 && pwarp == 0) {
                    StageInfo& si = sh->info[stage];
                    si.unit = u;
                    si.group = du.group;
                    si.k = k;
                    si.k1 = du.k1;
                    si.tok0 = du.tok0;
                    si.ntok = du.ntok;
                    si.qpos0 = du.qpos0;
                    si.nsplit = du.nsplit;
                    si.pbase = du.pbase;
                    si.split = du.split;
                    si.hb = hb;
                    si.nparts = du.nparts;
                    si.index = si_;
                    si.flags = (si_ == 0 ? kFirst : 0) | (si_ == nst - 1 ? kLast : 0);
                    if constexpr (CP) dev::mbar_arrive(&sh->full[stage]);
                    else dev::mbar_arrive_expect_tx(&sh->full[stage], (uint32_t)(2 * nk * stride));
                }
                armed |= 1u << stage;
                armed_par = (armed_par & ~(1u << stage)) | (phase << stage);
                __syncwarp();
                uint32_t slot[2];  // of the keys k + lane, k + lane + 32 (a pool has fewer than 2^32)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    slot[h] = r + 32 * h < nk ? (uint32_t)((checked(cur[h]) << p.page_shift) + ((k + r + 32 * h) & ps_mask)) : 0u;
                if constexpr (CP) {
                    // this warp's pool: rows 0 .. nk-1 of the stage, their chunks dealt to the lanes in order
                    const uint8_t* pool = reinterpret_cast<const uint8_t*>(pwarp ? p.v_pool : p.k_pool) + (int64_t)hb * stride;
                    const uint32_t dst = dev::smem_u32(ring) + stage * stage_bytes + pwarp * kKeys * stride;
                    int row = lane / nch, ch = lane % nch;
                    for (int e = 0; e < nk * nch; e += 32) {
                        const uint32_t s0 = __shfl_sync(0xffffffffu, slot[0], row & 31);
                        const uint32_t s1 = __shfl_sync(0xffffffffu, slot[1], row & 31);
                        if (row < nk)
                            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + row * stride + ch * 16),
                                         "l"(pool + (int64_t)(row < 32 ? s0 : s1) * p.mx_row_bytes + ch * 16));
                        row += ch_q;
                        ch += ch_r;
                        if (ch >= nch) ch -= nch, ++row;
                    }
                    arrive_copies(stage);
                } else {
                    // every head in the CTA: the rows of one page are contiguous in the pool and in the
                    // stage, and the lane of a page's first row copies them all
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int row = r + 32 * h, in_page = (k + row) & ps_mask;
                        if (row < nk && (row == 0 || in_page == 0)) {
                            const int64_t src = (int64_t)slot[h] * p.mx_row_bytes;
                            const uint32_t bytes = (uint32_t)(min(p.page_size - in_page, nk - row) * stride);
                            uint8_t* dst = ring + stage * stage_bytes + row * stride;
                            dev::bulk_g2s_hint(dst, reinterpret_cast<const uint8_t*>(p.k_pool) + src, bytes,
                                               &sh->full[stage], policy);
                            dev::bulk_g2s_hint(dst + kKeys * stride, reinterpret_cast<const uint8_t*>(p.v_pool) + src,
                                               bytes, &sh->full[stage], policy);
                        }
                    }
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
        // every copy issued must land before the CTA may exit
        if constexpr (CP) {
            asm volatile("cp.async.wait_all;" ::: "memory");
        } else {
            for (int s = 0; s < stages; ++s)
                if (armed & (1u << s)) (void)dev::mbar_wait(&sh->full[s], (armed_par >> s) & 1u);
        }
        if (wait_late) dev::grid_dep_wait();
        return;
    }

    // ==================================================================== consumers
    // A head's KW warps take a unit's stages in turn, each with its own running maximum, sum and
    // output; at the unit's end the others hand theirs to the first, which joins them.
    const int gl = warp % HB;  // kv head within the CTA's
    const int kw = warp / HB;
    const int gq = lane >> 2;  // MMA row group: a key of S^T, a run of dims of O^T, a query row of Q / P
    const int cq = lane & 3;   // MMA column pair
    const int group_bytes = min(HB, 8) * (D / 2 + NB);
    const int code_at = (gl >> 3) * group_bytes + (gl & 7) * (D / 2);  // of the head in a staged row
    const int scale_at = (gl >> 3) * group_bytes + min(HB, 8) * (D / 2) + (gl & 7) * NB;
    uint32_t qb[NQ][NB][4];    // query rows: per block two k-steps of B fragments
    float o[OT][NQ][4];
    float m[NQ][2], l[NQ][2], sl[NQ][2];
    int lim[NQ][2];
    int stage = 0;
    uint32_t phase = 0, xphase = 0;

    while (true) {
        if (!warp_wait(&sh->full[stage], phase, wlim, sh, err)) return;
        const StageInfo si = sh->info[stage];
        if (si.flags & kEnd) break;
        const int rows = si.ntok * G;
        const int g = si.hb * HB + gl;
        if (si.index == kw) {  // the warp's first stage of the unit
#pragma unroll
            for (int n = 0; n < NQ; ++n) {
                // B fragments of query row 8n + gq: block b, k-step t, columns (2cq, 2cq+1 | +8, +9) <-
                // dims 32b + 8cq + 4t + (0, 1 | 2, 3), the order the K fragments come in
                const int r = 8 * n + gq;
                uint4 w[NB];
                uint32_t amax = 0;
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    w[b] = make_uint4(0, 0, 0, 0);
                    if (r < rows)
                        w[b] = *reinterpret_cast<const uint4*>(
                            p.q + ((int64_t)(si.tok0 + r / G) * Hq + g * G + r % G) * D + 32 * b + 8 * cq);
                    const uint32_t ww[4] = {w[b].x, w[b].y, w[b].z, w[b].w};
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
                    const uint32_t ww[4] = {w[b].x, w[b].y, w[b].z, w[b].w};
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
        if (si.index % KW == kw) {
            const uint8_t* Ks = ring + stage * stage_bytes;
            const uint8_t* Vs = Ks + kKeys * stride;
            // ---- S^T = K Q^T, 16 keys a tile (in units of the row's scale sl)
            float s[kMT][NQ][4];
#pragma unroll
            for (int mt = 0; mt < kMT; ++mt) {
                const uint32_t ka = dev::smem_u32(Ks) + (mt * 16 + (lane & 15)) * stride + code_at + (lane >> 4) * 16;
                const uint8_t* kr = Ks + (mt * 16 + gq) * stride + scale_at;
                float f0[NB], f1[NB];  // scales of keys gq, gq + 8
                mx::scales_f32<NB>(kr, f0);
                mx::scales_f32<NB>(kr + 8 * stride, f1);
#pragma unroll
                for (int b2 = 0; b2 < NB; b2 += 2) {
                    uint32_t w[2][2];  // [block][keys 0-7 | 8-15]
                    dev::ldsm_x4(ka + b2 * 16, w[0][0], w[0][1], w[1][0], w[1][1]);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int b = b2 + i;
                        const uint32_t a0[4] = {mx::e2m1x2_to_f16x2<0>(w[i][0]), mx::e2m1x2_to_f16x2<0>(w[i][1]),
                                                mx::e2m1x2_to_f16x2<1>(w[i][0]), mx::e2m1x2_to_f16x2<1>(w[i][1])};
                        const uint32_t a1[4] = {mx::e2m1x2_to_f16x2<2>(w[i][0]), mx::e2m1x2_to_f16x2<2>(w[i][1]),
                                                mx::e2m1x2_to_f16x2<3>(w[i][0]), mx::e2m1x2_to_f16x2<3>(w[i][1])};
#pragma unroll
                        for (int n = 0; n < NQ; ++n) {
                            float c[4];
                            mma_f16_zero(c, a0, qb[n][b][0], qb[n][b][1]);
                            dev::mma_f16_16816(c, a1, qb[n][b][2], qb[n][b][3]);
                            float(&x)[4] = s[mt][n];
                            if (b == 0) {
                                x[0] = c[0] * f0[b], x[1] = c[1] * f0[b], x[2] = c[2] * f1[b], x[3] = c[3] * f1[b];
                            } else {
                                x[0] += c[0] * f0[b], x[1] += c[1] * f0[b], x[2] += c[2] * f1[b], x[3] += c[3] * f1[b];
                            }
                        }
                    }
                }
            }
            // a stage that crosses the range's end or the first token's diagonal
            if (si.k + kKeys > si.k1 || si.k + kKeys - 1 > si.qpos0) {
#pragma unroll
                for (int n = 0; n < NQ; ++n) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int last = min(lim[n][e & 1], si.k1 - 1) - si.k - gq - 8 * (e >> 1);
#pragma unroll
                        for (int mt = 0; mt < kMT; ++mt)
                            if (mt * 16 > last) s[mt][n][e] = -INFINITY;
                    }
                }
            }

            // ---- online softmax: P^T as f16, transposed to the next product's operand
            uint32_t pb[kMT][NQ][2];
#pragma unroll
            for (int n = 0; n < NQ; ++n) {
                float al[2], mu[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float mx = fmaxf(s[0][n][i], s[0][n][2 + i]);
#pragma unroll
                    for (int mt = 1; mt < kMT; ++mt) mx = dev::fmax3(mx, s[mt][n][i], s[mt][n][2 + i]);
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                    const float mn = fmaxf(m[n][i], mx * sl[n][i]);  // (sl > 0)
                    const float mz = mn == -INFINITY ? 0.f : mn;
                    al[i] = dev::fast_exp2(m[n][i] - mz);
                    m[n][i] = mn;
                    mu[i] = kPShift - mz;
                }
                float sum[2] = {0.f, 0.f};
#pragma unroll
                for (int mt = 0; mt < kMT; ++mt) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        s[mt][n][e] = dev::fast_exp2(fmaf(s[mt][n][e], sl[n][e & 1], mu[e & 1]));
                        sum[e & 1] += s[mt][n][e];
                    }
                    // (key gq, rows 2cq, 2cq+1) -> (row gq, keys 2cq, 2cq+1)
                    pb[mt][n][0] = movmatrix_t(dev::pack_f16x2(s[mt][n][0], s[mt][n][1]));
                    pb[mt][n][1] = movmatrix_t(dev::pack_f16x2(s[mt][n][2], s[mt][n][3]));
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) l[n][i] = l[n][i] * al[i] + sum[i];
#pragma unroll
                for (int t = 0; t < OT; ++t) {
                    o[t][n][0] *= al[0], o[t][n][1] *= al[1];
                    o[t][n][2] *= al[0], o[t][n][3] *= al[1];
                }
            }

            // ---- O^T += V^T P^T: the lane's keys 2cq, 2cq+1 | 2cq+8, 2cq+9, dims gq*D/8 .. +D/8-1
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
                if (si.k + kKeys > si.k1) {
                    // a row past the range's end holds what an earlier stage left: scale 0 (its P is 0)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (si.k + mt * 16 + 2 * cq + (i & 1) + (i >> 1) * 8 >= si.k1) ve[i] = 0;
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
                        for (int n = 0; n < NQ; ++n) dev::mma_f16_16816(o[4 * w + B][n], a, pb[mt][n][0], pb[mt][n][1]);
                    };
                    tile(IntTag<0>{});
                    tile(IntTag<1>{});
                    tile(IntTag<2>{});
                    tile(IntTag<3>{});
                }
            }
        }

        __syncwarp();
        if (lane == 0) dev::mbar_arrive(&sh->empty[stage]);
        if (++stage == stages) {
            stage = 0;
            phase ^= 1;
        }
        if (!(si.flags & kLast)) continue;

        // ================================================================ the head's warps' join
        if (KW > 1) {
            const int parts = min(KW, si.index + 1);  // warps that had a stage of the unit
            constexpr int kVals = OT * 4 * NQ + 4 * NQ;
            auto area = [&](int w) {
                return reinterpret_cast<float*>(smem + sp.exch) + ((int64_t)(w - 1) * HB + gl) * (kVals * 32) + lane;
            };
            if (kw > 0) {
                // the area is free once the first warp has taken the unit before
                if (!warp_wait(&xs->xempty[gl], xphase ^ 1, wlim, sh, err)) return;
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
                if (lane == 0) dev::mbar_arrive(&xs->xfull[gl]);
                xphase ^= 1;
                continue;
            }
            if (!warp_wait(&xs->xfull[gl], xphase, wlim, sh, err)) return;
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
            if (lane == 0) dev::mbar_arrive(&xs->xempty[gl]);
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
                    const int64_t slot = (int64_t)(si.pbase + si.split) * p.lay.rows_per_slot;
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
// groups fill the SMs by themselves), 4 up to 16, else 16.
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

template <int D, int NQ, bool CP>
cudaError_t launch_q(const ForwardParams& p, int ctas, cudaStream_t s) {
    const int Hkv = p.num_kv_heads;
    MxShape sp{};
    sp.hb = decode_mx_heads(Hkv, D, 8 * NQ);
    sp.kw = mx_consumers(D, NQ) / sp.hb;
    sp.pw = CP ? 2 : 1;
    // a head group of a row, or the row as the pool has it, padding included
    sp.stride = sp.hb < Hkv ? mx::group_bytes(Hkv, D) * (sp.hb / 8) : p.mx_row_bytes;
    const int head = (int)((sizeof(MxSmem) + 127) / 128 * 128);
    const int exch = (sp.kw - 1) * sp.hb * (D / 4 + 4) * NQ * 128;
    const int stage_bytes = 2 * kKeys * sp.stride;
    sp.stages = (220 * 1024 - 1024 - head - exch) / stage_bytes;
    sp.stages = sp.stages < 2 ? 2 : (sp.stages > 8 ? 8 : sp.stages);
    sp.exch = head + sp.stages * stage_bytes;
    const size_t smem = (size_t)sp.exch + exch;
    const cudaError_t e =
        cudaFuncSetAttribute(decode_mx_kernel<D, NQ, CP>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    return launch_programmatic(decode_mx_kernel<D, NQ, CP>, (unsigned)ctas, 32u * (sp.hb * sp.kw + sp.pw), smem, s, p, sp);
}

template <int D>
cudaError_t launch_dec(const ForwardParams& p, int ctas, cudaStream_t s) {
    const bool cp = decode_mx_small_pages(p.num_kv_heads, p.page_size, D) ||
                    decode_mx_heads(p.num_kv_heads, D, p.dec_rows) < p.num_kv_heads;
    if (p.dec_rows <= 8) return cp ? launch_q<D, 1, true>(p, ctas, s) : launch_q<D, 1, false>(p, ctas, s);
    return cp ? launch_q<D, 2, true>(p, ctas, s) : launch_q<D, 2, false>(p, ctas, s);
}

}  // namespace

// Whether the producers copy rows in 16-byte pieces: the copy engine takes about 70 cycles a bulk
// copy whatever its size, so a page's run has to be long to keep up with HBM.
bool decode_mx_small_pages(int num_kv_heads, int page_size, int head_dim) {
    return page_size * mx::row_bytes(num_kv_heads, head_dim) < 2048;
}

// kv heads a decode CTA serves: all of them, or a block of them when its warps are fewer.
int decode_mx_heads(int num_kv_heads, int head_dim, int rows) {
    if (num_kv_heads <= kDecHeadBlock) return num_kv_heads;
    return mx_consumers(head_dim, rows <= 8 ? 1 : 2) == 16 && num_kv_heads % 16 == 0 ? 16 : kDecHeadBlock;
}

cudaError_t launch_join_mx(const ForwardParams& p, int head_dim, int ctas, cudaStream_t s) {
    if (head_dim == 128) return launch_programmatic(join_kernel<128>, (unsigned)ctas, 32u * kJoinWarps, 0, s, p);
    if (head_dim == 64) return launch_programmatic(join_kernel<64>, (unsigned)ctas, 32u * kJoinWarps, 0, s, p);
    return cudaErrorInvalidValue;
}

cudaError_t launch_decode_mx(const ForwardParams& p, int head_dim, int ctas, cudaStream_t s) {
    if (head_dim == 128) return launch_dec<128>(p, ctas, s);
    if (head_dim == 64) return launch_dec<64>(p, ctas, s);
    return cudaErrorInvalidValue;
}

}  // namespace pva

// K9, K10, K12: linear attention's plan, its recurrence for requests of few new tokens, and the scan over a long
// request's segments.
//
// K10, for one (request, kv head): S <- e^{g_t} S + k_t v_t^T, o_t = scale q_t^T S_t, token by token, all
// in fp32.  The state is read once and written once for all of the request's new tokens, and the G q
// heads of the kv head share it.  Bound: HBM, 2 x 4 D^2 bytes a request and kv head (D = 128: 128 KiB
// against 2 KiB of activations); 64 requests of 32 heads, a token each: 270 MB in 42 us, 6.4 TB/s.  A thread
// keeps four columns of some rows in registers, so that a warp's accesses are whole rows and every load of the state
// is in flight before the first is used.  Of several tokens the next one's k, v and q are loaded while one is worked
// on (16 tokens of 64 requests, 32/8 heads: when it came in 90 us for 103, of 4 requests 14 for 22; now 88 and 13).  It also copies the
// starts of long requests that several CTAs of the tensor-core kernel behind it work on.
#include <cuda_runtime.h>

#include <type_traits>

#include "device_utils.cuh"
#include "linear.h"

namespace pva {
namespace {

// ---------------------------------------------------------------- K9: the plan

constexpr int kPlanThreads = 1024;
constexpr int kBuckets = 256;  // segments sorted by chunks (more: the first bucket)

// One CTA (10 us with 18 segments of one request).  Validates the batch, resolves each request's state slots, lists the long requests'
// segments, most tokens first, and notes each token's request.  A state slot is claimed by writing the
// request's index to it and looking who is there afterwards: what an earlier batch left in a slot that
// no one claimed is told by that request's own out slot being another.
__global__ void __launch_bounds__(kPlanThreads) linear_plan_kernel(const LinPlanParams p) {
    __shared__ int32_t hist[kBuckets], first[kBuckets];
    __shared__ int32_t n_items, n_pre, n_segs, n_cut, longest;
    __shared__ unsigned long long long_tokens;
    __shared__ uint32_t all_err;
    PlanHeader* hdr = reinterpret_cast<PlanHeader*>(p.ws + p.lay.header);
    int2* req_state = reinterpret_cast<int2*>(p.ws + p.lay.req_state);
    int32_t* req_base = reinterpret_cast<int32_t*>(p.ws + p.lay.req_base);
    int32_t* claim = reinterpret_cast<int32_t*>(p.ws + p.lay.claim);
    int32_t* tok_req = reinterpret_cast<int32_t*>(p.ws + p.lay.tok_req);
    LinItem* items = reinterpret_cast<LinItem*>(p.ws + p.lay.items);
    LinItem* pre = reinterpret_cast<LinItem*>(p.ws + p.lay.pre_items);
    LinItem* cuts = reinterpret_cast<LinItem*>(p.ws + p.lay.cut_items);
    const int tid = threadIdx.x, B = p.batch;
    for (int i = tid; i < kBuckets; i += kPlanThreads) hist[i] = 0;
    if (tid == 0) n_items = n_pre = n_segs = n_cut = longest = 0, long_tokens = 0, all_err = 0;

    uint32_t err = 0;
    for (int i = tid; i < B; i += kPlanThreads) {
        const int c0 = p.cu[i], c1 = p.cu[i + 1];
        if (c0 < 0 || c1 < c0 || c1 > p.total_tokens || (i == 0 && c0 != 0) || (i == B - 1 && c1 != p.total_tokens)) {
            err |= kErrCu;
            continue;
        }
        if (c1 - c0 > p.seqlens[i]) err |= kErrQgtKv;
        if (c1 - c0 > p.max_q_len) err |= kErrLimits;
    }
    if (B == 0 && tid == 0 && p.cu[0] != 0) err |= kErrCu;
    const bool fatal = __syncthreads_or(err != 0);
    if (err) atomicOr(&all_err, err);

    // slots: -1 nothing, -2 outside the pool
    auto slot_in = [&](int i) -> int {
        const int n = p.cu[i + 1] - p.cu[i];
        if (n <= 0 || p.state_in == nullptr || p.seqlens[i] <= n) return -1;  // starts from zero
        const int s = p.state_in[i];
        return s < -1 || s >= p.num_states ? -2 : s;
    };
    auto slot_out = [&](int i) -> int {
        if (p.cu[i + 1] - p.cu[i] <= 0 || p.state_out == nullptr) return -1;
        const int s = p.state_out[i];
        return s < -1 || s >= p.num_states ? -2 : s;
    };
    if (!fatal) {
        for (int i = tid; i < B; i += kPlanThreads) {
            const int in = slot_in(i), out = slot_out(i);
            const bool bad = in == -2 || out == -2;
            req_state[i] = bad ? make_int2(-2, -2) : make_int2(in, out);
            if (bad) atomicOr(&all_err, kErrState);
            if (!bad && out >= 0) claim[out] = i;
        }
        __syncthreads();
        // two requests of one out slot are both skipped, and one that writes where another reads; every
        // look is at the slots as given, so what is skipped depends on no order
        auto clash = [&](int j) {
            req_state[j].x = -2;
            atomicOr(&all_err, kErrState);
        };
        for (int i = tid; i < B; i += kPlanThreads) {
            const int in = slot_in(i), out = slot_out(i);
            if (in == -2 || out == -2) continue;
            if (out >= 0 && claim[out] != i) {
                clash(i);
                clash(claim[out]);
            }
            if (in >= 0) {
                const int j = claim[in];
                if (j >= 0 && j < B && j != i && slot_in(j) != -2 && slot_out(j) == in) clash(j);
            }
        }
        __syncthreads();
    }
    auto is_long = [&](int i, int* n) {
        *n = p.cu[i + 1] - p.cu[i];
        return *n > kStepTokens && req_state[i].x != -2;
    };
    if (!fatal) {
        // (those that are skipped too: how the others are cut, and so their bits, does not depend on them)
        for (int i = tid; i < B; i += kPlanThreads) {
            const int n = p.cu[i + 1] - p.cu[i];
            if (n <= kStepTokens) continue;
            atomicMax(&longest, n);
            atomicAdd(&long_tokens, (unsigned long long)n);
        }
        __syncthreads();
    }
    // how a request is cut: chunks of a segment, and segments
    const int seg_tokens = planned_segment_tokens(p.may_cut, (int64_t)long_tokens, longest, p.num_kv_heads, p.sm_count);
    auto cut = [&](int n, int* per) -> int {
        const int chunks = (n + kChunk - 1) / kChunk;
        const int want = (int)(((int64_t)n + seg_tokens - 1) / seg_tokens);
        *per = (chunks + want - 1) / want;
        return (chunks + *per - 1) / *per;
    };
    int parts = 1;
    if (!fatal) {
        for (int i = tid; i < B; i += kPlanThreads) {
            int n, per;
            if (!is_long(i, &n)) continue;
            const int nseg = cut(n, &per);
            for (int s = 0; s < nseg; ++s) {
                const int chunks = (min(per * kChunk, n - s * per * kChunk) + kChunk - 1) / kChunk;
                atomicAdd(&hist[kBuckets - min(chunks, kBuckets)], 1);
            }
        }
        __syncthreads();
        if (tid < 32) {  // where each bucket starts
            int sum = 0;
            for (int b0 = 0; b0 < kBuckets; b0 += 32) {
                const int v = hist[b0 + tid];
                int x = v;
#pragma unroll
                for (int d = 1; d < 32; d *= 2) {
                    const int y = __shfl_up_sync(0xffffffffu, x, d);
                    if (tid >= d) x += y;
                }
                first[b0 + tid] = sum + x - v;
                sum += __shfl_sync(0xffffffffu, x, 31);
            }
            if (tid == 0) n_items = sum;
        }
        __syncthreads();
        parts = head_parts(n_items, p.group, p.num_kv_heads, p.sm_count);
        for (int i = tid; i < B; i += kPlanThreads) {
            int n, per;
            req_base[i] = -1;
            if (!is_long(i, &n)) continue;
            const int nseg = cut(n, &per);
            const int at = nseg > 1 ? atomicAdd(&n_pre, nseg - 1) : 0;
            LinItem it;
            it.req = i;
            it.nseg = nseg;
            it.in = req_state[i].x;
            // several CTAs on one state: they start from a copy
            it.base = nseg > 1 || (parts > 1 && it.in >= 0) ? atomicAdd(&n_segs, nseg) : -1;
            if (it.in >= 0) req_base[i] = it.base;
            it.out = req_state[i].y;
            for (int s = 0; s < nseg; ++s) {
                it.seg = s;
                it.tok0 = p.cu[i] + s * per * kChunk;
                it.ntok = min(per * kChunk, n - s * per * kChunk);
                items[atomicAdd(&first[kBuckets - min((it.ntok + kChunk - 1) / kChunk, kBuckets)], 1)] = it;
                if (s < nseg - 1) pre[at + s] = it;
                if (s == 0 && nseg > 1) cuts[atomicAdd(&n_cut, 1)] = it;
            }
        }
        // requests of the tokens: a few tokens by one thread, many by the block
        for (int i = tid; i < B; i += kPlanThreads) {
            const int c0 = p.cu[i], n = p.cu[i + 1] - c0;
            if (n <= kStepTokens)
                for (int t = 0; t < n; ++t) tok_req[c0 + t] = i;
        }
        for (int i0 = 0; i0 < B; i0 += 32) {
            const int i = i0 + (tid & 31), c0 = i < B ? p.cu[i] : 0, n = i < B ? p.cu[i + 1] - c0 : 0;
            for (unsigned many = __ballot_sync(0xffffffffu, n > kStepTokens); many != 0; many &= many - 1) {
                const int l = __ffs(many) - 1;
                const int first_tok = __shfl_sync(0xffffffffu, c0, l), count = __shfl_sync(0xffffffffu, n, l);
                for (int t = tid; t < count; t += kPlanThreads) tok_req[first_tok + t] = i0 + l;
            }
        }
    }
    __syncthreads();
    if (tid == 0) {
        hdr->n_pre_tiles = fatal ? 0 : n_items;
        hdr->n_casc_tiles = fatal ? 0 : n_pre;
        hdr->n_casc_groups = fatal ? 0 : n_cut;
        hdr->n_casc_units = parts;
        hdr->wait_override = 0;
        hdr->error_bits = all_err;
    }
}

// ---------------------------------------------------------------- K10: token by token

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// 2 W consecutive bf16 (W = 2 or 4 words).
template <int W>
__device__ __forceinline__ void load_words(const uint16_t* src, uint32_t (&x)[W]) {
    if constexpr (W == 2) {
        const uint2 w = __ldg(reinterpret_cast<const uint2*>(src));
        x[0] = w.x, x[1] = w.y;
    } else {
        static_assert(W == 4, "8 or 16 bytes");
        const uint4 w = __ldg(reinterpret_cast<const uint4*>(src));
        x[0] = w.x, x[1] = w.y, x[2] = w.z, x[3] = w.w;
    }
}

constexpr int kHeadsAtOnce = 4;  // q heads whose results meet in shared memory together (and are loaded ahead)

// P: CTAs that share a state's columns.
template <int D, int P>
struct StepShape {
    static constexpr int kThreads = 2 * D;
    static constexpr int kCols = D / P;              // columns of a CTA
    static constexpr int kLanes = kCols / 4;         // lanes of a row
    static constexpr int kGroups = kThreads / kLanes;
    static constexpr int kRows = D / kGroups;        // rows of a thread
    static constexpr int kWarps = kThreads / 32;
};

// Where the warps' parts of the heads' results meet: two buffers.
template <int D, int P>
struct StepSums {
    alignas(16) float at[2][StepShape<D, P>::kWarps][kHeadsAtOnce][StepShape<D, P>::kCols];
};

template <int D, int P>
__device__ __noinline__ void steps_with_drops(const LinParams& p, StepSums<D, P>& red);

// DROPS: some token of the request is known to drop the state.
template <int D, int P, bool DROPS>
__device__ __forceinline__ void steps(const LinParams& p, StepSums<D, P>& red) {
    using L = StepShape<D, P>;
    constexpr int R = L::kRows, H = kHeadsAtOnce;
    const int req = blockIdx.y, kvh = blockIdx.x / P, col0 = (blockIdx.x % P) * L::kCols;
    const uint32_t errors = reinterpret_cast<const PlanHeader*>(p.ws + p.lay.header)->error_bits;
    const int2 slots = reinterpret_cast<const int2*>(p.ws + p.lay.req_state)[req];
    const int c0 = p.cu[req], n = p.cu[req + 1] - c0;
    if ((errors & kErrFatal) || n <= 0 || slots.x == -2) return;
    const int copy = n > kStepTokens ? reinterpret_cast<const int32_t*>(p.ws + p.lay.req_base)[req] : -1;
    if (n > kStepTokens && copy < 0) return;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int col = 4 * (tid % L::kLanes), row0 = (tid / L::kLanes) * R;

    const int64_t per_head = (int64_t)D * D;
    float4 S[R];
    if (slots.x >= 0) {
        const float* src = p.states + ((int64_t)slots.x * p.num_kv_heads + kvh) * per_head + row0 * D + col0 + col;
#pragma unroll
        for (int i = 0; i < R; ++i) S[i] = *reinterpret_cast<const float4*>(src + i * D);
    } else {
#pragma unroll
        for (int i = 0; i < R; ++i) S[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    if (copy >= 0) {
        // (as the tensor-core kernel reads it: four columns of a row, then those of the next row)
        float4* dst = reinterpret_cast<float4*>(reinterpret_cast<float*>(p.ws + p.lay.seg_state) +
                                                ((int64_t)copy * p.num_kv_heads + kvh) * per_head) + (col0 + col) / 4 * D + row0;
#pragma unroll
        for (int i = 0; i < R; ++i) dst[i] = S[i];
        return;
    }
    // what the next token and heads need is on its way while these are worked on
    uint32_t kw[R / 2], vw[2], qw[H][R / 2];
    float gw;
    auto load_token = [&](int64_t tok) {
        gw = p.log_decay[(p.ld_decay ? tok * p.ld_decay : 0) + kvh];
        load_words(p.k + tok * p.ld_k + kvh * D + row0, kw);
        load_words(p.v + tok * p.ld_v + kvh * D + col0 + col, vw);
    };
    auto load_head = [&](int h, int64_t tok, int head) {
        if (head < p.group) load_words(p.q + tok * p.ld_q + (kvh * p.group + head) * D + row0, qw[h]);
    };
    load_token(c0);
#pragma unroll
    for (int h = 0; h < H; ++h) load_head(h, c0, h);
    int buf = 0;
    auto tokens = [&](auto drops) {
        for (int t = 0; t < n; ++t) {
            const int64_t tok = c0 + t;
            const float lam = expf(gw);
            if constexpr (decltype(drops)::value) {
                if (gw <= kDropLogDecay) {
#pragma unroll
                    for (int i = 0; i < R; ++i) S[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                }
            }
            const float v[4] = {bf_lo(vw[0]), bf_hi(vw[0]), bf_lo(vw[1]), bf_hi(vw[1])};
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const float k = (i & 1) ? bf_hi(kw[i / 2]) : bf_lo(kw[i / 2]);
                S[i].x = fmaf(k, v[0], lam * S[i].x);
                S[i].y = fmaf(k, v[1], lam * S[i].y);
                S[i].z = fmaf(k, v[2], lam * S[i].z);
                S[i].w = fmaf(k, v[3], lam * S[i].w);
            }
            if (t + 1 < n) load_token(tok + 1);
            for (int h0 = 0; h0 < p.group; h0 += H, buf ^= 1) {
                const int heads = min(H, p.group - h0);
                const bool same = h0 + H < p.group;  // the next heads are this token's
                const int next0 = same ? h0 + H : t + 1 < n ? 0 : p.group;
#pragma unroll
                for (int h = 0; h < H; ++h) {
                    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                    for (int i = 0; i < R; ++i) {
                        const float x = (i & 1) ? bf_hi(qw[h][i / 2]) : bf_lo(qw[h][i / 2]);
                        o.x = fmaf(x, S[i].x, o.x);
                        o.y = fmaf(x, S[i].y, o.y);
                        o.z = fmaf(x, S[i].z, o.z);
                        o.w = fmaf(x, S[i].w, o.w);
                    }
                    load_head(h, same ? tok : tok + 1, next0 + h);
                    if (h >= heads) continue;
#pragma unroll
                    for (int m = L::kLanes; m < 32; m *= 2) {
                        o.x += __shfl_xor_sync(0xffffffffu, o.x, m);
                        o.y += __shfl_xor_sync(0xffffffffu, o.y, m);
                        o.z += __shfl_xor_sync(0xffffffffu, o.z, m);
                        o.w += __shfl_xor_sync(0xffffffffu, o.w, m);
                    }
                    if (lane < L::kLanes) *reinterpret_cast<float4*>(&red.at[buf][warp][h][col]) = o;
                }
                __syncthreads();
                // (the other buffer is written before the next barrier: nobody is more than one ahead)
                for (int x = tid; x < heads * L::kCols / 2; x += L::kThreads) {
                    const int h = x / (L::kCols / 2), c = 2 * (x % (L::kCols / 2));
                    float a = 0.f, b = 0.f;
#pragma unroll
                    for (int w = 0; w < L::kWarps; ++w) {
                        const float2 y = *reinterpret_cast<const float2*>(&red.at[buf][w][h][c]);
                        a += y.x, b += y.y;
                    }
                    *reinterpret_cast<uint32_t*>(p.out + (tok * p.num_qo_heads + kvh * p.group + h0 + h) * D + col0 + c) =
                        dev::pack_bf16x2(a * p.scale, b * p.scale);
                }
            }
        }
    };
    if constexpr (DROPS) {
        tokens(std::true_type{});
    } else {
        // Requests with a token that drops the state, whatever it holds, take a loop that looks at each token's decay: in one loop for
        // all 12 tokens of 64 requests, 16 heads of 64, took 33 us for 28, 64 decodes of 32 heads of 128 49 for 42.  For
        // D 64 that loop is a function of its own (in line 32 us), for D 128 it is not (a token of 64 requests, 32 heads, 44 us).
        const float g = lane < n ? p.log_decay[(p.ld_decay ? (c0 + lane) * p.ld_decay : 0) + kvh] : 0.f;
        if (!__any_sync(0xffffffffu, g <= kDropLogDecay)) {
            tokens(std::false_type{});
        } else if constexpr (D == 64) {
            steps_with_drops<D, P>(p, red);
            return;
        } else {
            tokens(std::true_type{});
        }
    }
    if (slots.y >= 0) {
        float* dst = p.states + ((int64_t)slots.y * p.num_kv_heads + kvh) * per_head + row0 * D + col0 + col;
#pragma unroll
        for (int i = 0; i < R; ++i) *reinterpret_cast<float4*>(dst + i * D) = S[i];
    }
}

template <int D, int P>
__device__ __noinline__ void steps_with_drops(const LinParams& p, StepSums<D, P>& red) {
    steps<D, P, true>(p, red);
}

template <int D, int P>
__global__ void __launch_bounds__(StepShape<D, P>::kThreads) linear_step_kernel(const __grid_constant__ LinParams p) {
    __shared__ StepSums<D, P> red;
    dev::grid_dep_wait();
    dev::grid_dep_launch();
    steps<D, P, false>(p, red);
}

// ---------------------------------------------------------------- K12: the scan over a request's segments
//
// Entry i of a request's segment states, i >= 2, holds the end of segment i - 1 from zero: X_i; it becomes that
// segment's end from the request's start, S_i = (decay over segment i - 1) S_{i-1} + X_i (X_i alone where that drops it).  Four elements of a state a
// thread, every segment's in turn, four loads in flight.  Bound: the L2's latency (18 segments of 8 heads of 128 x 128:
// 18 MB in 7.3 us; each segment's CTAs summing what lies before it took up to 20).
constexpr int kScanThreads = 256;

template <int D>
__global__ void __launch_bounds__(kScanThreads) linear_scan_kernel(const LinParams p) {
    dev::grid_dep_wait();
    dev::grid_dep_launch();
    const PlanHeader* hdr = reinterpret_cast<const PlanHeader*>(p.ws + p.lay.header);
    if (hdr->error_bits & kErrFatal) return;
    constexpr int kParts = D * D / 4 / kScanThreads;  // blocks of a state
    const int work = hdr->n_casc_groups * p.num_kv_heads * kParts;
    for (int x = blockIdx.x; x < work; x += gridDim.x) {
        const LinItem it = reinterpret_cast<const LinItem*>(p.ws + p.lay.cut_items)[x / (p.num_kv_heads * kParts)];
        const int kvh = x / kParts % p.num_kv_heads;
        const int64_t step = (int64_t)p.num_kv_heads * D * D / 4, first = (int64_t)it.base * p.num_kv_heads + kvh;
        float4* s = reinterpret_cast<float4*>(p.ws + p.lay.seg_state) + first * (D * D / 4) + x % kParts * kScanThreads + threadIdx.x;
        const float* decay = reinterpret_cast<const float*>(p.ws + p.lay.seg_decay) + first;
        float4 S = s[step];
        for (int i = 2; i < it.nseg; i += 4) {
            float4 y[4];
            float f[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (i + j < it.nseg) y[j] = s[(i + j) * step], f[j] = decay[(int64_t)(i + j) * p.num_kv_heads];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (i + j < it.nseg) {
                    if (f[j] < 0.f) S = make_float4(0.f, 0.f, 0.f, 0.f);  // (dropped)
                    S.x = fmaf(f[j], S.x, y[j].x), S.y = fmaf(f[j], S.y, y[j].y);
                    S.z = fmaf(f[j], S.z, y[j].z), S.w = fmaf(f[j], S.w, y[j].w);
                    s[(i + j) * step] = S;
                }
        }
    }
}

template <int D, int P>
cudaError_t launch_step(const LinParams& p, cudaStream_t s) {
    return launch_programmatic(linear_step_kernel<D, P>, dim3((unsigned)(p.num_kv_heads * P), (unsigned)p.batch),
                               (unsigned)StepShape<D, P>::kThreads, 0, s, p);
}

template <int D>
cudaError_t launch_step_d(const LinParams& p, cudaStream_t s) {
    // 64 columns a CTA, 8 rows a thread: its state and what is on its way take some 80 registers, three CTAs of 256 threads
    // an SM (a token of 64 requests, 32 heads of 128: 42 us, with 32 columns 45, with all 128 too).  32 columns where
    // that would leave half the SMs without work (4 requests of 8 heads of 128: 2.3 us for 2.8, of 16 tokens 13.4 for 19).
    constexpr int P = D / 64;
    const int64_t heads = (int64_t)p.batch * p.num_kv_heads;
    return 2 * heads > p.sm_count ? launch_step<D, P>(p, s) : launch_step<D, 2 * P>(p, s);
}

}  // namespace

cudaError_t launch_linear_plan(const LinPlanParams& p, cudaStream_t s) {
    linear_plan_kernel<<<1, kPlanThreads, 0, s>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_linear_scan(const LinParams& p, int head_dim, cudaStream_t s) {
    auto go = [&](auto kernel) { return launch_programmatic(kernel, dim3((unsigned)(4 * p.sm_count)), (unsigned)kScanThreads, 0, s, p); };
    if (head_dim == 128) return go(linear_scan_kernel<128>);
    if (head_dim == 64) return go(linear_scan_kernel<64>);
    return cudaErrorInvalidValue;
}

cudaError_t launch_linear_step(const LinParams& p, int head_dim, cudaStream_t s) {
    if (p.batch <= 0) return cudaSuccess;
    if (head_dim == 128) return launch_step_d<128>(p, s);
    if (head_dim == 64) return launch_step_d<64>(p, s);
    return cudaErrorInvalidValue;
}

}  // namespace pva

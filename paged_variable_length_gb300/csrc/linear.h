// Linear attention with a decay for each head: the plan's layout and the parameters of its kernels.
//
// For kv head h, token t and its q heads: S_t = e^{g_t} S_{t-1} + k_t v_t^T (D x D, fp32) and
// o_t = scale q_t^T S_t.  Requests of up to kStepTokens new tokens run the recurrence as it stands
// (linear_step.cu); longer ones in chunks of kChunk tokens on the tensor cores (linear_tc.cu), where
// with c_i the sum of g over the chunk's tokens up to i
//   o_i = scale (sum_{j <= i} e^{c_i - c_j} (q_i . k_j) v_j + e^{c_i} q_i^T S)
//   S'  = e^{c_end} S + sum_j e^{c_end - c_j} k_j v_j^T.
// A long request is cut into segments of whole chunks where its heads alone would not fill the GPU:
// a first pass finds the segments' states, a second starts each from what lies before it.
#pragma once

#include "pva_internal.h"

namespace pva {

constexpr int kStepTokens = 16;   // most new tokens of a request that runs token by token
constexpr int kChunk = 128;       // tokens of a tensor-core chunk
constexpr int kMaxSegments = 32;  // most segments of a request
constexpr uint32_t kErrState = PVA_DEVERR_STATE;
// Log decays below this are taken as this: e^-110 is 0 in fp32, and -inf - -inf is never formed.
constexpr float kLeastLogDecay = -110.f;

// A segment of a long request: tokens tok0 .. tok0 + ntok - 1.
struct LinItem {
    int32_t req;
    int32_t tok0;
    int32_t ntok;
    int32_t seg;     // index among the request's segments
    int32_t nseg;
    int32_t base;    // first of the request's nseg segment states in the workspace, -1: it has none (one CTA a kv head)
    int32_t in;      // state slot that the request starts from (-1: zero)
    int32_t out;     // state slot that receives its last state (-1: none)
};
static_assert(sizeof(LinItem) == 32, "LinItem is one 32-byte record");

// Workspace carve-up.  The header is a PlanHeader: error_bits, wait_override, n_pre_tiles (segments of
// long requests) and n_casc_tiles (those of them whose states the first pass finds).
struct LinLayout {
    size_t header;
    size_t tok_req;     // int32 [max_tokens]: request of each new token
    size_t req_state;   // int2 [max_batch]: state slots (in, out) of each request, in = -2: skipped
    size_t req_base;    // int32 [max_batch]: of a long request whose start is copied, its LinItem::base; else -1
    size_t claim;       // int32 [num_states]: the last request that claimed a slot as its out
    size_t items;       // LinItem [max_items], most tokens first
    size_t pre_items;   // LinItem [max_segs]: the segments of the first pass
    size_t seg_state;   // fp32 [max_segs][Hkv][D][D]: a request's entry 0: a copy of its start; s: segment s - 1's end
    size_t seg_decay;   // fp32 [max_segs][Hkv]: entry s: the decay over segment s - 1
    size_t total;
    int32_t max_items;
    int32_t max_segs;
};

struct LinPlanParams {
    const int32_t* cu;
    const int32_t* seqlens;
    const int32_t* state_in;   // or null: every request starts from zero
    const int32_t* state_out;  // or null: no state is kept
    int32_t batch;
    int32_t total_tokens;
    int32_t max_q_len;
    int32_t seg_tokens;        // most tokens of a segment
    int32_t head_parts;        // CTAs that share the q heads of a kv head
    int64_t num_states;
    uint8_t* ws;
    LinLayout lay;
};

struct LinParams {
    const uint16_t* q;         // bf16 bits [T, Hq, D], ld_q elements between tokens
    const uint16_t* k;
    const uint16_t* v;
    uint16_t* out;             // [T, Hq, D] contiguous
    int64_t ld_q, ld_k, ld_v;
    const float* log_decay;    // [Hkv], or [T, Hkv] with ld_decay elements between tokens
    int64_t ld_decay;
    float* states;             // [num_states, Hkv, D, D]
    const int32_t* cu;
    int32_t batch;
    int32_t total_tokens;
    int32_t num_qo_heads;
    int32_t num_kv_heads;
    int32_t group;
    int32_t sm_count;
    int32_t head_parts;
    float scale;
    uint8_t* ws;
    LinLayout lay;
};

// Host view of a prepared batch, stored inside pva_meta::opaque.
struct LinHost {
    uint64_t magic;
    pva_linear_config cfg;
    int32_t batch;
    int32_t total_tokens;
    int32_t max_q_len;
    int32_t sm_count;
    int32_t seg_tokens;
    int32_t head_parts;
    const int32_t* cu;
    const int32_t* seqlens;
    uint8_t* ws;
    void* stream;
    LinLayout lay;
};
static_assert(sizeof(LinHost) <= sizeof(pva_meta), "LinHost must fit in pva_meta");
constexpr uint64_t kLinMagic = 0x5056414c494e5231ull;  // "PVALINR1"

inline const LinHost* lin_of(const pva_meta* m) {
    if (m == nullptr) return nullptr;
    const LinHost* h = reinterpret_cast<const LinHost*>(m->opaque);
    return h->magic == kLinMagic ? h : nullptr;
}

// (linear_api.cu; the calls over a paged pool use them too)
pva_status check_rotation(const pva_rope* rope, const pva_qk_norm* norm, int64_t D);
void set_rotation(const pva_rope* rope, const pva_qk_norm* norm, RopeParams* rp);

cudaError_t launch_linear_plan(const LinPlanParams& p, cudaStream_t s);
cudaError_t launch_linear_step(const LinParams& p, int head_dim, cudaStream_t s);
// states: the first pass (the segments' states), else the outputs
cudaError_t launch_linear_chunks(const LinParams& p, int head_dim, bool states, int ctas, cudaStream_t s);

}  // namespace pva

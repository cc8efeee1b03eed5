// Linear attention with a decay for each head: the plan's layout and the parameters of its kernels.
//
// For kv head h, token t and its q heads: S_t = e^{g_t} S_{t-1} + k_t v_t^T (D x D, fp32) and
// o_t = scale q_t^T S_t.  Requests of up to kStepTokens new tokens run the recurrence as it stands
// (linear_step.cu); longer ones in chunks of kChunk tokens on the tensor cores (linear_tc.cu), where
// with c_i the sum of g over the chunk's tokens up to i
//   o_i = scale (sum_{j <= i} e^{c_i - c_j} (q_i . k_j) v_j + e^{c_i} q_i^T S)
//   S'  = e^{c_end} S + sum_j e^{c_end - c_j} k_j v_j^T.
// A long request is cut into segments of whole chunks where its heads alone would not fill the GPU: a first pass
// finds the segments' states, a scan what lies before each, and a second pass starts from there.
#pragma once

#include "pva_internal.h"

namespace pva {

constexpr int kChunk = 128;       // tokens of a tensor-core chunk
constexpr uint32_t kErrState = PVA_DEVERR_STATE;
// A log decay up to this drops the state, whatever it holds (e^-110 is 0 in fp32, but 0 times an infinity or a NaN is a
// NaN): what lies before the token has no part in anything from it on.
constexpr float kDropLogDecay = -110.f;

// Most new tokens of a request that runs token by token, between the lengths where the tensor cores catch up: 11 tokens
// of 64 requests of 32/8 heads of 128 (9 tokens 53 us for 60, 16 tokens 88 for 60), 16 of one such (13 us), 23 of
// 64 requests of 16/16 heads of 64 (16 tokens 34 us for 46, 24 tokens 48).  Their results keep fp32's accuracy.
constexpr int kStepTokens = 16;

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

// Tokens of a segment.  A long request is cut where its batch's heads and requests alone would leave SMs idle: the
// long requests' tokens dealt out evenly to as many segments as there are SMs for a kv head each, a chunk at least
// (with two at least a prompt of 700 tokens, 16/1 heads, takes 29 us for 22, two of 750-1500, 28/4 heads, 37 for 30,
// two of 150-300 the same 28.5).  A cut costs a first pass over K and V (about a third of the whole), so a batch
// whose longest request is not longer than two such shares, or than kWholeTokens, stays whole (8 prompts of 256-4096
// tokens and 32 heads take 169 us cut at one share and 168 whole; one of 16001 tokens and 8 kv heads 677 whole and 112
// cut).  In any other every request longer than a share is cut, so that none keeps the others' SMs waiting.
constexpr int kWholeSegment = 1 << 30;
constexpr int kWholeTokens = 4 * kChunk;
#ifdef __CUDACC__
__host__ __device__
#endif
inline int segment_share(int64_t long_tokens, int kv_heads, int sms) {
    const int64_t segments = sms / kv_heads > 0 ? sms / kv_heads : 1;
    const int64_t n = ((long_tokens + segments - 1) / segments + kChunk - 1) / kChunk * kChunk;
    return n < kChunk ? kChunk : n < kWholeSegment ? (int)n : kWholeSegment;
}
#ifdef __CUDACC__
__host__ __device__
#endif
inline int segment_tokens(int64_t long_tokens, int longest, int kv_heads, int sms) {
    const int n = segment_share(long_tokens, kv_heads, sms);
    return longest <= 2 * (int64_t)n || longest <= kWholeTokens ? kWholeSegment : n;
}

// Whether a batch's layer calls launch the states pass and the scan: known on the host from its bounds alone (the long
// requests have all tokens but kStepTokens of each short one at most).
inline bool may_cut(int64_t total_tokens, int64_t batch, int longest_bound, int kv_heads, int sms) {
    const int64_t least = total_tokens - kStepTokens * batch;
    return segment_tokens(least > 0 ? least : 0, longest_bound, kv_heads, sms) < kWholeSegment;
}

// What the plan goes by: it cuts only where those two kernels run, since the main pass starts a request's later
// segments from what they leave.
#ifdef __CUDACC__
__host__ __device__
#endif
inline int planned_segment_tokens(bool cuts_run, int64_t long_tokens, int longest, int kv_heads, int sms) {
    return cuts_run ? segment_tokens(long_tokens, longest, kv_heads, sms) : kWholeSegment;
}

// CTAs that share a kv head's q heads (two heads or more each), where the segments' kv heads are fewer than the SMs.
// Each of them finds the state for itself: two prompts of 500 tokens, 28/4 heads, take 39 us, with one CTA a kv
// head 67; one, 16/1 heads, 26 and 126.
#ifdef __CUDACC__
__host__ __device__
#endif
inline int head_parts(int64_t segments, int group, int kv_heads, int sms) {
    int64_t n = segments > 0 ? sms / (segments * kv_heads) : 1;
    if (n > group / 2) n = group / 2;
    return n < 1 ? 1 : (int)n;
}

// Workspace carve-up.  The header is a PlanHeader: error_bits, wait_override, n_pre_tiles (segments of long
// requests), n_casc_tiles (those of them whose states the first pass finds), n_casc_groups (requests with such) and
// n_casc_units (the CTAs that share a kv head's q heads).
struct LinLayout {
    size_t header;
    size_t tok_req;     // int32 [max_tokens]: request of each new token
    size_t req_state;   // int2 [max_batch]: state slots (in, out) of each request, in = -2: skipped
    size_t req_base;    // int32 [max_batch]: of a long request whose start is copied, its LinItem::base; else -1
    size_t claim;       // int32 [num_states]: the last request that claimed a slot as its out
    size_t items;       // LinItem [max_items], most tokens first
    size_t pre_items;   // LinItem [max_segs]: the segments of the first pass
    size_t cut_items;   // LinItem [max_segs]: the first segments of requests that are cut
    size_t seg_state;   // fp32 [max_segs][Hkv][D/4 (columns)][D (rows)][4]: a request's entry 0: a copy of its start; s:
                        // segment s - 1's end from zero, after the scan the request's state there
    size_t seg_decay;   // fp32 [max_segs][Hkv]: entry s: the decay over segment s - 1, -1: a token of it drops the state
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
    int32_t group;
    int32_t num_kv_heads;
    int32_t sm_count;
    int32_t may_cut;           // LinHost's
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
    int32_t may_cut;    // some request may be cut into segments
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
cudaError_t launch_linear_scan(const LinParams& p, int head_dim, cudaStream_t s);
// states: the first pass (the segments' states), else the outputs
cudaError_t launch_linear_chunks(const LinParams& p, int head_dim, bool states, int ctas, cudaStream_t s);

}  // namespace pva

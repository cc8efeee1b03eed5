// The C ABI of linear attention and of the norm of q and k (declared in include/pva.h): argument checks
// that need no GPU, workspace planning, and kernel launches.
#include <cuda_runtime.h>

#include <cmath>
#include <cstring>

#include "linear.h"

namespace pva {
namespace {

int device_sm_count() {
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    return sms;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

pva_status check_config(const pva_linear_config* c) {
    if (c == nullptr) return PVA_ERR_INVALID_ARG;
    if (c->num_qo_heads <= 0 || c->num_kv_heads <= 0 || c->num_states <= 0 || c->max_batch <= 0 || c->max_tokens < 0 ||
        c->num_qo_heads % c->num_kv_heads != 0 || std::isnan(c->scale) || std::isinf(c->scale))
        return PVA_ERR_INVALID_ARG;
    if ((c->head_dim != 64 && c->head_dim != 128) || c->max_batch > 65535 || c->num_states >= ((int64_t)1 << 31) ||
        c->num_qo_heads > 65535)
        return PVA_ERR_UNSUPPORTED;
    return PVA_OK;
}

LinLayout make_layout(const pva_linear_config* c, int sms) {
    LinLayout L{};
    L.max_items = (int32_t)(c->max_tokens / kChunk + c->max_batch + 1);
    // Segments with a state in the workspace.  Of a cut request: at most twice what its tokens fill (it is longer than
    // two shares), and all requests' tokens fill sms / Hkv shares or one; of whole ones whose q heads several CTAs
    // share: there are at most sms / (2 Hkv) of those.
    L.max_segs = 3 * (sms / c->num_kv_heads) + 3;
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off = align_up(off + bytes, 256);
        return at;
    };
    L.header = take(sizeof(PlanHeader));
    L.tok_req = take(sizeof(int32_t) * ((size_t)c->max_tokens + 1));
    L.req_state = take(sizeof(int2) * (size_t)c->max_batch);
    L.req_base = take(sizeof(int32_t) * (size_t)c->max_batch);
    L.claim = take(sizeof(int32_t) * (size_t)c->num_states);
    L.items = take(sizeof(LinItem) * (size_t)L.max_items);
    L.pre_items = take(sizeof(LinItem) * (size_t)L.max_segs);
    L.cut_items = take(sizeof(LinItem) * (size_t)L.max_segs);
    L.seg_state = take(sizeof(float) * (size_t)L.max_segs * c->num_kv_heads * c->head_dim * c->head_dim);
    L.seg_decay = take(sizeof(float) * (size_t)L.max_segs * c->num_kv_heads);
    L.total = off;
    return L;
}

// What attn_norm_rope and the linear calls need of a batch of either kind.
struct BatchView {
    const int32_t* cu;
    const int32_t* seqlens;
    const int32_t* tok_req;
    int32_t batch, total_tokens, num_qo_heads, num_kv_heads, head_dim, sm_count;
    uint8_t* header;
};

bool view_of(const pva_meta* meta, BatchView* v) {
    if (meta == nullptr) return false;
    if (const LinHost* l = lin_of(meta)) {
        *v = BatchView{l->cu, l->seqlens, reinterpret_cast<const int32_t*>(l->ws + l->lay.tok_req), l->batch,
                       l->total_tokens, l->cfg.num_qo_heads, l->cfg.num_kv_heads, l->cfg.head_dim, l->sm_count,
                       l->ws + l->lay.header};
        return true;
    }
    const MetaHost* h = reinterpret_cast<const MetaHost*>(meta->opaque);
    if (h->magic != kMetaMagic) return false;
    *v = BatchView{h->cu, h->seqlens, h->tok_req, h->batch, h->total_tokens, h->cfg.num_qo_heads, h->cfg.num_kv_heads,
                   h->cfg.head_dim, h->sm_count, h->ws + h->lay.header};
    return true;
}

// Memory from the first to the last element of T tokens' heads, ld elements between tokens.
struct Span {
    uintptr_t lo, hi;
};
Span span_of(const void* x, int64_t T, int64_t ld, int64_t row) {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(x);
    return x == nullptr || T <= 0 ? Span{0, 0} : Span{lo, lo + (uintptr_t)(((T - 1) * ld + row) * 2)};
}
bool meet(const Span& a, const Span& b) { return a.lo < b.hi && b.lo < a.hi; }

pva_status check_norm_rope(const BatchView& v, const pva_qk_norm* norm, const pva_rope* rope, const void* q, const void* k,
                           const void* q_out, const void* k_out) {
    const int64_t T = v.total_tokens, rq = (int64_t)v.num_qo_heads * v.head_dim, rk = (int64_t)v.num_kv_heads * v.head_dim;
    const pva_status st = check_rotation(rope, norm, v.head_dim);
    if (st != PVA_OK) return st;
    if (T > 0 && ((q == nullptr && k == nullptr) || (q != nullptr) != (q_out != nullptr) || (k != nullptr) != (k_out != nullptr)))
        return PVA_ERR_INVALID_ARG;
    if ((q != nullptr && (rope->ld_q < rq || rope->ld_q % 8 != 0)) || (k != nullptr && (rope->ld_k < rk || rope->ld_k % 8 != 0)))
        return PVA_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(q_out) || !aligned16(k_out)) return PVA_ERR_INVALID_ARG;
    const Span sq = span_of(q, T, rope->ld_q, rq), sk = span_of(k, T, rope->ld_k, rk);
    const Span oq = span_of(q_out, T, rq, rq), ok = span_of(k_out, T, rk, rk);
    const bool q_in_place = q == q_out && (T <= 1 || rope->ld_q == rq), k_in_place = k == k_out && (T <= 1 || rope->ld_k == rk);
    if ((!q_in_place && meet(oq, sq)) || (!k_in_place && meet(ok, sk)) || meet(oq, sk) || meet(ok, sq) || meet(oq, ok))
        return PVA_ERR_INVALID_ARG;
    return PVA_OK;
}

pva_status launch_flat(const BatchView& v, const pva_qk_norm* norm, const pva_rope* rope, const void* q, const void* k,
                       void* q_out, void* k_out, bool zero_refused, cudaStream_t s) {
    ForwardParams fp{};
    fp.k = static_cast<const uint16_t*>(k);
    fp.v = fp.k;  // (never read: there are no rows of v)
    fp.cu = v.cu;
    fp.seqlens = v.seqlens;
    fp.tok_req = v.tok_req;
    fp.total_tokens = v.total_tokens;
    fp.num_qo_heads = v.num_qo_heads;
    fp.num_kv_heads = v.num_kv_heads;
    fp.group = v.num_qo_heads / v.num_kv_heads;
    fp.ws = v.header;  // (its layout's header offset is 0)
    RopeParams rp{};
    rp.q = static_cast<const uint16_t*>(q);
    rp.q_out = static_cast<uint16_t*>(q_out);
    rp.k_out = static_cast<uint16_t*>(k_out);
    rp.ld_q = rope->ld_q;
    rp.ld_k = rope->ld_k;
    rp.batch = v.batch;
    rp.sm_count = v.sm_count;
    rp.zero_refused = zero_refused ? 1 : 0;
    set_rotation(rope, norm, &rp);
    return launch_norm_rope(fp, rp, v.head_dim, s) == cudaSuccess ? PVA_OK : PVA_ERR_CUDA;
}

pva_status check_linear(const LinHost* h, const pva_linear_args* a, const void* q, const void* k, const void* v,
                        const void* out, int64_t ld_q, int64_t ld_k, int64_t ld_v) {
    const int64_t T = h->total_tokens, D = h->cfg.head_dim, rq = h->cfg.num_qo_heads * D, rk = h->cfg.num_kv_heads * D;
    if (a == nullptr || a->log_decay == nullptr || a->states == nullptr) return PVA_ERR_INVALID_ARG;
    if (a->ld_decay != 0 && a->ld_decay < h->cfg.num_kv_heads) return PVA_ERR_INVALID_ARG;
    if (T > 0 && (q == nullptr || k == nullptr || v == nullptr || out == nullptr)) return PVA_ERR_INVALID_ARG;
    if (ld_q < rq || ld_k < rk || ld_v < rk || ld_q % 8 != 0 || ld_k % 8 != 0 || ld_v % 8 != 0) return PVA_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out) || !aligned16(a->states) ||
        (reinterpret_cast<uintptr_t>(a->log_decay) & 3u) != 0)
        return PVA_ERR_INVALID_ARG;
    if (T == 0) return PVA_OK;
    // rows of q, k, v and states are read while others' results, out's and the states', are written
    const Span o = span_of(out, T, rq, rq), sq = span_of(q, T, ld_q, rq), sk = span_of(k, T, ld_k, rk), sv = span_of(v, T, ld_v, rk);
    const int64_t decays = a->ld_decay ? (T - 1) * a->ld_decay + h->cfg.num_kv_heads : h->cfg.num_kv_heads;
    const uintptr_t g = reinterpret_cast<uintptr_t>(a->log_decay), st = reinterpret_cast<uintptr_t>(a->states);
    const Span states{st, st + (uintptr_t)(h->cfg.num_states * h->cfg.num_kv_heads * D * D * 4)};
    const Span sg{g, g + (uintptr_t)(decays * 4)};
    if (meet(o, states)) return PVA_ERR_INVALID_ARG;
    for (const Span& x : {sq, sk, sv, sg})
        if (meet(o, x) || meet(states, x)) return PVA_ERR_INVALID_ARG;
    return PVA_OK;
}

pva_status launch_linear(const LinHost* h, const pva_linear_args* a, const void* q, const void* k, const void* v, void* out,
                         int64_t ld_q, int64_t ld_k, int64_t ld_v, cudaStream_t s) {
    if (h->total_tokens == 0) return PVA_OK;
    LinParams p{};
    p.q = static_cast<const uint16_t*>(q);
    p.k = static_cast<const uint16_t*>(k);
    p.v = static_cast<const uint16_t*>(v);
    p.out = static_cast<uint16_t*>(out);
    p.ld_q = ld_q;
    p.ld_k = ld_k;
    p.ld_v = ld_v;
    p.log_decay = a->log_decay;
    p.ld_decay = a->ld_decay;
    p.states = a->states;
    p.cu = h->cu;
    p.batch = h->batch;
    p.total_tokens = h->total_tokens;
    p.num_qo_heads = h->cfg.num_qo_heads;
    p.num_kv_heads = h->cfg.num_kv_heads;
    p.group = h->cfg.num_qo_heads / h->cfg.num_kv_heads;
    p.sm_count = h->sm_count;
    p.scale = h->cfg.scale > 0.f ? h->cfg.scale : 1.0f / std::sqrt((float)h->cfg.head_dim);
    p.ws = h->ws;
    p.lay = h->lay;
    const int D = h->cfg.head_dim;
    // requests of few tokens first: their CTAs are short, and the tensor-core kernel's take whole SMs
    if (launch_linear_step(p, D, s) != cudaSuccess) return PVA_ERR_CUDA;
    if (h->max_q_len <= kStepTokens) return PVA_OK;
    if (h->may_cut && (launch_linear_chunks(p, D, true, h->sm_count, s) != cudaSuccess ||
                       launch_linear_scan(p, D, s) != cudaSuccess))
        return PVA_ERR_CUDA;
    return launch_linear_chunks(p, D, false, h->sm_count, s) == cudaSuccess ? PVA_OK : PVA_ERR_CUDA;
}

}  // namespace

// Host checks of a rotation and a norm (which may come without one) for heads of D.
pva_status check_rotation(const pva_rope* rope, const pva_qk_norm* norm, int64_t D) {
    if (rope == nullptr || rope->reserved != 0 || rope->rot_dim < 0 || rope->rot_dim > D) return PVA_ERR_INVALID_ARG;
    if (rope->rot_dim == 0 && norm == nullptr) return PVA_ERR_INVALID_ARG;
    if (rope->rot_dim > 0 && (rope->cos_sin == nullptr || rope->max_positions <= 0)) return PVA_ERR_INVALID_ARG;
    if (rope->rot_dim % 16 != 0) return PVA_ERR_UNSUPPORTED;
    if (!aligned16(rope->cos_sin) || (reinterpret_cast<uintptr_t>(rope->positions) & 3u) != 0) return PVA_ERR_INVALID_ARG;
    if (norm != nullptr && (norm->reserved != 0 || !(norm->eps >= 0.f) || std::isinf(norm->eps) || !aligned16(norm->q_gain) ||
                            !aligned16(norm->k_gain)))
        return PVA_ERR_INVALID_ARG;
    return PVA_OK;
}

void set_rotation(const pva_rope* rope, const pva_qk_norm* norm, RopeParams* rp) {
    rp->cos_sin = rope->cos_sin;
    rp->positions = rope->positions;
    rp->max_positions = rope->max_positions;
    rp->rot_dim = rope->rot_dim;
    rp->interleaved = rope->interleaved ? 1 : 0;
    if (norm != nullptr) {
        rp->norm = 1;
        rp->q_gain = norm->q_gain;
        rp->k_gain = norm->k_gain;
        rp->eps = norm->eps;
    }
}

}  // namespace pva

using namespace pva;

extern "C" {

size_t attn_linear_workspace_size(const pva_linear_config* cfg) {
    if (check_config(cfg) != PVA_OK) return 0;
    const int sms = device_sm_count();
    return sms > 0 ? make_layout(cfg, sms).total : 0;
}

pva_status attn_linear_prepare(const pva_linear_config* cfg, const int32_t* cu_seqlens_q, const int32_t* cache_seqlens,
                               const int32_t* state_in, const int32_t* state_out, int32_t batch, int32_t total_tokens,
                               int32_t max_q_len, void* workspace, size_t workspace_bytes, void* stream, pva_meta* meta) {
    const pva_status st = check_config(cfg);
    if (st != PVA_OK) return st;
    if (meta == nullptr || cu_seqlens_q == nullptr || (batch > 0 && cache_seqlens == nullptr)) return PVA_ERR_INVALID_ARG;
    if (batch < 0 || total_tokens < 0 || (batch == 0 && total_tokens != 0)) return PVA_ERR_INVALID_ARG;
    if (batch > cfg->max_batch || total_tokens > cfg->max_tokens) return PVA_ERR_INVALID_ARG;
    if (workspace == nullptr || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return PVA_ERR_INVALID_ARG;
    const int sms = device_sm_count();
    if (sms <= 0) return PVA_ERR_CUDA;
    LinHost h{};
    h.magic = kLinMagic;
    h.cfg = *cfg;
    h.lay = make_layout(cfg, sms);
    if (workspace_bytes < h.lay.total) return PVA_ERR_WORKSPACE_TOO_SMALL;
    h.batch = batch;
    h.total_tokens = total_tokens;
    h.max_q_len = max_q_len > 0 && max_q_len < total_tokens ? max_q_len : (total_tokens > 0 ? total_tokens : 1);
    h.sm_count = sms;
    h.may_cut = may_cut(total_tokens, batch, h.max_q_len, cfg->num_kv_heads, sms) ? 1 : 0;
    h.cu = cu_seqlens_q;
    h.seqlens = cache_seqlens;
    h.ws = static_cast<uint8_t*>(workspace);
    h.stream = stream;
    LinPlanParams pp{};
    pp.cu = cu_seqlens_q;
    pp.seqlens = cache_seqlens;
    pp.state_in = state_in;
    pp.state_out = state_out;
    pp.batch = batch;
    pp.total_tokens = total_tokens;
    pp.max_q_len = h.max_q_len;
    pp.group = cfg->num_qo_heads / cfg->num_kv_heads;
    pp.num_kv_heads = cfg->num_kv_heads;
    pp.sm_count = sms;
    pp.may_cut = h.may_cut;
    pp.num_states = cfg->num_states;
    pp.ws = h.ws;
    pp.lay = h.lay;
    if (launch_linear_plan(pp, static_cast<cudaStream_t>(stream)) != cudaSuccess) return PVA_ERR_CUDA;
    std::memset(meta, 0, sizeof(*meta));
    std::memcpy(meta->opaque, &h, sizeof(h));
    return PVA_OK;
}

pva_status attn_linear_forward(const pva_meta* meta, const pva_linear_args* args, const void* q, const void* k,
                               const void* v, void* out, void* stream) {
    const LinHost* h = lin_of(meta);
    if (h == nullptr) return PVA_ERR_NOT_PREPARED;
    if (args == nullptr) return PVA_ERR_INVALID_ARG;
    const pva_status st = check_linear(h, args, q, k, v, out, args->ld_q, args->ld_k, args->ld_v);
    if (st != PVA_OK) return st;
    return launch_linear(h, args, q, k, v, out, args->ld_q, args->ld_k, args->ld_v, static_cast<cudaStream_t>(stream));
}

pva_status attn_linear_forward_norm_rope(const pva_meta* meta, const pva_linear_args* args, const pva_qk_norm* norm,
                                         const pva_rope* rope, const void* q, const void* k, const void* v, void* q_rot,
                                         void* k_rot, void* out, void* stream) {
    const LinHost* h = lin_of(meta);
    if (h == nullptr) return PVA_ERR_NOT_PREPARED;
    BatchView view;
    (void)view_of(meta, &view);
    if (h->total_tokens > 0 && (q == nullptr || k == nullptr)) return PVA_ERR_INVALID_ARG;
    pva_status st = check_norm_rope(view, norm, rope, q, k, q_rot, k_rot);
    if (st != PVA_OK) return st;
    const int64_t D = h->cfg.head_dim, rq = h->cfg.num_qo_heads * D, rk = h->cfg.num_kv_heads * D, T = h->total_tokens;
    st = check_linear(h, args, q_rot, k_rot, v, out, rq, rk, rope->ld_v);
    if (st != PVA_OK) return st;
    // v, the decays and the states are read after q_rot and k_rot were written
    const int64_t decays = args->ld_decay ? (T - 1) * args->ld_decay + h->cfg.num_kv_heads : h->cfg.num_kv_heads;
    const uintptr_t g = reinterpret_cast<uintptr_t>(args->log_decay), s0 = reinterpret_cast<uintptr_t>(args->states);
    const Span sv = span_of(v, T, rope->ld_v, rk), sg{g, g + (uintptr_t)(decays * 4)};
    const Span ss{s0, s0 + (uintptr_t)(h->cfg.num_states * h->cfg.num_kv_heads * D * D * 4)};
    for (const Span& o : {span_of(q_rot, T, rq, rq), span_of(k_rot, T, rk, rk)})
        if (meet(o, sv) || meet(o, sg) || meet(o, ss)) return PVA_ERR_INVALID_ARG;
    if (T == 0) return PVA_OK;
    // (a refused token's rows become 0: what lay in q_rot and k_rot must not enter a state that is kept)
    st = launch_flat(view, norm, rope, q, k, q_rot, k_rot, true, static_cast<cudaStream_t>(stream));
    if (st != PVA_OK) return st;
    return launch_linear(h, args, q_rot, k_rot, v, out, rq, rk, rope->ld_v, static_cast<cudaStream_t>(stream));
}

pva_status attn_norm_rope(const pva_meta* meta, const pva_qk_norm* norm, const pva_rope* rope, const void* q,
                          const void* k, void* q_out, void* k_out, void* stream) {
    BatchView v;
    if (!view_of(meta, &v)) return PVA_ERR_NOT_PREPARED;
    const pva_status st = check_norm_rope(v, norm, rope, q, k, q_out, k_out);
    if (st != PVA_OK) return st;
    if (v.total_tokens == 0) return PVA_OK;
    return launch_flat(v, norm, rope, q, k, q_out, k_out, false, static_cast<cudaStream_t>(stream));
}

}  // extern "C"

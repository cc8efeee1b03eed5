"""Cases that measure the norm of q and k with the position rotation, and linear attention with decays.

Three kinds of call, each a layer's call of a serving engine on a prepared batch:
  append  norm q and k head by head, rotate them by position, write q out and append k / v to the
          paged pool (bf16 or E4M3);
  flat    the same without a pool: q and k to tensors of their own, as a linear layer takes them;
  linear  linear attention with a decay for each head over a pool of states: every token's output and
          the requests' new states.

``own`` False computes them with elementary torch operations in fp32 (sums of decays in 64 bits, one
rounding at the end), True calls the library.
"""
import math
import random

import torch

own = False

DEV = "cuda"
EPS = 1e-6


def _case(name, kind, hq, hkv, d, b, n, c, big=0, pool="bf16", ps=16, rot=0, inter=False, packed=False, gate="head", lens=1):
    """n / c: least and most new / cached tokens a request; with big, only so many requests have n, the others
    one token; gate: one decay a head, or one a head and token; lens: seed of the lengths."""
    return {"name": name, "kind": kind, "hq": hq, "hkv": hkv, "d": d, "b": b, "n_lo": n[0], "n_hi": n[1],
            "c_lo": c[0], "c_hi": c[1], "big": big, "pool": pool, "ps": ps, "rot": rot, "inter": inter, "packed": packed,
            "gate": gate, "lens": lens}


def listed():
    return [
        # one user's next token: latency of the call
        _case("append 1 token bf16", "append", 32, 8, 128, 1, (1, 1), (777, 777), rot=128),
        # a decode batch over a token-slot E4M3 pool, interleaved pairs, slices of one fused projection
        _case("append 64 decodes e4m3", "append", 28, 4, 128, 64, (1, 1), (0, 1000), pool="e4m3", ps=1, rot=128,
              inter=True, packed=True),
        # a prefill batch
        _case("append prefill bf16", "append", 32, 8, 128, 8, (256, 4096), (0, 0), rot=128, packed=True),
        # chunks of many requests on their way to a linear layer, half of the head rotated
        _case("flat chunks", "flat", 32, 32, 128, 16, (1, 1024), (0, 500), rot=64, packed=True),
        # a decode batch's
        _case("flat 64 decodes", "flat", 32, 32, 128, 64, (1, 1), (511, 4095), rot=128, packed=True),
        # one user's next token through a linear layer
        _case("linear 1 token", "linear", 32, 32, 128, 1, (1, 1), (777, 777)),
        # a decode batch: every state is read and written
        _case("linear 64 decodes", "linear", 32, 32, 128, 64, (1, 1), (511, 4095)),
        # a few tokens a request, gated by token
        _case("linear 40x4 tokens", "linear", 16, 16, 64, 40, (4, 4), (0, 300), gate="token"),
        # a prefill batch of fresh prompts
        _case("linear prefill", "linear", 32, 32, 128, 8, (256, 4096), (0, 0), packed=True),
        # one long prompt, grouped heads: few states, so the length is split
        _case("linear 1 x 16k", "linear", 32, 8, 128, 1, (16001, 16001), (0, 0), gate="token"),
        # chunks that go on from a state, odd lengths
        _case("linear chunks D64", "linear", 16, 16, 64, 12, (33, 900), (0, 1800), gate="token"),
        # decodes with two prompts' chunks among them
        _case("linear mixed", "linear", 28, 4, 128, 42, (700, 1500), (0, 3000), big=2, gate="token"),
    ]


def draw(rng):
    log = lambda lo, hi: int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    kind = rng.choice(["append", "append", "flat", "linear", "linear", "linear", "linear"])
    hq, hkv, d = rng.choice([(32, 32, 128), (32, 8, 128), (28, 4, 128), (16, 1, 128), (8, 8, 128), (64, 16, 128),
                             (16, 16, 64), (16, 2, 64), (4, 2, 64)])
    ps = rng.choice([1, 2, 4, 8, 16, 32, 64, 128])
    pool = rng.choice(["bf16", "e4m3"]) if kind == "append" else "bf16"
    rot = rng.choice([0, d, d, d // 2, 32]) if kind != "linear" else 0
    inter = bool(rot) and rng.random() < 0.4
    packed = rng.random() < 0.5
    gate = rng.choice(["head", "token"])
    big = 0
    if kind in ("append", "flat"):
        total = log(1, 12000 if kind == "append" else 7000)
        b = min(total, log(1, 100))
        mean = max(1, total // b)
        n = (max(1, mean // 2), max(1, mean + mean // 2))
        c = (0, log(1, 600))
    else:
        c = rng.choice([(0, 0), (0, log(1, 2000)), (1, log(2, 2000))])
        shape = rng.choice(["decode", "few", "prompts", "prompts", "long", "mixed"])
        if shape in ("decode", "few"):
            b = log(1, 64)
            k = 1 if shape == "decode" else rng.randint(2, 9)
            n = (k, k)
        elif shape == "prompts":
            b = log(1, 16)
            hi = log(20, min(100000, 16000 * 128 * 32 // (max(hq, 2 * hkv) * d)) // b)
            n = (max(1, hi // log(1, 8)), hi)
        elif shape == "long":
            b = 1
            hi = log(3000, min(100000, 16000 * 128 * 32 // (max(hq, 2 * hkv) * d)))
            n = (hi, hi)
        else:
            b = log(3, 60)
            big = rng.randint(1, 2)
            hi = log(40, 1800)
            n = (max(1, hi // 2), hi)
    return _case("", kind, hq, hkv, d, b, n, c, big=big, pool=pool, ps=ps, rot=rot, inter=inter, packed=packed, gate=gate,
                 lens=rng.randrange(1 << 20))


def _lengths(case):
    r = random.Random(case["lens"])
    q = [r.randint(case["n_lo"], case["n_hi"]) for _ in range(case["b"])]
    if case["big"]:
        at = r.sample(range(case["b"]), case["big"])
        q = [n if i in at else 1 for i, n in enumerate(q)]
    return q, [n + r.randint(case["c_lo"], case["c_hi"]) for n in q]


def work(case):
    q, kv = _lengths(case)
    hq, hkv, d, kind = case["hq"], case["hkv"], case["d"], case["kind"]
    T = sum(q)
    rope = min(T, max(kv)) * case["rot"] * 4 + 2 * d * 4
    if kind == "append":
        return {"bytes": 4 * T * hq * d + 4 * T * hkv * d + 2 * T * hkv * d * (2 if case["pool"] == "bf16" else 1) + rope,
                "flops": 0}
    if kind == "flat":
        return {"bytes": 4 * T * (hq + hkv) * d + rope, "flops": 0}
    states = hkv * d * d * 4 * (len(q) + sum(L > n for n, L in zip(q, kv)))
    byts = 2 * T * (2 * hq + 2 * hkv) * d + states + 4 * hkv * (T if case["gate"] == "token" else 1)
    return {"bytes": byts, "flops": 2 * d * d * (hq + hkv) * T}


# ------------------------------------------------------------------ inputs

class _State:
    pass


def prepare(case, seed):
    s = _State()
    s.case = case
    kind = case["kind"]
    q, kv = _lengths(case)
    hq, hkv, d, ps, B, T = case["hq"], case["hkv"], case["d"], case["ps"], case["b"], sum(q)
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 1000003 + 17)
    randn = lambda *shape: torch.randn(*shape, generator=g, device=DEV)
    rand = lambda *shape: torch.rand(*shape, generator=g, device=DEV)
    s.T, s.max_q, s.max_kv = T, max(q), max(kv)
    s.q_lens = torch.tensor(q, device=DEV)
    s.kv_lens = torch.tensor(kv, device=DEV)
    s.cu = torch.zeros(B + 1, dtype=torch.int32, device=DEV)
    s.cu[1:] = torch.cumsum(s.q_lens, 0)
    s.cache_seqlens = s.kv_lens.to(torch.int32)
    # each new token's request and position
    s.req = torch.repeat_interleave(torch.arange(B, device=DEV), s.q_lens, output_size=T)
    s.row = torch.arange(T, device=DEV) - s.cu[:-1].long()[s.req]
    s.pos = (s.kv_lens - s.q_lens)[s.req] + s.row
    # this step's activations, some channels larger: tensors of their own, or slices of one projection
    channel = 1.0 + 2.0 * rand(hq + 2 * hkv, d) ** 4
    x = (randn(T, hq + 2 * hkv, d) * channel).to(torch.bfloat16)
    s.q, s.k, s.v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    if not case["packed"]:
        s.q, s.k, s.v = s.q.contiguous(), s.k.contiguous(), s.v.contiguous()
    s.q_out, s.k_out = (torch.empty(T, h, d, dtype=torch.bfloat16, device=DEV) for h in (hq, hkv))
    s.out = torch.empty_like(s.q_out)
    if kind != "linear":
        s.q_gain, s.k_gain = 1.0 + 0.2 * randn(d), 1.0 + 0.2 * randn(d)
        s.cos_sin = None
        if case["rot"]:   # cos and sin of every position's angles, formed in 64 bits
            inv = 10000.0 ** (-torch.arange(0, case["rot"], 2, dtype=torch.float64, device=DEV) / case["rot"])
            ang = torch.arange(s.max_kv, dtype=torch.float64, device=DEV)[:, None] * inv
            s.cos_sin = torch.cat((ang.cos(), ang.sin()), 1).to(torch.float32).contiguous()
    if kind == "append":   # pages placed at random in a pool that earlier steps have filled
        need = (s.kv_lens + ps - 1) // ps
        s.pages = sum(-(-L // ps) for L in kv) + 3
        perm = torch.randperm(s.pages, generator=g, device=DEV)
        start = torch.cumsum(need, 0) - need
        j = torch.arange(-(-max(kv) // ps), device=DEV)
        s.table = torch.where(j < need[:, None], perm[(start[:, None] + j).clamp(max=s.pages - 1)], 0).to(torch.int32)
        s.slots = s.table.long()[s.req, s.pos // ps] * ps + s.pos % ps
        s.k_pool, s.v_pool = (randn(s.pages * ps, hkv, d).to(torch.bfloat16) for _ in range(2))
        s.k_scale = s.v_scale = None
        if case["pool"] == "e4m3":
            s.k_scale, s.v_scale = 0.01 + 0.02 * rand(hkv), 0.01 + 0.02 * rand(hkv)
            s.k_pool, s.v_pool = (x.to(torch.float8_e4m3fn).view(torch.uint8) for x in (s.k_pool, s.v_pool))
    if kind == "linear":
        # a pool of states: each request goes on from one and leaves its new one in another
        s.states = randn(2 * B + 1, hkv, d, d)
        perm = torch.randperm(2 * B + 1, generator=g, device=DEV).to(torch.int32)
        s.state_in, s.state_out = perm[:B].contiguous(), perm[B:2 * B].contiguous()
        # decays: from a few tokens' memory to some thousands, head by head; by token: spread around that
        slope = -(2.0 ** (-10.0 * (torch.arange(hkv, device=DEV) + rand(hkv)) / hkv))
        s.log_decay = slope if case["gate"] == "head" else slope * torch.nn.functional.softplus(2 * randn(T, hkv))
    if own:
        _plan(s)
    return s


def _plan(s):
    """The engine's handle of this batch, made once a step and used by every layer."""
    from paged_variable_length_gb300 import pva

    c = s.case
    if c["kind"] == "append":
        dtype = {"bf16": pva.KV_BF16, "e4m3": pva.KV_E4M3}[c["pool"]]
        s.engine = pva.PagedAttention(c["hq"], c["hkv"], c["d"], c["ps"], s.pages, max_batch=c["b"], max_tokens=s.T,
                                      max_kv_len=s.max_kv, device=DEV, kv_dtype=dtype)
        s.engine.prepare(s.cu, s.cache_seqlens, s.table, s.T, max_q_len=s.max_q)
    else:
        s.engine = pva.LinearAttention(c["hq"], c["hkv"], c["d"], 2 * c["b"] + 1, max_batch=c["b"], max_tokens=s.T,
                                       device=DEV)
        plain = c["kind"] == "flat"   # (no states are touched)
        s.engine.prepare(s.cu, s.cache_seqlens, s.T, None if plain else s.state_in, None if plain else s.state_out,
                         max_q_len=s.max_q)
    s.rope = s.norm = None
    if c["kind"] != "linear":
        s.norm = pva.QKNorm(s.q_gain, s.k_gain, eps=EPS)
        if c["rot"]:
            s.rope = pva.Rope(s.cos_sin, rot_dim=c["rot"], interleaved=c["inter"])


# ------------------------------------------------------------------ one pass

def run(s):
    kind = s.case["kind"]
    if kind == "append":
        if own:
            s.engine.append(s.q, s.k, s.v, s.k_pool, s.v_pool, s.rope, q_out=s.q_out, k_scale=s.k_scale,
                            v_scale=s.v_scale, norm=s.norm)
        else:
            s.q_out.copy_(_rotate(_norm(s.q, s.q_gain), s))
            k, v = _rotate(_norm(s.k, s.k_gain), s), s.v
            if s.case["pool"] == "e4m3":
                enc = lambda x, sc: (x / sc[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
                k, v = enc(k, s.k_scale), enc(v.float(), s.v_scale)
            s.k_pool[s.slots], s.v_pool[s.slots] = k.to(s.k_pool.dtype), v
        see = lambda x: x.view(torch.float8_e4m3fn) if s.case["pool"] == "e4m3" else x
        return {"q": s.q_out, "k": see(s.k_pool), "v": see(s.v_pool)}
    if kind == "flat":
        if own:
            s.engine.norm_rope(s.q, s.k, rope=s.rope, norm=s.norm, q_out=s.q_out, k_out=s.k_out)
        else:
            _flat(s)
        return {"q": s.q_out, "k": s.k_out}
    if own:
        s.engine.forward(s.q, s.k, s.v, s.log_decay, s.states, out=s.out)
    else:
        _linear(s)
    return {"out": s.out, "states": s.states}


def _norm(x, gain):
    x = x.float()
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * gain


def _rotate(x, s):
    rot = s.case["rot"]
    if not rot:
        return x
    cs = s.cos_sin[s.pos]
    c, sn = cs[:, None, :rot // 2], cs[:, None, rot // 2:]
    y = x.clone()
    if s.case["inter"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * c - b * sn, b * c + a * sn
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = a * c - b * sn, b * c + a * sn
    return y


def _flat(s):
    s.q_out.copy_(_rotate(_norm(s.q, s.q_gain), s))
    s.k_out.copy_(_rotate(_norm(s.k, s.k_gain), s))


def _linear(s):
    """All requests at once, padded to whole chunks of tokens: products inside a chunk, the chunks' own
    states, and the state before each chunk as a weighted sum of those before it."""
    c = s.case
    B, hq, hkv, d = c["b"], c["hq"], c["hkv"], c["d"]
    C = min(128, s.max_q)
    nc = -(-s.max_q // C)
    i = torch.arange(nc * C, device=DEV)
    held = i < s.q_lens[:, None]                                                   # [B, n]
    tok = torch.where(held, s.cu[:-1].long()[:, None] + i, 0)
    take = lambda x: torch.where(held[..., None, None], x[tok].float(), 0.0).reshape(B, nc, C, x.shape[1], d)
    qp = take(s.q).reshape(B, nc, C, hkv, hq // hkv, d)
    kp, vp = take(s.k), take(s.v)
    ld = s.log_decay.double()
    ld = ld[tok] if c["gate"] == "token" else ld.expand(B, nc * C, hkv)
    cum = torch.where(held[..., None], ld, 0.0).reshape(B, nc, C, hkv).cumsum(2)   # decay since the chunk's start
    end = cum[:, :, -1]                                                            # [B, nc, H]
    # the chunks' own states, and the state before each
    own_s = torch.einsum("bnchd,bnche->bnhde", kp * torch.exp(end[:, :, None] - cum).float()[..., None], vp)
    acc = end.cumsum(1)
    before = acc - end
    n = torch.arange(nc, device=DEV)
    w = torch.where((n[:, None] > n)[None, :, :, None], before[:, :, None] - acc[:, None], -math.inf)
    old = torch.where((s.kv_lens > s.q_lens)[:, None, None, None], s.states[s.state_in.long()], 0.0)
    prev = torch.einsum("bmnh,bnhde->bmhde", torch.exp(w).float(), own_s)
    prev = prev + torch.exp(before).float()[..., None, None] * old[:, None]
    # outputs
    j = torch.arange(C, device=DEV)
    u = cum.permute(0, 1, 3, 2)
    u = torch.where(j[:, None] >= j, u[..., :, None] - u[..., None, :], -math.inf)    # [B, nc, H, C, C]
    p = torch.einsum("bnihgd,bnjhd->bnhgij", qp, kp) * torch.exp(u).float()[:, :, :, None]
    o = torch.einsum("bnhgij,bnjhe->bnihge", p, vp)
    o = o + torch.einsum("bnihgd,bnhde->bnihge", qp, prev) * torch.exp(cum).float()[..., None, None]
    o = (o / math.sqrt(d)).reshape(B, nc * C, hq, d)
    s.out.copy_(o[s.req, s.row])
    s.states[s.state_out.long()] = prev[:, -1] * torch.exp(end[:, -1]).float()[..., None, None] + own_s[:, -1]


# ------------------------------------------------------------------ the definition, in 64 bits

def _turned(x, gain, s):
    """Each head over its root mean square, times the gain; then each pair as a complex number, times e^(i angle)."""
    rot = s.case["rot"]
    x = x.double()
    x = x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt() * gain.double()
    if not rot:
        return x
    w = torch.complex(s.cos_sin[s.pos, :rot // 2].double(), s.cos_sin[s.pos, rot // 2:].double())[:, None]
    head, tail = x[..., :rot], x[..., rot:]
    if s.case["inter"]:
        z = torch.view_as_complex(head.reshape(*head.shape[:-1], rot // 2, 2).contiguous()) * w
        head = torch.view_as_real(z).reshape(head.shape)
    else:
        z = torch.complex(*(h.contiguous() for h in head.chunk(2, -1))) * w
        head = torch.cat((z.real, z.imag), -1)
    return torch.cat((head, tail), -1)


def _grid8(x):
    """float64 -> the E4M3 values nearest to it (saturating)."""
    a = x.abs()
    step = 2.0 ** (torch.floor(torch.log2(a.clamp(min=2.0 ** -6))).clamp(-6, 8) - 3)
    return torch.sign(x) * (torch.round(a / step) * step).clamp(max=448.0)


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    kind = case["kind"]
    got = {}
    q, k, v = s.q.double(), s.k.double(), s.v.double()
    if kind != "linear":
        q, k = got["q"], got["k"] = _turned(s.q, s.q_gain, s), _turned(s.k, s.k_gain, s)
    if kind == "flat":
        return got
    if kind == "append":
        whole = lambda p: p.double()
        if case["pool"] == "e4m3":
            k, v = _grid8(k / s.k_scale.double()[:, None]), _grid8(v / s.v_scale.double()[:, None])
            whole = lambda p: p.view(torch.float8_e4m3fn).double()
        got["k"], got["v"] = whole(s.k_pool), whole(s.v_pool)
        got["k"][s.slots], got["v"][s.slots] = k, v
        return got
    # the recurrence, a token of every request that has one left at a time
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    n = s.q_lens.tolist()
    order = sorted(range(case["b"]), key=lambda i: -n[i])
    first = s.cu[:-1].long()[torch.tensor(order, device=DEV)]
    S = torch.where((s.kv_lens > s.q_lens)[:, None, None, None], s.states[s.state_in.long()].double(), 0.0)
    S = S[torch.tensor(order, device=DEV)]
    out = torch.empty(s.T, hq, d, dtype=torch.float64, device=DEV)
    live = case["b"]
    lam = torch.exp(s.log_decay.double())
    for t in range(s.max_q):
        while n[order[live - 1]] <= t:
            live -= 1
        at = first[:live] + t
        lt = lam[at] if case["gate"] == "token" else lam
        S[:live] *= lt[..., None, None]
        S[:live] += k[at][..., :, None] * v[at][..., None, :]
        out[at] = torch.matmul(q[at].reshape(live, hkv, hq // hkv, d), S[:live]).reshape(live, hq, d) / math.sqrt(d)
    states = s.states.double()
    states[s.state_out.long()[torch.tensor(order, device=DEV)]] = S
    return {"out": out, "states": states}

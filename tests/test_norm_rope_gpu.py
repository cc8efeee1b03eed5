"""GPU tests of the norm of q and k with the position rotation: on the way to the pools (attn_append_norm_rope,
attn_forward_norm_rope) and into tensors (attn_norm_rope), against the definition in 64 bits."""
import numpy as np
import pytest
import torch

import linear_reference as L
import mx_reference as R
import oracle
from harness import assert_close, make_engine
from paged_variable_length_gb300 import pva
from paged_variable_length_gb300 import workloads as W

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF16, E4M3, MX = pva.KV_BF16, pva.KV_E4M3, pva.KV_MXFP4
EPS = 1e-5


def positions_of(wl):
    return np.concatenate([np.arange(n, dtype=np.int64) + (L - n) for n, L in zip(wl.q_lens, wl.kv_lens)])


def expected(x, gain, table, pos, interleaved):
    """[T, H, D] in 64 bits, and how far fp32 may be off before the last rounding.  The sum of squares takes 16 fused
    additions and up to 4 more (each 2^-24 of it), its mean and eps two roundings, the reciprocal root 2 ulp, half of
    the sum's error passing through it; two products; then a rotation's three roundings of terms up to |y1| + |y2|:
    below 2^-24 * 32 of those."""
    y = L.norm_heads(x, gain, EPS).cpu().numpy()
    rot = 0 if table is None else table.shape[1]
    z = R.rotate(y, table.cpu().numpy(), pos, interleaved, np.float64) if rot else y
    pair = np.abs(y).copy()
    if rot:
        a, b = (np.s_[..., 0:rot:2], np.s_[..., 1:rot:2]) if interleaved else (np.s_[..., :rot // 2], np.s_[..., rot // 2:rot])
        both = pair[a] + pair[b]
        pair[a], pair[b] = both, both
    return z, 2.0 ** -24 * 32 * pair + 1e-38


def setup(case, seed=0, packed=False, positions=None):
    Hq, Hkv, D, ps, ql, kl, rot = case
    wl = W.custom(ql, kl, Hq, Hkv, D, ps, seed=Hq + D + seed)
    T = wl.total_tokens
    g = torch.Generator(device=DEV).manual_seed(wl.seed + 1)
    x = torch.randn(T, Hq + 2 * Hkv, D, generator=g, device=DEV) * torch.exp(2 * torch.randn(T, Hq + 2 * Hkv, 1, generator=g, device=DEV))
    x = x.to(torch.bfloat16)
    x[0, 0] = 0        # a head of zeros
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    if not packed:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    gains = [1 + 0.3 * torch.randn(D, generator=g, device=DEV) for _ in range(2)]
    pos = positions_of(wl) if positions is None else np.asarray(positions)
    table = pva.rope_table(int(pos.max()) + 1, rot, device=DEV) if rot else None
    cu, sl, pt = (torch.as_tensor(a, dtype=torch.int32, device=DEV) for a in (wl.cu_seqlens_q, wl.cache_seqlens, wl.page_table))
    return wl, (q, k, v), gains, pos, table, (cu, sl, pt)


CASES = [
    (32, 8, 128, 16, [1], [1], 128),
    (32, 8, 128, 16, [1, 1, 7, 0, 1], [1, 16, 17, 9, 700], 128),
    (28, 4, 128, 1, [3, 1, 40], [5, 2, 90], 64),
    (8, 8, 64, 4, [1, 9, 16], [3, 20, 16], 64),
    (4, 2, 64, 8, [5, 1, 1], [33, 1, 65], 32),
    (16, 1, 128, 32, [1, 5], [200, 5], 96),
    (24, 3, 128, 2, [2, 3], [11, 3], 48),
    (5, 5, 64, 64, [1, 2], [70, 129], 16),
    (32, 2, 128, 128, [1, 200], [300, 260], 112),
    (32, 32, 128, 16, [1, 150], [40, 300], 0),      # the norm alone
    (6, 3, 64, 16, [1, 3], [40, 3], 0),
]
IDS = [f"{c[0]}-{c[1]}-{c[2]}-ps{c[3]}-rot{c[6]}" for c in CASES]
KINDS = pytest.mark.parametrize("dtype", [BF16, E4M3, MX], ids=["bf16", "e4m3", "mxfp4"])


def check_bf16(got, z, lim):
    assert (np.abs(got.double().cpu().numpy() - z) <= 2.0 ** -8 * np.abs(z) + lim * (1 + 2.0 ** -8)).all()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_into_tensors(case, interleaved):
    """attn_norm_rope on plans of both kinds, strided and in place, with and without gains."""
    wl, (q, k, v), (gq, gk), pos, table, (cu, sl, pt) = setup(case, packed=interleaved)
    rope = None if table is None else pva.Rope(table, interleaved=interleaved)
    zq, zk = (expected(x, g, table, pos, interleaved) for x, g in ((q, gq), (k, gk)))
    paged = make_engine(wl)
    paged.prepare(cu, sl, pt, wl.total_tokens)
    lin = pva.LinearAttention(wl.num_qo_heads, wl.num_kv_heads, wl.head_dim, 1, wl.batch, wl.total_tokens)
    lin.prepare(cu, sl, wl.total_tokens)
    norm = pva.QKNorm(gq, gk, eps=EPS)
    first = None
    for eng in (paged, lin):
        q_out, k_out = eng.norm_rope(q, k, rope=rope, norm=norm)
        torch.cuda.synchronize()
        assert pva.attn_get_device_status(eng.meta) == 0
        check_bf16(q_out, *zq)
        check_bf16(k_out, *zk)
        if first is not None:
            assert torch.equal(first[0], q_out) and torch.equal(first[1], k_out)
        first = q_out, k_out
    # one of the two alone, in place, no gains
    q2, none = lin.norm_rope(q, None, rope=rope, norm=norm)
    assert none is None and torch.equal(q2, first[0])
    _, k2 = lin.norm_rope(None, k, rope=rope, norm=norm)
    assert torch.equal(k2, first[1])
    qc, kc = q.clone().contiguous(), k.clone().contiguous()
    lin.norm_rope(qc, kc, rope=rope, norm=norm, q_out=qc, k_out=kc)
    assert torch.equal(qc, first[0]) and torch.equal(kc, first[1])
    q3, k3 = lin.norm_rope(q, k, rope=rope, norm=pva.QKNorm(eps=EPS))
    ones = torch.ones(wl.head_dim, device=DEV)
    for got, x in ((q3, q), (k3, k)):
        check_bf16(got, *expected(x, None, table, pos, interleaved))
    q4, k4 = lin.norm_rope(q, k, rope=rope, norm=pva.QKNorm(ones, ones, eps=EPS))
    assert torch.equal(q3, q4) and torch.equal(k3, k4)
    if rope is not None:      # the rotation alone is attn_append_rope's
        q5, k5 = lin.norm_rope(q, k, rope=rope)
        cs = table.cpu().numpy()
        for got, x in ((q5, q), (k5, k)):
            want = R.rotate(x.float().cpu().numpy(), cs, pos, interleaved, np.float32)
            assert torch.equal(got.cpu(), torch.as_tensor(want).to(torch.bfloat16))


@KINDS
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_append(case, dtype):
    """The pools hold the normed and rotated k (as attn_norm_rope makes it, in the pool's type) and v, and nothing
    else changes."""
    interleaved = case[2] == 64
    wl, (q, k, v), (gq, gk), pos, table, (cu, sl, pt) = setup(case, packed=True)
    Hkv, D, T = wl.num_kv_heads, wl.head_dim, wl.total_tokens
    rope = None if table is None else pva.Rope(table, interleaved=interleaved)
    norm = pva.QKNorm(gq, gk, eps=EPS)
    per = {BF16: Hkv * D * 2, E4M3: Hkv * D, MX: R.row_layout(Hkv, D)[2]}[dtype]
    g = torch.Generator(device=DEV).manual_seed(9)
    kp, vp = (torch.randint(0, 256, (wl.num_slots, per), generator=g, device=DEV, dtype=torch.uint8) for _ in range(2))
    before = [x.clone() for x in (kp, vp)]
    ks = vs = None
    if dtype == E4M3:
        ks, vs = (torch.rand(Hkv, generator=g, device=DEV) * 0.05 + 0.013 for _ in range(2))
    eng = make_engine(wl, kv_dtype=dtype)
    eng.prepare(cu, sl, pt, T)
    q_out = eng.append(q, k, v, kp, vp, rope, k_scale=ks, v_scale=vs, norm=norm)
    torch.cuda.synchronize()
    assert pva.attn_get_device_status(eng.meta) == 0
    flat_q, flat_k = eng.norm_rope(q, k, rope=rope, norm=norm)
    assert torch.equal(q_out, flat_q)
    slots = torch.as_tensor(oracle.slot_mapping(wl.cu_seqlens_q, wl.cache_seqlens, wl.page_table, wl.page_size), device=DEV)
    used = Hkv * (D // 2 + D // 32) if dtype == MX else per
    kept = torch.ones(wl.num_slots, dtype=torch.bool, device=DEV)
    kept[slots] = False
    for pool, was in ((kp, before[0]), (vp, before[1])):
        assert torch.equal(pool[kept], was[kept]) and torch.equal(pool[slots, used:], was[slots, used:])
    z, lim = expected(k, gk, table, pos, interleaved)
    if dtype == BF16:
        assert torch.equal(kp[slots].view(torch.bfloat16).view(T, Hkv, D), flat_k)
        assert torch.equal(vp[slots].view(torch.bfloat16).view(T, Hkv, D), v)
    elif dtype == E4M3:
        # between the codes of the ends of what fp32 may have made of it (the codec is monotone)
        s = ks.double().cpu().numpy()[None, :, None]
        div = lambda x: np.float32(x / s)
        lo, hi = (oracle.e4m3_decode(oracle.e4m3_encode(div(x))) for x in (z - lim * 1.01, z + lim * 1.01))
        got = oracle.e4m3_decode(kp[slots].cpu().numpy().reshape(T, Hkv, D))
        assert (got >= np.minimum(lo, hi)).all() and (got <= np.maximum(lo, hi)).all()
        want = oracle.e4m3_encode((v.float().cpu().numpy() / vs.cpu().numpy()[None, :, None]).astype(np.float32))
        assert np.array_equal(vp[slots].cpu().numpy().reshape(T, Hkv, D), want)
    else:
        # Codes of a value as near as fp32 leaves it.  With S the larger of the scales that a block's largest
        # magnitude may give (a power of two may lie between what fp32 and 64 bits make of it), half a code step is
        # S/4 up to 2 S, S/2 up to 3 S and S up to 6 S, which stands for all above; with S/2 the largest code is 3 S,
        # and what it stands for reaches 4 S.
        kb, vb = eng.load(kp, vp)
        got = kb.double().cpu().numpy()
        blocks, err = np.abs(z).reshape(T, Hkv, D // 32, 32), lim.reshape(T, Hkv, D // 32, 32)
        top = (blocks + err).max(-1)[..., None]
        S = 2.0 ** (np.floor(np.log2(top)) - 2).clip(-22, 13)
        room = S * np.where(blocks <= 2 * S, 0.25, np.where(blocks <= 3 * S, 0.5, 1.0))
        room = np.maximum(room, blocks - 6 * S)
        assert (np.abs(got - z) <= (room.reshape(z.shape) + lim) * (1 + 2.0 ** -8)).all()
        assert np.array_equal(vb.double().cpu().numpy(), R.unpack_rows(R.pack_rows(v.float().cpu().numpy()), Hkv, D))


@pytest.mark.parametrize("dtype", [BF16, E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("ql,kl", [([1, 1, 4, 1], [700, 33, 40, 1]), ([40, 1, 130], [40, 900, 300])], ids=["decode", "prefill"])
def test_layer_call_equals_its_parts(dtype, ql, kl):
    """attn_forward_norm_rope: the append's q and pools, then the attention of those (against the oracle)."""
    wl = W.custom(ql, kl, 16, 4, 128, 16, seed=len(ql))
    T = wl.total_tokens
    t = W.make_tensors(wl, DEV, poison_unused=True)
    if dtype == E4M3:
        kp, vp, ks, vs = W.make_fp8_pools(wl, DEV, poison_unused=True)
    else:
        kp, vp, ks, vs = t["k_pool"], t["v_pool"], None, None
    gains = [1 + 0.3 * torch.randn(128, device=DEV) for _ in range(2)]
    norm, rope = pva.QKNorm(*gains), pva.Rope(pva.rope_table(max(kl), 128, device=DEV))
    eng = make_engine(wl, kv_dtype=dtype)
    eng.prepare(t["cu_seqlens_q"], t["cache_seqlens"], t["page_table"], T)
    kp2, vp2 = kp.clone(), vp.clone()
    q_rot = eng.append(t["q"], t["k"], t["v"], kp2, vp2, rope, k_scale=ks, v_scale=vs, norm=norm)
    lse = torch.empty(T, 16, dtype=torch.float32, device=DEV)
    q_in = torch.empty_like(t["q"])
    out = eng.forward(t["q"], t["k"], t["v"], kp, vp, lse=lse, k_scale=ks, v_scale=vs, rope=rope, norm=norm, q_rot=q_in)
    torch.cuda.synchronize()
    assert pva.attn_get_device_status(eng.meta) == 0
    assert torch.equal(q_in, q_rot)
    assert torch.equal(kp.view(torch.uint8), kp2.view(torch.uint8)) and torch.equal(vp.view(torch.uint8), vp2.view(torch.uint8))
    args = (wl.cu_seqlens_q, wl.cache_seqlens, wl.page_table, wl.page_size)
    if dtype == BF16:
        ref_o, ref_l, _, _ = oracle.forward(q_rot.cpu(), t["k"].cpu(), t["v"].cpu(), kp2.cpu(), vp2.cpu(), *args,
                                            slots=np.full(T, -1, np.int64))
    else:
        ref_o, ref_l = oracle.attention_fp8(q_rot.cpu(), kp2.cpu(), vp2.cpu(), ks.cpu(), vs.cpu(), *args)
    assert_close(out, lse, ref_o, ref_l)


def test_far_explicit_and_foreign_positions():
    case = (4, 1, 64, 128, [2, 1], [200_001, 131_073], 64)
    wl, (q, k, v), (gq, gk), pos, table, (cu, sl, pt) = setup(case)
    norm = pva.QKNorm(gq, gk, eps=EPS)
    lin = pva.LinearAttention(4, 1, 64, 1, 2, 3)
    lin.prepare(cu, sl, 3)
    q_out, k_out = lin.norm_rope(q, k, rope=pva.Rope(table), norm=norm)
    check_bf16(q_out, *expected(q, gq, table, pos, False))
    given = torch.tensor([5, 0, 77], dtype=torch.int32, device=DEV)
    q_out, k_out = lin.norm_rope(q, k, rope=pva.Rope(table, positions=given), norm=norm)
    check_bf16(k_out, *expected(k, gk, table, given.cpu().numpy(), False))
    assert pva.attn_get_device_status(lin.meta) == 0
    # a position outside the table is reported, and its token's rows stay
    q_out.fill_(7.0), k_out.fill_(7.0)
    lin.norm_rope(q, k, rope=pva.Rope(table, positions=torch.tensor([5, -1, 200_001], dtype=torch.int32, device=DEV)), norm=norm,
                  q_out=q_out, k_out=k_out)
    torch.cuda.synchronize()
    assert pva.attn_get_device_status(lin.meta) == 0x40
    assert bool((q_out[1:] == 7).all()) and bool((k_out[1:] == 7).all()) and not bool((q_out[0] == 7).all())


def test_nan_stays_in_its_head():
    wl, (q, k, v), (gq, gk), pos, table, (cu, sl, pt) = setup((8, 2, 128, 16, [5], [9], 96))
    norm, rope = pva.QKNorm(gq, gk, eps=EPS), pva.Rope(table)
    lin = pva.LinearAttention(8, 2, 128, 1, 1, 5)
    lin.prepare(cu, sl, 5)
    want = lin.norm_rope(q, k, rope=rope, norm=norm)
    q2 = q.clone()
    q2[3, 5, 100] = float("nan")
    got = lin.norm_rope(q2, k, rope=rope, norm=norm)
    assert bool(torch.isnan(got[0][3, 5]).all())
    got[0][3, 5] = want[0][3, 5]
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])

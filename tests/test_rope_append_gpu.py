"""GPU tests of the rotary append (attn_append_rope, attn_forward_rope).

The kernel's arithmetic is fixed (fp32 products and sums, each rounded by itself, one rounding
into what holds the result), so q_out and the pools are compared bit for bit with the same steps
in numpy, and with the definition in 64 bits within what those steps allow."""
import numpy as np
import pytest
import torch

import mx_reference as R
import oracle
from harness import assert_close, make_engine
from paged_variable_length_gb300 import pva
from paged_variable_length_gb300 import workloads as W

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF16, E4M3, MX = pva.KV_BF16, pva.KV_E4M3, pva.KV_MXFP4


def bf16(x):
    return torch.as_tensor(np.asarray(x, np.float32)).to(torch.bfloat16)


def bits(t):
    return t.detach().cpu().contiguous().view(torch.int16).numpy()


def pools(wl, dtype, seed=0):
    """Pools of arbitrary bytes: what the append does not write stays as it was."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    per = {BF16: wl.num_kv_heads * wl.head_dim * 2, E4M3: wl.num_kv_heads * wl.head_dim,
           MX: R.row_layout(wl.num_kv_heads, wl.head_dim)[2]}[dtype]
    kp, vp = (torch.randint(0, 256, (wl.num_slots, per), generator=g, device=DEV, dtype=torch.uint8) for _ in range(2))
    if dtype == BF16:
        shape = (wl.num_slots, wl.num_kv_heads, wl.head_dim)
        kp, vp = kp.view(torch.bfloat16).view(shape), vp.view(torch.bfloat16).view(shape)
    elif dtype == E4M3:
        kp, vp = (x.view(wl.num_slots, wl.num_kv_heads, wl.head_dim) for x in (kp, vp))
    return kp, vp


def positions_of(wl):
    return np.concatenate([np.arange(L - n, L) for n, L in zip(wl.q_lens, wl.kv_lens)]).astype(np.int64)


def rows_of(x, dtype, scale):
    """fp32 [T, Hkv, D] -> the pool rows' bytes [T, ...]."""
    T = x.shape[0]
    if dtype == BF16:
        return bf16(x).view(torch.uint8).numpy().reshape(T, -1)
    if dtype == E4M3:
        return oracle.e4m3_encode((x / scale[None, :, None]).astype(np.float32)).reshape(T, -1)
    return R.pack_rows(x)


def check_append(wl, dtype, rot, interleaved=False, packed=False, slot_mapping=None, positions=None, in_place=False,
                 forward=False):
    T, Hq, Hkv, D = wl.total_tokens, wl.num_qo_heads, wl.num_kv_heads, wl.head_dim
    g = torch.Generator(device=DEV).manual_seed(wl.seed + 1)
    if packed:
        qkv = torch.randn(T, Hq + 2 * Hkv, D, generator=g, device=DEV).to(torch.bfloat16)
        q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    else:
        q, k, v = (torch.randn(T, h, D, generator=g, device=DEV).to(torch.bfloat16) for h in (Hq, Hkv, Hkv))
    hq, hk, hv = (x.float().cpu().numpy() for x in (q, k, v))
    kp, vp = pools(wl, dtype)
    before = [x.clone().view(torch.uint8).cpu().numpy().reshape(wl.num_slots, -1) for x in (kp, vp)]
    ks = vs = None
    if dtype == E4M3:
        ks, vs = (torch.rand(Hkv, generator=g, device=DEV) * 0.05 + 0.013 for _ in range(2))
    pos = positions_of(wl) if positions is None else np.asarray(positions)
    table = pva.rope_table(int(pos.max()) + 1 if T else 1, rot, device=DEV)
    rope = pva.Rope(table, interleaved=interleaved, positions=None if positions is None else
                    torch.as_tensor(pos, dtype=torch.int32, device=DEV))
    eng = make_engine(wl, kv_dtype=dtype)
    cu, sl, pt = (torch.as_tensor(x, dtype=torch.int32, device=DEV) for x in (wl.cu_seqlens_q, wl.cache_seqlens, wl.page_table))
    sm = None if slot_mapping is None else torch.as_tensor(slot_mapping, dtype=torch.int64, device=DEV)
    eng.prepare(cu, sl, pt, T, sm)
    q_out = q if in_place else torch.empty(T, Hq, D, dtype=torch.bfloat16, device=DEV)
    got = eng.append(q, k, v, kp, vp, rope, q_out=q_out, k_scale=ks, v_scale=vs)
    torch.cuda.synchronize()
    assert got is q_out and pva.attn_get_device_status(eng.meta) == 0
    cs = table.cpu().numpy()
    yq, yk = (R.rotate(x, cs, pos, interleaved, np.float32) for x in (hq, hk))
    assert np.array_equal(bits(q_out), bits(bf16(yq))), "rotated q"
    # and the definition in 64 bits: three fp32 roundings of terms up to |x1| + |x2|, then half a bf16 step
    ref = R.rotate(hq, cs, pos, interleaved, np.float64)
    lim = 2.0 ** -8 * np.abs(ref) + 2.0 ** -22 * (np.abs(hq).max() * 2) + 2.0 ** -133
    assert (np.abs(q_out.float().cpu().numpy() - ref) <= lim).all()
    slots = oracle.slot_mapping(wl.cu_seqlens_q, wl.cache_seqlens, wl.page_table, wl.page_size) \
        if slot_mapping is None else np.asarray(slot_mapping)
    for pool, was, x, sc, name in ((kp, before[0], yk, ks, "K"), (vp, before[1], hv, vs, "V")):
        want = was.copy()
        new = rows_of(x, dtype, None if sc is None else sc.cpu().numpy())
        if dtype == MX:  # the row's padding is not written
            used = Hkv * (D // 2 + D // 32)
            want[slots[slots >= 0], :used] = new[slots >= 0, :used]
        else:
            want[slots[slots >= 0]] = new[slots >= 0]
        assert np.array_equal(pool.view(torch.uint8).cpu().numpy().reshape(wl.num_slots, -1), want), f"{name} pool"
    return eng, (q, k, v, q_out, kp, vp, ks, vs, rope)


# (Hq, Hkv, D, ps, q_lens, kv_lens, rot)
CASES = [
    (32, 8, 128, 16, [1], [1], 128),
    (32, 8, 128, 16, [1, 1, 7, 0, 1], [1, 16, 17, 9, 700], 128),
    (28, 4, 128, 1, [3, 1, 40], [5, 2, 90], 64),
    (8, 8, 64, 4, [1, 9, 16], [3, 20, 16], 64),
    (4, 2, 64, 8, [5, 1, 1], [33, 1, 65], 32),
    (16, 1, 128, 32, [1, 5], [200, 5], 96),
    (24, 3, 128, 2, [2, 3], [11, 3], 48),       # 3 chunks apart
    (5, 5, 64, 64, [1, 2], [70, 129], 16),      # 1 chunk apart
    (32, 2, 128, 128, [1, 200], [300, 260], 112),
    (32, 32, 128, 16, [1, 3], [40, 3], 128),
    (16, 16, 64, 1, [1, 1, 1], [9, 1, 7], 64),
]
IDS = [f"{c[0]}-{c[1]}-{c[2]}-ps{c[3]}-rot{c[6]}" for c in CASES]


@pytest.mark.parametrize("dtype", [BF16, E4M3, MX], ids=["bf16", "e4m3", "mxfp4"])
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_append(case, dtype):
    Hq, Hkv, D, ps, ql, kl, rot = case
    wl = W.custom(ql, kl, Hq, Hkv, D, ps, seed=Hq + D)
    check_append(wl, dtype, rot)
    check_append(wl, dtype, rot, interleaved=True, packed=True)


@pytest.mark.parametrize("dtype", [BF16, E4M3, MX], ids=["bf16", "e4m3", "mxfp4"])
def test_append_in_place_strided_and_explicit(dtype):
    wl = W.custom([3, 1, 20], [40, 1, 20], 8, 2, 128, 4, seed=3)
    check_append(wl, dtype, 128, in_place=True)
    check_append(wl, dtype, 64, packed=True, positions=[(7 * t) % 101 for t in range(wl.total_tokens)])
    slots = oracle.slot_mapping(wl.cu_seqlens_q, wl.cache_seqlens, wl.page_table, wl.page_size)[::-1].copy()
    slots[2] = slots[11] = -1   # padding tokens: q is rotated, nothing is stored
    check_append(wl, dtype, 128, slot_mapping=slots, interleaved=True)


def test_append_without_q_and_an_empty_batch():
    wl = W.custom([3, 1], [40, 1], 8, 2, 64, 4, seed=3)
    eng, (q, k, v, _, kp, vp, _, _, rope) = check_append(wl, BF16, 64)
    want = kp.clone(), vp.clone()
    for x in (kp, vp):
        x.zero_()
    assert eng.append(None, k, v, kp, vp, rope) is None
    torch.cuda.synchronize()
    sl = torch.as_tensor(oracle.slot_mapping(wl.cu_seqlens_q, wl.cache_seqlens, wl.page_table, wl.page_size), device=DEV)
    assert torch.equal(kp[sl], want[0][sl]) and torch.equal(vp[sl], want[1][sl])
    eng.prepare(torch.zeros(1, dtype=torch.int32, device=DEV), torch.zeros(0, dtype=torch.int32, device=DEV),
                torch.zeros(0, 1, dtype=torch.int32, device=DEV), 0)
    eng.append(q[:0], k[:0], v[:0], kp, vp, rope)
    eng.forward(q[:0], k[:0], v[:0], kp, vp, rope=rope)
    torch.cuda.synchronize()
    assert pva.attn_get_device_status(eng.meta) == 0


def test_far_positions():
    """A position past 2^17 in a long request (the table holds 64-bit angles), few tokens."""
    wl = W.custom([2, 1], [200_001, 131_073], 4, 1, 64, 128, seed=2)
    check_append(wl, BF16, 64)


def test_a_position_outside_the_table_is_reported_and_skipped():
    wl = W.custom([3, 1], [10, 1], 8, 2, 64, 4, seed=3)
    eng, (q, k, v, q_out, kp, vp, _, _, rope) = check_append(wl, BF16, 64)
    table = rope.cos_sin[:9].contiguous()     # request 0's last token is position 9
    q_out.fill_(7.0)
    was_k = kp.clone().fill_(3.0)
    kp.fill_(3.0)
    eng.append(q, k, v, kp, vp, pva.Rope(table), q_out=q_out)
    torch.cuda.synchronize()
    assert pva.attn_get_device_status(eng.meta) == 0x40
    assert (q_out[2] == 7.0).all() and not (q_out[1] == 7.0).all()
    slots = oracle.slot_mapping(wl.cu_seqlens_q, wl.cache_seqlens, wl.page_table, wl.page_size)
    assert torch.equal(kp[int(slots[2])], was_k[int(slots[2])]) and not (kp[int(slots[1])] == 3.0).all()
    # a negative explicit position
    cu, sl, pt = (torch.as_tensor(x, dtype=torch.int32, device=DEV) for x in (wl.cu_seqlens_q, wl.cache_seqlens, wl.page_table))
    eng.prepare(cu, sl, pt, wl.total_tokens)
    pos = torch.tensor([0, -1, 2, 3], dtype=torch.int32, device=DEV)
    eng.append(q, k, v, kp, vp, pva.Rope(table, positions=pos), q_out=q_out)
    assert pva.attn_get_device_status(eng.meta) == 0x40


def test_bad_pages_and_slots_are_reported():
    wl = W.custom([1, 1], [10, 3], 8, 2, 64, 4, seed=3)
    for dtype in (BF16, MX):
        eng, (q, k, v, q_out, kp, vp, _, _, rope) = check_append(wl, dtype, 64)
        cu, sl = (torch.as_tensor(x, dtype=torch.int32, device=DEV) for x in (wl.cu_seqlens_q, wl.cache_seqlens))
        pt = torch.as_tensor(wl.page_table, dtype=torch.int32, device=DEV).clone()
        good = pt.clone()
        pt[0, 2] = wl.num_pages       # the page of request 0's new token
        eng.prepare(cu, sl, pt, 2)
        was = kp.clone()
        eng.append(q, k, v, kp, vp, rope, q_out=q_out)
        assert pva.attn_get_device_status(eng.meta) & 0x04
        same = (kp.view(torch.uint8) == was.view(torch.uint8)).reshape(wl.num_slots, -1).all(1)
        slots = oracle.slot_mapping(wl.cu_seqlens_q, wl.cache_seqlens, wl.page_table, wl.page_size)
        assert bool(same[[i for i in range(wl.num_slots) if i != slots[1]]].all())
        eng.prepare(cu, sl, good, 2, torch.tensor([wl.num_slots, -2], device=DEV))
        eng.append(q, k, v, kp, vp, rope, q_out=q_out)
        assert pva.attn_get_device_status(eng.meta) & 0x08


def test_refusals_launch_nothing():
    wl = W.custom([3, 1], [10, 1], 8, 2, 64, 4, seed=3)
    eng, (q, k, v, q_out, kp, vp, _, _, rope) = check_append(wl, BF16, 64, packed=True)
    eng8, _ = check_append(wl, E4M3, 64)
    out = torch.empty_like(q_out)

    def refused(status, engine=eng, **kw):
        a = dict(q=q, k=k, v=v, q_out=q_out, kp=kp, vp=vp, ks=None, vs=None)
        a.update({n: x for n, x in kw.items() if n in a})
        args = rope.args(q, k, v)
        for n, x in kw.items():
            if n not in a:
                setattr(args, n, x)
        with pytest.raises(pva.PvaError) as e:
            pva._check(pva.load().attn_append_rope(engine.meta, args, *[pva._ptr(a[n]) for n in (
                "q", "k", "v", "q_out", "kp", "vp", "ks", "vs")], pva._stream(None)), "append")
        assert e.value.status == status
        with pytest.raises(pva.PvaError) as e:
            pva._check(pva.load().attn_forward_rope(engine.meta, args, *[pva._ptr(a[n]) for n in (
                "q", "k", "v", "q_out", "kp", "vp", "ks", "vs")], pva._ptr(out), None, pva._stream(None)), "forward")
        assert e.value.status == status

    was = kp.clone()
    refused(1, cos_sin=None)
    refused(1, cos_sin=rope.cos_sin.data_ptr() + 4)
    refused(1, max_positions=0)
    refused(1, rot_dim=0)
    refused(1, rot_dim=80)
    refused(2, rot_dim=24)
    refused(1, reserved=1)
    refused(1, ld_q=8 * 64 - 8)
    refused(1, ld_k=2 * 64 + 4)
    refused(1, ld_v=64)
    refused(1, k=None)
    refused(1, v=None)
    refused(1, q_out=None)
    refused(1, kp=None)
    refused(1, q_out=q)                          # in place, but q is strided
    refused(1, q_out=k)                          # overlaps k
    refused(1, engine=eng8)                      # an E4M3 pool needs its scales
    assert torch.equal(kp.view(torch.int16), was.view(torch.int16))
    with pytest.raises(pva.PvaError):
        eng.load(kp, vp)                         # not an MXFP4 plan
    with pytest.raises(pva.PvaError):
        pva.attn_forward_mxfp4kv(eng.meta, q_out, k, v, kp, vp, out)


@pytest.mark.parametrize("dtype", [BF16, E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("ql,kl", [([1, 1, 4, 1], [700, 33, 40, 1]), ([40, 1, 130], [40, 900, 300])],
                         ids=["decode", "prefill"])
def test_forward_rope_equals_append_and_attention(dtype, ql, kl):
    """A layer's call over bf16 and E4M3 pools, against the oracle on rotated inputs."""
    wl = W.custom(ql, kl, 16, 4, 128, 16, seed=len(ql))
    T, Hkv, D = wl.total_tokens, 4, 128
    t = W.make_tensors(wl, DEV, poison_unused=True)
    if dtype == E4M3:
        kp, vp, ks, vs = W.make_fp8_pools(wl, DEV, poison_unused=True)
    else:
        kp, vp, ks, vs = t["k_pool"], t["v_pool"], None, None
    h = {n: x.detach().cpu().clone() for n, x in dict(t, kp=kp, vp=vp).items()}
    table = pva.rope_table(max(kl), 128, device=DEV)
    rope = pva.Rope(table)
    eng = make_engine(wl, kv_dtype=dtype)
    eng.prepare(t["cu_seqlens_q"], t["cache_seqlens"], t["page_table"], T)
    qkv = torch.cat((t["q"], t["k"], t["v"]), 1)
    lse = torch.empty(T, 16, dtype=torch.float32, device=DEV)
    q_rot = torch.empty_like(t["q"])
    out = eng.forward(qkv[:, :16], qkv[:, 16:20], qkv[:, 20:], kp, vp, lse=lse, k_scale=ks, v_scale=vs, rope=rope,
                      q_rot=q_rot)
    torch.cuda.synchronize()
    assert pva.attn_get_device_status(eng.meta) == 0
    pos, cs = positions_of(wl), table.cpu().numpy()
    yq = bf16(R.rotate(h["q"].float().numpy(), cs, pos, False, np.float32))
    yk = R.rotate(h["k"].float().numpy(), cs, pos, False, np.float32)
    assert np.array_equal(bits(q_rot), bits(yq))
    args = (wl.cu_seqlens_q, wl.cache_seqlens, wl.page_table, wl.page_size)
    if dtype == BF16:
        ref_o, ref_l, ref_kp, ref_vp = oracle.forward(yq, bf16(yk), h["v"], h["kp"], h["vp"], *args)
        assert np.array_equal(kp.cpu().view(torch.int16).numpy().view(np.uint16), ref_kp)
    else:
        slots = oracle.slot_mapping(*args)
        kc, vc = h["kp"].numpy().copy(), h["vp"].numpy().copy()
        kc[slots] = oracle.e4m3_encode((yk / ks.cpu().numpy()[None, :, None]).astype(np.float32))
        vc[slots] = oracle.e4m3_encode((h["v"].float().numpy() / vs.cpu().numpy()[None, :, None]).astype(np.float32))
        assert np.array_equal(kp.cpu().numpy(), kc) and np.array_equal(vp.cpu().numpy(), vc)
        ref_o, ref_l = oracle.attention_fp8(yq, torch.as_tensor(kc), torch.as_tensor(vc), ks.cpu(), vs.cpu(), *args)
    assert_close(out, lse, ref_o, ref_l)


def test_append_captured_with_the_plan_and_replayed():
    """prepare + two layers' forward_rope in one graph, replayed with new activations."""
    wl = W.custom([1, 3, 1], [50, 9, 700], 16, 4, 128, 16, seed=8)
    t = W.make_tensors(wl, DEV)
    eng = make_engine(wl)
    rope = pva.Rope(pva.rope_table(max(wl.kv_lens), 128, device=DEV), interleaved=True)
    layers = [(t["k_pool"].clone(), t["v_pool"].clone()) for _ in range(2)]
    outs = [torch.empty_like(t["q"]) for _ in range(2)]
    rot = [torch.empty_like(t["q"]) for _ in range(2)]

    def step(stream=None):
        eng.prepare(t["cu_seqlens_q"], t["cache_seqlens"], t["page_table"], wl.total_tokens, stream=stream)
        for (kp, vp), o, r in zip(layers, outs, rot):
            eng.forward(t["q"], t["k"], t["v"], kp, vp, out=o, rope=rope, q_rot=r, stream=stream)

    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step(s)
    for seed in (1, 2):
        for n in ("q", "k", "v"):
            t[n].copy_(torch.randn_like(t[n].float()).to(torch.bfloat16))
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in outs], [kp.clone() for kp, _ in layers]
        step()
        torch.cuda.synchronize()
        for i in range(2):
            assert torch.equal(got[0][i], outs[i]) and torch.equal(got[1][i], layers[i][0])


def test_forward_rope_refuses_an_output_over_the_rotated_q():
    wl = W.custom([3, 1], [10, 1], 8, 2, 64, 4, seed=3)
    eng, (q, k, v, q_out, kp, vp, _, _, rope) = check_append(wl, BF16, 64)
    room = torch.zeros(2, *q_out.shape, dtype=torch.bfloat16, device=DEV).view(-1)
    n, was = q_out.numel(), kp.clone()
    q_rot = room[:n].view(q_out.shape)
    for at in (0, 8, n - 8):
        with pytest.raises(pva.PvaError) as e:
            eng.forward(q, k, v, kp, vp, out=room[at:at + n].view(q_out.shape), rope=rope, q_rot=q_rot)
        assert e.value.status == 1
    torch.cuda.synchronize()
    assert torch.equal(kp.view(torch.int16), was.view(torch.int16)) and not bool(room.any())
    eng.forward(q, k, v, kp, vp, out=room[n:].view(q_out.shape), rope=rope, q_rot=q_rot)   # side by side
    torch.cuda.synchronize()
    assert torch.equal(q_rot, q_out)


def test_outputs_of_calls_on_another_stream():
    """Tensors that the binding allocates belong to the stream that writes them."""
    wl = W.custom([1, 300], [1, 300], 16, 4, 128, 16, seed=3)
    eng, (q, k, v, q_out, kp, vp, _, _, rope) = check_append(wl, MX, 128)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream, 0):
        got = eng.append(q, k, v, kp, vp, rope, stream=stream)
        k2, v2 = eng.load(kp, vp, stream=stream)
        out = torch.empty_like(q)
        eng.forward(q, k, v, kp, vp, out=out, rope=rope, stream=stream)
        noise = torch.empty_like(q).fill_(3.0)   # current stream: must not be given the rotated q's memory
        side.synchronize()
        torch.cuda.synchronize()
        assert torch.equal(got, q_out) and bool(torch.isfinite(out.float()).all()) and bool((noise == 3.0).all())
        assert torch.equal(eng.load(kp, vp)[0], k2) and torch.equal(eng.load(kp, vp)[1], v2)
        torch.cuda.synchronize()


def test_binding_refuses_strided_outputs_and_short_pools():
    wl = W.custom([3, 1], [10, 1], 8, 2, 64, 4, seed=3)
    eng, (q, k, v, q_out, kp, vp, _, _, rope) = check_append(wl, MX, 64)
    wide = torch.empty(wl.total_tokens, 8, 128, dtype=torch.bfloat16, device=DEV)
    for call in (lambda: eng.append(q, k, v, kp, vp, rope, q_out=wide[..., :64]),
                 lambda: eng.forward(q, k, v, kp, vp, out=wide[..., 64:], rope=rope),
                 lambda: eng.forward(wide[..., :64], k, v, kp, vp),
                 lambda: eng.load(kp, vp, k=wide[:, :2, :64], v=v.clone()),
                 lambda: eng.store(wide[:, :2, :64], v, kp, vp),
                 lambda: eng.store(k, v, kp[:-1], vp),
                 lambda: eng.append(q, k, v, kp, vp[1:], rope),
                 lambda: eng.load(kp[:0], vp),
                 lambda: eng.forward(q, k, v, kp[:4], vp, rope=rope)):
        with pytest.raises(pva.PvaError) as e:
            call()
        assert e.value.status == 1

"""GPU tests of the MXFP4 pool: store and read-back bit for bit, attention against the definition
in 64 bits over the same quantised values, within bounds formed from the kernels' roundings
(mx_reference.tolerances).  Slots that hold no request's key are arbitrary bytes (NaN scales among
them), and page-table columns past a request's last page point outside the pool."""
import numpy as np
import pytest
import torch

import mx_reference as R
import oracle
from harness import make_engine
from paged_variable_length_gb300 import pva
from paged_variable_length_gb300 import workloads as W

pytestmark = pytest.mark.gpu

DEV = "cuda"
MX = pva.KV_MXFP4


def make(wl, seed=0, spread=1.0):
    """q, k, v on the device and pools whose used slots hold quantised values of several magnitudes."""
    rng = np.random.default_rng(seed + 17)
    T, Hq, Hkv, D, ps = wl.total_tokens, wl.num_qo_heads, wl.num_kv_heads, wl.head_dim, wl.page_size
    rb = R.row_layout(Hkv, D)[2]
    kp, vp = (rng.integers(0, 256, (wl.num_slots, rb), dtype=np.uint8) for _ in range(2))
    mag = np.exp(spread * rng.standard_normal((1, Hkv, D // 32, 1)))
    for i, L in enumerate(wl.kv_lens):
        if L == 0:
            continue
        sl = slots_of(wl, i)
        for pool in (kp, vp):
            x = rng.standard_normal((L, Hkv, D // 32, 32)) * mag * np.exp(0.5 * rng.standard_normal((L, 1, 1, 1)))
            pool[sl] = R.pack_rows(x.reshape(L, Hkv, D).astype(np.float32))
    t = {n: torch.as_tensor(rng.standard_normal((T, h, D)).astype(np.float32)).to(torch.bfloat16).to(DEV)
         for n, h in (("q", Hq), ("k", Hkv), ("v", Hkv))}
    t["k"], t["v"] = (t["k"].float() * 1.7).to(torch.bfloat16), (t["v"].float() * 0.3).to(torch.bfloat16)
    t["kp"], t["vp"] = torch.as_tensor(kp).to(DEV), torch.as_tensor(vp).to(DEV)
    return t


def slots_of(wl, i):
    j = np.arange(wl.kv_lens[i])
    return wl.page_table[i].astype(np.int64)[j // wl.page_size] * wl.page_size + j % wl.page_size


def prepared(wl, slot_mapping=None, max_q_len=0, **kw):
    eng = make_engine(wl, kv_dtype=MX, **kw)
    cu, sl, pt = (torch.as_tensor(x, dtype=torch.int32, device=DEV) for x in (wl.cu_seqlens_q, wl.cache_seqlens, wl.page_table))
    sm = None if slot_mapping is None else torch.as_tensor(slot_mapping, dtype=torch.int64, device=DEV)
    eng.prepare(cu, sl, pt, wl.total_tokens, sm, max_q_len)
    return eng


def check(wl, t, out, lse, scale=None, rows=None):
    """out and lse against 64 bits, on the pool as it is now; rows: requests to look at."""
    kp, vp = t["kp"].cpu().numpy(), t["vp"].cpu().numpy()
    Hkv, D = wl.num_kv_heads, wl.head_dim
    q_lens = wl.q_lens if rows is None else [n if i in rows else 0 for i, n in enumerate(wl.q_lens)]
    cu = wl.cu_seqlens_q
    sel = np.concatenate([np.arange(cu[i], cu[i] + n) for i, n in enumerate(q_lens)]).astype(int)
    ref = R.attention(t["q"].float().cpu().numpy()[sel], lambda s: R.unpack_rows(kp[s], Hkv, D),
                      lambda s: R.unpack_rows(vp[s], Hkv, D), q_lens, wl.kv_lens, lambda i: slots_of(wl, i), Hkv, scale)
    tol, ltol = R.tolerances(*ref, D)
    got, gl = out.float().cpu().numpy()[sel], lse.cpu().numpy()[sel]
    assert np.isfinite(got).all() and np.isfinite(gl).all()
    over = np.abs(got - ref[0]) / tol
    assert over.max() <= 1.0, f"out is off by {over.max():.2f} times what the roundings allow"
    lover = np.abs(gl - ref[1]) / ltol
    assert lover.max() <= 1.0, f"lse is off by {lover.max():.2f} times what the roundings allow"


def run(wl, t, eng, **kw):
    out = torch.full_like(t["q"], float("nan"))
    lse = torch.full(t["q"].shape[:2], float("nan"), device=DEV)
    eng.forward(t["q"], t["k"], t["v"], t["kp"], t["vp"], out=out, lse=lse, **kw)
    torch.cuda.synchronize()
    assert pva.attn_get_device_status(eng.meta) == 0
    return out, lse


def full_case(wl, scale=None, slot_mapping=False, max_q_len=0, **kw):
    t = make(wl, wl.seed)
    before = t["kp"].cpu().numpy().copy(), t["vp"].cpu().numpy().copy()
    W.set_junk_columns(wl, 2 ** 31 - 1)
    slots = oracle.slot_mapping(wl.cu_seqlens_q, wl.cache_seqlens, wl.page_table, wl.page_size)
    eng = prepared(wl, slots if slot_mapping else None, max_q_len, **({"sm_scale": scale} if scale else {}), **kw)
    out, lse = run(wl, t, eng)
    used = wl.num_kv_heads * (wl.head_dim // 2 + wl.head_dim // 32)
    for name, was, x in (("kp", before[0], t["k"]), ("vp", before[1], t["v"])):
        was[slots, :used] = R.pack_rows(x.float().cpu().numpy())[:, :used]
        assert np.array_equal(t[name].cpu().numpy(), was), f"{name} after the store"
    check(wl, t, out, lse, scale)
    return eng, t


CASES = [
    # (Hq, Hkv, D, ps, q_lens, kv_lens)
    (32, 8, 128, 16, [1], [1]),
    (32, 8, 128, 16, [1, 1, 1, 1, 3], [1, 16, 17, 700, 33]),
    (28, 4, 128, 1, [1, 2, 1, 1], [5, 2, 1000, 257]),
    (8, 8, 64, 4, [1, 9, 0, 16, 1], [3, 20, 5, 16, 77]),
    (16, 1, 128, 32, [1, 5, 1], [4096, 5, 31]),            # MQA
    (2, 1, 64, 2, [1, 1], [63, 64]),
    (16, 16, 64, 2, [1, 1, 7], [9, 1, 7]),                 # MHA
    (32, 2, 128, 8, [1, 1], [1500, 5]),                    # group 16
    (24, 3, 128, 16, [1, 1, 2], [100, 31, 300]),           # three kv heads
    (25, 5, 64, 1, [1, 3], [130, 33]),                     # five
    (32, 8, 128, 64, [1, 1, 3], [5000, 64, 3]),            # pages of 64 slots, split
    (32, 16, 128, 128, [1, 1, 5], [3000, 129, 200]),       # two head groups
    (64, 32, 64, 16, [1, 2], [700, 65]),                   # four
    (32, 8, 128, 16, [4] * 6, [4, 5, 40, 300, 1030, 2000]),   # speculative verify: 16 rows
    (16, 4, 128, 16, [40, 1, 130], [40, 900, 300]),        # prefills and a chunk
    (8, 1, 64, 4, [300, 17], [300, 1000]),
    (4, 4, 128, 1, [129, 2, 200], [129, 700, 333]),
]


@pytest.mark.parametrize("case", CASES, ids=[f"{c[0]}-{c[1]}-{c[2]}-ps{c[3]}-{i}" for i, c in enumerate(CASES)])
def test_attention(case):
    Hq, Hkv, D, ps, ql, kl = case
    full_case(W.custom(ql, kl, Hq, Hkv, D, ps, seed=len(ql) + D + Hq))


@pytest.mark.parametrize("seed", range(6))
def test_random_batches(seed):
    rng = np.random.default_rng(1000 + seed)
    Hkv = int(rng.choice([1, 2, 4, 6, 8, 16]))
    G, D = int(rng.choice([1, 2, 3, 5, 8, 11])), int(rng.choice([64, 128]))
    B = int(rng.integers(2, 9))
    ql = [int(x) for x in rng.choice([0, 1, 1, 1, 2, 4, 9, 65, 140], B)]
    kl = [n + int(x) for n, x in zip(ql, (10 ** rng.uniform(0, 3.2, B)).astype(int))]
    full_case(W.custom(ql, kl, G * Hkv, Hkv, D, int(2 ** rng.integers(0, 8)), seed=seed))


def test_explicit_slots_no_split_scale_and_hint():
    wl = lambda: W.custom([1, 1, 4], [3000, 700, 2500], 32, 8, 128, 16, seed=5)
    full_case(wl(), slot_mapping=True)
    full_case(wl(), enable_split_kv=False)
    full_case(wl(), scale=0.031)
    full_case(wl(), max_q_len=4)


def test_one_long_request_is_split_over_the_grid():
    wl = W.custom([1], [60_001], 8, 2, 128, 64, seed=2)
    eng, _ = full_case(wl)
    assert pva.attn_debug_plan_counts(eng.meta)["partial_slots"] > 50


def test_lengths_around_a_stage_and_a_page():
    kl = [1, 15, 16, 17, 31, 32, 33, 47, 48, 63, 64, 65, 95, 96, 97, 127, 128, 129]
    for ps in (1, 16, 128):
        full_case(W.custom([1] * len(kl), kl, 8, 2, 128, ps, seed=ps))


def test_store_and_load_are_exact():
    wl = W.custom([5, 0, 1, 33], [9, 4, 1, 40], 8, 4, 128, 8, seed=4)
    t = make(wl, 4)
    k = t["k"].clone()
    # a block of zeros, one beyond the largest scale, one below the smallest, NaN, infinity, signed zeros
    k[0, 0, :32] = 0
    k[0, 1, 32:64] = 3e5
    k[0, 2, 64:96] = 1e-9
    k[1, 0, 5] = float("nan")
    k[1, 1, 40] = float("inf")
    k[2, 0, :32] = -0.0
    k[2, 3, :8] = torch.tensor([4.0, 0.25, 0.75, 1.25, 2.5, 5.0, 7.9, -3.5], dtype=torch.bfloat16)
    eng = prepared(wl)
    eng.store(k, t["v"], t["kp"], t["vp"])
    k2, v2 = eng.load(t["kp"], t["vp"])
    torch.cuda.synchronize()
    assert pva.attn_get_device_status(eng.meta) == 0
    for x, got, pool in ((k, k2, "kp"), (t["v"], v2, "vp")):
        rows = R.pack_rows(x.float().cpu().numpy())
        slots = oracle.slot_mapping(wl.cu_seqlens_q, wl.cache_seqlens, wl.page_table, wl.page_size)
        used = 4 * (64 + 4)
        assert np.array_equal(t[pool].cpu().numpy()[slots, :used], rows[:, :used])
        want = R.unpack_rows(rows, 4, 128)
        np.testing.assert_array_equal(got.float().cpu().numpy(), want.astype(np.float32))
    assert torch.isnan(k2[1, 0, :32]).all() and torch.isnan(k2[1, 1, 32:64]).all() and torch.isnan(k2).sum() == 64


def test_load_leaves_unstored_tokens_and_gathers_whole_requests():
    wl = W.custom([3, 2], [30, 11], 8, 2, 64, 4, seed=4)
    t = make(wl, 4)
    slots = oracle.slot_mapping(wl.cu_seqlens_q, wl.cache_seqlens, wl.page_table, wl.page_size).copy()
    slots[1] = -1
    eng = prepared(wl, slots)
    k = torch.full_like(t["k"], 5.0)
    v = torch.full_like(t["v"], 6.0)
    eng.load(t["kp"], t["vp"], k, v)
    assert (k[1] == 5.0).all() and (v[1] == 6.0).all() and not (k[0] == 5.0).all()
    whole = W.Workload("whole", [30, 11], [30, 11], 8, 2, 64, 4, wl.num_pages, wl.page_table)
    eng = prepared(whole)
    k, v = eng.load(t["kp"], t["vp"])
    sl = np.concatenate([slots_of(wl, 0), slots_of(wl, 1)])
    np.testing.assert_array_equal(k.float().cpu().numpy(), R.unpack_rows(t["kp"].cpu().numpy()[sl], 2, 64))
    np.testing.assert_array_equal(v.float().cpu().numpy(), R.unpack_rows(t["vp"].cpu().numpy()[sl], 2, 64))


def test_nan_stays_in_its_request():
    """A NaN among one request's values reaches that request's heads and no other's."""
    wl = W.custom([1, 1, 1], [40, 70, 33], 8, 2, 128, 16, seed=4)
    t = make(wl, 4)
    t["v"][1, 0, 3] = float("nan")     # request 1, kv head 0, block 0
    t["k"][2, 1, 3] = float("nan")     # request 2, kv head 1
    eng = prepared(wl)
    out = torch.zeros_like(t["q"])
    lse = torch.zeros(3, 8, device=DEV)
    eng.forward(t["q"], t["k"], t["v"], t["kp"], t["vp"], out=out, lse=lse)
    torch.cuda.synchronize()
    nan = torch.isnan(out).cpu().numpy()
    want = np.zeros((3, 8, 128), bool)
    want[1, :4, :32] = True
    want[2, 4:] = True
    assert np.array_equal(nan, want)
    assert np.array_equal(torch.isnan(lse).cpu().numpy(), want.all(-1))


def test_query_range():
    """Queries far beyond f16's range, or far below it, keep their precision."""
    wl = W.custom([1, 1, 1], [300, 70, 5], 8, 2, 128, 16, seed=6)
    for mul, scale in ((2.0 ** 40, 2.0 ** -43), (2.0 ** -60, 2.0 ** 57)):
        t = make(wl, 6)
        t["q"] = (t["q"].float() * mul).to(torch.bfloat16)
        eng = prepared(wl, sm_scale=scale)
        out, lse = run(wl, t, eng)
        check(wl, t, out, lse, scale)


def test_entry_points_refuse_other_pool_types():
    wl = W.custom([1, 3], [40, 9], 8, 2, 64, 4, seed=3)
    t = make(wl)
    out = torch.empty_like(t["q"])
    eng = prepared(wl)
    s = torch.ones(2, device=DEV)
    for call in (lambda: pva.attn_forward(eng.meta, t["q"], t["k"], t["v"], t["kp"], t["vp"], out),
                 lambda: pva.attn_forward_fp8kv(eng.meta, t["q"], t["k"], t["v"], t["kp"], t["vp"], s, s, out),
                 lambda: pva.attn_store_kvcache(eng.meta, t["k"], t["v"], t["kp"], t["vp"]),
                 lambda: pva.attn_forward_mxfp4kv(eng.meta, t["q"], t["k"], t["v"], None, t["vp"], out),
                 lambda: pva.attn_forward_mxfp4kv(eng.meta, None, t["k"], t["v"], t["kp"], t["vp"], out),
                 lambda: pva.attn_load_kvcache_mxfp4kv(eng.meta, t["kp"], t["vp"], None, t["v"]),
                 lambda: pva.attn_store_kvcache_mxfp4kv(eng.meta, t["k"], None, t["kp"], t["vp"])):
        with pytest.raises(pva.PvaError) as e:
            call()
        assert e.value.status == 1
    e16 = make_engine(wl)
    e16.prepare(*(torch.as_tensor(x, dtype=torch.int32, device=DEV) for x in (
        wl.cu_seqlens_q, wl.cache_seqlens, wl.page_table)), wl.total_tokens)
    with pytest.raises(pva.PvaError):
        pva.attn_store_kvcache_mxfp4kv(e16.meta, t["k"], t["v"], t["kp"], t["vp"])


def test_bad_pages_are_reported():
    for D, ps in ((64, 4), (128, 16)):
        wl = W.custom([1, 1, 1], [40, 9, 90], 8, 2, D, ps, seed=3)
        t = make(wl)
        wl.page_table[0, 1] = wl.num_pages + 5    # in the middle of request 0's keys
        wl.page_table[2, 0] = -7
        eng = prepared(wl)
        out = torch.zeros_like(t["q"])
        eng.forward(t["q"], t["k"], t["v"], t["kp"], t["vp"], out=out)
        assert pva.attn_get_device_status(eng.meta) == 0x04


def test_two_engines_on_two_streams_and_repeated_runs_agree():
    wls = [W.custom([1] * 9, [77 + 300 * i for i in range(9)], 16, 4, 128, 16, seed=s) for s in (1, 2)]
    ts = [make(w, w.seed) for w in wls]
    engs = [prepared(w) for w in wls]
    want = [run(w, t, e) for w, t, e in zip(wls, ts, engs)]
    outs = [[torch.empty_like(t["q"]) for _ in range(4)] for t in ts]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for rep in range(4):
        for i in range(2):
            engs[i].forward(ts[i]["q"], ts[i]["k"], ts[i]["v"], ts[i]["kp"], ts[i]["vp"], out=outs[i][rep],
                            stream=streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        for o in outs[i]:
            assert torch.equal(o, want[i][0])   # fixed order: bit for bit


def test_captured_and_replayed():
    wl = W.custom([1] * 5, [700, 33, 40, 1300, 1], 16, 4, 128, 16, seed=8)
    t = make(wl, 8)
    eng = prepared(wl)
    out = torch.empty_like(t["q"])
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        eng.forward(t["q"], t["k"], t["v"], t["kp"], t["vp"], out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        eng.forward(t["q"], t["k"], t["v"], t["kp"], t["vp"], out=out, stream=s)
    for seed in (1, 2):
        fresh = make(wl, 20 + seed)
        for n in t:
            t[n].copy_(fresh[n])
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        ref, lse = run(wl, t, eng)
        assert torch.equal(got, ref)
        check(wl, t, ref, lse)


def test_static_scratch():
    wl = W.custom([1, 3, 1], [700, 40, 2500], 32, 8, 128, 16, seed=3)
    t = make(wl, 3)
    ref, rl = run(wl, t, prepared(wl))
    cfg = pva.make_config(32, 8, 128, 16, wl.num_pages, 3, wl.total_tokens, 2500, kv_dtype=MX)
    meta = pva.attn_prepare_metadata_static(cfg, *(torch.as_tensor(x, dtype=torch.int32, device=DEV) for x in (
        wl.cu_seqlens_q, wl.cache_seqlens, wl.page_table)), None, 3, wl.total_tokens, 3)
    out, lse = torch.empty_like(ref), torch.empty_like(rl)
    pva.attn_forward_mxfp4kv(meta, t["q"], t["k"], t["v"], t["kp"], t["vp"], out, lse)
    torch.cuda.synchronize()
    assert pva.attn_get_device_status(meta) == 0
    check(wl, t, out, lse)


@pytest.mark.parametrize("ql,kl", [([1] * 4, [3000, 2000, 40, 999]), ([200, 1], [200, 900])], ids=["decode", "prefill"])
def test_waits_that_run_out_end_with_a_status(ql, kl):
    wl = W.custom(ql, kl, 32, 8, 128, 16, seed=3)
    t = make(wl, 3)
    eng = prepared(wl)
    pva.attn_debug_set_wait_limit(eng.meta, 0)
    out = torch.zeros_like(t["q"])
    eng.forward(t["q"], t["k"], t["v"], t["kp"], t["vp"], out=out)
    assert pva.attn_get_device_status(eng.meta) & 0x20
    eng = prepared(wl)
    out, lse = run(wl, t, eng)
    check(wl, t, out, lse)


def test_rotated_step_over_the_pool():
    """A whole layer call (rotate, append, attend) for three steps of a growing batch, and the same
    by its parts."""
    Hq, Hkv, D, ps = 16, 4, 128, 16
    wl = W.custom([20, 1, 5], [20, 300, 40], Hq, Hkv, D, ps, seed=9, slack_pages=16)
    wl.page_table = np.concatenate([wl.page_table, np.zeros((3, 2), np.int32)], 1)
    free = [p for p in range(wl.num_pages) if p not in set(wl.used_pages().tolist())]
    for i, L in enumerate(wl.kv_lens):     # room for three more tokens
        if -(-L // ps) < -(-(L + 3) // ps):
            wl.page_table[i, -(-L // ps)] = free.pop()
    t = make(wl, 9)
    rope = pva.Rope(pva.rope_table(400, 64, device=DEV))
    rng = np.random.default_rng(3)
    kl = list(wl.kv_lens)
    for step in range(3):
        ql = wl.q_lens if step == 0 else [1, 1, 1]
        kl = kl if step == 0 else [L + 1 for L in kl]
        w = W.Workload("step", list(ql), list(kl), Hq, Hkv, D, ps, wl.num_pages, wl.page_table)
        T = w.total_tokens
        qkv = torch.as_tensor(rng.standard_normal((T, Hq + 2 * Hkv, D)).astype(np.float32)).to(torch.bfloat16).to(DEV)
        q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        eng = prepared(w)
        parts = {"kp": t["kp"].clone(), "vp": t["vp"].clone()}
        q_rot, lse = torch.empty(T, Hq, D, dtype=torch.bfloat16, device=DEV), torch.empty(T, Hq, device=DEV)
        out = eng.forward(q, k, v, t["kp"], t["vp"], lse=lse, rope=rope, q_rot=q_rot)
        torch.cuda.synchronize()
        assert pva.attn_get_device_status(eng.meta) == 0
        check(w, dict(t, q=q_rot), out, lse)
        r2 = eng.append(q, k, v, parts["kp"], parts["vp"], rope)
        torch.cuda.synchronize()
        assert torch.equal(parts["kp"], t["kp"]) and torch.equal(parts["vp"], t["vp"]) and torch.equal(r2, q_rot)
        # and the read-back is what the next step's attention sees
        k2, _ = eng.load(t["kp"], t["vp"])
        pos = np.concatenate([np.arange(L - n, L) for n, L in zip(ql, kl)])
        yk = R.rotate(k.float().cpu().numpy(), rope.cos_sin.cpu().numpy(), pos, False, np.float32)
        np.testing.assert_array_equal(k2.float().cpu().numpy(), R.unpack_rows(R.pack_rows(yk), Hkv, D).astype(np.float32))


def _shared(wl, **kw):
    """A batch with shared prefixes: with the prefix pass and without, both against 64 bits."""
    t = make(wl, wl.seed)
    counts = []
    for cascade in (True, False):
        eng = prepared(wl, enable_cascade=cascade, **kw)
        out, lse = run(wl, t, eng)
        check(wl, t, out, lse)
        counts.append(pva.attn_debug_plan_counts(eng.meta))
    assert counts[0]["casc_groups"] > 0 and counts[1]["casc_groups"] == 0
    return counts[0]


def test_shared_prefix_groups():
    from test_parity_gpu import _cascade_batch

    _shared(_cascade_batch(seed=4))


def test_shared_prefix_trees():
    from test_parity_gpu import _deep_tree, _tree3_batch

    _shared(_tree3_batch(seed=4))
    assert _shared(_deep_tree(31, 4, 2))["casc_levels"] == 4


@pytest.mark.parametrize("Hq,Hkv,D,ps", [(32, 8, 128, 16), (28, 4, 128, 1), (16, 1, 64, 64), (16, 16, 128, 4),
                                         (32, 2, 64, 128)])
def test_prefill_lengths_around_a_tile(Hq, Hkv, D, ps):
    """Chunks whose queries and keys end around the tensor cores' 128-row and 128-key tiles."""
    ql = [17, 31, 32, 33, 64, 65, 127, 128, 129]
    kl = [17, 128, 160, 161, 64, 300, 127, 256, 385]
    eng, _ = full_case(W.custom(ql, kl, Hq, Hkv, D, ps, seed=ps))
    assert pva.attn_debug_plan_counts(eng.meta)["pre_tiles"] > 0


def test_many_chunks_share_the_queue_with_decodes():
    rng = np.random.default_rng(5)
    ql = [int(x) for x in rng.integers(1, 90, 40)]
    kl = [n + int(x) for n, x in zip(ql, rng.integers(0, 200, 40))]
    full_case(W.custom(ql + [1] * 20, kl + [1 + 13 * i for i in range(20)], 8, 2, 64, 16, seed=5))


@pytest.mark.parametrize("Hq,Hkv,D,ps,n", [(48, 16, 128, 4, 4), (80, 16, 64, 1, 3), (48, 24, 64, 2, 1), (120, 24, 128, 16, 3),
                                           (32, 32, 128, 2, 1), (64, 32, 64, 1, 1), (16, 1, 128, 1, 1), (15, 1, 64, 64, 1),
                                           (12, 1, 128, 16, 1)])
def test_head_blocks_row_tiles_and_page_sizes(Hq, Hkv, D, ps, n):
    """Several CTAs a unit, one or two tiles of query rows, copies of a row or of a page."""
    kl = [n, 31 + n, 32 + n, 64 + n, 65, 700, 1301, 2000]
    eng, t = full_case(W.custom([n] * len(kl), kl, Hq, Hkv, D, ps, seed=Hq + ps))
    assert pva.attn_debug_plan_counts(eng.meta)["dec_units"] > 0


@pytest.mark.parametrize("ps", [1, 16])
def test_layers_of_one_plan(ps):
    """Several layer calls of one prepared batch (a queue of decode units beside prefill tiles)."""
    wl = W.custom([150, 1, 1, 3, 1], [150, 900, 33, 40, 2500], 16, 8, 64, ps, seed=12)
    eng = prepared(wl)
    for layer in range(3):
        t = make(wl, 20 + layer)
        out, lse = run(wl, t, eng)
        check(wl, t, out, lse)
    again, _ = run(wl, t, eng)
    assert torch.equal(again, out)


def test_rows_past_the_batch_stay():
    """Buffers longer than the batch: what lies behind the last token is neither read nor written."""
    wl = W.custom([1, 40, 1], [700, 40, 33], 16, 4, 128, 16, seed=3)
    t = make(wl, 3)
    want, wl_lse = run(wl, t, prepared(wl))
    T, pad = wl.total_tokens, 70
    long = {n: torch.cat([t[n], torch.full((pad, *t[n].shape[1:]), float("nan"), dtype=torch.bfloat16, device=DEV)])
            for n in ("q", "k", "v")}
    out = torch.full_like(long["q"], 7.0)
    lse = torch.full(long["q"].shape[:2], 7.0, device=DEV)
    eng = prepared(wl)
    eng.forward(long["q"], long["k"], long["v"], t["kp"], t["vp"], out=out, lse=lse)
    k2, v2 = torch.full_like(long["k"], 7.0), torch.full_like(long["v"], 7.0)
    eng.load(t["kp"], t["vp"], k=k2, v=v2)
    torch.cuda.synchronize()
    assert pva.attn_get_device_status(eng.meta) == 0
    assert torch.equal(out[:T], want) and torch.equal(lse[:T], wl_lse)
    for x in (out, lse, k2, v2):
        assert bool((x[T:] == 7.0).all())


def test_pools_past_4_gib():
    """Slots whose byte offset needs more than 32 bits (decodes, a chunk, a prefill, the store)."""
    Hq, Hkv, D, ps = 16, 8, 128, 16
    wl = W.custom([1, 40, 1, 130], [700, 90, 33, 130], Hq, Hkv, D, ps, seed=3)
    t = make(wl, 3)
    near, far = {n: x.clone() for n, x in t.items()}, dict(t)
    want, want_lse = run(wl, near, prepared(wl))
    rb = pva.mxfp4_row_bytes(Hkv, D)
    first = -(-(2 ** 32 + 2 ** 20) // (rb * ps))            # pages before the used ones
    for n in ("kp", "vp"):
        far[n] = torch.empty(first * ps + wl.num_slots, rb, dtype=torch.uint8, device=DEV)
        far[n][first * ps:] = t[n]
    w = W.Workload("far", list(wl.q_lens), list(wl.kv_lens), Hq, Hkv, D, ps, wl.num_pages + first,
                   (wl.page_table + first).astype(np.int32))
    out, lse = run(w, far, prepared(w))
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    for n in ("kp", "vp"):
        assert torch.equal(far[n][first * ps:], near[n])


def test_bad_pages_of_a_prefill_are_reported():
    """Page ids outside the pool among the keys of a chunk and of a prefill: flagged, the others' results
    as they were."""
    for D, ps in ((64, 1), (128, 16)):
        wl = W.custom([40, 150, 70], [300, 150, 200], 8, 2, D, ps, seed=3)
        t = make(wl)
        ref, _ = run(wl, {n: x.clone() for n, x in t.items()}, prepared(wl))
        wl.page_table[0, 2] = wl.num_pages + 5
        wl.page_table[0, 4] = -1
        eng = prepared(wl)
        out = torch.zeros_like(t["q"])
        eng.forward(t["q"], t["k"], t["v"], t["kp"], t["vp"], out=out)
        assert pva.attn_get_device_status(eng.meta) == 0x04
        assert torch.equal(out[40:], ref[40:])


@pytest.mark.parametrize("Hq,Hkv,D,ps,ql,kl", [(16, 16, 64, 1, [1] * 4, [3000, 2000, 40, 999]),
                                               (48, 24, 128, 2, [1] * 3, [700, 33, 1000]),
                                               (16, 1, 128, 1, [1] * 3, [700, 33, 1000])],
                         ids=["slots", "head-blocks", "one-head"])
def test_waits_of_several_producers_that_run_out(Hq, Hkv, D, ps, ql, kl):
    wl = W.custom(ql, kl, Hq, Hkv, D, ps, seed=3)
    t = make(wl, 3)
    eng = prepared(wl)
    pva.attn_debug_set_wait_limit(eng.meta, 0)
    eng.forward(t["q"], t["k"], t["v"], t["kp"], t["vp"], out=torch.zeros_like(t["q"]))
    assert pva.attn_get_device_status(eng.meta) & 0x20
    eng = prepared(wl)
    out, lse = run(wl, t, eng)
    check(wl, t, out, lse)


@pytest.mark.parametrize("Hq,Hkv,D,ps", [(16, 1, 128, 32), (16, 1, 64, 16), (64, 4, 128, 16), (24, 2, 64, 1), (4, 1, 128, 4),
                                         (8, 2, 64, 8), (32, 8, 128, 16)])
def test_many_units_a_cta_of_unlike_lengths(Hq, Hkv, D, ps):
    """CTAs that take several units, some too short for all of a head's warps, before longer ones."""
    rng = np.random.default_rng(Hq + D)
    kl = [int(x) for x in rng.choice([1, 20, 33, 64, 65, 130, 300, 700, 1500], 330)]
    eng, _ = full_case(W.custom([1] * len(kl), kl, Hq, Hkv, D, ps, seed=ps))
    assert pva.attn_debug_plan_counts(eng.meta)["dec_units"] > 330
    full_case(W.custom([1] * len(kl), kl, Hq, Hkv, D, ps, seed=ps), enable_split_kv=False)
    full_case(W.custom([1] * len(kl), kl, Hq, Hkv, D, ps, seed=ps), max_q_len=1)   # (one tile of query rows)

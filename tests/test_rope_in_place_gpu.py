"""GPU test: the rotated q in q's own place, through the C ABI with any token stride for one token."""
import pytest
import torch

from harness import make_engine
from paged_variable_length_gb300 import pva
from paged_variable_length_gb300 import workloads as W

pytestmark = pytest.mark.gpu

DEV = "cuda"


def test_one_token_of_a_fused_projection_in_place():
    """One token's q is contiguous whatever the stride between tokens says."""
    Hq, Hkv, D = 8, 2, 128
    wl = W.custom([1], [40], Hq, Hkv, D, 16, seed=3)
    t = W.make_tensors(wl, DEV)
    eng = make_engine(wl)
    eng.prepare(t["cu_seqlens_q"], t["cache_seqlens"], t["page_table"], 1)
    rope = pva.Rope(pva.rope_table(64, D, device=DEV))
    qkv = torch.cat((t["q"], t["k"], t["v"]), 1)
    kept = qkv.clone()
    want = eng.append(qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], t["k_pool"], t["v_pool"], rope)
    pool = t["k_pool"].clone()
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    args = rope.args(q, k, v)
    args.ld_q = args.ld_k = args.ld_v = (Hq + 2 * Hkv) * D
    st = pva.load().attn_append_rope(eng.meta, args, q.data_ptr(), k.data_ptr(), v.data_ptr(), q.data_ptr(),
                                     t["k_pool"].data_ptr(), t["v_pool"].data_ptr(), None, None, pva._stream(None))
    torch.cuda.synchronize()
    assert st == 0 and pva.attn_get_device_status(eng.meta) == 0
    assert torch.equal(qkv[:, :Hq], want) and torch.equal(qkv[:, Hq:], kept[:, Hq:]) and torch.equal(t["k_pool"], pool)


def test_several_strided_tokens_in_place_are_refused():
    Hq, Hkv, D = 8, 2, 128
    wl = W.custom([2], [40], Hq, Hkv, D, 16, seed=3)
    t = W.make_tensors(wl, DEV)
    eng = make_engine(wl)
    eng.prepare(t["cu_seqlens_q"], t["cache_seqlens"], t["page_table"], 2)
    rope = pva.Rope(pva.rope_table(64, D, device=DEV))
    qkv = torch.cat((t["q"], t["k"], t["v"]), 1)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    st = pva.load().attn_append_rope(eng.meta, rope.args(q, k, v), q.data_ptr(), k.data_ptr(), v.data_ptr(), q.data_ptr(),
                                     t["k_pool"].data_ptr(), t["v_pool"].data_ptr(), None, None, pva._stream(None))
    assert st == 1

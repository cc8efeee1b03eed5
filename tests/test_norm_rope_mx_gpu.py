"""GPU tests of attn_forward_norm_rope over an MXFP4 pool: the append's q and pools, and the attention of those
against 64 bits on the same quantised values."""
import numpy as np
import pytest
import torch

import mx_reference as R
from harness import make_engine
from paged_variable_length_gb300 import pva
from paged_variable_length_gb300 import workloads as W

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.mark.parametrize("rot,interleaved", [(None, False), (0, False), (0, True), (32, False), (48, False)],
                         ids=["norm", "split", "inter", "low", "part"])
@pytest.mark.parametrize("ql,kl", [([1, 1, 4, 1], [700, 33, 40, 1]), ([40, 1, 130], [40, 900, 300])], ids=["decode", "prefill"])
@pytest.mark.parametrize("heads", [(16, 4, 128), (6, 3, 64)], ids=["128", "64"])
def test_layer_call_over_an_mxfp4_pool(heads, ql, kl, rot, interleaved):
    Hq, Hkv, D = heads
    wl = W.custom(ql, kl, Hq, Hkv, D, 16, seed=len(ql) + D)
    T = wl.total_tokens
    g = torch.Generator(device=DEV).manual_seed(7)
    qkv = torch.randn(T, Hq + 2 * Hkv, D, generator=g, device=DEV).to(torch.bfloat16)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    old = torch.randn(2, wl.num_slots, Hkv, D, generator=g, device=DEV).cpu().numpy()
    pools = [torch.as_tensor(R.pack_rows(x)).to(DEV) for x in old]
    norm = pva.QKNorm(*(1 + 0.3 * torch.randn(D, generator=g, device=DEV) for _ in range(2)), eps=1e-5)
    rope = None if rot is None else pva.Rope(pva.rope_table(max(kl), rot or D, device=DEV), interleaved=interleaved)
    eng = make_engine(wl, kv_dtype=pva.KV_MXFP4)
    cu, sl, pt = (torch.as_tensor(x, dtype=torch.int32, device=DEV) for x in (wl.cu_seqlens_q, wl.cache_seqlens, wl.page_table))
    eng.prepare(cu, sl, pt, T)
    apart = [x.clone() for x in pools]
    want_q = eng.append(q, k, v, apart[0], apart[1], rope, norm=norm)
    q_rot, out = torch.empty_like(want_q), torch.full_like(want_q, float("nan"))
    lse = torch.full((T, Hq), float("nan"), device=DEV)
    eng.forward(q, k, v, pools[0], pools[1], out=out, lse=lse, rope=rope, norm=norm, q_rot=q_rot)
    torch.cuda.synchronize()
    assert pva.attn_get_device_status(eng.meta) == 0
    assert torch.equal(q_rot, want_q) and all(torch.equal(a, b) for a, b in zip(pools, apart))
    kp, vp = (x.cpu().numpy() for x in pools)

    def slots(i):
        j = np.arange(wl.kv_lens[i])
        return wl.page_table[i].astype(np.int64)[j // 16] * 16 + j % 16

    ref = R.attention(q_rot.float().cpu().numpy(), lambda s: R.unpack_rows(kp[s], Hkv, D), lambda s: R.unpack_rows(vp[s], Hkv, D),
                      wl.q_lens, wl.kv_lens, slots, Hkv)
    tol, ltol = R.tolerances(*ref, D)
    assert (np.abs(out.float().cpu().numpy() - ref[0]) <= tol).all()
    assert (np.abs(lse.cpu().numpy() - ref[1]) <= ltol).all()

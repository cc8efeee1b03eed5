"""GPU test of a model's layers as they run: one plan, every layer's rotated call behind the one before
on one stream with the same q_rot and output buffers, prefills and decodes in one batch."""
import numpy as np
import pytest
import torch

import mx_reference as R
from harness import make_engine
from paged_variable_length_gb300 import pva
from paged_variable_length_gb300 import workloads as W

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.mark.parametrize("kind", [pva.KV_BF16, pva.KV_E4M3, pva.KV_MXFP4], ids=["bf16", "e4m3", "mxfp4"])
@pytest.mark.parametrize("ql,kl", [([150, 1, 1, 3, 1], [150, 900, 33, 40, 2500]), ([1] * 6, [700, 33, 2000, 1, 65, 128])],
                         ids=["mixed", "decode"])
def test_layers_back_to_back_equal_layers_alone(kind, ql, kl):
    Hq, Hkv, D, layers = 16, 4, 128, 6
    wl = W.custom(ql, kl, Hq, Hkv, D, 16, seed=len(ql))
    T = wl.total_tokens
    g = torch.Generator(device=DEV).manual_seed(5)
    qkv = [torch.randn(T, Hq + 2 * Hkv, D, generator=g, device=DEV).to(torch.bfloat16) for _ in range(layers)]
    old = [torch.randn(2, wl.num_slots, Hkv, D, generator=g, device=DEV) for _ in range(layers)]
    scale = torch.full((Hkv,), 0.02, device=DEV) if kind == pva.KV_E4M3 else None

    def pools():
        if kind == pva.KV_BF16:
            return [x.to(torch.bfloat16) for x in old]
        if kind == pva.KV_E4M3:
            return [(x / 0.02).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8) for x in old]
        return [torch.stack([torch.as_tensor(R.pack_rows(y.cpu().numpy())) for y in x]).to(DEV) for x in old]

    rope = pva.Rope(pva.rope_table(max(kl), D, device=DEV))
    eng = make_engine(wl, kv_dtype=kind)
    cu, sl, pt = (torch.as_tensor(x, dtype=torch.int32, device=DEV) for x in (wl.cu_seqlens_q, wl.cache_seqlens, wl.page_table))
    eng.prepare(cu, sl, pt, T)

    def call(i, pool, q_rot, out):
        x = qkv[i]
        eng.forward(x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], pool[0], pool[1], out=out, rope=rope, q_rot=q_rot,
                    k_scale=scale, v_scale=scale)

    alone, pool = [], pools()
    for i in range(layers):
        q_rot, out = (torch.empty(T, Hq, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        torch.cuda.synchronize()
        call(i, pool[i], q_rot, out)
        torch.cuda.synchronize()
        alone.append((q_rot, out, pool[i]))
    pool = pools()
    q_rot, outs = torch.empty(T, Hq, D, dtype=torch.bfloat16, device=DEV), [torch.empty_like(alone[0][1]) for _ in range(layers)]
    torch.cuda.synchronize()
    for _ in range(3):
        for i in range(layers):
            call(i, pool[i], q_rot, outs[i])
    torch.cuda.synchronize()
    assert pva.attn_get_device_status(eng.meta) == 0
    for i in range(layers):
        assert torch.equal(outs[i], alone[i][1]), f"layer {i}"
        assert torch.equal(pool[i], alone[i][2])
    assert torch.equal(q_rot, alone[-1][0])
    assert bool(torch.isfinite(outs[0].float()).all()) and not np.array_equal(outs[0].cpu().float(), outs[1].cpu().float())

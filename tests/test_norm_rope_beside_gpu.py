"""GPU tests of attn_norm_rope beside other calls of the same plan."""
import pytest
import torch

from harness import make_engine
from paged_variable_length_gb300 import pva
from paged_variable_length_gb300 import workloads as W

pytestmark = pytest.mark.gpu

DEV = "cuda"


def batch(ql, kl):
    wl = W.custom(ql, kl, 16, 4, 128, 16, seed=3)
    t = W.make_tensors(wl, DEV)
    eng = make_engine(wl)
    eng.prepare(t["cu_seqlens_q"], t["cache_seqlens"], t["page_table"], wl.total_tokens)
    return wl, t, eng


@pytest.mark.parametrize("with_norm", [True, False])
def test_the_plan_stays_as_it_is(with_norm):
    """Every word of the workspace, the tickets that a running attention draws among them."""
    wl, t, eng = batch([40, 1, 130, 1], [40, 900, 300, 2000])
    torch.cuda.synchronize()
    words = eng.workspace[:256].view(torch.int32)      # the plan's header: tickets in words 13 and 14
    words[13:15] = torch.tensor([1234, 77], dtype=torch.int32, device=DEV)
    was = eng.workspace.clone()
    rope = pva.Rope(pva.rope_table(2000, 64, device=DEV))
    eng.norm_rope(t["q"], t["k"], rope=rope, norm=pva.QKNorm() if with_norm else None)
    torch.cuda.synchronize()
    assert torch.equal(eng.workspace, was)


def test_beside_a_running_attention():
    """Layer calls on one stream, norms of the same plan on another: the same bits as alone."""
    wl, t, eng = batch([700, 1, 1, 130, 1] + [1] * 20, [700, 9000, 900, 300, 2000] + [3000] * 20)
    rope, norm = pva.Rope(pva.rope_table(9000, 128, device=DEV)), pva.QKNorm()
    want = eng.forward(t["q"], t["k"], t["v"], t["k_pool"], t["v_pool"])
    normed = eng.norm_rope(t["q"], t["k"], rope=rope, norm=norm)
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    outs = [torch.empty_like(want) for _ in range(30)]
    qs, ks = ([torch.empty_like(x) for _ in range(30)] for x in normed)
    torch.cuda.synchronize()
    for o, q, k in zip(outs, qs, ks):
        eng.forward(t["q"], t["k"], t["v"], t["k_pool"], t["v_pool"], out=o, stream=a)
        for _ in range(3):
            eng.norm_rope(t["q"], t["k"], rope=rope, norm=norm, q_out=q, k_out=k, stream=b)
    torch.cuda.synchronize()
    assert pva.attn_get_device_status(eng.meta) == 0
    for o, q, k in zip(outs, qs, ks):
        assert torch.equal(o, want) and torch.equal(q, normed[0]) and torch.equal(k, normed[1])

"""GPU test: forward's own output tensor belongs to the stream that writes it."""
import pytest
import torch

from harness import make_engine
from paged_variable_length_gb300 import pva
from paged_variable_length_gb300 import workloads as W

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.mark.parametrize("kind", ["bf16", "bf16-rope", "mxfp4"])
def test_forward_without_out_on_another_stream(kind):
    """A block that the current stream let go while its work is pending is not the side stream's output;
    nor is the output's memory, once let go, the current stream's while the side stream writes."""
    wl = W.custom([1, 300], [1, 300], 16, 4, 128, 16, seed=3)
    t = W.make_tensors(wl, DEV)
    dtype = pva.KV_MXFP4 if kind == "mxfp4" else pva.KV_BF16
    kp, vp = t["k_pool"], t["v_pool"]
    if kind == "mxfp4":
        kp, vp = (torch.zeros(wl.num_slots, pva.mxfp4_row_bytes(4, 128), dtype=torch.uint8, device=DEV) for _ in range(2))
    rope = pva.Rope(pva.rope_table(300, 128, device=DEV)) if kind.endswith("rope") else None
    eng = make_engine(wl, kv_dtype=dtype)
    eng.prepare(t["cu_seqlens_q"], t["cache_seqlens"], t["page_table"], wl.total_tokens)
    want = eng.forward(t["q"], t["k"], t["v"], kp, vp, out=torch.empty_like(t["q"]), rope=rope).clone()
    busy = torch.randn(6000, 6000, device=DEV)
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        torch.cuda.synchronize()
        let_go = [torch.empty_like(t["q"]) for _ in range(3)]
        where = {x.data_ptr() for x in let_go}
        for _ in range(8):
            busy @ busy                      # the current stream is at work for a while
        for x in let_go:
            x.fill_(3.0)                     # pending
        del let_go, x
        out = eng.forward(t["q"], t["k"], t["v"], kp, vp, rope=rope, stream=stream)
        assert out.data_ptr() not in where
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        mine = out.data_ptr()
        del out
        again = [torch.empty_like(t["q"]) for _ in range(3)]
        assert mine not in {x.data_ptr() for x in again}
        del again

"""GPU tests of layer calls made by two host threads at once (ctypes lets go of the interpreter lock
during a call): engines of unlike head layouts, whose kernels are the same function."""
import threading

import pytest
import torch

from harness import make_engine
from paged_variable_length_gb300 import pva
from paged_variable_length_gb300 import workloads as W

pytestmark = pytest.mark.gpu

DEV = "cuda"


def layer(Hq, Hkv, D, ps, kv_dtype, seed):
    """A decode batch of its own engine, pools and stream: (call, its output)."""
    wl = W.custom([1] * 3, [40, 300, 65], Hq, Hkv, D, ps, seed=seed)
    t = W.make_tensors(wl, DEV)
    kp, vp = t["k_pool"], t["v_pool"]
    if kv_dtype == pva.KV_MXFP4:
        kp, vp = (torch.zeros(wl.num_slots, pva.mxfp4_row_bytes(Hkv, D), dtype=torch.uint8, device=DEV) for _ in range(2))
    eng = make_engine(wl, kv_dtype=kv_dtype)
    eng.prepare(t["cu_seqlens_q"], t["cache_seqlens"], t["page_table"], wl.total_tokens, max_q_len=1)
    out, stream = torch.empty_like(t["q"]), torch.cuda.Stream()
    torch.cuda.synchronize()
    return lambda: eng.forward(t["q"], t["k"], t["v"], kp, vp, out=out, stream=stream), out


def at_once(layers, times=1500):
    wants = []
    for call, out in layers:
        call()
        torch.cuda.synchronize()
        wants.append(out.clone())
    failed, start = [], threading.Barrier(len(layers))

    def work(call):
        start.wait()
        try:
            for i in range(times):
                call()
                if i % 200 == 0:
                    torch.cuda.synchronize()
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=work, args=(call,)) for call, _ in layers]
    for x in threads:
        x.start()
    for x in threads:
        x.join()
    torch.cuda.synchronize()
    assert not failed, failed
    for (_, out), want in zip(layers, wants):
        assert torch.equal(out, want)


def test_mxfp4_layouts_of_one_kernel():
    """Two tiles of query rows at one and at two kv heads (148 and 204 KB of shared memory), and three and
    seven heads of one tile."""
    at_once([layer(16, 1, 128, 16, pva.KV_MXFP4, 1), layer(32, 2, 128, 16, pva.KV_MXFP4, 2)])
    at_once([layer(12, 3, 128, 16, pva.KV_MXFP4, 3), layer(28, 7, 128, 16, pva.KV_MXFP4, 4)])


def test_bf16_layouts_of_one_kernel():
    """One and eight kv heads (several CTAs of an SM against one)."""
    at_once([layer(4, 1, 128, 16, pva.KV_BF16, 1), layer(32, 8, 128, 16, pva.KV_BF16, 2)], times=6000)


def test_plans_of_unlike_batches():
    """Batches of 1100 and of 1500 requests, whose plans take unlike amounts of shared memory."""
    def plan(B, seed):
        wl = W.custom([1] * B, [1 + i % 7 for i in range(B)], 4, 1, 64, 1, seed=seed)
        cu, sl, pt = (torch.as_tensor(x, dtype=torch.int32, device=DEV) for x in (wl.cu_seqlens_q, wl.cache_seqlens,
                                                                                 wl.page_table))
        eng, stream = make_engine(wl), torch.cuda.Stream()
        torch.cuda.synchronize()
        return lambda: eng.prepare(cu, sl, pt, wl.total_tokens, max_q_len=1, stream=stream), torch.zeros(1, device=DEV)

    at_once([plan(1100, 1), plan(1500, 2)], times=3000)

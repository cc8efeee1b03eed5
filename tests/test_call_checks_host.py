"""What the binding refuses of the rotary and MXFP4 calls before anything is launched (no GPU: the
batch is said to be on the CPU, and a call whose tensors pass gets as far as the library, which
answers that the batch was never prepared)."""
import pytest
import torch

from paged_variable_length_gb300 import build, pva

T, HQ, HKV, D, PS, PAGES = 5, 4, 2, 64, 4, 6
BF, F32 = torch.bfloat16, torch.float32
NOT_PREPARED = 6


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return pva.load()


def batch_of(kv_dtype, device=-1):
    meta = pva.Meta()
    meta.batch = pva.Batch(HQ, HKV, D, PS * PAGES, kv_dtype, T, device)
    return meta


def tensors(kv_dtype):
    row = {pva.KV_BF16: 2 * HKV * D, pva.KV_E4M3: HKV * D, pva.KV_MXFP4: pva.mxfp4_row_bytes(HKV, D)}[kv_dtype]
    e = lambda *s, dtype=BF: torch.empty(*s, dtype=dtype)
    a = dict(q=e(T, HQ, D), k=e(T, HKV, D), v=e(T, HKV, D), q_rot=e(T, HQ, D), out=e(T, HQ, D), lse=e(T, HQ, dtype=F32),
             k_pool=e(PAGES * PS, row, dtype=torch.uint8), v_pool=e(PAGES * PS, row, dtype=torch.uint8),
             k_scale=None, v_scale=None, rope=pva.Rope(torch.zeros(64, D)))
    if kv_dtype == pva.KV_E4M3:
        a["k_scale"], a["v_scale"] = torch.ones(HKV), torch.ones(HKV)
    return a


def calls(kv_dtype):
    """name -> (the tensors it takes, the call)."""
    out = {
        "append": (("q", "k", "v", "q_rot", "k_pool", "v_pool", "k_scale", "v_scale"),
                   lambda m, a: pva.attn_append_rope(m, a["rope"], a["q"], a["k"], a["v"], a["q_rot"], a["k_pool"], a["v_pool"],
                                                     a["k_scale"], a["v_scale"], stream=0)),
        "forward_rope": (("q", "k", "v", "q_rot", "k_pool", "v_pool", "out", "lse", "k_scale", "v_scale"),
                         lambda m, a: pva.attn_forward_rope(m, a["rope"], a["q"], a["k"], a["v"], a["q_rot"], a["k_pool"],
                                                            a["v_pool"], a["out"], a["lse"], a["k_scale"], a["v_scale"], stream=0)),
    }
    if kv_dtype == pva.KV_MXFP4:
        out["forward"] = (("q", "k", "v", "k_pool", "v_pool", "out", "lse"),
                          lambda m, a: pva.attn_forward_mxfp4kv(m, a["q"], a["k"], a["v"], a["k_pool"], a["v_pool"], a["out"],
                                                                a["lse"], stream=0))
        out["store"] = (("k", "v", "k_pool", "v_pool"),
                        lambda m, a: pva.attn_store_kvcache_mxfp4kv(m, a["k"], a["v"], a["k_pool"], a["v_pool"], stream=0))
        out["load"] = (("k", "v", "k_pool", "v_pool"),
                       lambda m, a: pva.attn_load_kvcache_mxfp4kv(m, a["k_pool"], a["v_pool"], a["k"], a["v"], stream=0))
    return out


def status(call, meta, a):
    try:
        call(meta, a)
    except ValueError:
        return 1
    except pva.PvaError as e:
        return e.status
    return 0


KINDS = [pva.KV_BF16, pva.KV_E4M3, pva.KV_MXFP4]


@pytest.mark.parametrize("kv_dtype", KINDS)
def test_what_passes(kv_dtype):
    for name, (_, call) in calls(kv_dtype).items():
        meta, a = batch_of(kv_dtype), tensors(kv_dtype)
        assert status(call, meta, a) == NOT_PREPARED, name
        for n, x in list(a.items()):      # longer than the batch, and slices of one projection
            if isinstance(x, torch.Tensor):
                a[n] = torch.cat((x, x))
        assert status(call, meta, a) == NOT_PREPARED, name
        if name in ("append", "forward_rope"):
            qkv = torch.empty(T, HQ + 2 * HKV, D, dtype=BF)
            a.update(q=qkv[:, :HQ], k=qkv[:, HQ:HQ + HKV], v=qkv[:, HQ + HKV:])
            assert status(call, meta, a) == NOT_PREPARED, name


@pytest.mark.parametrize("kv_dtype", KINDS)
def test_tensors_shorter_than_the_batch(kv_dtype):
    for name, (takes, call) in calls(kv_dtype).items():
        for n in takes:
            a = tensors(kv_dtype)
            if a[n] is None:
                continue
            a[n] = a[n][:-1]
            assert status(call, batch_of(kv_dtype), a) == 1, (name, n)
        if name in ("append", "forward_rope"):   # all of them short alike, positions too
            a = tensors(kv_dtype)
            for n in ("q", "k", "v", "q_rot", "out", "lse"):
                a[n] = a[n][:3]
            a["rope"].set_positions(torch.zeros(3, dtype=torch.int32))
            assert status(call, batch_of(kv_dtype), a) == 1, name


@pytest.mark.parametrize("kv_dtype", KINDS)
def test_other_types_and_head_layouts(kv_dtype):
    for name, (takes, call) in calls(kv_dtype).items():
        for n in takes:
            a = tensors(kv_dtype)
            if a[n] is None or n.endswith("pool"):
                continue
            a[n] = a[n].to(torch.float16)
            assert status(call, batch_of(kv_dtype), a) == 1, (name, n)
        for n, heads in (("q", HQ - 1), ("k", HKV + 1), ("v", 1)):
            if name in ("append", "forward_rope"):
                a = tensors(kv_dtype)
                a[n] = torch.empty(T, heads, D, dtype=BF)
                assert status(call, batch_of(kv_dtype), a) == 1, (name, n)


@pytest.mark.parametrize("kv_dtype", KINDS)
def test_tensors_on_another_device(kv_dtype):
    """A host table, host positions or host activations of a batch on a GPU."""
    for name, (takes, call) in calls(kv_dtype).items():
        assert status(call, batch_of(kv_dtype, device=0), tensors(kv_dtype)) == 1, name
        for n in takes:
            a = tensors(kv_dtype)
            if a[n] is None:
                continue
            a[n] = SomewhereElse(a[n])
            assert status(call, batch_of(kv_dtype), a) == 1, (name, n)


@pytest.mark.parametrize("kv_dtype", KINDS)
def test_a_batch_on_another_device_than_the_current_one(kv_dtype, monkeypatch):
    """Refused on any stream: the library launches on the current device."""
    current = [0]
    monkeypatch.setattr(pva, "_raw_stream", (lambda dev: 0, lambda: current[0]))
    for name, (_, call) in calls(kv_dtype).items():
        a = {n: SomewhereElse(x) if isinstance(x, torch.Tensor) else x for n, x in tensors(kv_dtype).items()}
        a["rope"] = pva.Rope(SomewhereElse(torch.zeros(64, D)))
        current[0] = 0
        assert status(call, batch_of(kv_dtype, device=3), a) == 1, name
        current[0] = 3
        assert status(call, batch_of(kv_dtype, device=3), a) == NOT_PREPARED, name


def test_a_table_or_positions_on_another_device():
    a = tensors(pva.KV_MXFP4)
    table = SomewhereElse(torch.zeros(64, D))
    with pytest.raises(ValueError):
        pva.Rope(table, positions=torch.zeros(T, dtype=torch.int32))
    rope = pva.Rope(table)
    with pytest.raises(ValueError):
        rope.args(a["q"], a["k"], a["v"])
    with pytest.raises(ValueError):
        pva.Rope(torch.zeros(64, D), positions=SomewhereElse(torch.zeros(T, dtype=torch.int32)))


def test_a_prepared_meta_makes_its_batch_when_first_asked():
    """From what the config said at prepare, whatever it is changed to later."""
    cfg = pva.make_config(HQ, HKV, D, PS, PAGES, 2, T, 64, kv_dtype=pva.KV_MXFP4)
    meta = pva.Meta()
    assert meta.of_batch() is None
    meta._sizes = pva._batch_sizes(cfg, T, -1)
    cfg.num_qo_heads, cfg.kv_dtype = 99, pva.KV_BF16
    b = meta.of_batch()
    assert b is meta.batch and (b.tokens, b.q_heads, b.kv_heads, b.head_dim, b.device) == (T, HQ, HKV, D, -1)
    assert b.pool_bytes == PS * PAGES * pva.mxfp4_row_bytes(HKV, D) and not b.scaled


class SomewhereElse(torch.Tensor):
    """A tensor that says it is on GPU 3."""

    @staticmethod
    def __new__(cls, x):
        return x.as_subclass(cls)

    def get_device(self):
        return 3

"""The rotary append and the MXFP4 pool without a GPU: structures, refusals that need no device,
the rotation table, and the references the GPU tests compare with."""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

import mx_reference as R
from paged_variable_length_gb300 import build, pva

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    build.build()
    return pva.load()


def test_rope_struct_matches_the_header(tmp_path):
    fields = [f for f, _ in pva.RopeArgs._fields_]
    src = tmp_path / "probe.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "pva.h"\nint main(void){\n'
                   'printf("%zu\\n", sizeof(pva_rope));\n'
                   + "".join(f'printf("%zu\\n", offsetof(pva_rope, {f}));\n' for f in fields) + "return 0;}\n")
    exe = tmp_path / "probe"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    vals = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert vals == [ctypes.sizeof(pva.RopeArgs)] + [getattr(pva.RopeArgs, f).offset for f in fields]


@pytest.mark.parametrize("Hkv,D", [(1, 64), (1, 128), (2, 64), (3, 128), (4, 128), (5, 64), (8, 64), (8, 128), (16, 128), (32, 64)])
def test_row_bytes(lib, Hkv, D):
    hb, group, rb = R.row_layout(Hkv, D)
    assert pva.mxfp4_row_bytes(Hkv, D) == rb and rb % 16 == 0
    if Hkv > 8:
        assert group % 16 == 0 and rb == Hkv // 8 * group   # a head group is a piece of its own


@pytest.mark.parametrize("Hkv,D", [(0, 128), (-1, 64), (12, 128), (8, 96), (8, 0), (9, 64)])
def test_row_bytes_of_a_layout_that_is_not_built(lib, Hkv, D):
    with pytest.raises(pva.PvaError):
        pva.mxfp4_row_bytes(Hkv, D)


def test_the_new_calls_need_a_prepared_meta(lib):
    meta, d = pva.Meta(), ctypes.c_void_p(256)
    rope = pva.RopeArgs(256, None, 64, 64, 64, 16, 32, 0, 0)
    m, r = ctypes.byref(meta), ctypes.byref(rope)
    assert lib.attn_forward_mxfp4kv(m, d, d, d, d, d, d, None, None) == 6
    assert lib.attn_store_kvcache_mxfp4kv(m, d, d, d, d, None) == 6
    assert lib.attn_load_kvcache_mxfp4kv(m, d, d, d, d, None) == 6
    assert lib.attn_append_rope(m, r, d, d, d, d, d, d, None, None, None) == 6
    assert lib.attn_forward_rope(m, r, d, d, d, d, d, d, None, None, d, None, None) == 6
    assert lib.attn_append_rope(None, r, d, d, d, d, d, d, None, None, None) == 6


def test_config_takes_the_mxfp4_pool_type(lib):
    """The host checks pass the pool type (the call stops at the 16-byte workspace, or for want of a
    device), and still refuse one that does not exist."""
    meta, d = pva.Meta(), ctypes.c_void_p(256)
    for dtype, want in ((pva.KV_MXFP4, (3, 4)), (3, (2,))):
        cfg = pva.make_config(32, 8, 128, 16, 100, 4, 16, 1024, kv_dtype=dtype)
        st = lib.attn_prepare_metadata(ctypes.byref(cfg), d, d, d, 8, None, 1, 1, 1, d, 16, None, ctypes.byref(meta))
        assert st in want


def test_rope_table_is_formed_in_64_bits():
    """Far positions: the table's fp32 entries are the nearest to the true cosine (0.5 ulp)."""
    t = pva.rope_table(200_001, 64, base=10000.0, device="cpu")
    assert t.shape == (200_001, 64) and t.dtype == torch.float32
    for p in (0, 1, 777, 65_537, 200_000):
        ang = np.longdouble(p) * np.longdouble(10000.0) ** (-np.arange(0, 64, 2, dtype=np.longdouble) / 64)
        ref = np.concatenate((np.cos(ang), np.sin(ang))).astype(np.float64)
        # angle: 2^-52 relative of up to 2e5; then half an fp32 step of a value up to 1
        assert np.abs(t[p].numpy() - ref).max() <= 2e5 * 2.0 ** -52 + 2.0 ** -25


def test_rope_refuses_what_it_cannot_read():
    t = pva.rope_table(32, 64, device="cpu")
    k = torch.zeros(5, 2, 64, dtype=torch.bfloat16)
    for bad in (t.double(), t[0], t[:, :32]):
        with pytest.raises(ValueError):
            pva.Rope(bad)
    with pytest.raises(ValueError):
        pva.Rope(t, rot_dim=32)
    with pytest.raises(ValueError):
        pva.Rope(t, positions=torch.zeros(5, dtype=torch.int64))
    with pytest.raises(ValueError):
        pva.Rope(t, positions=torch.zeros(4, dtype=torch.int32)).args(None, k, k)
    with pytest.raises(ValueError):  # heads apart
        pva.Rope(t).args(None, torch.zeros(5, 4, 64)[:, ::2], k)
    with pytest.raises(ValueError):  # a strided head dim
        pva.Rope(t).args(None, torch.zeros(5, 2, 128)[..., ::2], k)


def test_rope_reads_token_strides():
    t = pva.rope_table(32, 64, device="cpu")
    qkv = torch.zeros(5, 8, 64, dtype=torch.bfloat16)
    a = pva.Rope(t, interleaved=True).args(qkv[:, :4], qkv[:, 4:6], qkv[:, 6:])
    assert (a.ld_q, a.ld_k, a.ld_v, a.max_positions, a.rot_dim, a.interleaved) == (512, 512, 512, 32, 64, 1)
    a = pva.Rope(t).args(qkv[:1, :4], qkv[:1, 4:6], qkv[:1, 6:])   # one token: the stride does not matter
    assert (a.ld_q, a.ld_k, a.ld_v) == (256, 128, 128)


def test_reference_quantiser_on_the_formats_own_values():
    """Every code times every scale comes back as itself; ties, saturation, tiny and NaN blocks."""
    mags = np.concatenate((R.MAGNITUDES, -R.MAGNITUDES))
    for e in (R.E_LO, 120, 127, R.E_HI):
        block = np.zeros((1, 1, 32), np.float32)
        block[0, 0, :16] = mags * 2.0 ** (e - 127.0)
        rows = R.pack_rows(np.tile(block, (1, 1, 2)))
        assert np.array_equal(R.unpack_rows(rows, 1, 64)[0, 0, :16], block[0, 0, :16].astype(np.float64))
    x = np.zeros(32, np.float32)
    x[:10] = [4.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.9, -0.25]
    code, e = R.quantise(x)
    assert e == 127 and list(code[:10]) == [6, 0, 2, 2, 4, 4, 6, 6, 7, 8]
    code, e = R.quantise(np.full(32, 1e9, np.float32))
    assert e == R.E_HI and (code == 7).all()
    code, e = R.quantise(np.full(32, 1e-12, np.float32))
    assert e == R.E_LO and (code == 0).all()
    for bad in (np.nan, np.inf):
        y = x.copy()
        y[3] = bad
        code, e = R.quantise(y)
        assert e == R.E_NAN and (code == 0).all()


def test_reference_rotation_is_a_rotation():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((6, 3, 64))
    cs = pva.rope_table(50, 32, device="cpu").double().numpy()
    for inter in (False, True):
        y = R.rotate(x, cs, np.arange(10, 16), inter, np.float64)
        assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1), rtol=1e-6)
        assert np.array_equal(y[..., 32:], x[..., 32:])
        # a pair's angle is the position times its frequency
        a, b = (0, 1) if inter else (0, 16)
        ang = np.arctan2(y[:, :, b], y[:, :, a]) - np.arctan2(x[:, :, b], x[:, :, a])
        assert np.allclose(np.cos(ang), np.cos(np.arange(10, 16))[:, None], atol=1e-6)

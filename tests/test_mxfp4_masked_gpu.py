"""GPU tests of NaN and infinite values in an MXFP4 pool behind the causal mask: a token's output
depends on the keys it sees and on no others, whatever those hold."""
import numpy as np
import pytest
import torch

import mx_reference as R
from paged_variable_length_gb300 import pva
from paged_variable_length_gb300 import workloads as W
from test_mxfp4_gpu import DEV, make, prepared, run

pytestmark = pytest.mark.gpu


def masked_case(wl, bad, **kw):
    """bad: (request, new token, kv head, dim, of V, value).  Against the same batch without them:
    the rows that see a bad V block are NaN in its 32 dims, those that see a bad K block are NaN,
    and everything else is what it was, bit for bit."""
    Hq, Hkv, D = wl.num_qo_heads, wl.num_kv_heads, wl.head_dim
    G, cu = Hq // Hkv, wl.cu_seqlens_q
    t = make(wl, wl.seed)
    clean, clean_lse = run(wl, {n: x.clone() for n, x in t.items()}, prepared(wl, **kw))
    want = np.zeros((wl.total_tokens, Hq, D), bool)
    want_lse = np.zeros((wl.total_tokens, Hq), bool)
    for i, r, h, d, is_v, value in bad:
        t["v" if is_v else "k"][cu[i] + r, h, d] = value
        rows, heads, b = slice(cu[i] + r, cu[i + 1]), slice(h * G, (h + 1) * G), d // 32 * 32
        if is_v:
            want[rows, heads, b:b + 32] = True
        else:
            want[rows, heads] = True
            want_lse[rows, heads] = True
    out, lse = run(wl, t, prepared(wl, **kw))
    nan, nan_lse = torch.isnan(out).cpu().numpy(), torch.isnan(lse).cpu().numpy()
    assert np.array_equal(nan, want), "outputs that are NaN"
    assert np.array_equal(nan_lse, want_lse), "LSE that are NaN"
    ok, okl = torch.as_tensor(~want).to(DEV), torch.as_tensor(~want_lse).to(DEV)
    assert torch.equal(out[ok], clean[ok]) and torch.equal(lse[okl], clean_lse[okl])


NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("Hq,Hkv,D,ps", [(32, 8, 128, 16), (16, 4, 64, 1), (8, 1, 128, 32), (16, 16, 64, 4), (48, 16, 128, 2),
                                         (24, 3, 64, 16)])
def test_hidden_values_of_small_groups(Hq, Hkv, D, ps):
    """Verify batches: several new tokens a request in one tile of rows (and over several parts)."""
    n = min(4, 16 // (Hq // Hkv))
    wl = W.custom([n, n, n, 1], [n, 63 + n, 700, 40], Hq, Hkv, D, ps, seed=Hq + D)
    h = Hkv - 1
    masked_case(wl, [(0, n - 1, 0, 3, True, NAN), (1, 1, h, D - 1, True, INF), (2, n - 1, h, 33, True, -INF),
                     (2, 1, h, 40, True, NAN)])
    masked_case(wl, [(0, n - 1, h, 5, False, NAN), (2, 1, 0, 63, False, INF), (1, n - 1, 0, 0, True, NAN)],
                max_q_len=n)
    masked_case(wl, [(2, n - 1, 0, 7, True, NAN), (2, 0, h, 34, True, NAN)], enable_split_kv=False)


@pytest.mark.parametrize("Hq,Hkv,D,ps", [(32, 8, 128, 16), (8, 4, 64, 1), (16, 1, 128, 64), (16, 16, 64, 4)])
def test_hidden_values_of_prefills(Hq, Hkv, D, ps):
    """Prefills and chunks on the tensor cores: keys hidden inside a tile and in the next one, several
    units of one request and of others on a CTA."""
    wl = W.custom([300, 130, 90, 1], [300, 400, 90, 50], Hq, Hkv, D, ps, seed=Hq + D)
    h = Hkv - 1
    masked_case(wl, [(0, 1, 0, 3, True, NAN), (0, 150, h, 40, True, INF), (0, 299, 0, D - 1, True, NAN),
                     (1, 129, h, 0, True, -INF), (1, 5, 0, 33, True, NAN), (1, 6, 0, 33, True, NAN)])
    masked_case(wl, [(0, 200, 0, 3, False, NAN), (0, 17, h, 3, True, NAN), (1, 64, h, 63, False, INF),
                     (2, 89, h, 5, True, NAN)])


def test_hidden_values_of_many_units():
    """More units than CTAs, a NaN in every third request: none reaches a unit that follows on its CTA."""
    B = 60
    wl = W.custom([40] * B, [40 + 3 * i for i in range(B)], 32, 8, 128, 16, seed=4)
    masked_case(wl, [(i, 10 + i % 30, i % 8, (37 * i) % 128, True, NAN) for i in range(0, B, 3)])


def test_hidden_values_of_every_unit():
    """Every unit of a long queue holds a NaN."""
    B = 700
    wl = W.custom([17] * B, [17 + i % 5 for i in range(B)], 8, 8, 64, 4, seed=4)
    masked_case(wl, [(i, i % 17, h, (37 * i) % 64, True, NAN) for i in range(B) for h in range(8)], max_q_len=17)


def test_values_of_a_shared_prefix():
    """A NaN in a prefix that several decodes share reaches each of them, in its block and nowhere else."""
    from test_parity_gpu import _cascade_batch

    wl = _cascade_batch(seed=4)
    t = make(wl, wl.seed)
    Hkv, D = wl.num_kv_heads, wl.head_dim
    G = wl.num_qo_heads // Hkv
    clean, _ = run(wl, {n: x.clone() for n, x in t.items()}, prepared(wl))
    hb, group, _ = R.row_layout(Hkv, D)
    pos, h, b = 21, Hkv - 1, 1
    slot = int(wl.page_table[0][pos // wl.page_size]) * wl.page_size + pos % wl.page_size
    at = h // hb * group + hb * (D // 2) + (h % hb) * (D // 32) + b
    codes = h // hb * group + (h % hb) * (D // 2) + b * 16
    t["vp"][slot, at] = 255
    t["vp"][slot, codes:codes + 16] = 0
    sees = np.array([L > pos and wl.page_table[i][pos // wl.page_size] == wl.page_table[0][pos // wl.page_size]
                     for i, L in enumerate(wl.kv_lens)])
    assert sees.sum() > 1
    for cascade in (True, False):
        out, _ = run(wl, {n: x.clone() for n, x in t.items()}, prepared(wl, enable_cascade=cascade))
        want = np.zeros(out.shape, bool)
        for i in np.flatnonzero(sees):
            for tok in range(wl.cu_seqlens_q[i], wl.cu_seqlens_q[i + 1]):
                first = wl.kv_lens[i] - wl.q_lens[i]
                if first + tok - wl.cu_seqlens_q[i] >= pos:
                    want[tok, h * G:(h + 1) * G, b * 32:b * 32 + 32] = True
        assert np.array_equal(torch.isnan(out).cpu().numpy(), want)
        if cascade:
            ok = torch.as_tensor(~want).to(DEV)
            assert torch.equal(out[ok], clean[ok])


def test_hidden_values_of_more_units_than_a_cta_lists():
    """160 000 units, each with a NaN: more than a thousand on a CTA."""
    B, Hq, Hkv, D = 20_000, 128, 8, 64
    wl = W.Workload("many", [2] * B, [2] * B, Hq, Hkv, D, 2, B, np.arange(B, dtype=np.int32)[:, None])
    g = torch.Generator(device=DEV).manual_seed(1)
    q, k, v = (torch.randn(2 * B, h, D, generator=g, device=DEV).to(torch.bfloat16) for h in (Hq, Hkv, Hkv))
    t = {"q": q, "k": k, "v": v}
    for n in ("kp", "vp"):
        t[n] = torch.zeros(2 * B, R.row_layout(Hkv, D)[2], dtype=torch.uint8, device=DEV)
    eng = prepared(wl, max_q_len=2, enable_cascade=False)
    clean, clean_lse = run(wl, t, eng)
    v[1::2, :, 40] = NAN                    # the second token's, in every head's second block
    out, lse = run(wl, t, eng)
    nan = torch.isnan(out)
    assert bool(nan[1::2, :, 32:].all()) and not bool(nan[1::2, :, :32].any()) and not bool(nan[::2].any())
    assert torch.equal(out[~nan], clean[~nan]) and torch.equal(lse, clean_lse)
    assert pva.attn_debug_plan_counts(eng.meta)["pre_tiles"] > 1024 * torch.cuda.get_device_properties(0).multi_processor_count

"""GPU tests of NaN and infinite values in an MXFP4 pool behind the causal mask: a token's output
depends on the keys it sees and on no others, whatever those hold."""
import numpy as np
import pytest
import torch

from test_mxfp4_gpu import DEV, make, prepared, run
from paged_variable_length_gb300 import workloads as W

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

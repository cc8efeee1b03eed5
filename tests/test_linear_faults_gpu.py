"""GPU tests of linear attention where one request or token of a batch is at fault: what the others keep."""
import pytest
import torch

from paged_variable_length_gb300 import pva
from test_linear_gpu import Case

pytestmark = pytest.mark.gpu

DEV = "cuda"


def i32(*x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("hint", [False, True], ids=["no-hint", "hint"])
@pytest.mark.parametrize("heads,lens,bad", [
    ((32, 32, 128), [1024, 1100], {1: 1 << 30}),
    ((32, 32, 128), [2000] * 8, {i: -7 for i in range(1, 8)}),
    ((32, 32, 64), [1500] * 3, {0: 5, 2: 5}),           # two requests at one slot
    ((16, 4, 128), [3000, 5, 2500, 700], {2: 99}),      # a batch that is cut
    ((16, 4, 128), [3000, 5, 2500, 700], {0: 99, 2: 99}),
    ((64, 8, 64), [200] * 9, {i: -2 for i in range(1, 7)}),      # the others' q heads shared by more CTAs than without the fault
], ids=["two", "eight", "clash", "cut", "cut-longest", "parts"])
def test_long_requests_beside_skipped_ones(heads, lens, bad, hint):
    """Requests with bad state slots are skipped; how the others are cut, and their bits, do not depend on them,
    whatever an earlier batch left in the workspace."""
    c = Case(heads, lens, [3] * len(lens), gate="token", seed=4)
    n = len(lens)
    c.state_in = i32(*range(n))
    c.state_out = i32(*range(n, 2 * n))
    kw = dict(max_q_len=max(lens)) if hint else {}
    was, want = c.run(**kw)
    if len(lens) < 8:
        c.check(was, want)
    after = c.states.clone()
    outs = [bad.get(i, n + i) for i in range(n)]
    c.state_out = i32(*outs)
    c.states.copy_(was)
    c.eng.workspace.fill_(255)      # (as fp32: NaN)
    c.prepare(**kw)
    out = c.forward()
    torch.cuda.synchronize()
    assert pva.attn_get_device_status(c.eng.meta) == 0x80
    at = 0
    for i, m in enumerate(lens):
        rows = out[at:at + m]
        if i in bad:
            assert bool((rows == 7).all()) and torch.equal(c.states[n + i], was[n + i])
        else:
            assert torch.equal(rows, want[at:at + m]) and torch.equal(c.states[n + i], after[n + i])
        at += m
    assert torch.equal(c.states[:n], was[:n]) and torch.equal(c.states[2 * n:], was[2 * n:])


@pytest.mark.parametrize("with_norm", [True, False], ids=["norm", "rotation"])
@pytest.mark.parametrize("rot,interleaved", [(64, False), (64, True), (32, False), (48, False)], ids=["split", "inter", "low", "part"])
@pytest.mark.parametrize("heads,lens", [((4, 2, 64), [3, 5, 2]), ((6, 3, 128), [1, 300, 20]), ((64, 64, 64), [500, 1100, 700])],
                         ids=["few", "long", "four-rows-a-warp"])
def test_a_bad_position_leaves_nothing_in_the_states(heads, lens, rot, interleaved, with_norm):
    """A layer's call with positions outside the table: those tokens are reported and count as q = k = 0, whatever
    q_rot and k_rot held; every other row, the outputs and the states are as of the call on such q and k."""
    Hq, Hkv, D = heads
    c = Case(heads, lens, [3] * len(lens), gate="token", seed=8, packed=True)
    T, end = c.T, sum(lens[:2])
    table = pva.rope_table(4000, rot, device=DEV)
    good = torch.arange(T, dtype=torch.int32, device=DEV)
    bad = [0, lens[0] + lens[1] - 1, end, T - 1] if T > 10 else [1, 4, 9]
    given = good.clone()
    given[bad] = i32(*[-1, 4000, 1 << 30, -(1 << 31)][:len(bad)])
    norm = pva.QKNorm(1 + 0.1 * torch.randn(D, device=DEV), None) if with_norm else None
    was = c.states.clone()
    c.prepare()
    # what the other tokens' rows are, and with 0 in the bad ones' place the recurrence of those
    q, k = c.eng.norm_rope(c.q, c.k, rope=pva.Rope(table, interleaved=interleaved, positions=good), norm=norm)
    q[bad], k[bad] = 0, 0
    want = c.eng.forward(q, k, c.v, c.log_decay, c.states)
    after = c.states.clone()
    assert pva.attn_get_device_status(c.eng.meta) == 0
    c.states.copy_(was)
    q_rot, k_rot = torch.full_like(q, float("nan")), torch.full_like(k, float("nan"))
    out = c.forward(rope=pva.Rope(table, interleaved=interleaved, positions=given), norm=norm, q_rot=q_rot, k_rot=k_rot)
    torch.cuda.synchronize()
    assert pva.attn_get_device_status(c.eng.meta) == 0x40
    assert torch.equal(q_rot, q) and torch.equal(k_rot, k)
    assert torch.equal(out, want) and torch.equal(c.states, after)
    assert bool((out[bad] == 0).all()) and bool(torch.isfinite(c.states).all())

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
], ids=["two", "eight", "clash", "cut", "cut-longest"])
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

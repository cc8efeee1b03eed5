"""GPU tests of linear attention's tokens that drop the state (log decays of -inf): whatever lay before them, infinities
and NaN among it, has no part in anything from them on."""
import pytest
import torch

import linear_reference as R
from paged_variable_length_gb300 import pva
from test_linear_gpu import Case

pytestmark = pytest.mark.gpu

DEV = "cuda"
INF, NAN = float("inf"), float("nan")


def last_reset(resets, n):
    """For each of a request's n tokens the last of `resets` (indices in the request) up to it, -1: none."""
    return torch.tensor([max([r for r in resets if r <= t], default=-1) for t in range(n)], device=DEV)


def reset_case(heads, lens, resets, seed, packed=False):
    """resets: for each request the tokens at which every second kv head (from the first) drops its state."""
    c = Case(heads, lens, [5] * len(lens), gate="token", seed=seed, packed=packed)
    at = 0
    for n, rs in zip(lens, resets):
        for r in rs:
            c.log_decay[at + r, ::2] = -INF
        at += n
    return c


SHAPES = [
    ((4, 2, 128), [1, 5, 16], [[0], [2], [0, 9]]),
    ((6, 3, 64), [1, 5, 16], [[0], [2], [15]]),
    ((4, 2, 128), [300, 130, 17], [[0], [129], [16]]),
    ((8, 4, 64), [300, 260, 128], [[37, 200], [128, 255], [127]]),
    ((2, 1, 128), [5200, 300], [[1300, 4000], [31]]),             # segments
    ((16, 2, 64), [2600, 700], [[128, 129, 2000], [690]]),        # q heads dealt out
]
IDS = ["few", "few-64", "edges", "chunks-64", "segments", "parts"]


@pytest.mark.parametrize("value", [NAN, INF, -INF], ids=["nan", "inf", "-inf"])
@pytest.mark.parametrize("heads,lens,resets", SHAPES, ids=IDS)
def test_a_reset_drops_a_state_that_is_not_finite(heads, lens, resets, value):
    """From the reset on outputs and states have the bits that a finite state before it leaves."""
    c = reset_case(heads, lens, resets, seed=21)
    Hkv, G = c.Hkv, c.Hq // c.Hkv
    was, want = c.run()
    c.check(was, want)
    after = c.states.clone()
    c.states.copy_(was)
    for i in range(c.B):      # of every head, the heads without resets too
        c.states[int(c.state_in[i]), :, 3, 5] = value
        c.states[int(c.state_in[i]), :, 40] = value
    out = c.forward()
    torch.cuda.synchronize()
    assert pva.attn_get_device_status(c.eng.meta) == 0
    at = 0
    for i, n in enumerate(lens):
        for h in range(Hkv):
            first = resets[i][0] if h % 2 == 0 else n
            rows = slice(at + first, at + n)
            assert torch.equal(out[rows, h * G:(h + 1) * G], want[rows, h * G:(h + 1) * G])
            slot = int(c.state_out[i])
            if h % 2 == 0:
                assert torch.equal(c.states[slot, h], after[slot, h])
            else:
                assert not bool(torch.isfinite(c.states[slot, h, 40]).any())
        at += n


@pytest.mark.parametrize("name", ["v", "k", "g"])
@pytest.mark.parametrize("value", [NAN, INF], ids=["nan", "inf"])
@pytest.mark.parametrize("heads,lens,resets", SHAPES[2:], ids=IDS[2:])
def test_a_reset_drops_odd_tokens(heads, lens, resets, value, name):
    """An infinity or a NaN in v, k or a decay of tokens before a reset: in no output from it on, and not in the state."""
    c = reset_case(heads, lens, resets, seed=22, packed=True)
    G = c.Hq // c.Hkv
    c.log_decay[:, 1:] -= 0.2
    was, want = c.run()
    after, gates, v, k = c.states.clone(), c.log_decay.clone(), c.v.clone(), c.k.clone()
    ref, S, mag, A = R.attend(c.q, k, v, gates, c.starts(was), lens)
    lim, slim = R.out_limit(ref, mag, gates, lens), R.state_limit(A, lens)
    # one odd token before each reset (none before a reset at token 0): at a distance, and right before it
    odd = torch.zeros(c.T, dtype=torch.bool, device=DEV)
    at = 0
    for n, rs in zip(lens, resets):
        for j, r in enumerate(rs):
            if r > 0:
                odd[at + (r - 1 if j else r // 2)] = True
        at += n
    for t in odd.nonzero().flatten().tolist():
        if name == "g":
            if float(c.log_decay[t, 0]) != -INF:
                c.log_decay[t, 0] = value
        else:
            (c.v if name == "v" else c.k)[t, 0, 7] = value
    c.states.copy_(was)
    _, out = c.run()
    at = 0
    for i, n in enumerate(lens):
        last = last_reset(resets[i], n)
        t = torch.arange(n, device=DEV)
        # clean: no odd token between the last reset (or the start) and the row
        seen = torch.cumsum(odd[at:at + n].int(), 0)
        before = torch.where(last > 0, seen[(last - 1).clamp(min=0)], 0)
        clean = seen == before
        rows, err = at + t[clean], (out.double() - ref).abs()
        assert bool((err[rows][:, :G] <= lim[rows][:, :G]).all()), "a row after a reset"
        assert bool((err[at:at + n, G:] <= lim[at:at + n, G:]).all()), "another head"
        slot = int(c.state_out[i])
        if bool(clean[-1]):
            assert bool(((c.states[slot, 0].double() - S[i, 0]).abs() <= slim[i, 0]).all()), "the state"
        if c.Hkv > 1:
            assert torch.equal(c.states[slot, 1:], after[slot, 1:])
        at += n


@pytest.mark.parametrize("heads", [(4, 2, 128), (2, 2, 64)], ids=["128", "64"])
def test_many_resets_cost_no_accuracy(heads):
    """A reset at every third token: sums start anew at each, so the bound counts the decays between them alone."""
    lens = [700, 129, 40]
    c = Case(heads, lens, [0, 3, 9], gate="token", seed=23)
    c.log_decay[1::3, 0] = -INF
    c.log_decay[::50, 1] = -200.0
    c.log_decay[:, 1] += 0.05       # (the state grows in between)
    was, out = c.run()
    ref, S, mag, A = R.attend(c.q, c.k, c.v, c.log_decay, c.starts(was), lens)
    gates = torch.where(c.log_decay <= -110, torch.zeros_like(c.log_decay), c.log_decay)
    assert bool(((out.double() - ref).abs() <= R.out_limit(ref, mag, gates, lens)).all())
    slim = R.state_limit(A, lens)
    for i in range(c.B):
        assert bool(((c.states[int(c.state_out[i])].double() - S[i]).abs() <= slim[i]).all())

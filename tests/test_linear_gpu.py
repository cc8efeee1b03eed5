"""GPU tests of linear attention with decays (attn_linear_prepare, attn_linear_forward), against the recurrence
in 64 bits."""
import pytest
import torch

import linear_reference as R
from paged_variable_length_gb300 import pva

pytestmark = pytest.mark.gpu

DEV = "cuda"


def decays(kind, T, Hkv, g):
    if kind == "none":
        return torch.zeros(Hkv, device=DEV)
    slope = -(2.0 ** (-9.0 * torch.rand(Hkv, generator=g, device=DEV)))
    if kind == "head":
        return slope
    if kind == "strong":      # a few tokens' memory, down to none
        return -torch.exp(torch.linspace(-1, 6, Hkv, device=DEV))
    x = slope * torch.nn.functional.softplus(2 * torch.randn(T, Hkv, generator=g, device=DEV))
    if kind == "resets":      # tokens that drop the state, -inf among them
        drop = torch.rand(T, Hkv, generator=g, device=DEV)
        x = torch.where(drop < 0.03, -float("inf"), torch.where(drop < 0.05, -300.0, x))
    return x


class Case:
    def __init__(self, heads, q_lens, cached, gate="head", seed=0, packed=False, in_place=True, scale=0.0):
        Hq, Hkv, D = self.Hq, self.Hkv, self.D = heads
        self.q_lens, self.cached = list(q_lens), list(cached)
        B, T = self.B, self.T = len(q_lens), sum(q_lens)
        g = torch.Generator(device=DEV).manual_seed(100 + seed)
        x = torch.randn(T, Hq + 2 * Hkv, D, generator=g, device=DEV).to(torch.bfloat16)
        self.q, self.k, self.v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
        if not packed:
            self.q, self.k, self.v = self.q.contiguous(), self.k.contiguous(), self.v.contiguous()
        self.log_decay = decays(gate, T, Hkv, g)
        self.num_states = 2 * B + 3
        self.states = torch.randn(self.num_states, Hkv, D, D, generator=g, device=DEV)
        perm = torch.randperm(self.num_states, generator=g, device=DEV).to(torch.int32)
        self.state_in = perm[:B].contiguous()
        self.state_out = self.state_in if in_place else perm[B:2 * B].contiguous()
        self.cu = torch.tensor([sum(q_lens[:i]) for i in range(B + 1)], dtype=torch.int32, device=DEV)
        self.lens = torch.tensor([n + c for n, c in zip(q_lens, cached)], dtype=torch.int32, device=DEV)
        self.scale = scale
        self.eng = pva.LinearAttention(Hq, Hkv, D, self.num_states, max(B, 1), max(T, 1), scale=scale)

    def prepare(self, **kw):
        a = dict(state_in=self.state_in, state_out=self.state_out)
        a.update(kw)
        return self.eng.prepare(self.cu, self.lens, self.T, **a)

    def starts(self, states):
        S = torch.zeros(self.B, self.Hkv, self.D, self.D, dtype=torch.float64, device=DEV)
        for i, c in enumerate(self.cached):
            if c > 0 and self.q_lens[i] > 0 and int(self.state_in[i]) >= 0:
                S[i] = states[int(self.state_in[i])].double()
        return S

    def forward(self, out=None, **kw):
        out = torch.full((self.T, self.Hq, self.D), 7.0, dtype=torch.bfloat16, device=DEV) if out is None else out
        return self.eng.forward(self.q, self.k, self.v, self.log_decay, self.states, out=out, **kw)

    def run(self, **kw):
        """(states before, out)"""
        was = self.states.clone()
        self.prepare(**kw)
        out = self.forward()
        torch.cuda.synchronize()
        assert pva.attn_get_device_status(self.eng.meta) == 0
        return was, out

    def check(self, was, out):
        scale = self.scale if self.scale > 0 else None
        ref, S, mag, A = R.attend(self.q, self.k, self.v, self.log_decay, self.starts(was), self.q_lens, scale)
        err = (out.double() - ref).abs()
        lim = R.out_limit(ref, mag, self.log_decay, self.q_lens)
        assert bool((err <= lim).all()), f"out: {float((err / lim).max()):.2f} of the limit"
        want, lim = was.double(), torch.zeros_like(was, dtype=torch.float64)
        slim = R.state_limit(A, self.q_lens)
        for i in range(self.B):
            slot = int(self.state_out[i])
            if self.q_lens[i] > 0 and slot >= 0:
                want[slot], lim[slot] = S[i], slim[i]
        err = (self.states.double() - want).abs()
        assert bool((err <= lim).all()), f"states: {float((err / lim.clamp(min=1e-30)).max()):.2f} of the limit"


HEADS = [(4, 4, 128), (8, 2, 128), (4, 4, 64), (6, 2, 64), (16, 1, 128), (3, 3, 64)]
LENS = [
    ([1], [0]),
    ([1, 1, 0, 2, 16], [0, 5, 9, 0, 3]),
    ([17, 1, 128, 129, 3], [0, 5, 0, 7, 2]),
    ([300, 5, 0, 700], [11, 0, 3, 0]),
]


@pytest.mark.parametrize("lens", LENS, ids=["one", "few", "edges", "long"])
@pytest.mark.parametrize("gate", ["none", "head", "token", "strong", "resets"])
@pytest.mark.parametrize("heads", HEADS, ids=["-".join(map(str, h)) for h in HEADS])
def test_against_the_recurrence(heads, gate, lens):
    c = Case(heads, *lens, gate=gate, seed=len(lens[0]), packed=gate == "token", in_place=gate != "head")
    c.check(*c.run())


@pytest.mark.parametrize("heads", [(4, 2, 128), (2, 2, 64)], ids=["128", "64"])
@pytest.mark.parametrize("where", [("v", 200), ("v", 3), ("k", 200), ("q", 150), ("g", 210)], ids=lambda w: f"{w[0]}{w[1]}")
@pytest.mark.parametrize("value", [float("nan"), float("inf")], ids=["nan", "inf"])
@pytest.mark.parametrize("fast", [0.0, 0.6, 2.0])
def test_hidden_infinities_and_nan(heads, where, value, fast):
    """An infinity or a NaN in one token's v, k, q or decay changes no token before it, no other request, and
    of the tokens after it (in v's case) only the columns that it lies in."""
    lens, cached = [300, 130, 9], [5, 0, 2]
    c = Case(heads, lens, cached, gate="token", seed=3)
    c.log_decay[:, 1] -= fast       # (chunks whose sums go further than one power for all rows reaches, or not)
    was, want = c.run()
    after, gates = c.states.clone(), c.log_decay.clone()
    ref, _, mag, _ = R.attend(c.q, c.k, c.v, c.log_decay, c.starts(was), lens)
    name, t = where
    x = {"v": c.v, "k": c.k, "q": c.q, "g": c.log_decay}[name]
    if name == "g":
        x[t, 1] = value
    else:
        x[t, 1, 7] = value
    c.states.copy_(was)
    _, out = c.run()
    bad = ~torch.isfinite(out.float())
    odd = torch.zeros_like(bad)
    G = c.Hq // c.Hkv
    if name == "q":
        odd[t, 1] = True
    elif name == "v":
        odd[t:300, G:2 * G, 7] = True
    else:
        odd[t:300, G:2 * G] = True
    assert bool((~bad | odd).all())
    # (their sums may be taken in another order)
    lim = R.out_limit(ref, mag, gates, lens)
    assert bool(((out.double() - ref).abs() <= lim)[~odd].all())
    assert torch.equal(out[300:], want[300:]) and torch.equal(out[:128 * (t // 128)], want[:128 * (t // 128)])
    if name == "v" and fast == 0:   # it stays in every later token's sum
        assert bool(bad[t:300, G:2 * G, 7].all())
    same = torch.ones(c.num_states, dtype=torch.bool, device=DEV)
    same[int(c.state_out[0])] = False
    assert torch.equal(c.states[same], after[same])
    i = int(c.state_out[0])
    assert torch.equal(c.states[i, 0], after[i, 0])

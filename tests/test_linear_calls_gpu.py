"""GPU tests of linear attention's calls: state slots, errors, refusals, graphs, streams, waits that run out, many
segments, and a hybrid model's layers (softmax and linear, q and k normed and rotated) over one batch."""
import pytest
import torch

import linear_reference as R
from paged_variable_length_gb300 import pva
from test_linear_gpu import Case

pytestmark = pytest.mark.gpu

DEV = "cuda"


def i32(*x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


# ------------------------------------------------------------------ lengths and layouts

@pytest.mark.parametrize("heads,lens,cached", [
    ((2, 1, 128), [5200, 1, 300], [0, 3, 9]),          # many segments
    ((8, 1, 64), [2600, 2, 0, 1100], [7, 0, 1, 0]),    # q heads dealt out
    ((16, 4, 128), [513], [4]),
    ((7, 7, 64), [128, 256, 384, 16, 17], [0, 0, 1, 2, 3]),
    ((12, 3, 128), [2000, 700], [0, 11]),
], ids=["segments", "head-parts", "one", "whole-chunks", "odd-heads"])
@pytest.mark.parametrize("gate", ["head", "resets"])
def test_long_requests(heads, lens, cached, gate):
    c = Case(heads, lens, cached, gate=gate, seed=7, packed=True)
    c.check(*c.run())
    again = c.states.clone()
    c = Case(heads, lens, cached, gate=gate, seed=7, packed=True)     # the same once more: bit for bit
    c.run()
    assert torch.equal(c.states, again)


@pytest.mark.parametrize("heads,lens", [((32, 8, 128), [16001]), ((28, 4, 128), [1400, 700, 1100, 500]),
                                        ((16, 16, 64), [900, 800, 850, 600, 500, 700, 300])], ids=["long", "prompts", "64"])
def test_many_runs_are_the_same(heads, lens):
    """Bit for bit, with the work of every SM's roles in as many orders as the runs make."""
    c = Case(heads, lens, [0] * len(lens), gate="token", seed=11)
    c.log_decay *= 0.05
    was, want = c.run()
    c.check(was, want)
    after = c.states.clone()
    for _ in range(40):
        c.states.copy_(was)
        assert torch.equal(c.forward(), want) and torch.equal(c.states, after)
    assert pva.attn_get_device_status(c.eng.meta) == 0


def test_scale_and_many_requests():
    g = torch.Generator().manual_seed(3)
    lens = [int(n) for n in torch.randint(0, 40, (300,), generator=g)]
    cached = [int(n) for n in torch.randint(0, 3, (300,), generator=g)]
    c = Case((2, 2, 64), lens, cached, gate="token", scale=0.37, in_place=False)
    c.check(*c.run())


@pytest.mark.parametrize("hint", [0, 16, 4])
def test_a_hint_of_few_tokens(hint):
    c = Case((4, 2, 128), [1, 4, 2], [3, 0, 9])
    c.check(*c.run(max_q_len=hint))


def test_strong_growth_and_decay_of_one_head():
    """Decays from token to token far apart, some above 0 (the state grows)."""
    c = Case((2, 2, 128), [300, 40], [4, 0], gate="token")
    c.log_decay[:, 0] = torch.linspace(-2.0, 0.4, 340, device=DEV)
    c.log_decay[::7, 1] = 3.0
    c.log_decay[3::7, 1] = -3.5
    c.check(*c.run())


def test_longer_buffers_and_strides():
    """Rows past the batch's tokens and states past the config's stay as they were; decays strided by token."""
    c = Case((4, 2, 64), [20, 3], [0, 2], gate="token")
    wide = torch.randn(60, 7, device=DEV)
    wide[:23, :2] = c.log_decay
    c.log_decay = wide[:, :2]
    pad = lambda x: torch.cat((x, torch.full_like(x, float("nan"))))
    c.q, c.k, c.v = pad(c.q), pad(c.k), pad(c.v)
    was = c.states.clone()
    more = torch.full_like(c.states, 5.0)
    c.states = torch.cat((c.states, more))
    c.prepare()
    out = torch.full((46, 4, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    c.forward(out)
    assert pva.attn_get_device_status(c.eng.meta) == 0
    assert bool((out[23:] == 7).all()) and torch.equal(c.states[c.num_states:], more)
    c.states, c.q, c.k, c.v, c.log_decay = c.states[:c.num_states], c.q[:23], c.k[:23], c.v[:23], c.log_decay[:23]
    c.check(was, out[:23])


# ------------------------------------------------------------------ states

def test_requests_that_go_on_from_one_state_and_keep_none():
    """A shared prefix's state read by several, a draft that is not kept, and fresh requests in a slot of NaN."""
    lens, cached = [3, 200, 1, 2], [9, 9, 9, 0]
    c = Case((4, 4, 64), lens, cached)
    c.state_in, c.state_out = i32(2, 2, 2, 5), i32(3, 4, -1, 5)
    c.states[5] = float("nan")      # a fresh request does not read its slot
    was, out = c.run()
    was[5] = c.states[5]            # (NaN before: what it holds now is checked below)
    c.check(was, out)
    assert bool(torch.isfinite(c.states[5]).all())


def test_without_states():
    c = Case((4, 4, 64), [3, 150], [9, 0])
    was = c.states.clone()
    c.prepare(state_in=None, state_out=None)
    out = c.forward()
    torch.cuda.synchronize()
    c.state_in, c.state_out = i32(-1, -1), i32(-1, -1)
    c.check(was, out)


@pytest.mark.parametrize("n", [2, 40], ids=["few", "many"])
def test_bad_slots_skip_their_requests(n):
    """A slot outside the pool, two requests at one, and a slot written that another reads: reported, nothing of the
    requests at fault written, the others as ever."""
    lens, cached = [n, 3, n, n, 2, n], [5, 5, 5, 5, 5, 5]
    for ins, outs, bad in (([0, 1, 2, 3, 4, 99], [0, 1, 2, 3, 4, 5], [5]),
                           ([0, 1, 2, 3, 4, 5], [0, 1, -2, 3, 4, 5], [2]),
                           ([0, 1, 2, 3, 4, 5], [0, 7, 2, 7, 4, 7], [1, 3, 5]),
                           ([0, 1, 2, 3, 4, 5], [0, 1, 4, 3, 6, 5], [2]),
                           ([0, 1, 2, 3, 4, 5], [0, 1, 2, 3, 4, 1 << 30], [5])):
        c = Case((2, 2, 64), lens, cached)
        c.state_in, c.state_out = i32(*ins), i32(*outs)
        was = c.states.clone()
        c.prepare()
        out = c.forward()
        torch.cuda.synchronize()
        assert pva.attn_get_device_status(c.eng.meta) == 0x80
        starts = torch.stack([was[s].double() if 0 <= s < c.num_states else was[0].double() * 0 for s in ins])
        ref, S, mag, A = R.attend(c.q, c.k, c.v, c.log_decay, starts, lens)
        lim = R.out_limit(ref, mag, c.log_decay, lens)
        at, want = 0, was.double()
        for i, m in enumerate(lens):
            if i in bad:
                assert bool((out[at:at + m] == 7).all())
            else:
                assert bool(((out[at:at + m].double() - ref[at:at + m]).abs() <= lim[at:at + m]).all())
                want[outs[i]] = S[i]
            at += m
        assert float((c.states.double() - want).abs().max()) <= float(R.state_limit(A, lens).max())


def test_errors_of_the_batch():
    c = Case((2, 2, 64), [3, 40], [5, 0])
    good_cu, good_lens, was = c.cu, c.lens, c.states.clone()
    for cu, lens, hint, bits in ((i32(0, 3, 42), good_lens, 0, 0x01), (i32(1, 3, 43), good_lens, 0, 0x01),
                                 (i32(0, 50, 43), good_lens, 0, 0x01), (good_cu, i32(2, 40), 0, 0x02),
                                 (good_cu, good_lens, 39, 0x10)):
        c.cu, c.lens = cu, lens
        c.prepare(max_q_len=hint)
        out = c.forward()
        assert pva.attn_get_device_status(c.eng.meta) & bits
        assert bool((out == 7).all()) and torch.equal(c.states, was)


def test_empty_batches():
    c = Case((2, 2, 64), [0, 0], [5, 0])
    was = c.states.clone()
    c.prepare()
    c.forward(torch.empty(0, 2, 64, dtype=torch.bfloat16, device=DEV))
    c.eng.prepare(i32(0), i32(), 0, i32(), i32())
    c.forward(torch.empty(0, 2, 64, dtype=torch.bfloat16, device=DEV))
    assert pva.attn_get_device_status(c.eng.meta) == 0 and torch.equal(c.states, was)


# ------------------------------------------------------------------ refusals

def test_refusals_launch_nothing():
    c = Case((4, 2, 64), [3, 40], [5, 0], gate="token", packed=True)
    c.prepare()
    was, out = c.states.clone(), torch.full((43, 4, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    lib = pva.load()

    def refused(status, call=None, **kw):
        a = dict(q=c.q.data_ptr(), k=c.k.data_ptr(), v=c.v.data_ptr(), out=out.data_ptr())
        f = dict(log_decay=c.log_decay.data_ptr(), ld_decay=2, ld_q=8 * 64, ld_k=8 * 64, ld_v=8 * 64, states=c.states.data_ptr())
        a.update({n: x for n, x in kw.items() if n in a})
        f.update({n: x for n, x in kw.items() if n in f})
        st = lib.attn_linear_forward(c.eng.meta, pva.LinearArgs(*[f[n] for n, _ in pva.LinearArgs._fields_]), a["q"], a["k"],
                                     a["v"], a["out"], pva._stream(None))
        assert st == status, kw

    for n in ("q", "k", "v", "out", "log_decay", "states"):
        refused(1, **{n: None})
        refused(1, **{n: {"q": c.q, "k": c.k, "v": c.v, "out": out, "log_decay": c.log_decay, "states": c.states}[n].data_ptr() + 2})
    refused(1, ld_q=4 * 64 - 8)
    refused(1, ld_k=8 * 64 + 4)
    refused(1, ld_v=64)
    refused(1, ld_decay=1)
    refused(1, ld_decay=-2)
    for x in (c.q, c.k, c.v, c.states, c.log_decay):      # an output over an input
        refused(1, out=x.data_ptr() // 16 * 16)
    refused(1, out=c.q.data_ptr() - 43 * 4 * 64 * 2 + 16)
    end = c.states.data_ptr() + c.states.numel() * 4
    for n in ("q", "k", "v", "log_decay"):                # an input in the pool of states
        refused(1, **{n: end - 16})
    assert lib.attn_linear_forward(pva.Meta(), pva.LinearArgs(), None, None, None, None, None) == 6
    paged = pva.PagedAttention(4, 2, 64, 16, 4, 2, 43, 64)
    paged.prepare(c.cu, c.lens, torch.zeros(2, 4, dtype=torch.int32, device=DEV), 43)
    with pytest.raises(pva.PvaError) as e:                # a plan of the other kind
        pva.attn_linear_forward(paged.meta, c.q, c.k, c.v, c.log_decay, torch.zeros(16, 16, 64, 64, device=DEV), out)
    assert e.value.status == 6
    with pytest.raises(pva.PvaError) as e:
        pva.attn_forward(c.eng.meta, c.q, c.k, c.v, out, out, out)
    assert e.value.status == 6
    torch.cuda.synchronize()
    assert torch.equal(c.states, was) and bool((out == 7).all())


def test_refusals_of_the_norm():
    c = Case((4, 2, 64), [3, 4], [5, 0])
    c.prepare()
    norm, rope = pva.QKNorm(torch.ones(64, device=DEV)), pva.Rope(pva.rope_table(64, 64, device=DEV))
    qo, ko = torch.empty_like(c.q), torch.empty_like(c.k)
    room = torch.zeros(3 * c.q.numel(), dtype=torch.bfloat16, device=DEV)
    at = lambda i, like: room[i:i + like.numel()].view(like.shape)
    for kw in (dict(q_out=at(0, c.q), k_out=at(64, c.k)), dict(q_out=c.k.new_empty(7, 4, 64)[:, :2]), dict(q_out=qo[:6]),
               dict(k_out=ko.float())):
        with pytest.raises(pva.PvaError) as e:
            c.eng.norm_rope(c.q, c.k, rope=rope, norm=norm, **{"q_out": qo, "k_out": ko, **kw})
        assert e.value.status == 1
    for q, k in ((at(0, c.q), at(c.q.numel() - 64, c.k)), (at(0, c.q), c.k)):
        with pytest.raises(pva.PvaError) as e:            # an output over the other input
            c.eng.norm_rope(q, k, rope=rope, norm=norm, q_out=qo, k_out=at(8, c.k))
        assert e.value.status == 1
    with pytest.raises(ValueError):
        c.eng.norm_rope(c.q, c.k)                         # neither a norm nor a rotation
    with pytest.raises(ValueError):
        c.eng.norm_rope(c.q, c.k, norm=pva.QKNorm(torch.ones(128, device=DEV)))
    # a layer call whose q_rot is v, or out
    v = c.v.clone()
    for kw in (dict(k_rot=v), dict(q_rot=at(0, c.q), out=at(8, c.q))):
        with pytest.raises(pva.PvaError) as e:
            c.eng.forward(c.q, c.k, v, c.log_decay, c.states, rope=rope, norm=norm, **kw)
        assert e.value.status == 1
    assert pva.attn_get_device_status(c.eng.meta) == 0


# ------------------------------------------------------------------ graphs, streams, waits

def test_prepare_and_layers_captured_and_replayed():
    """One graph of a plan and two layers' calls, replayed with other activations, lengths and slots; a second
    graph on an engine of its own beside it."""
    lens = [[1, 700, 3, 40], [300, 2, 441, 1]]
    cases = [Case((8, 2, 64), ln, [4, 0, 9, 1], gate="token", seed=i) for i, ln in enumerate(lens)]
    live = Case((8, 2, 64), lens[0], [4, 0, 9, 1], gate="token", seed=5)
    twin = Case((8, 2, 64), lens[0], [4, 0, 9, 1], gate="token", seed=5)
    layers = []
    graphs = []
    s = torch.cuda.Stream()
    for c in (live, twin):
        states = [torch.zeros_like(c.states) for _ in range(2)]
        outs = [torch.zeros(c.T, 8, 64, dtype=torch.bfloat16, device=DEV) for _ in range(2)]

        def step(stream=None, c=c, states=states, outs=outs):
            c.prepare(max_q_len=744, stream=stream)
            for st, o in zip(states, outs):
                c.eng.forward(c.q, c.k, c.v, c.log_decay, st, out=o, stream=stream)

        with torch.cuda.stream(s):
            step()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            step(s)
        layers.append((states, outs))
        graphs.append(g)
    names = ("q", "k", "v", "log_decay", "cu", "lens", "state_in")
    for c in cases:
        assert c.T == live.T
        want = c.states.clone()
        for (states, outs), target in zip(layers, (live, twin)):
            for n in names:
                getattr(target, n).copy_(getattr(c, n))
            target.state_out.copy_(c.state_out)
            for st in states:
                st.copy_(want)
        torch.cuda.synchronize()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        was, out = c.run()
        c.check(was, out)
        for (states, outs), target in zip(layers, (live, twin)):
            assert pva.attn_get_device_status(target.eng.meta) == 0
            for st, o in zip(states, outs):
                assert torch.equal(st, c.states) and torch.equal(o, out)


def test_calls_on_another_stream():
    c = Case((4, 4, 128), [200, 1], [3, 9])
    norm = pva.QKNorm(eps=1e-6)
    c.prepare()
    was = c.states.clone()
    want = c.eng.forward(c.q, c.k, c.v, c.log_decay, c.states, norm=norm)
    after = c.states.clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream, 0):
        c.states.copy_(was)
        torch.cuda.synchronize()
        out = torch.empty_like(want)
        c.eng.forward(c.q, c.k, c.v, c.log_decay, c.states, out=out, norm=norm, stream=stream)
        noise = torch.empty_like(want).fill_(3.0)   # current stream: must not be given q_rot's memory
        qn, kn = c.eng.norm_rope(c.q, c.k, norm=norm, stream=stream)
        side.synchronize()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(c.states, after) and bool((noise == 3.0).all())
        assert torch.equal(qn, c.eng.norm_rope(c.q, c.k, norm=norm)[0])
        torch.cuda.synchronize()


def test_waits_that_run_out_end_with_a_status():
    """With a limit of 0 the tensor-core kernel's waits give up; the next plan's calls are as ever."""
    c = Case((8, 2, 128), [1500, 300, 2], [0, 3, 1], gate="token")
    was, want = c.run()
    after = c.states.clone()
    c.states.copy_(was)
    c.prepare()
    pva.attn_debug_set_wait_limit(c.eng.meta, 0)
    c.forward()
    torch.cuda.synchronize()
    assert pva.attn_get_device_status(c.eng.meta) == 0x20
    c.states.copy_(was)
    got_was, got = c.run()
    assert torch.equal(got, want) and torch.equal(c.states, after)


def test_two_threads():
    """Two threads' calls of unlike layouts, each on its own stream and engine."""
    import threading

    cases = [Case((4, 4, 128), [300, 2], [1, 1]), Case((8, 2, 64), [1, 40, 260], [3, 0, 1], gate="token")]
    wants = []
    for c in cases:
        was, out = c.run()
        wants.append((was, out, c.states.clone()))
    bad = []

    def work(c, was, want, after):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(50):
                c.states.copy_(was)
                c.prepare()
                out = c.forward()
                s.synchronize()
                if not (torch.equal(out, want) and torch.equal(c.states, after)):
                    bad.append(c.Hq)

    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(c, *w)) for c, w in zip(cases, wants)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not bad


# ------------------------------------------------------------------ a hybrid model's layers

def test_hybrid_layers_back_to_back():
    """Softmax layers over a paged pool and linear layers over states, all with normed and rotated q and k, of one
    batch of prompts and decodes, back to back on one stream and the same buffers: as each layer alone, and the
    linear ones as the recurrence of what attn_norm_rope makes."""
    Hq, Hkv, D, ps = 16, 4, 128, 16
    ql, kl = [300, 1, 1, 20, 1], [300, 700, 33, 60, 1]
    T, B = sum(ql), len(ql)
    g = torch.Generator(device=DEV).manual_seed(2)
    cu = i32(*[sum(ql[:i]) for i in range(B + 1)])
    lens = i32(*kl)
    pages = [-(-n // ps) for n in kl]
    perm = torch.randperm(sum(pages), generator=g, device=DEV).to(torch.int32)
    table = torch.zeros(B, max(pages), dtype=torch.int32, device=DEV)
    at = 0
    for i, n in enumerate(pages):
        table[i, :n] = perm[at:at + n]
        at += n
    soft = pva.PagedAttention(Hq, Hkv, D, ps, sum(pages), B, T, max(kl))
    soft.prepare(cu, lens, table, T)
    lin = pva.LinearAttention(Hq, Hkv, D, B, B, T)
    slots = torch.randperm(B, generator=g, device=DEV).to(torch.int32)
    lin.prepare(cu, lens, T, slots, slots)
    rope = pva.Rope(pva.rope_table(max(kl), 64, device=DEV))
    layers = 6
    x = [torch.randn(T, Hq + 2 * Hkv, D, generator=g, device=DEV).to(torch.bfloat16) for _ in range(layers)]
    norms = [pva.QKNorm(*(1 + 0.2 * torch.randn(D, generator=g, device=DEV) for _ in range(2))) for _ in range(layers)]
    decay = [-torch.rand(T, Hkv, generator=g, device=DEV) * 0.2 for _ in range(layers)]
    pools = [torch.randn(2, sum(pages) * ps, Hkv, D, generator=g, device=DEV).to(torch.bfloat16) for _ in range(layers)]
    states = [torch.randn(B, Hkv, D, D, generator=g, device=DEV) for _ in range(layers)]
    q_rot, k_rot = torch.empty(T, Hq, D, dtype=torch.bfloat16, device=DEV), torch.empty(T, Hkv, D, dtype=torch.bfloat16, device=DEV)

    def call(i, out, pool, state):
        q, k, v = x[i][:, :Hq], x[i][:, Hq:Hq + Hkv], x[i][:, Hq + Hkv:]
        if i % 2:
            soft.forward(q, k, v, pool[0], pool[1], out=out, rope=rope, norm=norms[i], q_rot=q_rot)
        else:
            lin.forward(q, k, v, decay[i], state, out=out, rope=rope, norm=norms[i], q_rot=q_rot, k_rot=k_rot)

    alone = []
    for i in range(layers):
        pool, state, out = pools[i].clone(), states[i].clone(), torch.empty_like(q_rot)
        torch.cuda.synchronize()
        call(i, out, pool, state)
        torch.cuda.synchronize()
        alone.append((out, pool, state))
        if i % 2 == 0:
            q, k, v = x[i][:, :Hq], x[i][:, Hq:Hq + Hkv], x[i][:, Hq + Hkv:]
            qn, kn = lin.norm_rope(q, k, rope=rope, norm=norms[i])
            starts = torch.stack([states[i][int(slots[b])].double() * (kl[b] > ql[b]) for b in range(B)])
            ref, S, mag, A = R.attend(qn, kn, v, decay[i], starts, ql)
            assert bool(((out.double() - ref).abs() <= R.out_limit(ref, mag, decay[i], ql)).all())
            assert bool(((state[slots.long()].double() - S).abs() <= R.state_limit(A, ql)).all())
    outs = [torch.empty_like(q_rot) for _ in range(layers)]
    torch.cuda.synchronize()
    for i in range(layers):
        call(i, outs[i], pools[i], states[i])
    torch.cuda.synchronize()
    assert pva.attn_get_device_status(soft.meta) == 0 and pva.attn_get_device_status(lin.meta) == 0
    for i in range(layers):
        assert torch.equal(outs[i], alone[i][0]), f"layer {i}"
        assert torch.equal(pools[i], alone[i][1] if i % 2 else pools[i]) and torch.equal(states[i], states[i] if i % 2 else alone[i][2])


# ------------------------------------------------------------------ large sizes

def test_states_past_32_bit_offsets():
    """Slots of a pool of more than 2^31 elements, read and written by both forms: as in a small pool."""
    lens, cached = [200, 3, 17], [5, 4, 0]
    small = Case((32, 32, 128), lens, cached, in_place=False)
    was, want = small.run()
    after = small.states.clone()
    n = (1 << 31) // (32 * 128 * 128) + 40
    big = Case((32, 32, 128), lens, cached, in_place=False)
    big.num_states, big.states = n, torch.empty(n, 32, 128, 128, device=DEV)
    big.eng = pva.LinearAttention(32, 32, 128, n, 3, big.T)
    shift = n - small.num_states
    big.state_in, big.state_out = small.state_in + shift, small.state_out + shift
    big.states[shift:] = was
    big.prepare()
    out = big.forward()
    assert pva.attn_get_device_status(big.eng.meta) == 0
    assert torch.equal(out, want) and torch.equal(big.states[shift:], after)


def test_tokens_past_32_bit_offsets():
    """The last requests of a batch of more than 2^31 elements of q: as in a batch of their own."""
    heads, tail = (64, 1, 128), [200, 5]
    first = (1 << 31) // (64 * 128) + 1000
    alone = Case(heads, tail, [3, 2], gate="token")
    was, want = alone.run()
    T = first + sum(tail)
    q, k, v = (torch.empty(T, h, 128, dtype=torch.bfloat16, device=DEV).fill_(0.01) for h in (64, 1, 1))
    q[first:], k[first:], v[first:] = alone.q, alone.k, alone.v
    decay = torch.full((T, 1), -0.01, device=DEV)
    decay[first:] = alone.log_decay
    states = torch.cat((was, torch.zeros_like(was[:1])))
    eng = pva.LinearAttention(64, 1, 128, states.shape[0], 3, T)
    slot = was.shape[0]
    ins = torch.cat((i32(slot), alone.state_in))
    eng.prepare(i32(0, first, first + 200, T), i32(first, 203, 7), T, ins, ins)
    qn, kn = eng.norm_rope(q, k, norm=pva.QKNorm(), rope=pva.Rope(torch.zeros(first, 128, device=DEV) + 1.0))
    out = eng.forward(q, k, v, decay, states)
    assert pva.attn_get_device_status(eng.meta) == 0
    assert torch.equal(out[first:], want) and torch.equal(states[:slot], alone.states)
    rope = pva.Rope(torch.ones(400, 128, device=DEV))
    alone.prepare()
    qs, ks = alone.eng.norm_rope(alone.q, alone.k, norm=pva.QKNorm(), rope=rope)
    assert torch.equal(qn[first:], qs) and torch.equal(kn[first:], ks)
    # the first one's: q, k and v of one value, so o_t = scale D x^2 v sum_{s <= t} e^{-0.01 (t - s)}
    x = float(torch.tensor(0.01, dtype=torch.bfloat16))
    for t in (0, 1000, first - 1):
        ref = 128 ** 0.5 * x ** 3 * (1 - 2.718281828459045 ** (-0.01 * (t + 1))) / (1 - 2.718281828459045 ** -0.01)
        assert bool(((out[t].double() - ref).abs() <= 2.0 ** -6 * ref).all())

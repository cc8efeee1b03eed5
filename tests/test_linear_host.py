"""Linear attention and the norm of q and k without a GPU: structures, refusals that need no device, and the
plan's rules."""
import ctypes
import os
import subprocess

import pytest
import torch

from paged_variable_length_gb300 import build, pva

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    build.build()
    return pva.load()


@pytest.mark.parametrize("name,mirror", [("pva_qk_norm", pva.QKNormArgs), ("pva_linear_config", pva.LinearConfig),
                                         ("pva_linear_args", pva.LinearArgs)])
def test_structs_match_the_header(tmp_path, name, mirror):
    fields = [f for f, _ in mirror._fields_]
    src = tmp_path / "probe.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "pva.h"\nint main(void){\n'
                   f'printf("%zu\\n", sizeof({name}));\n'
                   + "".join(f'printf("%zu\\n", offsetof({name}, {f}));\n' for f in fields) + "return 0;}\n")
    exe = tmp_path / "probe"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    vals = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert vals == [ctypes.sizeof(mirror)] + [getattr(mirror, f).offset for f in fields]


def test_the_calls_need_a_prepared_meta(lib):
    meta, d = pva.Meta(), ctypes.c_void_p(256)
    rope, norm = pva.RopeArgs(256, None, 64, 64, 64, 16, 32, 0, 0), pva.QKNormArgs(None, None, 1e-6, 0)
    lin = pva.LinearArgs(256, 0, 64, 64, 64, 256)
    for m in (meta, None):
        assert lib.attn_append_norm_rope(m, norm, rope, d, d, d, d, d, d, None, None, None) == 6
        assert lib.attn_forward_norm_rope(m, norm, rope, d, d, d, d, d, d, None, None, d, None, None) == 6
        assert lib.attn_norm_rope(m, norm, rope, d, d, d, d, None) == 6
        assert lib.attn_linear_forward(m, lin, d, d, d, d, None) == 6
        assert lib.attn_linear_forward_norm_rope(m, lin, norm, rope, d, d, d, d, d, d, None) == 6


GOOD = dict(num_qo_heads=8, num_kv_heads=2, head_dim=128, num_states=10, max_batch=4, max_tokens=64)


@pytest.mark.parametrize("kw,status", [(dict(head_dim=96), 2), (dict(num_qo_heads=9), 1), (dict(num_kv_heads=0), 1),
                                       (dict(num_states=0), 1), (dict(num_states=1 << 31), 2), (dict(max_batch=0), 1),
                                       (dict(max_batch=65536), 2), (dict(max_tokens=-1), 1), (dict(scale=float("nan")), 1),
                                       (dict(scale=float("inf")), 1)])
def test_configs_that_are_refused(lib, kw, status):
    cfg = pva.make_linear_config(**{**GOOD, **kw})
    assert pva.attn_linear_workspace_size(cfg) == 0
    d = ctypes.c_void_p(256)
    assert lib.attn_linear_prepare(ctypes.byref(cfg), d, d, d, d, 1, 1, 1, d, 1 << 20, None, ctypes.byref(pva.Meta())) == status


def test_prepare_refuses_on_the_host(lib):
    cfg, d = pva.make_linear_config(**GOOD), ctypes.c_void_p(256)
    meta = pva.Meta()
    prepare = lambda cu=d, lens=d, batch=1, tokens=1, ws=d, m=ctypes.byref(meta): lib.attn_linear_prepare(
        ctypes.byref(cfg), cu, lens, None, None, batch, tokens, 0, ws, 16, None, m)
    assert prepare() in (3, 4)      # a workspace of 16 bytes, or no device
    assert prepare(lens=None, batch=0, tokens=0) in (3, 4)
    for kw in (dict(cu=None), dict(lens=None), dict(batch=5), dict(tokens=65), dict(batch=-1), dict(tokens=-1),
               dict(batch=0), dict(ws=None), dict(ws=ctypes.c_void_p(264)), dict(m=None)):
        assert prepare(**kw) == 1, kw


def test_what_the_binding_of_prepare_refuses(lib):
    cfg, batch = pva.make_linear_config(8, 2, 64, 10, 4, 64), 3
    i32 = lambda n: torch.zeros(n, dtype=torch.int32)
    room = torch.empty(1024, dtype=torch.uint8)
    room = room[-room.data_ptr() % 256:]

    def prepare(**kw):
        a = {**dict(cu=i32(batch + 1), lens=i32(batch), ins=i32(batch), outs=i32(batch)), **kw}
        try:
            pva.attn_linear_prepare(cfg, a["cu"], a["lens"], a["ins"], a["outs"], batch, 9, 0,
                                    room, stream=0)
        except pva.PvaError as e:
            return e.status
        return 0

    assert prepare() != 1 and prepare(ins=None, outs=None) != 1      # (no device, or the workspace is too small)
    for name, n in (("cu", batch + 1), ("lens", batch), ("ins", batch), ("outs", batch)):
        for bad in (i32(n - 1), i32(n).long(), i32(2 * n)[::2], i32(n).float()):
            assert prepare(**{name: bad}) == 1, name


T, HQ, HKV, D = 5, 4, 2, 64


def batch_of(device=-1):
    meta = pva.Meta()
    meta.batch = pva.Batch(HQ, HKV, D, 3, pva._STATES, T, device)
    return meta


def tensors():
    e = lambda *s, dtype=torch.bfloat16: torch.empty(*s, dtype=dtype)
    return dict(q=e(T, HQ, D), k=e(T, HKV, D), v=e(T, HKV, D), out=e(T, HQ, D), q_rot=e(T, HQ, D), k_rot=e(T, HKV, D),
                log_decay=torch.zeros(HKV), states=torch.zeros(3, HKV, D, D))


CALLS = {
    "forward": (("q", "k", "v", "out", "log_decay", "states"),
                lambda m, a: pva.attn_linear_forward(m, a["q"], a["k"], a["v"], a["log_decay"], a["states"], a["out"], stream=0)),
    "layer": (("q", "k", "v", "out", "q_rot", "k_rot", "log_decay", "states"),
              lambda m, a: pva.attn_linear_forward_norm_rope(m, pva.QKNorm(), None, a["q"], a["k"], a["v"], a["q_rot"],
                                                             a["k_rot"], a["log_decay"], a["states"], a["out"], stream=0)),
    "norm": (("q", "k", "q_rot", "k_rot"),
             lambda m, a: pva.attn_norm_rope(m, pva.QKNorm(torch.ones(D)), None, a["q"], a["k"], a["q_rot"], a["k_rot"], stream=0)),
}


def status(call, meta, a):
    try:
        call(meta, a)
    except ValueError:
        return 1
    except pva.PvaError as e:
        return e.status
    return 0


@pytest.mark.parametrize("name", CALLS)
def test_what_the_binding_passes_and_refuses(lib, name):
    takes, call = CALLS[name]
    assert status(call, batch_of(), tensors()) == 6      # gets as far as the library
    for n in takes:
        for change in (lambda x: x[:-1], lambda x: x.to(torch.float16), lambda x: x.new_empty(*x.shape[:-1], 2 * x.shape[-1])[..., ::2]):
            a = tensors()
            a[n] = change(a[n])
            if n == "log_decay" and a[n].shape == (HKV,) and a[n].dtype == torch.float32 and a[n].is_contiguous():
                continue
            assert status(call, batch_of(), a) == 1, n
    assert status(call, batch_of(device=0), tensors()) == 1     # host tensors of a batch on a GPU
    if "log_decay" in takes:
        for good in (torch.zeros(T, HKV), torch.zeros(T + 2, 2 * HKV)[:, :HKV]):
            assert status(call, batch_of(), {**tensors(), "log_decay": good}) == 6
        for bad in (torch.zeros(T - 1, HKV), torch.zeros(HKV, T).T, torch.zeros(T, HKV + 1), torch.zeros(1, T, HKV)):
            assert status(call, batch_of(), {**tensors(), "log_decay": bad}) == 1
        a = tensors()
        qkv = torch.empty(T, HQ + 2 * HKV, D, dtype=torch.bfloat16)
        a.update(q=qkv[:, :HQ], k=qkv[:, HQ:HQ + HKV], v=qkv[:, HQ + HKV:])
        assert status(call, batch_of(), a) == 6


def test_norms_that_are_refused():
    for bad in (dict(q_gain=torch.ones(64, dtype=torch.float16)), dict(k_gain=torch.ones(2, 64)), dict(q_gain=torch.ones(128)[::2]),
                dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf"))):
        with pytest.raises(ValueError):
            pva.QKNorm(**bad)
    with pytest.raises(ValueError):
        pva.QKNorm(torch.ones(64)).args(128, -1)
    with pytest.raises(ValueError):
        pva.QKNorm(torch.ones(64)).args(64, 0)


def test_segments_never_outgrow_their_workspace(tmp_path):
    """The plan's rules, compiled for the host: whatever the lengths, a batch's segments with a state in the workspace
    fit it (3 (sms / Hkv) + 3 of them), and a request stays whole or is cut into pieces that cover it."""
    src = tmp_path / "rules.cpp"
    src.write_text(r'''
#include <cstdio>
#include <cstdlib>
#include "linear.h"
using namespace pva;
int main() {
    srand(3);
    for (int round = 0; round < 20000; ++round) {
        const int sms = 152, hkv = 1 + rand() % 40, group = 1 + rand() % 16, B = 1 + rand() % (round % 2 ? 5 : 200);
        int n[200]; long long total = 0; int longest = 0;
        for (int i = 0; i < B; ++i) {
            n[i] = kStepTokens + 1 + rand() % (rand() % 3 ? 900 : 1 + rand() % 30000);
            total += n[i];
            if (n[i] > longest) longest = n[i];
        }
        const int seg = segment_tokens(total, longest, hkv, sms);
        long long items = 0, with_state = 0;
        for (int i = 0; i < B; ++i) {
            const int chunks = (n[i] + kChunk - 1) / kChunk, want = (int)(((long long)n[i] + seg - 1) / seg);
            const int per = (chunks + want - 1) / want, nseg = (chunks + per - 1) / per;
            if ((long long)(nseg - 1) * per * kChunk >= n[i] || (long long)nseg * per * kChunk < n[i]) return printf("cover\n"), 1;
            items += nseg;
            if (nseg > 1) with_state += nseg;
        }
        const int parts = head_parts(items, group, hkv, sms);
        if (parts > 1)
            for (int i = 0; i < B; ++i) with_state += n[i] <= seg;
        if (with_state > 3 * (sms / hkv) + 3) return printf("%lld states, Hkv %d\n", with_state, hkv), 1;
        if (parts < 1 || (parts > 1 && parts > group / 2)) return printf("parts\n"), 1;
        // fewer tokens known for certain: never whole where the plan cuts
        const long long least = total - rand() % 500;
        if (segment_tokens(least > 0 ? least : 0, longest, hkv, sms) == kWholeSegment && seg != kWholeSegment) return printf("cut\n"), 1;
    }
    return 0;
}
''')
    exe = tmp_path / "rules"
    subprocess.run(["g++", "-std=c++17", "-I", os.path.join(build.CSRC), "-I", "/usr/local/cuda/include", str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout

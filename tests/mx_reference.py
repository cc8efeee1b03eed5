"""Plain references of the MXFP4 pool and the rotary append, in numpy, written from the formats'
and the rotation's definitions: 64-bit values, and the fp32 steps where the bits are defined."""
from __future__ import annotations

import numpy as np

E_LO, E_HI, E_NAN = 105, 140, 255
MAGNITUDES = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], np.float64)


def row_layout(Hkv, D):
    """(heads per group, bytes of a group, bytes of a row)."""
    hb = min(Hkv, 8)
    group = hb * (D // 2 + D // 32)
    return hb, group, -(-(Hkv // hb * group) // 16) * 16


def quantise(x):
    """fp32 [..., 32] blocks -> (codes uint8 [..., 32], scale bytes uint8 [...])."""
    x = np.asarray(x, np.float32)
    a = np.abs(x)
    finite = np.isfinite(x).all(-1)
    top = np.where(finite, a.max(-1), 1.0).astype(np.float64)
    _, ex = np.frexp(top)
    e = np.where(top == 0, E_LO, np.clip(ex - 1 - 2 + 127, E_LO, E_HI))
    u = a.astype(np.float64) * 2.0 ** (127.0 - e)[..., None]
    # nearest magnitude; a tie goes to the even code
    d = np.abs(u[..., None] - MAGNITUDES)
    near = d.min(-1, keepdims=True)
    tie = d == near
    code = np.where(tie & (np.arange(8) % 2 == 0), np.arange(8), np.where(tie, np.arange(8) + 100, 1000)).min(-1) % 100
    code = code.astype(np.uint8) | (np.signbit(x).astype(np.uint8) << 3)
    code = np.where(finite[..., None], code, 0).astype(np.uint8)
    return code, np.where(finite, e, E_NAN).astype(np.uint8)


def pack_rows(x):
    """fp32 [N, Hkv, D] -> rows uint8 [N, row_bytes] (padding zero)."""
    N, Hkv, D = x.shape
    hb, group, rb = row_layout(Hkv, D)
    code, e = quantise(x.reshape(N, Hkv, D // 32, 32))
    code = code.reshape(N, Hkv, D)
    byte = (code[..., 0::2] | (code[..., 1::2] << 4)).astype(np.uint8)
    rows = np.zeros((N, rb), np.uint8)
    for h in range(Hkv):
        g0, i = h // hb * group, h % hb
        rows[:, g0 + i * (D // 2): g0 + (i + 1) * (D // 2)] = byte[:, h]
        s0 = g0 + hb * (D // 2) + i * (D // 32)
        rows[:, s0:s0 + D // 32] = e[:, h]
    return rows


def unpack_rows(rows, Hkv, D):
    """rows uint8 [N, row_bytes] -> float64 [N, Hkv, D]."""
    N = rows.shape[0]
    hb, group, _ = row_layout(Hkv, D)
    out = np.empty((N, Hkv, D))
    for h in range(Hkv):
        g0, i = h // hb * group, h % hb
        byte = rows[:, g0 + i * (D // 2): g0 + (i + 1) * (D // 2)]
        code = np.stack((byte & 15, byte >> 4), -1).reshape(N, D)
        s0 = g0 + hb * (D // 2) + i * (D // 32)
        e = rows[:, s0:s0 + D // 32].astype(np.int64)
        scale = np.where(e == E_NAN, np.nan, 2.0 ** (e - 127.0))
        val = MAGNITUDES[code & 7] * np.where(code & 8, -1.0, 1.0)
        out[:, h] = (val.reshape(N, D // 32, 32) * scale[..., None]).reshape(N, D)
    return out


def rotate(x, cos_sin, positions, interleaved, dtype):
    """x [T, H, D] rotated, in `dtype` arithmetic (every product and sum rounded by itself)."""
    x = np.asarray(x, dtype)
    rot = cos_sin.shape[1]
    cs = np.asarray(cos_sin, dtype)[np.asarray(positions)]
    c, s = cs[:, None, :rot // 2], cs[:, None, rot // 2:]
    y = x.copy()
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * c - b * s, b * c + a * s
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = a * c - b * s, b * c + a * s
    return y


def attention(q, k_rows, v_rows, q_lens, kv_lens, slots_of, Hkv, scale=None, k_new=None, v_new=None):
    """Causal (bottom-right) GQA attention in float64, request by request.

    q [T, Hq, D]; k_rows / v_rows: functions of a slot list giving float64 [n, Hkv, D];
    slots_of(i): the slots of request i's positions 0 .. kv_len - 1.
    Returns (out, lse, spread, reach, small): spread = sum_j p_j |v_jd|, reach = the largest sum
    over d of |q_d k_jd| * scale of a row, small = sum_j |v_jd|, from which tolerances are formed.
    """
    T, Hq, D = q.shape
    G = Hq // Hkv
    scale = 1.0 / np.sqrt(D) if scale is None else scale
    q = np.asarray(q, np.float64)
    out, spread, small = np.zeros((T, Hq, D)), np.zeros((T, Hq, D)), np.zeros((T, Hq, D))
    lse, reach = np.zeros((T, Hq)), np.zeros((T, Hq))
    t = 0
    for i, (n, L) in enumerate(zip(q_lens, kv_lens)):
        if n == 0:
            continue
        sl = slots_of(i)
        K, V = k_rows(sl), v_rows(sl)
        seen = np.arange(L)[None, :] <= (L - n) + np.arange(n)[:, None]
        for h in range(Hkv):
            qh = q[t:t + n, h * G:(h + 1) * G]                       # [n, G, D]
            x = np.einsum("ngd,ld->ngl", qh, K[:, h]) * scale
            x = np.where(seen[:, None, :], x, -np.inf)
            m = x.max(-1, keepdims=True)
            p = np.exp(x - m)
            l = p.sum(-1, keepdims=True)
            p = p / l
            # masked keys weigh nothing, whatever they hold
            Vh = np.where(seen.any(0)[:, None], V[:, h], 0.0)
            out[t:t + n, h * G:(h + 1) * G] = np.einsum("ngl,ld->ngd", p, Vh)
            spread[t:t + n, h * G:(h + 1) * G] = np.einsum("ngl,ld->ngd", p, np.abs(Vh))
            small[t:t + n, h * G:(h + 1) * G] = np.abs(Vh).sum(0)
            lse[t:t + n, h * G:(h + 1) * G] = (m + np.log(l))[..., 0]
            reach[t:t + n, h * G:(h + 1) * G] = np.where(
                seen[:, None, :], np.einsum("ngd,ld->ngl", np.abs(qh), np.abs(K[:, h])), 0.0).max(-1) * scale
        t += n
    return out, lse, spread, reach, small


def tolerances(out, lse, spread, reach, small, D):
    """What the kernels' roundings allow, from first principles:
    - a score is a sum of D products in fp32, in any order: off by at most (D + 8) 2^-24 of the
      sum of magnitudes (`reach`); a weight p_j is then off by e^(2 x that) at most, plus 2^-20 for
      exp2 and its argument;
    - P, held as 2^7 (tensor cores; at most 2^8 under their lazily raised maximum) or 2^15 (decode)
      times a weight relative to a maximum not above the row's largest, is rounded to f16: 2^-11
      relative, and below f16's normal range half of its smallest step, 2^-25 / 2^7 = 2^-32 of the
      largest weight (so at most 2^-32 sum_j |v_j| in all); products and sums in fp32 add less
      than 2^-13;
    - out is rounded to bf16 (2^-8, and half a step of its subnormals)."""
    ds = (D + 8) * 2.0 ** -24 * reach
    dp = np.expm1(2 * ds) + 2.0 ** -20
    tol = 2.0 ** -8 * np.abs(out) + (dp[..., None] + 2.0 ** -11 + 2.0 ** -13) * spread * (1 + 2.0 ** -8) \
        + 2.0 ** -32 * small + 2.0 ** -134
    return tol, ds + 2.0 ** -20 * (1 + np.abs(lse))

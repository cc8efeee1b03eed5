"""Linear attention with decays and the norm of q and k, plain and in 64 bits (torch, any device)."""
import math

import torch


def norm_heads(x, gain, eps):
    """[T, H, D] -> each head over its root mean square, times the gain."""
    x = x.double()
    y = x / (x.pow(2).mean(-1, keepdim=True) + eps).sqrt()
    return y if gain is None else y * gain.double()


def attend(q, k, v, log_decay, starts, q_lens, scale=None):
    """The recurrence, token by token.  starts: float64 [B, Hkv, D, D]; log_decay [Hkv] or [T, Hkv].  Returns out
    [T, Hq, D], the states [B, Hkv, D, D] and, of each, the sums of the terms' absolute values."""
    q, k, v, g = (x.double() for x in (q, k, v, log_decay))
    (T, Hq, D), Hkv = q.shape, k.shape[1]
    scale = 1 / math.sqrt(D) if scale is None else scale
    out, mag = torch.zeros(2, T, Hq, D, dtype=torch.float64, device=q.device)
    S, A = starts.double().clone(), starts.double().abs()
    lam = torch.exp(g)
    at = 0
    for b, n in enumerate(q_lens):
        for t in range(at, at + n):
            decay = (lam[t] if g.dim() == 2 else lam)[:, None, None]
            new = k[t][:, :, None] * v[t][:, None, :]
            S[b] = torch.where(decay == 0, 0.0, decay * S[b]) + new
            A[b] = torch.where(decay == 0, 0.0, decay * A[b]) + new.abs()
            qt = q[t].reshape(Hkv, Hq // Hkv, D)
            out[t] = scale * torch.matmul(qt, S[b]).reshape(Hq, D)
            mag[t] = scale * torch.matmul(qt.abs(), A[b]).reshape(Hq, D)
        at += n
    return out, S, mag, A


def chunk_depth(log_decay, q_lens):
    """Largest |sum of log2 decays| over a 128-token chunk of any request (-inf counts as the kernels take it)."""
    g = log_decay.double().clamp(min=-110.0) / math.log(2)
    if g.dim() == 1:
        return float(g.abs().max()) * min(128, max(q_lens))
    worst, t = 0.0, 0
    for n in q_lens:
        for c in range(0, n, 128):
            worst = max(worst, float(g[t + c:t + min(c + 128, n)].sum(0).abs().max()))
        t += n
    return worst


def out_limit(ref, mag, log_decay, q_lens):
    """How far an output may be off.  Rounding it to bf16: half a step, 2^-8 of it.  Requests of more than 16 tokens:
    the weights within a chunk and the copy of the state are rounded to bf16 before the products (2^-8 of every
    term), and their exponents are differences of two fp32 sums (2^-24 of the chunk's depth each, times ln 2), the
    exponential itself 2^-22.  fp32 products and sums: every term passes at most D + 128 additions and the state's
    own (state_limit's)."""
    lim = torch.empty_like(ref)
    depth = chunk_depth(log_decay, q_lens)
    t = 0
    for n in q_lens:
        steps = 32 * math.ceil(n / 128) if n > 16 else 6 * n
        rel = 2.0 ** -24 * (ref.shape[-1] + 128 + 256 + steps)
        if n > 16:
            rel += 2.0 ** -8 + 2 * 2.0 ** -24 * depth * math.log(2) + 2.0 ** -22
        lim[t:t + n] = ref[t:t + n].abs() * 2.0 ** -8 + mag[t:t + n] * rel * (1 + 2.0 ** -7) + 1e-38
        t += n
    return lim


def state_limit(A, q_lens):
    """How far a state may be off, beside the sums A of its terms' absolute values: fp32 throughout.  A weight is an
    exponential of a fp32 argument of at most 160 (2^-24 of it, times ln 2) within 2 ulp; the three parts of a
    weighted key hold it whole; a chunk's sum takes 24 additions of 16 products each, whose roundings (to nearest
    or towards zero) come to at most 2^-22 of the terms for each; each chunk or token then two roundings and a
    decay."""
    n = torch.tensor(q_lens, dtype=torch.float64, device=A.device)
    steps = torch.where(n > 16, 32 * torch.ceil(n / 128), 6 * n)
    return A * (2.0 ** -24 * (256 + steps))[:, None, None, None] + 1e-38

"""Plain forms in 64 bits of rotary positions, prompt attention, gathered weight and the choice of
the heaviest tokens, with error bounds from the arithmetic that include/kvc.h states.  Test
infrastructure only; torch tensors on any device."""
import math

import torch

F64 = torch.float64
# Half a step of bf16, of fp32 and a whole one of fp32 (what truncates), relative to the value.
BF, HALF, STEP = 2.0 ** -8, 2.0 ** -24, 2.0 ** -23


def frequencies(dim, base=10000.0, scaling="none", factor=1.0, low=1.0, high=4.0, original=0.0):
    """Radians a token of each pair."""
    out = []
    for i in range(dim // 2):
        b = base * factor ** (dim / (dim - 2)) if scaling == "ntk" else base
        f = b ** (-2 * i / dim)
        if scaling == "linear":
            f /= factor
        if scaling == "bands":
            m = min(max((original * f / (2 * math.pi) - low) / (high - low), 0.0), 1.0)
            f = (1 - m) * f / factor + m * f
        out.append(f)
    return out


def rotary(x, pos, f, interleaved, magnitude=1.0):
    """x [..., n, d], pos [..., n] (broadcast against x's leading axes), f: radians a token of each
    pair -> rows and their bound.  Angles are off by 2^-29 + 2^-51 |a| (and this form's own products
    by 2^-52 |a|), fp32 sines by 2 steps each, times the magnitude (one rounding), products and
    their sum (the second is fused) by one rounding each; the result is rounded to bf16."""
    x, dim = x.to(F64), 2 * len(f)
    a = pos.to(F64)[..., None] * torch.tensor(f, dtype=F64, device=x.device)
    cos, sin = a.cos() * magnitude, a.sin() * magnitude
    y, lead = x.clone(), torch.zeros_like(x)
    i = torch.arange(dim // 2, device=x.device)
    p, q = (2 * i, 2 * i + 1) if interleaved else (i, i + dim // 2)
    y[..., p] = x[..., p] * cos - x[..., q] * sin
    y[..., q] = x[..., p] * sin + x[..., q] * cos
    off = (2.0 ** -29 + 2.0 ** -50 * a.abs() + 8 * STEP) * magnitude * (x[..., p].abs() + x[..., q].abs())
    lead[..., p] = off
    lead[..., q] = off
    turned = torch.zeros(x.shape[-1], dtype=torch.bool, device=x.device)
    turned[:dim] = True
    return y, torch.where(turned, lead + BF * (y.abs() + lead), 0.0)


def attention(q, k, v, scale):
    """One head of one prompt: q, k, v [m, d] -> out, lse and their bounds.

    A logit is off by d products summed in fp32 (steps, since a tensor core may truncate) and its
    scaling: (d + 8) STEP scale sum |q k|, by fp32's roundings of x = log2(e) z, of x - M and of M:
    STEP of |z| + |z|max, and the exponential's own 2^-21.  A weight is rounded to bf16 for the
    product with v, sums over m tokens are fp32, the output is rounded to bf16.  A weight that a
    type's smallest number ends is below 2^-100 of the largest."""
    q, k, v = q.to(F64), k.to(F64), v.to(F64)
    m, d = q.shape
    sees = torch.ones((m, m), dtype=torch.bool, device=q.device).tril()
    z = (q @ k.T * scale).masked_fill(~sees, -math.inf)
    top = z.amax(-1, keepdim=True)
    w = (z - top).exp()
    total = w.sum(-1, keepdim=True)
    p, lse = w / total, (top + total.log())[:, 0]
    out = p @ v
    zmax = torch.where(sees, z.abs(), 0).amax(-1, keepdim=True)
    dz = STEP * (d + 8) * scale * (q.abs() @ k.abs().T) + STEP * 2 * zmax + 2.0 ** -21
    de = torch.expm1(dz.clamp(max=50.0))
    sums = m * STEP + 2.0 ** -20
    low = (p * de).sum(-1, keepdim=True) + sums
    num = (p * (de + BF * (1 + de) + sums)) @ v.abs() + 2.0 ** -100 * v.abs().sum(0)
    err = (num + low * out.abs()) * (1 + 2 * low.clamp(max=1.0))
    return (out, lse, err + BF * (out.abs() + err) + 1e-30,
            (low * (1 + low))[:, 0] + STEP * (zmax[:, 0] + 64) + STEP * lse.abs())


def weigh(q, k, lse, old, decay, scale, factor_bound=None):
    """One KV head: q [G, n, d] (the newest n tokens' queries), k [m, d] (codes times scales), lse
    [G, n], old [m] -> weights and their bound (the terms of attention(); q may be held to 2^-25 of
    its row's largest; lse is rounded with its factor log2(e); G n terms are summed in fp32)."""
    q, k, lse, old = q.to(F64), k.to(F64), lse.to(F64), old.to(F64)
    G, n, d = q.shape
    m = k.shape[0]
    t = torch.arange(m, device=k.device)
    sees = t <= (m - n) + torch.arange(n, device=k.device)[:, None]
    z = q @ k.T * scale
    gone = torch.isinf(lse)[..., None] | ~sees
    y = torch.where(torch.isinf(lse), 0.0, lse)[..., None]
    p = torch.where(gone, 0.0, (z - y).exp())
    dz = (STEP * (d + 8) * scale * (q.abs() @ k.abs().T) + 2.0 ** -25 * scale *
          q.abs().amax(-1, keepdim=True) * k.abs().sum(-1) + STEP * 2 * (z.abs() + y.abs()) + 2.0 ** -21)
    err = (p * (torch.expm1(dz.clamp(max=50.0)) + (G * n + 4) * STEP)).sum((0, 1))
    kept = decay * old if decay else torch.zeros_like(old)
    new = kept + p.sum((0, 1))
    return new, err + 3 * STEP * (kept.abs() + new.abs()) + 1e-36


def heaviest(w, length, budget, n_sink, n_recent):
    """One unit: weights (any floats) -> kept positions, by the definition."""
    n = min(length, budget)
    recent = min(n_recent, budget)
    must = set(range(max(length - recent, 0), length)) | set(range(min(n_sink, budget - recent, length)))
    rest = [t for t in range(length) if t not in must]
    rest.sort(key=lambda t: (-w[t] if w[t] == w[t] else math.inf, w[t] != w[t], t))
    return sorted(list(must) + rest[:n - len(must)])

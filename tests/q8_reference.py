"""Plain 64-bit forms of the rotating append and of the 8-bit paged cache, with the elementwise
error bounds of the kernels' roundings.

U = 2^-24 is half a step of fp32, B = 2^-8 half a step of bf16, both relative; half a step of e4m3
is 2^-4 relative and at least 2^-10 (codes).  The attention's bounds count, from the kernel's
formulas: scores as fp32 sums of d products; q as an e4m3 and an e5m2 term (half the least e5m2, 2^-17,
where the row's largest is at least 2^7: 2^-24 of it); exponents of fp32 arguments, an argument
made of a score, log2 of the value scale and the running maximum; a weight as f16 (2^-11) of which
three e5m2 terms are taken (half a step of each is 2^-3 of what is left: 2^-9; and half the least
e5m2, 2^-17, where the largest weight of a row is at least 2^9: 2^-26 of it; f16's own end is 2^-25
there, 2^-34), fp32 sums, and a bf16 output rounded once.
"""
import math

import torch

from tests.span_reference import B, NEG, U

E_MIN, E_MAX, TOP = -60, 60, 448.0
P_REL, P_ABS = 2.0 ** -11 + 2.0 ** -9, 2.0 ** -26 + 2.0 ** -34


def rotate(x, inv_freq, pos, interleaved):
    """x [tokens, heads, d] in 64 bits, rotated at integer positions; and the error bound of a
    kernel that turns in fp32 and rounds nothing else: two products and a sum, with a sine and a cosine
    good to 4 U and an angle cut at 2^-32 turns."""
    n = inv_freq.numel()
    a = pos.double()[:, None] * inv_freq.double()
    cos, sin = torch.cos(a)[:, None], torch.sin(a)[:, None]
    out, err = x.clone(), torch.zeros_like(x)
    for i in range(n):
        j, k = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
        u, v = x[..., j], x[..., k]
        c, s = cos[..., i], sin[..., i]
        out[..., j], out[..., k] = u * c - v * s, u * s + v * c
        err[..., j] = err[..., k] = 8 * U * (u.abs() + v.abs())
    return out, err


def scale_for(top):
    """Least power of two s, 2^-60 <= s <= 2^60, with top <= 448 s."""
    e = E_MIN
    while e < E_MAX and top > TOP * 2.0 ** e:
        e += 1
    return 2.0 ** e


def code(x):
    """e4m3 of x (nearest, ties to even, saturating) by its definition, as numbers."""
    x = x.double()
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -20))).clamp(min=-6)
    e = torch.where(torch.ldexp(torch.ones_like(x), e + 1) <= x.abs(), e + 1, e)  # log2 rounded down too far
    step = torch.ldexp(torch.ones_like(x), e - 3)
    return (torch.round(x / step) * step).clamp(-TOP, TOP)


def store(codes, scales, first, new):
    """One block: codes [block, d] and a scale, new values [n, d] (64 bits) at rows first...; returns
    the codes and the scale after it."""
    finite = new[torch.isfinite(new)].abs()
    need = scale_for(float(finite.max()) if finite.numel() else 0.0)
    codes = codes.clone()
    s = need if first == 0 else max(need, scales)
    if first and s > scales:
        codes[:first] = code(codes[:first] * (scales / s))
    codes[first:first + new.shape[0]] = code(new / s)
    return codes, s


def attend(q, kc, ks, vc, vs, see, scale):
    """q [Q, H, d], codes [n, Hkv, d] and their scales [n, Hkv] in 64 bits, see [Q, n] -> o, lse and
    their error bounds."""
    Q, H, d = q.shape
    n, hk = kc.shape[:2]
    r = H // hk
    o, lse = torch.zeros(Q, H, d, dtype=torch.float64), torch.full((Q, H), NEG, dtype=torch.float64)
    eo, el = torch.zeros_like(o), torch.zeros(Q, H, dtype=torch.float64)
    for h in range(H):
        kk, c, sv = kc[:, h // r] * ks[:, h // r, None], vc[:, h // r], vs[:, h // r]
        s = (q[:, h] @ kk.T * scale).masked_fill(~see, NEG)
        some = see.any(1)
        lse[:, h] = torch.logsumexp(s, 1) if n else NEG
        p = torch.where(see & some[:, None], torch.exp(s - torch.where(some, lse[:, h], 0.0)[:, None]), 0.0)
        w = p * sv
        o[:, h] = w @ c
        if not n:
            continue
        mag = ((q[:, h].abs() @ kk.abs().T) * scale).masked_fill(~see, 0.0).max(1).values
        q_cut = (2.0 ** -24 * q[:, h].abs().max(1).values[:, None] * kk.abs().sum(1) * scale).masked_fill(~see, 0.0)
        logs = torch.log(sv).abs().max()
        es = (d + 16) * U * mag + q_cut.max(1).values + 8 * U * (mag + logs)
        rel = 2 * es + 2.0 ** -19 + n * U
        eo[:, h] = ((P_REL + rel)[:, None] * (w @ c.abs()) + P_ABS * w.max(1).values[:, None] * (see.double() @ c.abs())
                    + B * o[:, h].abs() * (1 + rel[:, None] + P_REL))
        el[:, h] = rel + 4 * U * (lse[:, h].masked_fill(~some, 0.0).abs() + logs)
    return o, lse, eo, el

"""Plain 64-bit forms of the paged-cache and sink-window operators, one sequence at a time,
with the elementwise error bounds of the kernels' roundings.

U = 2^-24 is half a step of fp32, B = 2^-8 half a step of bf16 (both relative).  The bounds
count, from the kernels' formulas: scores as fp32 sums of d products (error d U times the sum
of |q k|), base-2 exponentials of fp32 arguments (an argument's absolute error is the result's
relative error; ex2.approx itself 2^-22), fp32 sums of n terms (n U relative to the sum of
magnitudes), P and dS rounded once to bf16 and a bf16 output rounded once.
"""
import math

import torch

U, B = 2.0 ** -24, 2.0 ** -8
NEG = float("-inf")


def visible(pos, n_keys, window, n_sink):
    """[queries, keys]: key j <= p, and j > p - window or j < n_sink when window > 0."""
    j = torch.arange(n_keys)[None, :]
    p = torch.as_tensor(pos)[:, None]
    see = j <= p
    return see & ((j > p - window) | (j < n_sink)) if window else see


def attend(q, k, v, see, scale):
    """q [Q, H, d], k, v [n, Hkv, d] (64 bits), see [Q, n] -> o, lse and their error bounds."""
    Q, H, d = q.shape
    n, hk = k.shape[:2]
    r = H // hk
    o, lse = torch.zeros(Q, H, d, dtype=torch.float64), torch.full((Q, H), NEG, dtype=torch.float64)
    eo, el = torch.zeros_like(o), torch.zeros(Q, H, dtype=torch.float64)
    for h in range(H):
        kk, vv = k[:, h // r], v[:, h // r]
        s = (q[:, h] @ kk.T * scale).masked_fill(~see, NEG)
        some = see.any(1)
        lse[:, h] = torch.logsumexp(s, 1) if n else NEG
        p = torch.where(see & some[:, None], torch.exp(s - torch.where(some, lse[:, h], 0.0)[:, None]), 0.0)
        o[:, h] = p @ vv
        # largest absolute error of a score (in the exponent), with the scale's own rounding
        mag = ((q[:, h].abs() @ kk.abs().T) * scale).masked_fill(~see, 0.0)
        es = (d + 8) * U * (mag.max(1).values if n else torch.zeros(Q))
        rel = 2 * es + 2.0 ** -20 + n * U  # p's numerator and the sum it is divided by
        eo[:, h] = (B + rel)[:, None] * (p @ vv.abs()) + B * o[:, h].abs() * (1 + rel[:, None])
        el[:, h] = rel + 4 * U * lse[:, h].masked_fill(~some, 0.0).abs()
    return o, lse, eo, el


def key_weights(q, k, see, lse, scale):
    """Sum over queries and group heads of exp(s - lse): [n, Hkv] and its error bound."""
    Q, H, d = q.shape
    n, hk = k.shape[:2]
    r = H // hk
    w, e = torch.zeros(n, hk, dtype=torch.float64), torch.zeros(n, hk, dtype=torch.float64)
    for h in range(H):
        kk = k[:, h // r]
        some = see & torch.isfinite(lse[:, h])[:, None]
        s = q[:, h] @ kk.T * scale
        p = torch.where(some, torch.exp(s - torch.where(torch.isfinite(lse[:, h]), lse[:, h], 0.0)[:, None]), 0.0)
        mag = (q[:, h].abs() @ kk.abs().T) * scale
        arg = (d + 8) * U * mag + 4 * U * torch.where(torch.isfinite(lse[:, h]), lse[:, h], 0.0).abs()[:, None]
        w[:, h // r] += p.sum(0)
        e[:, h // r] += (p * (arg + 2.0 ** -20 + Q * r * U)).sum(0)
    return w, e


def gradients(q, k, v, do, o, lse, see, scale, eo=None):
    """dq, dk, dv with D = sum_j p_j dp_j, and their error bounds.  The kernel takes D = dO.o for
    dq where a row's keys are many; eo bounds its stored o's distance from the exact one."""
    Q, H, d = q.shape
    n, hk = k.shape[:2]
    r = H // hk
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    eq, ek, ev = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    for h in range(H):
        g = h // r
        kk, vv, qq, dd = k[:, g], v[:, g], q[:, h], do[:, h]
        p = torch.where(see, torch.exp(qq @ kk.T * scale - lse[:, h][:, None]), 0.0)
        dp = dd @ vv.T
        dsum = (p * dp).sum(1, keepdim=True)
        ds = p * (dp - dsum)
        dq[:, h] = scale * ds @ kk
        dk[:, g] += scale * ds.T @ qq
        dv[:, g] += p.T @ dd
        arg = (d + 8) * U * (qq.abs() @ kk.abs().T) * scale + 4 * U * lse[:, h].abs()[:, None] + 2.0 ** -20
        # |dp - D| is known to within d U of the magnitudes that make it up, D to within the
        # errors of the p that it sums
        mag = dd.abs() @ vv.abs().T
        ed = ((arg + n * U) * p * mag).sum(1, keepdim=True) + (dd * o[:, h]).abs().sum(1, keepdim=True) * (d + n) * U
        eds = ds.abs() * (B + arg) + p * ((d + 4) * U * mag + ed)
        far = 0.0 if eo is None else p * (dd.abs() * eo[:, h]).sum(1, keepdim=True)
        eq[:, h] = scale * (eds + far + n * U * ds.abs()) @ kk.abs()
        ek[:, g] += scale * (eds + Q * r * U * ds.abs()).T @ qq.abs()
        ev[:, g] += (p * (B + arg + Q * r * U)).T @ dd.abs()
    return (dq, dk, dv), tuple(e + B * x.abs() * (1 + 2 * B) for e, x in zip((eq, ek, ev), (dq, dk, dv)))


def choose(weights, L, budget, n_sink, n_recent):
    """Kept positions of one kv-head by definition: sinks, recents, then the heaviest, equal
    weights to the lower position, NaN lowest.  weights: Python floats of the L positions."""
    if L <= budget:
        return list(range(L))
    forced = [i for i in range(L) if i < n_sink or i >= L - n_recent]
    rest = [i for i in range(L) if n_sink <= i < L - n_recent]
    rest.sort(key=lambda i: (0, 0.0, i) if not math.isnan(weights[i]) and weights[i] == math.inf else
              (2, 0.0, i) if math.isnan(weights[i]) else (1, -weights[i], i))
    return sorted(forced + rest[:budget - len(forced)])


def within(got, ref, bound, what):
    """got (any type) within the bound of ref, infinities and zeros in the same places."""
    got = got.detach().cpu().double()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    inf = torch.isinf(ref)
    assert torch.equal(got[inf], ref[inf]), f"{what}: infinities"
    assert torch.isfinite(got[~inf]).all(), f"{what}: {int((~torch.isfinite(got[~inf])).sum())} values are not finite"
    err = (got - ref).abs().masked_fill(inf, 0.0)
    over = err - bound.masked_fill(inf, 0.0)
    if over.numel() and over.max() > 0:
        at = tuple(int(x) for x in torch.unravel_index(over.argmax(), over.shape))
        raise AssertionError(f"{what}: {int((over > 0).sum())} of {over.numel()} out of bounds; worst at {at}: got "
                             f"{got[at]!r}, exact {ref[at]!r}, bound {float(bound[at]):.3g}")

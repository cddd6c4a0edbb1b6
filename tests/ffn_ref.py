"""Plain 64-bit forms of token quantisation, the scaled W8A8 matmul and the gated feed-forward
block, each with a bound on how far a right kernel may be from it.

Roundings counted by the bounds (u: half a step of the 16-bit result type, eps / 2):
  - every fp32 operation is off by at most 2^-24 of its result (2^-23 for one addition inside a
    tensor-core sum, which may cut instead of rounding): a sum of n products by at most
    (n + 2) 2^-23 sum |x w|;
  - the activations and their derivatives by 2^-18 relative (the fast exponential is off by
    about |x| 2^-23, |x| <= 16 where the result matters) plus 2^-22 absolute for a derivative;
  - a result rounded to 16 bits by u |result|, or half the smallest subnormal.
"""
import math

import numpy as np
import torch

TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def sum_slack(n):
    return (n + 2) * 2.0 ** -23


def quant(x):
    """Codes and scales by the definition's binary32 steps, in numpy; x: [M, K] float32 values."""
    x = np.asarray(x, dtype=np.float32)
    with np.errstate(all="ignore"):
        amax = np.abs(x).max(axis=1)
        bad = ~np.isfinite(x).all(axis=1)
        up = np.where(amax < np.float32(2.0 ** -60), np.float32(2.0 ** 64), np.float32(1))
        scale = np.where(amax == 0, np.float32(1), amax / np.float32(127))
        inv = np.where(amax == 0, np.float32(0), np.float32(127) / (amax * up))
        q = np.rint((x * up[:, None]) * inv[:, None])
    q[bad] = 0
    scale[bad] = np.nan
    return q.astype(np.int8), scale.astype(np.float32)


def _tanh_arg(g):
    """2 sqrt(2/pi) (g + 0.044715 g^3): 0.5 (1 + tanh(x / 2)) is the logistic function of it."""
    return 2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)


def value(g, act):
    """In forms without cancellation far below 0 (1 + erf and 1 + tanh lose everything there)."""
    if act == "silu":
        return g * torch.sigmoid(g)
    if act == "gelu":
        return 0.5 * g * torch.special.erfc(-g / math.sqrt(2))
    return g * torch.sigmoid(_tanh_arg(g))


def slope(g, act):
    if act == "silu":
        return torch.sigmoid(g) * (1 + g * torch.sigmoid(-g))
    if act == "gelu":
        return 0.5 * torch.special.erfc(-g / math.sqrt(2)) + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    x = _tanh_arg(g)
    return torch.sigmoid(x) * (1 + g * torch.sigmoid(-x) * 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * g * g))


def rounded(ref, err, dtype):
    """The bound after the rounding to `dtype` of a value within err of ref."""
    return err + half_step(dtype) * (ref.abs() + err) + TINY[dtype]


def scaled(A, W, sa, sw, bias, dtype):
    p = (A.double() @ W.double().T) * sa.double()[:, None] * sw.double()
    ref = p if bias is None else p + bias.double()
    err = 3.1 * 2.0 ** -24 * p.abs() + (0 if bias is None else 1.1 * 2.0 ** -24 * ref.abs())
    return ref, rounded(ref, err, dtype)


def _gate(g, eg, u, eu, act, dtype):
    """H and its bound from pre-activations with errors eg, eu."""
    v = value(g, act)
    ref = v * u
    ev = 1.13 * eg + 2.0 ** -18 * (v.abs() + 1.13 * eg)      # |act'| <= 1.13
    err = ev * (u.abs() + eu) + v.abs() * eu + 2.0 ** -23 * ref.abs()
    return ref, rounded(ref, err, dtype)


def gated8(A, Wg, Wu, sa, sg, su, act, dtype):
    a = A.double()
    g = (a @ Wg.double().T) * sa.double()[:, None] * sg.double()
    u = (a @ Wu.double().T) * sa.double()[:, None] * su.double()
    slack = 3.1 * 2.0 ** -24
    return _gate(g, slack * g.abs(), u, slack * u.abs(), act, dtype)


def gated(X, Wg, Wu, act):
    """{"H", "G", "U"}: (reference, bound)."""
    x, wg, wu = X.double(), Wg.double(), Wu.double()
    k = sum_slack(X.shape[1])
    g, u = x @ wg.T, x @ wu.T
    eg, eu = k * (x.abs() @ wg.abs().T), k * (x.abs() @ wu.abs().T)
    return {"H": _gate(g, eg, u, eu, act, X.dtype), "G": (g, rounded(g, eg, X.dtype)),
            "U": (u, rounded(u, eu, X.dtype))}


def backward(dH, X, Wg, Wu, G, U, act):
    """{"dX", "dWg", "dWu"}: (reference, bound). dG and dU are rounded to the 16-bit type."""
    dt, M, F = X.dtype, X.shape[0], Wg.shape[0]
    dh, x, wg, wu, g, u = (t.double() for t in (dH, X, Wg, Wu, G, U))
    s, v = slope(g, act), value(g, act)
    dg, du = dh * u * s, dh * v
    edg = rounded(dg, (dh * u).abs() * (2.0 ** -18 * s.abs() + 2.0 ** -22) + 2.0 ** -22 * dg.abs(), dt)
    edu = rounded(du, 2.0 ** -17 * du.abs(), dt)

    def product(a, ea, b, n):
        return a @ b, ea @ b.abs() + sum_slack(n) * ((a.abs() + ea) @ b.abs())

    p, ep = product(dg, edg, wg, 2 * F)
    q, eq = product(du, edu, wu, 2 * F)
    out = {"dX": (p + q, rounded(p + q, ep + eq, dt))}
    for name, d, e in (("dWg", dg, edg), ("dWu", du, edu)):
        r, er = product(d.T, e.T, x, M)
        out[name] = (r, rounded(r, er, dt))
    return out


def check(got, ref_bound, what=""):
    """Every element within its bound, non-finite ones where the reference has them."""
    ref, bound = ref_bound
    got = got.double()
    off = (got - ref).abs()
    bad = ~(off <= bound) & torch.isfinite(ref)
    assert not bad.any(), (what, int(bad.sum()), float((off / bound)[bad].max()), bad.nonzero()[:4].tolist())
    assert torch.equal(torch.isfinite(got), torch.isfinite(ref)), what

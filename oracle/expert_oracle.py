"""CPU oracle of the experts' own products: linear layers of rows sorted by
expert with their activation, the gradients, and 4-bit weights.

TEST INFRASTRUCTURE ONLY, numpy in 64 bits, written from the definitions.
Functions that return computed numbers return beside each a bound on what an
evaluation in 32 bits may be off by, ``err``, made of
  * a sum of n products: 2 (n + 8) u of the sum of their magnitudes, in any
    order, the accumulator's roundings taken as whole steps;
  * an activation evaluated in 32 bits at g: (|g|^3 + 4 g^2 + 8 |g| + 32) u of
    its magnitude (the arguments of exp and erfc are at most cubic in g, their
    roundings are multiplied by the argument);
  * what it was evaluated at being off itself, to first order by its
    derivative, to second by 2 (1 + |up|) (no second derivative of these
    functions is larger), or, at a clamp, by the jump of the derivative;
with u = 2^-24.
"""
import math

import numpy as np

U = 2.0 ** -24
GATED = ("silu", "gelu", "gelu_tanh", "swigluoai", "swiglustep")
SINGLE = ("silu_no_mul", "gelu_no_mul", "gelu_tanh_no_mul", "relu2_no_mul")
_erfc = np.vectorize(math.erfc, otypes=[float])


def sum_rel(n):
    return 2.0 * (n + 8) * U


def act_rel(g):
    a = np.abs(g)
    return (a ** 3 + 4.0 * a ** 2 + 8.0 * a + 32.0) * U


def _sigmoid(x):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-x))


def curve(kind, x):
    """(f, f') of an activation without its clamps."""
    kind = kind.replace("_no_mul", "")
    if kind in ("silu", "swiglustep", "swigluoai"):
        a = 1.702 if kind == "swigluoai" else 1.0
        s = _sigmoid(a * x)
        return x * s, s + a * x * s * _sigmoid(-a * x)
    if kind == "gelu":
        phi = 0.5 * _erfc(-x / math.sqrt(2.0)) if np.size(x) else np.zeros_like(x)
        return x * phi, phi + x * np.exp(-0.5 * x * x) / math.sqrt(2.0 * math.pi)
    if kind == "gelu_tanh":
        c = 2.0 * math.sqrt(2.0 / math.pi)
        y = c * (x + 0.044715 * x ** 3)
        s = _sigmoid(y)
        return x * s, s + x * s * _sigmoid(-y) * c * (1.0 + 3.0 * 0.044715 * x * x)
    assert kind == "relu2", kind
    r = np.maximum(x, 0.0)
    return r * r, 2.0 * r


def default_limit(kind, limit):
    return limit or 7.0 if kind in ("swigluoai", "swiglustep") else limit


def activate(kind, pre, limit=0.0):
    """(F, dF/dgate, dF/dup) with pre [R, wide]; dF/dup is None without an up half."""
    if kind == "none":
        return pre, np.ones_like(pre), None
    if kind not in GATED:
        f, df = curve(kind, pre)
        return f, df, None
    n = pre.shape[1] // 2
    g, u = pre[:, :n], pre[:, n:]
    L = default_limit(kind, limit)
    live_g = live_u = np.ones_like(g)
    if L > 0.0:
        live_u = (np.abs(u) <= L).astype(float)
        u = np.clip(u, -L, L)
        if kind != "swiglustep":
            live_g = (g <= L).astype(float)
            g = np.minimum(g, L)
    f, df = curve(kind, g)
    if kind == "swiglustep":
        live_g = (f <= L).astype(float)
        f = np.minimum(f, L)
    if kind == "swigluoai":
        u = u + 1.0
    return f * u, df * live_g * u, f * live_u


def activated(kind, pre, err, limit=0.0):
    """(values, err) of F at pre, which is off by at most err."""
    f, dg, du = activate(kind, pre, limit)
    if kind == "none":
        return f, err
    if du is None:
        return f, err * (np.abs(dg) + 4.0 * err) + act_rel(pre) * (np.abs(f) + np.abs(pre))
    n = f.shape[1]
    eg, eu, up = err[:, :n], err[:, n:], 2.0 * (1.0 + np.abs(pre[:, n:]))
    return f, eg * (np.abs(dg) + eg * up) + eu * (np.abs(du) + eu) \
        + act_rel(pre[:, :n]) * (np.abs(f) + np.abs(du))


def ranges(offsets, R, E):
    if offsets is None:
        return [(0, 0, R)]
    return [(e, int(offsets[e]), int(offsets[e + 1])) for e in range(E)]


def linear(x, w, offsets, kind="none", limit=0.0):
    """{"out": (values, err), "pre_act": ...} with NaN in rows of no expert."""
    R, (E, wide, K) = x.shape[0], w.shape
    pre, mag = np.full((R, wide), np.nan), np.full((R, wide), np.nan)
    for e, a, b in ranges(offsets, R, E):
        pre[a:b] = x[a:b] @ w[e].T
        mag[a:b] = np.abs(x[a:b]) @ np.abs(w[e]).T
    err = sum_rel(K) * mag
    return {"out": activated(kind, pre, err, limit), "pre_act": (pre, err)}


def linear_grad(x, w, offsets, grad_out, pre=None, kind="none", limit=0.0, step=0.0):
    """{"grad_x": (values, err), "grad_weight": ...}; step: the half step that
    d is rounded by, relative (0 without an activation)."""
    R, (E, wide, K) = x.shape[0], w.shape
    if kind == "none":
        d, derr = grad_out, np.zeros_like(grad_out)
    else:
        _, dg, du = activate(kind, pre, limit)
        g = pre if du is None else pre[:, :grad_out.shape[1]]
        d = grad_out * dg
        mag = np.abs(grad_out) * (np.abs(dg) + (1.0 if du is None else
                                                1.0 + np.abs(pre[:, grad_out.shape[1]:])))
        derr = act_rel(g) * mag
        if du is not None:
            d = np.concatenate([d, grad_out * du], axis=1)
            derr = np.concatenate([derr, act_rel(g) * np.abs(grad_out * du)], axis=1)
        derr = derr + step * np.abs(d) * 1.01
    gx, gxe = np.full((R, K), np.nan), np.full((R, K), np.nan)
    gw, gwe = np.zeros(w.shape), np.zeros(w.shape)
    for e, a, b in ranges(offsets, R, E):
        aw, ax, ad = np.abs(w[e]), np.abs(x[a:b]), np.abs(d[a:b])
        gx[a:b] = d[a:b] @ w[e]
        gxe[a:b] = sum_rel(wide) * (ad @ aw) + derr[a:b] @ aw
        gw[e] = d[a:b].T @ x[a:b]
        gwe[e] = sum_rel(b - a) * (ad.T @ ax) + derr[a:b].T @ ax
    return {"grad_x": (gx, gxe), "grad_weight": (gw, gwe)}


E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6])


def dequant_w4(codes, scales, form, zeros=None):
    """(weights [E, wide, K], magnitudes that a product with x may pass through):
    int4 codes may be carried as 128 + q of the group's own scale."""
    E, wide, half = codes.shape
    q = np.empty((E, wide, 2 * half), dtype=np.int64)
    q[..., 0::2], q[..., 1::2] = codes & 15, codes >> 4
    group = 2 * half // scales.shape[2]
    if form == "mxfp4":
        s = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(float) - 127.0))
        v = E2M1[q] * np.repeat(s, group, axis=2)
        return v, np.abs(v)
    z = np.full(scales.shape, 8) if zeros is None else zeros.astype(np.int64)
    s = np.repeat(scales, group, axis=2)
    z = np.repeat(z, group, axis=2)
    return s * (q - z), np.abs(s) * (144.0 + np.abs(z))


def linear_w4(x, w, mag, offsets, kind="none", limit=0.0):
    """(values, err) of out; w, mag: from dequant_w4."""
    R, K = x.shape
    wide = w.shape[1]
    pre, err = np.full((R, wide), np.nan), np.full((R, wide), np.nan)
    for e, a, b in ranges(offsets, R, w.shape[0]):
        pre[a:b] = x[a:b] @ w[e].T
        err[a:b] = sum_rel(K) * (np.abs(x[a:b]) @ mag[e].T)
    return activated(kind, pre, err, limit)

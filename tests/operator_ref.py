"""Plain 64-bit implementations (numpy) of the 16-bit operators around the int3
layer -- dense product, expert-order moves, router gradient -- and the error
bounds their kernels are held to.

Bounds.  u(t) = half a step of type t relative to the value (bf16 2^-8, fp16
2^-11, fp32 2^-24); an fp16 result below 2^-14 is off by at most 2^-25.
- a sum of n fp32 terms in any order: n * 2^-24 * sum |terms|;
- a product over C on the tensor cores: the 16 products of an MMA step are
  exact, are aligned and added with truncation, and join an fp32 accumulator,
  also by truncation: at most 2^-22 of the terms' magnitude per step, C / 16
  steps, plus the joins of up to 16 partial accumulators;
- activations: the fp32 formulas are within 2^-20 (|z| + 1) of the function
  (a few roundings of numbers no larger than |z| + 1, expf and erff within 2^-22),
  and no activation here has a slope above 1.13.
"""
import math

import numpy as np

U = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}
TINY = {"bf16": 2.0 ** -133, "f16": 2.0 ** -25, "f32": 2.0 ** -149}
SLOPE = 1.13
_erf = np.vectorize(math.erf, otypes=[np.float64])


def _sigmoid(z):
    e = np.exp(-np.abs(z))
    return np.where(z >= 0, 1.0, e) / (1.0 + e)


def act(name, z):
    if name == "relu":
        return np.maximum(z, 0.0)
    if name == "silu":
        return z * _sigmoid(z)
    if name == "gelu":
        return 0.5 * z * (1.0 + _erf(z / math.sqrt(2.0)))
    if name == "gelu_tanh":
        return 0.5 * z * (1.0 + np.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3)))
    return z


def dact(name, z):
    if name == "relu":
        return (z > 0).astype(np.float64)
    if name == "silu":
        g = _sigmoid(z)
        return g * (1.0 + z * (1.0 - g))
    if name == "gelu":
        return 0.5 * (1.0 + _erf(z / math.sqrt(2.0))) + z * np.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if name == "gelu_tanh":
        c = math.sqrt(2.0 / math.pi)
        t = np.tanh(c * (z + 0.044715 * z ** 3))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * z * z)
    return np.ones_like(z)


def _rounded(v, err, dt):
    """Bound of a value with error err, rounded to dt."""
    return err + U[dt] * (np.abs(v) + err) + TINY[dt]


def _mma(C):
    return (C / 16 + 16) * 2.0 ** -22


def linear(x, W, bias, act_name, residual, dt, out_dt):
    """(y, bound of y, z, bound of z)."""
    z = x @ W.T
    mag = np.abs(x) @ np.abs(W).T
    if bias is not None:
        z = z + bias
        mag = mag + np.abs(bias)
    ez = _mma(x.shape[1]) * mag + 2.0 ** -24 * np.abs(z)
    y = act(act_name, z)
    ey = ez if act_name == "none" else SLOPE * ez + 2.0 ** -20 * (np.abs(z) + 1.0)
    if residual is not None:
        y = y + residual
        ey = ey + 2.0 ** -24 * np.abs(y)
    return y, _rounded(y, ey, out_dt), z, _rounded(z, ez, dt)


def linear_backward(dy, x, W, act_name, z, dt, exact_dz):
    """{name: (gradient, bound)}; exact_dz: dy enters the products unrounded."""
    dz = dy if act_name == "none" else dy * dact(act_name, z)
    e32 = np.zeros_like(dz) if act_name == "none" else 2.0 ** -20 * np.abs(dy) * (np.abs(z) + 1.0)
    edz = e32 if exact_dz else _rounded(dz, e32, dt)
    adz = np.abs(dz) + edz
    out = {}
    for name, a, b, ea, aa in (("dx", dz, W, edz, adz), ("dW", dz.T, x, edz.T, adz.T)):
        g = a @ b
        out[name] = (g, _rounded(g, ea @ np.abs(b) + _mma(a.shape[1]) * (aa @ np.abs(b)), dt))
    db = dz.sum(0)
    out["db"] = (db, _rounded(db, e32.sum(0) + dz.shape[0] * 2.0 ** -24 * np.abs(dz).sum(0), dt))
    return out


def dispatch(x, inv, w, out_dt, xs0):
    """(xs, bound): rows that no slot points to keep xs0."""
    T, k = inv.shape
    xs, b = xs0.copy(), np.zeros_like(xs0)
    for t in range(T):
        for j in range(k):
            if inv[t, j] >= 0:
                v = x[t] * (1.0 if w is None else w[t, j])
                xs[inv[t, j]] = v
                b[inv[t, j]] = _rounded(v, 0.0 if w is None else 2.0 ** -24 * np.abs(v), out_dt)
    return xs, b


def combine(ys, inv, w, residual, out_dt):
    T, k = inv.shape
    y = np.zeros((T, ys.shape[1])) if residual is None else residual.copy()
    mag = np.abs(y)
    for t in range(T):
        for j in range(k):
            if inv[t, j] >= 0:
                v = ys[inv[t, j]] * (1.0 if w is None else w[t, j])
                y[t] += v
                mag[t] += np.abs(v)
    return y, _rounded(y, (k + 2) * 2.0 ** -24 * mag, out_dt)


def slot_dots(tok, rows, inv):
    """(dw, bound): dw[t, j] = <tok[t], rows[inv[t, j]]>, 0 for a dropped slot."""
    T, k = inv.shape
    d, b = np.zeros((T, k)), np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            if inv[t, j] >= 0:
                d[t, j] = tok[t] @ rows[inv[t, j]]
                b[t, j] = (tok.shape[1] + 1) * 2.0 ** -24 * (np.abs(tok[t]) @ np.abs(rows[inv[t, j]]))
    return d, b


def route_weights(logits, ids, renorm):
    e = np.exp(logits - logits.max(1, keepdims=True))
    pk = np.take_along_axis(e, ids, 1)
    return pk / (pk.sum(1, keepdims=True) if renorm else e.sum(1, keepdims=True))


def route_backward(logits, ids, w, dw, E, renorm, out_dt):
    """(dl, bound).  fp32: w dw, its sum over k picks, the softmax (expf within
    2^-22 of an exponent up to 2^-18 off for |l - max| <= 64, E terms in its
    denominator) and two products."""
    T, k = ids.shape
    g = w * dw
    s = g.sum(1, keepdims=True)
    sm = np.abs(g).sum(1, keepdims=True)
    if renorm:
        q = np.zeros((T, E))
        np.put_along_axis(q, ids, w, 1)
    else:
        e = np.exp(logits - logits.max(1, keepdims=True))
        q = e / e.sum(1, keepdims=True)
    hot = np.zeros((T, E))
    np.put_along_axis(hot, ids, g, 1)
    dl = hot - q * s
    err = (k + 4) * 2.0 ** -24 * (np.abs(hot) + q * sm) + (2.0 ** -18 + E * 2.0 ** -24) * q * np.abs(s)
    return dl, _rounded(dl, err, out_dt)

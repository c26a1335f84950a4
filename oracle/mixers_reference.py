"""Float64 CPU oracle of the token-by-token mixers: causal convolution, selective scan, and
sliding-window attention with sinks over a sequence or a rolling cache.

TEST INFRASTRUCTURE, shared with nothing in the CUDA library.  Each function follows its
definition token by token and also returns what a rounding analysis of the result needs:
the sums of absolute values behind every output.
"""

import math

import numpy as np


def causal_conv(x, weight, bias=None, state=None, silu=True):
    """x [T, D], weight [D, W], state [W - 1, D] -> out [T, D], new state, and the absolute sums."""
    x, w = np.asarray(x, np.float64), np.asarray(weight, np.float64)
    T, D = x.shape
    W = w.shape[1]
    st = np.zeros((W - 1, D)) if state is None else np.asarray(state, np.float64)
    b = np.zeros(D) if bias is None else np.asarray(bias, np.float64)
    rows = np.concatenate([st, x])
    out, mag = np.zeros((T, D)), np.zeros((T, D))
    for t in range(T):
        terms = rows[t:t + W] * w.T
        y = b + terms.sum(0)
        mag[t] = np.abs(b) + np.abs(terms).sum(0)
        out[t] = y / (1.0 + np.exp(-y)) if silu else y
    return out, rows[T:], mag


def softplus(x):
    return np.logaddexp(0.0, x)


def selective_scan(x, dt, A, Bm, Cm, skip=None, z=None, dt_bias=None, state=None, dt_softplus=True,
                   arg_eps=2.0 ** -20, exp_eps=2.0 ** -22, add_eps=2.0 ** -23):
    """One sequence: x, dt, z [T, D], Bm, Cm [T, N], A and state [D, N].

    Returns y, the last state, and first-order bounds on what float32 arithmetic may add to each:
    exp(delta A) off by |delta A| arg_eps + exp_eps of its value, the two roundings of the update by
    add_eps, carried along the recurrence.  In units of 2^-24: an approximate exponential and a quotient
    are off by 3 and 4, so softplus through u = e^-|x|, u / (2 + u) and its odd series is off by
    3 + 1 + 4 for the quotient and 2 for the last products, 10 together, and delta A or delta x by 2
    products more: 12, below 16 = arg_eps.
    """
    x, dt, A, Bm, Cm = (np.asarray(v, np.float64) for v in (x, dt, A, Bm, Cm))
    T, D = x.shape
    N = A.shape[1]
    h = np.zeros((D, N)) if state is None else np.asarray(state, np.float64).copy()
    sk = np.zeros(D) if skip is None else np.asarray(skip, np.float64)
    bias = np.zeros(D) if dt_bias is None else np.asarray(dt_bias, np.float64)
    err = np.zeros_like(h)
    y, yerr = np.zeros((T, D)), np.zeros((T, D))
    for t in range(T):
        delta = dt[t] + bias
        if dt_softplus:
            delta = softplus(delta)
        arg = delta[:, None] * A
        a = np.exp(arg)
        new = (delta * x[t])[:, None] * Bm[t][None]
        err = a * err + np.abs(a * h) * (np.abs(arg) * arg_eps + exp_eps) + \
            np.abs(new) * arg_eps + (np.abs(a * h) + np.abs(new)) * add_eps
        h = a * h + new
        v = h @ Cm[t] + sk * x[t]
        ve = err @ np.abs(Cm[t]) + (np.abs(h) @ np.abs(Cm[t]) + np.abs(sk * x[t])) * (N + 2) * add_eps
        if z is not None:
            zt = np.asarray(z[t], np.float64)
            g = zt / (1.0 + np.exp(-zt))
            ve = np.abs(g) * ve + np.abs(v * g) * 2.0 ** -20
            v = v * g
        y[t], yerr[t] = v, ve
    return y, h, yerr, err


def window_keys(t, window, sinks):
    """The tokens that token t sees, in order."""
    lo = max(0, t - window + 1)
    return np.concatenate([np.arange(min(sinks, lo)), np.arange(lo, t + 1)])


def _attend(q, k, v, scale):
    s = (k @ q) * scale
    p = np.exp(s - s.max())
    p /= p.sum()
    return p @ v, p @ np.abs(v)


def window_attention(q, k, v, window, sinks=0, scale=None):
    """One sequence: q [Tq, Hq, d_k] (the last Tq tokens), k, v [Tk, Hkv, d] -> out and sum p |v|."""
    q, k, v = (np.asarray(a, np.float64) for a in (q, k, v))
    Tq, Hq, dk = q.shape
    Tk, Hkv, dv = v.shape
    scale = 1.0 / math.sqrt(dk) if scale is None else scale
    out, mag = np.zeros((Tq, Hq, dv)), np.zeros((Tq, Hq, dv))
    for i in range(Tq):
        at = window_keys(Tk - Tq + i, window, sinks)
        for h in range(Hq):
            g = h // (Hq // Hkv)
            out[i, h], mag[i, h] = _attend(q[i, h], k[at, g], v[at, g], scale)
    return out, mag


def slot(p, window, sinks):
    return p if p < sinks else sinks + (p - sinks) % window

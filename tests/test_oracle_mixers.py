"""Pins of the token-by-token mixers' oracle: hand-derived values, other formulas of the same
quantity, composition of a sequence from its pieces, and the rolling cache against a simulation."""

import math

import numpy as np
import pytest

from oracle import mixers_reference as M


def rng(seed):
    return np.random.default_rng(seed)


@pytest.mark.parametrize("W", [2, 3, 4])
def test_conv_is_a_correlation_and_composes(W):
    r = rng(W)
    x, w, b, st = r.normal(size=(11, 5)), r.normal(size=(5, W)), r.normal(size=5), r.normal(size=(W - 1, 5))
    y, new, _ = M.causal_conv(x, w, b, st, silu=False)
    rows = np.concatenate([st, x])
    for c in range(5):
        assert np.allclose(y[:, c], np.correlate(rows[:, c], w[c], "valid") + b[c], atol=1e-13)
    y1, s1, _ = M.causal_conv(x[:4], w, b, st)
    y2, s2, _ = M.causal_conv(x[4:], w, b, s1)
    assert np.allclose(np.concatenate([y1, y2]), M.causal_conv(x, w, b, st)[0], atol=1e-14)
    assert np.array_equal(s2, new)


def test_conv_silu_by_hand():
    y, new, _ = M.causal_conv([[1.0], [2.0]], [[0.5, 1.0]], [1.0], silu=True)
    assert np.allclose(y[:, 0], [2.0 / (1 + math.exp(-2.0)), 3.5 / (1 + math.exp(-3.5))])
    assert new.tolist() == [[2.0]]


def test_scan_by_hand_and_in_closed_form():
    # one state, A = -1, delta = ln 2 (no softplus): h halves each token and gains ln 2 * x * B
    L = math.log(2.0)
    y, h, _, _ = M.selective_scan([[1.0], [3.0]], [[L], [L]], [[-1.0]], [[2.0], [1.0]], [[1.0], [5.0]], skip=[10.0],
                                  state=[[4.0]], dt_softplus=False)
    h1 = 2.0 + 2 * L
    h2 = h1 / 2 + 3 * L
    assert np.allclose(y[:, 0], [h1 + 10, 5 * h2 + 30]) and np.allclose(h, [[h2]])
    # softplus(0) = ln 2, and a constant input's geometric series
    y, h, _, _ = M.selective_scan(np.ones((30, 1)), np.zeros((30, 1)), [[-1.0]], np.ones((30, 1)), np.ones((30, 1)))
    assert np.isclose(h[0, 0], L * (1 - 0.5 ** 30) / 0.5)


def test_scan_composes_and_is_linear_in_the_state_and_input():
    r = rng(5)
    T, D, N = 9, 3, 8
    x, dt, z = (r.normal(size=(T, D)) for _ in range(3))
    A, B, C = -np.exp(r.normal(size=(D, N))), r.normal(size=(T, N)), r.normal(size=(T, N))
    h0, sk, bias = r.normal(size=(D, N)), r.normal(size=D), r.normal(size=D)
    full = M.selective_scan(x, dt, A, B, C, sk, z, bias, h0)
    p1 = M.selective_scan(x[:4], dt[:4], A, B[:4], C[:4], sk, z[:4], bias, h0)
    p2 = M.selective_scan(x[4:], dt[4:], A, B[4:], C[4:], sk, z[4:], bias, p1[1])
    assert np.allclose(np.concatenate([p1[0], p2[0]]), full[0]) and np.allclose(p2[1], full[1])
    free = M.selective_scan(0 * x, dt, A, B, C, sk, z, bias, h0)
    forced = M.selective_scan(x, dt, A, B, C, sk, z, bias)
    assert np.allclose(free[0] + forced[0], full[0]) and np.allclose(free[1] + forced[1], full[1])


def test_window_attention_limits():
    r = rng(3)
    T, H, d = 12, 4, 16
    q, k, v = r.normal(size=(T, H, d)), r.normal(size=(T, 2, d)), r.normal(size=(T, 2, d))
    # a window of one token without sinks returns that token's value
    out, _ = M.window_attention(q, k, v, 1)
    assert np.allclose(out, v[:, [0, 0, 1, 1]])
    # q = 0 averages what is seen: window 3 plus 2 sinks
    out, _ = M.window_attention(0 * q, k, v, 3, 2)
    assert np.allclose(out[7, 0], v[[0, 1, 5, 6, 7], 0].mean(0)) and np.allclose(out[1, 3], v[:2, 1].mean(0))
    # a window as long as the sequence is causal attention, with or without sinks
    s = np.einsum("tgd,sd->gts", q[:, :2], k[:, 0]) / 4.0
    s[:, np.triu_indices(T, 1)[0], np.triu_indices(T, 1)[1]] = -np.inf
    p = np.exp(s - s.max(-1, keepdims=True))
    full = np.einsum("gts,sd->tgd", p / p.sum(-1, keepdims=True), v[:, 0])
    assert np.allclose(M.window_attention(q, k, v, T)[0][:, :2], full)
    assert np.allclose(M.window_attention(q, k, v, 5, T)[0][:, :2], full)
    # the last queries of a sequence are the whole sequence's
    assert np.allclose(M.window_attention(q[8:], k, v, 4, 1)[0], M.window_attention(q, k, v, 4, 1)[0][8:])


@pytest.mark.parametrize("window,sinks", [(1, 0), (3, 0), (4, 2), (5, 1), (1, 3)])
def test_rolling_slots_hold_exactly_what_a_position_sees(window, sinks):
    cache = {}
    for p in range(40):
        cache[M.slot(p, window, sinks)] = p
        seen = min(window + sinks, p + 1)
        assert sorted(cache) == list(range(seen))
        assert sorted(cache.values()) == M.window_keys(p, window, sinks).tolist()

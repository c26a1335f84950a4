"""The token-by-token mixers on values at the ends of the number range: masks by the type's lowest
value or an infinity, growing and infinite states, NaN and infinities in tokens that a query does not
see, sums that could overflow, idle sessions; and that a call repeats itself bit for bit.

Compared with the float64 oracle under the tolerances of test_gpu_mixers.py; where the oracle's value
is not finite, the kernel's has to be the same infinity or NaN.
"""

import numpy as np
import pytest
import torch

import hybrid_linear_attention_frame_b200 as G
from oracle import mixers_reference as M
from test_gpu_mixers import (HALF, TYPES, Guarded, assert_near, attn_inputs, attn_tol, check_scan, done, gen, ids, normal,
                             np64, scan_inputs)

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


def same_kind(got, ref, tol, what):
    """Finite values within the tolerance, the others alike."""
    on = np.isfinite(ref)
    assert np.array_equal(got[~on], ref[~on], equal_nan=True), f"{what}: infinities and NaN differ"
    assert_near(got[on], ref[on], tol[on], what)


def run_scan(p, form, softplus=True, lengths=None):
    """A scan in one of its forms: tokens at once ("prompt"; "cut" where a cluster shares the sequence) or
    one at a time; y [B, T, D] and the last state in 64 bits."""
    if form == "step":
        h, y = p["state"].clone(), []
        for t in range(p["x"].shape[1]):
            s = {k: None if p[k] is None else p[k][:, t] for k in ("x", "dt", "z", "Bm", "Cm")}
            y.append(G.selective_scan_step(s["x"], s["dt"], p["A"], s["Bm"], s["Cm"], h, p["D"], s["z"], p["dt_bias"],
                                           softplus))
        y = torch.stack(y, 1)
    else:
        y, h = G.selective_scan(p["x"], p["dt"], p["A"], p["Bm"], p["Cm"], p["D"], p["z"], p["dt_bias"], p["state"],
                                softplus, lengths)
    done()
    return np64(y), np64(h)


TOKENS = {"prompt": 21, "cut": 1100, "step": 5}


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("form", ["prompt", "cut", "step"])
def test_scan_masks_by_the_lowest_value(cuda, dtype, form):
    """softplus of the lowest value of a type and of -inf is 0, so such a token leaves the state as it is;
    above, softplus is its argument (here with x = 0, which empties the state)."""
    g = gen(101)
    T = TOKENS[form]
    p = scan_inputs(g, 1, T, 16, 16, dtype)
    p["dt_bias"] = None
    low = torch.finfo(dtype).min
    for c, v in enumerate((low, -INF, -2.37e38)):
        p["dt"][0, :, c] = v                          # every token masked
        p["dt"][0, 1::3, 4 + c] = v                   # some
    if form != "cut":
        p["dt"][0, 2, 8], p["x"][0, 2, 8] = -low, 0.0
        p["dt"][0, 3, 9], p["x"][0, 3, 9] = 2.37e38, 0.0
    y, h = run_scan(p, form)
    check_scan(p, [T], y, h, dtype, f"masked scan, {form}")
    assert np.array_equal(h[0, :3], np64(p["state"][0, :3]))


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("form", ["prompt", "step"])
def test_scan_keeps_nan_steps(cuda, dtype, form):
    """A NaN step is the caller's to see: its channel becomes NaN, no other one."""
    g = gen(103)
    p = scan_inputs(g, 1, 5, 16, 16, dtype)
    p["dt"][0, 1, 3] = NAN
    y, h = run_scan(p, form)
    assert np.isnan(h[0, 3]).all() and np.isnan(y[0, 1:, 3]).all()
    assert np.isfinite(np.delete(h[0], 3, 0)).all() and np.isfinite(np.delete(y[0], 3, 1)).all()


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("form,lengths", [("prompt", None), ("prompt", [13, 21]), ("step", None)])
def test_scan_keeps_an_infinite_state(cuda, dtype, form, lengths):
    """exp(.) inf + . is inf, also through small and zero steps and through the padding of a group of tokens."""
    g = gen(104)
    T = TOKENS[form]
    p = scan_inputs(g, 2, T, 16, 8, dtype)
    p["A"].clamp_(min=-2)                             # (no decay that underflows)
    n = [T, T] if lengths is None else lengths
    p["dt"][:, 1] = torch.finfo(dtype).min if dtype == torch.float32 else -200.0
    p["state"][0, 2, 3], p["state"][1, 5, 0] = INF, -INF
    ln = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device=cuda)
    y, h = run_scan(p, form, lengths=ln)
    for b, c, s in ((0, 2, 3), (1, 5, 0)):
        assert h[b, c, s] == np64(p["state"])[b, c, s]
        sign = np.sign(np64(p["Cm"][b, :n[b], s]) * np64(p["z"][b, :n[b], c])) * h[b, c, s]
        assert np.array_equal(y[b, :n[b], c], sign)
        p["state"][b, c] = 0.0                        # the channel's other states, and everything else: the oracle
        y[b, :, c], h[b, c] = 0.0, 0.0
        p["x"][b, :, c] = 0.0
    check_scan(p, n, y, h, dtype, f"infinite states, {form}")


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("form", ["prompt", "step"])
def test_scan_of_an_infinite_step_is_infinite(cuda, dtype, form):
    g = gen(102)
    p = scan_inputs(g, 1, 5, 16, 16, dtype)
    p["dt_bias"] = None
    p["A"].clamp_(min=-2)                             # (no decay that underflows)
    p["dt"][0, 1, 3] = INF
    _, h = run_scan(p, form)
    want = np.sign(np64(p["x"][0, 1, 3]) * np64(p["Bm"][0, 1])) * INF
    assert np.array_equal(h[0, 3], want)
    assert np.isfinite(np.delete(h[0], 3, 0)).all()


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("form", ["prompt", "cut", "step"])
def test_scan_of_an_unbounded_decay(cuda, dtype, form):
    """A = -inf forgets at every token with a step, and keeps the state where there is none: padding, masks."""
    g = gen(105)
    T = TOKENS[form]
    p = scan_inputs(g, 2, T, 16, 8, dtype)
    n = [T, T - 2] if form != "step" else [T, T]
    p["dt"][0, T // 2, 4] = -INF                      # a masked token
    p["A"][4, 2], p["A"][5, 0], p["A"][6, 1] = -INF, torch.finfo(torch.float32).min, -3e38
    y, h = run_scan(p, form, lengths=None if form == "step" else torch.tensor(n, dtype=torch.int32, device=cuda))
    p["A"][4, 2] = p["A"][5, 0] = p["A"][6, 1] = -1e30   # (as good, and finite times the oracle's zero steps)
    check_scan(p, n, y, h, dtype, f"unbounded decay, {form}")


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("T", [40, 600, 1100])
def test_scan_growth_of_nothing_is_nothing(cuda, dtype, T):
    """A growing channel whose inputs begin late stays 0 until then, however much a segment would grow it."""
    g = gen(106)
    p = scan_inputs(g, 1, T, 8, 16, dtype)
    p["state"], p["dt_bias"] = None, None
    p["A"][:, :4] = 0.5
    p["dt"][:] = 1.0
    p["x"][:, :T - 20] = 0.0
    y, h = run_scan(p, "prompt", softplus=False)
    check_scan(p, [T], y, h, dtype, "late growth", softplus=False)


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("T", [40, 600, 1100])
def test_scan_decay_of_infinity_is_infinity(cuda, dtype, T):
    """An infinite state stays infinite however much a segment decays it."""
    g = gen(108)
    p = scan_inputs(g, 1, T, 8, 16, dtype)
    p["dt_bias"] = None
    p["A"].clamp_(min=-2)                             # (no step of the recurrence underflows)
    p["dt"][:] = 1.0
    p["state"][0, 1, 4] = -INF
    _, h = run_scan(p, "prompt", softplus=False)
    assert h[0, 1, 4] == -INF
    h[0, 1, 4] = 0.0
    assert np.isfinite(h).all()


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("T", [600, 1100])
def test_scan_with_steps_that_sum_past_the_range(cuda, dtype, T):
    """Steps of the largest value (with x = 0: the state is emptied), several in a segment and in a group of tokens."""
    g = gen(107)
    p = scan_inputs(g, 1, T, 8, 16, dtype)
    p["dt_bias"] = None
    p["A"][:, 3] = 0.0                                # keeps its state whatever the step
    top = torch.finfo(dtype).max
    for c, at in enumerate(([3, 300, 301], [0, 1], [500], [130, 260, 390])):
        p["dt"][0, at, c], p["x"][0, at, c] = top, 0.0
    y, h = run_scan(p, "prompt")
    check_scan(p, [T], y, h, dtype, "largest steps")


def step_inputs(g, B, Hq, Hkv, d, window, sinks, pos):
    t, cap = torch.bfloat16, window + sinks
    q, k, v = normal(g, B, Hq, d, dtype=t), normal(g, B, Hkv, d, dtype=t), normal(g, B, Hkv, d, dtype=t)
    kc, vc = normal(g, B, cap, Hkv, d, dtype=t), normal(g, B, cap, Hkv, d, dtype=t)
    return q, k, v, kc, vc, torch.tensor(pos, dtype=torch.int32, device="cuda")


def check_step(q, kc, vc, pos, out, window, sinks, what):
    for i, p in enumerate(pos.tolist()):
        m = min(window + sinks, p + 1)
        with np.errstate(invalid="ignore"):
            ref, mag = M.window_attention(np64(q[i])[None], np64(kc[i, :m]), np64(vc[i, :m]), m)
        same_kind(out[i], ref[0], attn_tol(ref, mag)[0], f"{what}[{i}]")


@pytest.mark.parametrize("value", [-INF, torch.finfo(torch.bfloat16).min])
@pytest.mark.parametrize("Hq,Hkv,window,sinks", [(4, 2, 880, 16), (40, 2, 100, 0), (2, 2, 70, 5)])
def test_window_step_with_keys_of_minus_infinity(cuda, value, Hq, Hkv, window, sinks):
    """Keys whose score is -inf weigh nothing, also where they are all that a warp or a block has; a row that
    sees no others is NaN, as the formula is."""
    g = gen(110)
    cap = window + sinks
    q, k, v, kc, vc, pos = step_inputs(g, 5, Hq, Hkv, 64, window, sinks, [cap - 1, 3 * cap, cap // 2, cap + 40, 20])
    q[..., 7] = 2.0
    kc[0, :cap // 2, :, 7] = value                    # the first half of the slots
    kc[1, 16:32, :, 7] = value                        # one tile
    kc[2, 5:, :, 7] = value                           # the later ones; the new token's is finite
    kc[3, :, :, 7] = value                            # all but the new token
    kc[4, :, :, 7], k[4, :, 7] = value, value         # all
    out = G.window_attention_step(q, k, v, kc, vc, pos, window, sinks)
    done()
    check_step(q, kc, vc, pos, np64(out), window, sinks, "step with -inf keys") if value == -INF else \
        check_step(q[:4], kc[:4], vc[:4], pos[:4], np64(out)[:4], window, sinks, "step with the lowest keys")


@pytest.mark.parametrize("pos", [15, 16, 17, 31, 32, 100])
def test_window_step_shows_a_nan_key(cuda, pos):
    """A NaN key that a position sees makes its heads' outputs NaN, wherever its slot lies."""
    g = gen(111)
    q, k, v, kc, vc, p = step_inputs(g, 2, 4, 2, 64, 90, 10, [pos, pos])
    k[0, 1, 3] = NAN
    out = G.window_attention_step(q, k, v, kc, vc, p, 90, 10)
    done()
    assert torch.isnan(out[0, 2:]).all() and torch.isfinite(out[0, :2]).all() and torch.isfinite(out[1]).all()


@pytest.mark.parametrize("value", [-INF, torch.finfo(torch.bfloat16).min])
@pytest.mark.parametrize("Hq,Hkv", [(2, 2), (4, 2)])
def test_window_attention_with_keys_of_minus_infinity(cuda, value, Hq, Hkv):
    """Whole key tiles, a sink and single tokens with scores of -inf; queries that see no others are NaN."""
    g = gen(112)
    T, window, sinks = 500, 140, 3
    q, k, v = attn_inputs(g, 1, T, T, Hq, Hkv, 64, 64)
    q[..., 7] = 2.0
    for s in (slice(100, 300), 400):
        k[0, s, :, 7] = value
    if value == -INF:
        k[0, :3, :, 7] = value                        # all sinks: queries 239 to 299 see nothing else
    o = np64(G.window_attention(q, k, v, window, sinks))
    done()
    with np.errstate(invalid="ignore"):
        ref, mag = M.window_attention(np64(q[0]), np64(k[0]), np64(v[0]), window, sinks)
    assert np.isnan(ref).any() == (value == -INF)
    same_kind(o[0], ref, attn_tol(ref, mag), "prompt with -inf keys")


@pytest.mark.parametrize("size", [1e30, 1e35, 1e-30, 1e-37])
@pytest.mark.parametrize("rise", [0.0, 10.0, 14.0, 20.0, 40.0])
def test_window_attention_over_the_range_of_values(cuda, size, rise):
    """Values near the ends of bf16's range, and scores that rise by `rise` (base e) from tile to tile: no sum
    overflows on the way, and small values are not lost.  (2^-133 is bf16's smallest step.)"""
    g = gen(113)
    T, d = 600, 64
    q, k, v = attn_inputs(g, 1, T, T, 2, 1, d, d, std=0.5)
    v = (v.float() * size).to(torch.bfloat16)
    q[..., 0] = 8.0                                   # its score is the key's first element
    k[0, :, 0, 0] = torch.arange(T, device=cuda).div(128, rounding_mode="floor").to(torch.bfloat16) * rise
    o = np64(G.window_attention(q, k, v, 400, 4))
    done()
    ref, mag = M.window_attention(np64(q[0]), np64(k[0]), np64(v[0]), 400, 4)
    S = 8.0 * 4 * rise / 8.0 + 8.0
    tol = 2.0 ** -8 * (np.abs(ref) + mag) + (2.0 ** -12 + 2 * S * 2.0 ** -20) * mag + 4 * 2.0 ** -133
    assert_near(o[0], ref, tol, "values at the ends of the range")


@pytest.mark.parametrize("value", [NAN, INF, -INF])
@pytest.mark.parametrize("Tq,Tk,Hq,Hkv,dv,window,sinks,lengths", [
    (300, 300, 2, 2, 64, 40, 3, None), (300, 300, 4, 2, 112, 200, 0, None), (700, 700, 3, 1, 128, 150, 40, [700, 650]),
    (70, 330, 2, 1, 48, 90, 20, None), (33, 33, 2, 2, 16, 1, 0, None),
])
def test_unseen_values_stay_unseen(cuda, value, Tq, Tk, Hq, Hkv, dv, window, sinks, lengths):
    """NaN and infinities in v reach the queries that see their token and no others: not those before it,
    not those whose window has passed it."""
    g = gen(114)
    B = 1 if lengths is None else len(lengths)
    q, k, v = attn_inputs(g, B, Tq, Tk, Hq, Hkv, 64, dv)
    at = sorted({Tk - 1, Tk - Tq + Tq // 2, max(0, Tk - Tq - 10), Tk // 3})
    for i, s in enumerate(at):
        v[:, s, i % Hkv, (5 * i) % dv] = value
    v[:, Tk - 3, 0] = value
    ln = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device=cuda)
    o = np64(G.window_attention(q, k, v, window, sinks, ln))
    done()
    seen = 0
    for b in range(B):
        n = Tk if lengths is None else lengths[b]
        m = min(Tq, n - (Tk - Tq))
        with np.errstate(invalid="ignore"):
            ref, mag = M.window_attention(np64(q[b, :m]), np64(k[b, :n]), np64(v[b, :n]), window, sinks)
        same_kind(o[b, :m], ref, attn_tol(ref, mag), f"values of {value}")
        seen += int((~np.isfinite(ref)).sum())
    assert seen


@pytest.mark.parametrize("value", [NAN, INF])
def test_unseen_values_stay_unseen_in_a_step(cuda, value):
    g = gen(115)
    q, k, v, kc, vc, pos = step_inputs(g, 2, 4, 2, 64, 30, 4, [20, 12])
    vc[:, 21:] = value
    kc[:, 21:] = value
    vc[1, 13:], kc[1, 13:] = value, value
    out = G.window_attention_step(q, k, v, kc, vc, pos, 30, 4)
    done()
    check_step(q, kc, vc, pos, np64(out), 30, 4, "step beside unused slots")


@pytest.mark.parametrize("value", [NAN, INF])
def test_unseen_keys_stay_unseen(cuda, value):
    """The same of keys; with NaN in all of v, every row is NaN."""
    g = gen(119)
    T, window, sinks = 400, 60, 2
    q, k, v = attn_inputs(g, 1, T, T, 4, 2, 96, 96)
    k[0, 50, 0, 3], k[0, 51, 1, 9], k[0, 399, :, 0], v[0, 51, 1, 9] = value, value, value, NAN
    o = np64(G.window_attention(q, k, v, window, sinks))
    done()
    with np.errstate(invalid="ignore"):
        ref, mag = M.window_attention(np64(q[0]), np64(k[0]), np64(v[0]), window, sinks)
    for rows in (np.isfinite(ref), np.isnan(ref)):
        assert rows.any()
    same_kind(o[0], ref, attn_tol(ref, mag), f"keys of {value}")
    o = G.window_attention(q, torch.zeros_like(k), torch.full_like(v, NAN), window, sinks)
    done()
    assert torch.isnan(o).all()


def test_idle_sessions_get_zeros_unless_out_is_given(cuda):
    """New memory is not handed out as it is: an idle session's row of a new `out` is zero; a given one stays."""
    g = gen(116)
    q, k, v, kc, vc, pos = step_inputs(g, 6, 4, 2, 64, 30, 4, [-1, 3, -7, 100, -(2 ** 31), 0])
    for _ in range(3):
        junk = torch.full((6, 4, 64), NAN, dtype=torch.bfloat16, device=cuda)
        del junk                                      # (its memory is the next call's)
        before = kc.clone(), vc.clone()
        out = G.window_attention_step(q, k, v, kc, vc, pos, 30, 4)
        done()
        idle = pos < 0
        assert (out[idle] == 0).all() and torch.isfinite(out[~idle]).all() and (out[~idle] != 0).any()
        assert torch.equal(kc[idle], before[0][idle]) and torch.equal(vc[idle], before[1][idle])
    given = Guarded((6, 4, 64), torch.bfloat16, 5.0)
    G.window_attention_step(q, k, v, kc, vc, pos, 30, 4, out=given.t)
    done()
    o = given.check()
    assert (o[idle.cpu().numpy()] == 5.0).all() and np.array_equal(o[~idle.cpu().numpy()], np64(out[~idle]))


def test_sizes_past_an_int_are_refused(cuda):
    """A window or sink count that a C int cannot hold is refused, not cut to its low bits."""
    g = gen(117)
    q, k, v = attn_inputs(g, 1, 20, 20, 2, 2, 64, 64)
    for kw in (dict(window=2 ** 32 + 5), dict(window=2 ** 31), dict(window=5, sinks=2 ** 32 + 1), dict(window=2 ** 32)):
        with pytest.raises(ValueError):
            G.window_attention(q, k, v, **kw)
    o = G.window_attention(q, k, v, 2 ** 31 - 1, 2 ** 31 - 1)
    done()
    assert torch.equal(o, G.window_attention(q, k, v, 20))
    kc, vc = G.window_cache(1, 2, 64, 64, 8, 2, cuda)
    with pytest.raises(ValueError):
        G.window_cache_append(k, v, kc, vc, None, 2 ** 32 + 8, 2 - 2 ** 32)
    with pytest.raises(ValueError):
        G.window_attention_step(q[:, 0], k[:, 0], v[:, 0], kc, vc, torch.zeros(1, dtype=torch.int32, device=cuda),
                                2 ** 32 + 8, 2 - 2 ** 32)


def test_calls_repeat_themselves(cuda):
    """The same bits every time: no result depends on which block or warp comes first."""
    g = gen(118)
    p = scan_inputs(g, 1, 1500, 64, 16, torch.bfloat16)
    q, k, v = attn_inputs(g, 2, 1100, 1100, 8, 2, 128, 128, std=3.0)
    s = step_inputs(g, 3, 32, 8, 128, 1000, 16, [1015, 4000, 500])
    q2, k2, v2 = attn_inputs(g, 1, 333, 333, 3, 3, 112, 112, std=8.0)

    def calls():
        return [*G.selective_scan(p["x"], p["dt"], p["A"], p["Bm"], p["Cm"], p["D"], p["z"], p["dt_bias"], p["state"]),
                G.window_attention(q, k, v, 300, 20), G.window_attention(q2, k2, v2, 100, 1),
                G.window_attention_step(*s, 1000, 16)]

    first = calls()
    others = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    runs = []
    for i in range(30):
        with torch.cuda.stream(others[i % 3]):
            runs.append(calls())
    done()
    assert all(torch.equal(a, b) for r in runs for a, b in zip(first, r))


def test_a_block_after_the_cache_has_rolled(cuda):
    """The next block of a session whose earlier tokens are only in the rolling cache: the sinks, the window's
    last tokens and the block, in order, stand for the whole sequence."""
    g = gen(120)
    window, sinks, n, new = 150, 6, 700, 90
    q, k, v = attn_inputs(g, 1, n + new, n + new, 4, 2, 64, 64)
    kc, vc = G.window_cache(1, 2, 64, 64, window, sinks, cuda)
    G.window_cache_append(k[:, :n], v[:, :n], kc, vc, None, window, sinks)
    order = [*range(sinks), *(M.slot(p, window, sinks) for p in range(n - window, n))]
    kk, vv = torch.cat([kc[:, order], k[:, n:]], 1), torch.cat([vc[:, order], v[:, n:]], 1)
    got = np64(G.window_attention(q[:, n:], kk, vv, window, sinks))
    done()
    ref, mag = M.window_attention(np64(q[0, n:]), np64(k[0]), np64(v[0]), window, sinks)
    assert_near(got[0], ref, attn_tol(ref, mag), "a block after the cache")

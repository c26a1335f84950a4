"""GPU parity of the token-by-token mixers against the float64 oracle, element by element.

Tolerances are counted, not fitted.  A rounding to bf16 is off by at most 2^-8 of the value, one
to float32 by 2^-24.
  * convolution: W + 2 float32 roundings of the absolute sum, the SiLU (slope at most 1.1, its
    exponential and division good to 2^-20), one rounding to the output type;
  * scan: the oracle carries a first-order bound along the recurrence (exponent, exponential,
    update, output sum, gate), plus one rounding to the output type;
  * attention: each weight rounded to bf16 (2^-8 of sum p |v|), scores of d float32 products and
    the exponential (2^-12 of sum p |v| covers scores up to a few tens), one output rounding.
Outputs and states sit between guard bands and are NaN-filled first; rows of padding hold NaN.
"""

import numpy as np
import pytest
import torch

import hybrid_linear_attention_frame_b200 as G
from oracle import mixers_reference as M

pytestmark = pytest.mark.gpu

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
TYPES = [torch.bfloat16, torch.float32]
NAN = float("nan")


def ids(t):
    return str(t).split(".")[-1] if isinstance(t, torch.dtype) else None


def np64(t):
    return t.double().cpu().numpy()


class Guarded:
    """A contiguous tensor with 64 guard elements on either side."""

    def __init__(self, shape, dtype, fill=NAN):
        n = int(np.prod(shape))
        self.buf = torch.full((n + 128,), 7.0, dtype=dtype, device="cuda")
        self.t = self.buf[64:64 + n].view(shape)
        self.t.fill_(fill)

    def check(self):
        assert bool((self.buf[:64] == 7.0).all()) and bool((self.buf[-64:] == 7.0).all()), "write outside an output"
        return np64(self.t)


def assert_near(got, ref, tol, what):
    bad = ~(np.abs(got - ref) <= tol)
    if bad.any():
        i = tuple(int(v) for v in np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {bad.sum()} of {bad.size} off, first at {i}: {got[i]!r} vs {ref[i]!r}, "
                             f"tolerance {np.broadcast_to(tol, ref.shape)[i]:.3e}")


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(g, *shape, dtype=torch.float32, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def strided(x, extra):
    """The same values as a slice of wider rows."""
    wide = torch.full((*x.shape[:-1], x.shape[-1] + extra), NAN, dtype=x.dtype, device=x.device)
    wide[..., :x.shape[-1]] = x
    return wide[..., :x.shape[-1]]


def done():
    torch.cuda.synchronize()
    assert G.gdn_get_last_device_status() == G.GDN_OK


# ------------------------------------------------------------------------------------- convolution

def conv_tol(ref, mag, W, half):
    return 1.1 * mag * (W + 2) * 2.0 ** -24 + np.abs(ref) * (half + 2.0 ** -20) + 1e-30


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("B,T,D,W,silu,lengths", [
    (1, 1, 8, 4, True, None), (2, 2, 16, 4, False, None), (1, 15, 24, 3, True, None), (1, 16, 24, 2, True, None),
    (3, 17, 40, 4, True, [17, 0, 2]), (2, 33, 1032, 3, False, [1, 33]), (2, 131, 264, 4, True, [130, 16]),
    (1, 700, 56, 4, True, None),
])
def test_conv(cuda, dtype, B, T, D, W, silu, lengths):
    g = gen(T * 100 + D)
    x, w, b = normal(g, B, T, D, dtype=dtype), normal(g, D, W, std=0.7), normal(g, D)
    st = normal(g, B, W - 1, D, dtype=dtype)
    n = [T] * B if lengths is None else lengths
    for i in range(B):
        x[i, n[i]:] = NAN
    ln = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device=cuda)
    out, so = Guarded((B, T, D), dtype, 5.0), Guarded((B, W - 1, D), dtype)
    for state, bias in ((st, b), (None, None)):
        out.t.fill_(5.0)
        G.causal_conv(strided(x, 8), w, bias, state, silu, ln, out=out.t, state_out=so.t)
        done()
        o, s = out.check(), so.check()
        for i in range(B):
            ref, new, mag = M.causal_conv(np64(x[i, :n[i]]), np64(w), None if bias is None else np64(bias),
                                          None if state is None else np64(state[i]), silu)
            assert_near(o[i, :n[i]], ref, conv_tol(ref, mag, W, HALF[dtype]), f"conv out[{i}]")
            assert np.array_equal(s[i], new), "conv state"
            assert (o[i, n[i]:] == 5.0).all(), "a padded row was written"


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
def test_conv_pieces_and_steps_equal_the_prompt(cuda, dtype):
    g = gen(9)
    B, T, D, W = 3, 41, 72, 4
    x, w, b = normal(g, B, T, D, dtype=dtype), normal(g, D, W), normal(g, D)
    whole, last = G.causal_conv(x, w, b)
    state = torch.zeros(B, W - 1, D, dtype=dtype, device=cuda)
    got = []
    for t0, t1 in ((0, 2), (2, 3), (3, 20), (20, 20), (20, 36)):
        y, same = G.causal_conv(x[:, t0:t1], w, b, state, state_out=state)
        assert same is state
        got.append(y)
    for t in range(36, T):
        got.append(G.causal_conv_step(x[:, t], w, b, state)[:, None])
    done()
    assert torch.equal(torch.cat(got, 1), whole) and torch.equal(state, last)


def test_conv_extreme_values(cuda):
    """SiLU of large magnitudes is 0 or the value, and an infinity stays in its channel."""
    x = torch.zeros(1, 6, 16, device=cuda)
    x[0, 2, 0], x[0, 2, 1], x[0, 2, 2] = 3e38, -3e38, float("inf")
    w = torch.ones(16, 2, device=cuda) * 0.5
    y, _ = G.causal_conv(x, w)
    done()
    y = y.cpu()
    assert y[0, 2, 0] == 1.5e38 and y[0, 2, 1] == 0 and torch.isinf(y[0, 2, 2])
    assert (y[0, :, 3:] == 0).all()


# ------------------------------------------------------------------------------------- scan

def scan_inputs(g, B, T, D, N, dtype):
    step = torch.exp(torch.rand(D, generator=g, device="cuda") * 4.6 - 6.9)
    return dict(x=normal(g, B, T, D, dtype=dtype), dt=normal(g, B, T, D, dtype=dtype, std=0.7),
                A=-torch.exp(normal(g, D, N)) * torch.arange(1, N + 1, device="cuda"),
                Bm=normal(g, B, T, N, dtype=dtype), Cm=normal(g, B, T, N, dtype=dtype), D=normal(g, D),
                z=normal(g, B, T, D, dtype=dtype, std=2.0), dt_bias=torch.log(torch.expm1(step)),
                state=normal(g, B, D, N))


def check_scan(p, n, y, h, dtype, what, softplus=True):
    for i in range(len(n)):
        k = n[i]
        get = lambda name: None if p[name] is None else np64(p[name])
        row = lambda name: None if p[name] is None else np64(p[name][i, :k])
        ref, last, yerr, herr = M.selective_scan(row("x"), row("dt"), get("A"), row("Bm"), row("Cm"), get("D"),
                                                 row("z"), get("dt_bias"),
                                                 None if p["state"] is None else np64(p["state"][i]), softplus)
        assert_near(y[i, :k], ref, yerr + np.abs(ref) * HALF[dtype] + 1e-30, f"{what} y[{i}]")
        assert_near(h[i], last, herr + 1e-30, f"{what} state[{i}]")


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("B,T,D,N,lengths", [
    (1, 1, 8, 16, None), (2, 3, 24, 8, None), (1, 31, 40, 32, None), (1, 32, 16, 64, None), (2, 33, 136, 16, [33, 7]),
    (4, 65, 72, 16, [0, 1, 64, 65]), (1, 300, 264, 16, None), (1, 257, 48, 64, None), (5, 100, 200, 8, [3, 100, 50, 99, 32]),
    # long enough that a cluster shares a sequence, also one that leaves some of its blocks without tokens
    (1, 512, 24, 16, None), (1, 1025, 8, 16, None), (2, 1100, 40, 8, [1100, 130]), (2, 600, 16, 32, [600, 0]),
    (1, 1300, 24, 64, None),
])
def test_scan(cuda, dtype, B, T, D, N, lengths):
    g = gen(T * 7 + N)
    p = scan_inputs(g, B, T, D, N, dtype)
    n = [T] * B if lengths is None else lengths
    for i in range(B):
        for name in ("x", "dt", "z", "Bm", "Cm"):
            p[name][i, n[i]:] = NAN
    ln = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device=cuda)
    y, h = Guarded((B, T, D), dtype), Guarded((B, D, N), torch.float32)
    plain = dict(p, D=None, z=None, dt_bias=None, state=None)
    for q in (p, plain):
        y.t.fill_(5.0)
        a = {k: (strided(v, 16) if k in ("x", "dt", "z", "Bm", "Cm") and v is not None else v) for k, v in q.items()}
        G.selective_scan(a["x"], a["dt"], a["A"], a["Bm"], a["Cm"], a["D"], a["z"], a["dt_bias"], a["state"],
                         lengths=ln, out=y.t, state_out=h.t)
        done()
        yo, ho = y.check(), h.check()
        check_scan(q, n, yo, ho, dtype, f"scan {'full' if q is p else 'plain'}")
        for i in range(B):
            assert (yo[i, n[i]:] == 5.0).all(), "a padded row was written"


def test_scan_without_softplus_and_with_growth(cuda):
    """delta as given, zero and tiny deltas, a positive A (a growing state)."""
    g = gen(77)
    p = scan_inputs(g, 1, 50, 32, 16, torch.float32)
    p["dt"] = torch.rand(1, 50, 32, generator=g, device=cuda) * 0.2
    p["dt"][:, ::3] = 0.0
    p["dt"][:, 1::7] = 1e-9
    p["dt_bias"] = None
    p["A"][:, :4] = 0.5
    p["A"][:, 4] = 0.0
    y, h = G.selective_scan(p["x"], p["dt"], p["A"], p["Bm"], p["Cm"], p["D"], p["z"], None, p["state"], False)
    done()
    check_scan(p, [50], np64(y), np64(h), torch.float32, "scan as given", softplus=False)


def test_scan_extreme_steps(cuda):
    """softplus of far arguments: 0 below (the state stays), the argument above (the state is replaced)."""
    g = gen(78)
    p = scan_inputs(g, 1, 20, 16, 16, torch.float32)
    p["dt_bias"] = None
    p["dt"][0, :, 0], p["dt"][0, :, 1], p["dt"][0, :, 2] = -200.0, 90.0, -18.0
    y, h = G.selective_scan(p["x"], p["dt"], p["A"], p["Bm"], p["Cm"], p["D"], p["z"], None, p["state"])
    done()
    check_scan(p, [20], np64(y), np64(h), torch.float32, "scan far steps")
    assert torch.equal(h[0, 0], p["state"][0, 0])


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("N", [8, 16, 32, 64])
def test_scan_pieces_and_steps(cuda, dtype, N):
    """A prompt in pieces, then token by token, against the oracle over the whole sequence."""
    g = gen(N)
    B, T, D = 2, 70, 88
    p = scan_inputs(g, B, T, D, N, dtype)
    state, got = p["state"].clone(), []
    for t0, t1 in ((0, 1), (1, 40), (40, 40), (40, 64)):
        s = {k: p[k][:, t0:t1] for k in ("x", "dt", "z", "Bm", "Cm")}
        y, same = G.selective_scan(s["x"], s["dt"], p["A"], s["Bm"], s["Cm"], p["D"], s["z"], p["dt_bias"], state,
                                   state_out=state)
        assert same is state
        got.append(y)
    for t in range(64, T):
        s = {k: p[k][:, t] for k in ("x", "dt", "z", "Bm", "Cm")}
        got.append(G.selective_scan_step(s["x"], s["dt"], p["A"], s["Bm"], s["Cm"], state, p["D"], s["z"],
                                         p["dt_bias"])[:, None])
    done()
    check_scan(p, [T] * B, np64(torch.cat(got, 1)), np64(state), dtype, f"scan in pieces, N {N}")


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("B,D,N", [(1, 8, 16), (7, 136, 8), (300, 24, 16), (301, 2240, 32), (3, 264, 32), (2, 72, 64)])
def test_scan_step(cuda, dtype, B, D, N):
    g = gen(B + D)
    p = scan_inputs(g, B, 1, D, N, dtype)
    y, h = Guarded((B, D), dtype), Guarded((B, D, N), torch.float32)
    for q in (p, dict(p, D=None, z=None, dt_bias=None)):
        h.t.copy_(p["state"])
        s = {k: None if q[k] is None else strided(q[k][:, 0], 8) for k in ("x", "dt", "z", "Bm", "Cm")}
        G.selective_scan_step(s["x"], s["dt"], q["A"], s["Bm"], s["Cm"], h.t, q["D"], s["z"], q["dt_bias"], out=y.t)
        done()
        check_scan(q, [1] * B, y.check()[:, None], h.check(), dtype, "scan step")


# ------------------------------------------------------------------------------------- window attention

def attn_tol(ref, mag):
    return 2.0 ** -8 * (np.abs(ref) + mag) + 2.0 ** -12 * mag + 1e-30


def attn_inputs(g, B, Tq, Tk, Hq, Hkv, dk, dv, std=1.0):
    t = torch.bfloat16
    return normal(g, B, Tq, Hq, dk, dtype=t, std=std), normal(g, B, Tk, Hkv, dk, dtype=t), normal(g, B, Tk, Hkv, dv, dtype=t)


# B, Tq, Tk, Hq, Hkv, dk, dv, window, sinks, lengths
ATTN = [
    (1, 1, 1, 1, 1, 16, 16, 1, 0, None), (1, 1, 1, 2, 1, 128, 128, 5, 3, None), (2, 5, 5, 4, 2, 64, 64, 3, 1, None),
    (1, 127, 127, 2, 2, 112, 112, 40, 4, None), (1, 128, 128, 3, 1, 64, 128, 128, 0, None),
    (1, 129, 129, 2, 2, 112, 112, 1000, 0, None), (1, 200, 200, 7, 1, 96, 48, 1, 0, None),
    (1, 200, 200, 2, 2, 80, 80, 1, 9, None), (1, 300, 300, 5, 5, 112, 112, 130, 0, None),
    (1, 300, 300, 4, 1, 128, 128, 17, 200, None), (1, 520, 520, 2, 1, 112, 112, 256, 128, None),
    (1, 520, 520, 2, 2, 32, 32, 128, 129, None), (3, 260, 260, 4, 2, 64, 64, 100, 5, [260, 129, 1]),
    (2, 150, 150, 2, 2, 128, 112, 300, 0, [0, 150]), (4, 90, 90, 6, 3, 16, 128, 20, 30, [90, 64, 65, 3]),
    (1, 3, 400, 4, 2, 112, 112, 90, 7, None), (2, 130, 391, 4, 4, 64, 64, 150, 0, [391, 300]),
    (1, 1, 1000, 8, 2, 128, 128, 400, 4, None), (1, 257, 700, 2, 2, 112, 112, 64, 600, None),
    (2, 64, 200, 2, 1, 48, 80, 30, 2, [100, 170]),
    # query tiles side by side whose windows start in different key tiles, sinks apart from the window
    (1, 700, 700, 3, 3, 64, 64, 150, 5, None), (2, 900, 900, 1, 1, 112, 112, 1, 130, [900, 640]),
    (1, 900, 900, 2, 2, 128, 128, 290, 300, None),
]


@pytest.mark.parametrize("case", range(len(ATTN)))
def test_window_attention(cuda, case):
    B, Tq, Tk, Hq, Hkv, dk, dv, window, sinks, lengths = ATTN[case]
    g = gen(1000 + case)
    q, k, v = attn_inputs(g, B, Tq, Tk, Hq, Hkv, dk, dv)
    n = [Tk] * B if lengths is None else lengths
    for i in range(B):
        k[i, n[i]:], v[i, n[i]:] = NAN, NAN
        q[i, max(0, n[i] - (Tk - Tq)):] = NAN
    ln = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device=cuda)
    out = Guarded((B, Tq, Hq, dv), torch.bfloat16, 5.0)
    G.window_attention(q, k, v, window, sinks, ln, out=out.t)
    done()
    o = out.check()
    for i in range(B):
        m = min(Tq, max(0, n[i] - (Tk - Tq)))
        if m:
            ref, mag = M.window_attention(np64(q[i, :m]), np64(k[i, :n[i]])[:Tk - Tq + m], np64(v[i, :n[i]])[:Tk - Tq + m],
                                          window, sinks)
            assert_near(o[i, :m], ref, attn_tol(ref, mag), f"window attention[{i}]")
        assert (o[i, m:] == 5.0).all(), "a padded row was written"


def test_window_attention_layouts_agree(cuda):
    """Slices of a fused projection and the [B, H, T, d] order give the same bits as contiguous tensors."""
    g = gen(5)
    B, T, Hq, Hkv, d = 2, 300, 4, 2, 112
    qkv = normal(g, B, T, (Hq + 2 * Hkv) * d, dtype=torch.bfloat16).view(B, T, Hq + 2 * Hkv, d)
    q, k, v = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv], qkv[:, :, Hq + Hkv:]
    a = G.window_attention(q, k, v, 100, 5)
    b = G.window_attention(q.contiguous(), k.contiguous(), v.contiguous(), 100, 5)
    c = G.window_attention(*(t.transpose(1, 2).contiguous().transpose(1, 2) for t in (q, k, v)), 100, 5)
    done()
    assert torch.equal(a, b) and torch.equal(a, c)


def test_window_attention_large_scores_and_scale(cuda):
    """Peaked softmaxes, scores in the hundreds of either sign, a scale of one's own, equal scores."""
    g = gen(6)
    q, k, v = attn_inputs(g, 1, 300, 300, 2, 2, 112, 112, std=8.0)
    k[:, 100:130] *= 4
    for scale in (None, 0.5):
        o = np64(G.window_attention(q, k, v, 200, 3, scale=scale))
        done()
        ref, mag = M.window_attention(np64(q[0]), np64(k[0]), np64(v[0]), 200, 3, scale)
        # scores up to S: their float32 error d 2^-24 S moves a weight by that much
        S = np.abs(np64(q[0])).max() * np.abs(np64(k[0])).max() * 112 * (112 ** -0.5 if scale is None else scale)
        assert_near(o[0], ref, attn_tol(ref, mag) + 2 * S * 2.0 ** -20 * mag, "large scores")
    o = np64(G.window_attention(torch.zeros_like(q), k, v, 200, 3))
    ref, mag = M.window_attention(0 * np64(q[0]), np64(k[0]), np64(v[0]), 200, 3)
    assert_near(o[0], ref, attn_tol(ref, mag), "equal scores")


# B, Hq, Hkv, dk, dv, window, sinks, positions
STEP = [
    (1, 1, 1, 16, 16, 1, 0, [0]), (3, 4, 2, 64, 64, 8, 2, [0, 5, 300]), (1, 20, 20, 112, 112, 880, 16, [895]),
    (2, 8, 1, 128, 128, 500, 4, [250, 100000]), (4, 14, 2, 80, 48, 63, 1, [-1, 62, 63, 64]),
    (2, 5, 5, 32, 128, 64, 64, [127, 128]), (2, 32, 2, 96, 96, 130, 0, [129, 2 ** 31 - 1]), (1, 6, 2, 112, 64, 1, 300, [700]),
    (2, 40, 2, 128, 128, 700, 33, [731, 5000]), (5, 3, 3, 128, 128, 1000, 0, [0, 1, 31, 32, 33]),
]


@pytest.mark.parametrize("case", range(len(STEP)))
def test_window_step(cuda, case):
    B, Hq, Hkv, dk, dv, window, sinks, pos = STEP[case]
    g = gen(2000 + case)
    t, cap = torch.bfloat16, window + sinks
    q, k, v = normal(g, B, Hq, dk, dtype=t), normal(g, B, Hkv, dk, dtype=t), normal(g, B, Hkv, dv, dtype=t)
    kc, vc, out = Guarded((B, cap, Hkv, dk), t), Guarded((B, cap, Hkv, dv), t), Guarded((B, Hq, dv), t, 5.0)
    kc.t.copy_(normal(g, B, cap, Hkv, dk, dtype=t))
    vc.t.copy_(normal(g, B, cap, Hkv, dv, dtype=t))
    for i, p in enumerate(pos):                       # slots that no token has reached hold NaN
        kc.t[i, max(0, min(cap, p)):], vc.t[i, max(0, min(cap, p)):] = NAN, NAN
        if p >= cap:
            kc.t[i, M.slot(p, window, sinks)] = NAN
    kref, vref = kc.t.clone(), vc.t.clone()
    for i, p in enumerate(pos):
        if p >= 0:
            kref[i, M.slot(p, window, sinks)], vref[i, M.slot(p, window, sinks)] = k[i], v[i]
    G.window_attention_step(q, k, v, kc.t, vc.t, torch.tensor(pos, dtype=torch.int32, device=cuda), window, sinks,
                            out=out.t)
    done()
    o = out.check()
    assert np.array_equal(kc.check(), np64(kref), equal_nan=True) and np.array_equal(vc.check(), np64(vref), equal_nan=True)
    for i, p in enumerate(pos):
        if p < 0:
            assert (o[i] == 5.0).all()
            continue
        m = min(cap, p + 1)
        ref, mag = M.window_attention(np64(q[i])[None], np64(kref[i, :m]), np64(vref[i, :m]), m)
        assert_near(o[i], ref[0], attn_tol(ref, mag)[0], f"window step[{i}]")


@pytest.mark.parametrize("B,T,window,sinks,start,lengths", [
    (2, 1, 5, 0, None, None), (1, 40, 16, 4, None, None), (3, 9, 16, 4, [0, 2, 30], [9, 0, 5]),
    (2, 100, 7, 3, [0, 50], [100, 61]), (2, 6, 1, 0, [3, -1], None), (1, 20, 16, 4, [3], None), (1, 21, 16, 4, [3], None),
    (2, 64, 8, 40, [0, 20], [64, 10]),
])
def test_append(cuda, B, T, window, sinks, start, lengths):
    g = gen(T + window)
    H, dk, dv, t = 3, 32, 48, torch.bfloat16
    k, v = normal(g, B, T, H, dk, dtype=t), normal(g, B, T, H, dv, dtype=t)
    kc, vc = Guarded((B, window + sinks, H, dk), t), Guarded((B, window + sinks, H, dv), t)
    kr, vr = kc.t.clone(), vc.t.clone()
    for b in range(B):
        s = 0 if start is None else start[b]
        n = T if lengths is None else lengths[b]
        for i in range(n if s >= 0 else 0):
            p = s + i
            if p < sinks or p >= s + n - window:
                kr[b, M.slot(p, window, sinks)], vr[b, M.slot(p, window, sinks)] = k[b, i], v[b, i]
    dev = lambda a: None if a is None else torch.tensor(a, dtype=torch.int32, device=cuda)
    G.window_cache_append(strided(k.reshape(B, T, -1), 8).unflatten(2, (H, dk)), v, kc.t, vc.t, dev(start), window,
                          sinks, dev(lengths))
    done()
    assert np.array_equal(kc.check(), np64(kr), equal_nan=True) and np.array_equal(vc.check(), np64(vr), equal_nan=True)


# ------------------------------------------------------------------------------------- together

def test_session_prompt_then_steps(cuda):
    """A hybrid layer pair as a session runs it: convolution, scan and window attention over a padded
    batch of prompts, then token by token, against the same operators over the whole sequences."""
    g = gen(42)
    B, T, S, D, N, W, H, Hkv, d, window, sinks = 3, 90, 30, 64, 16, 4, 4, 2, 16, 24, 3
    t = torch.bfloat16
    n = [90, 1, 57]
    x = normal(g, B, T + S, D, dtype=t)
    w, b = normal(g, D, W, std=0.5), normal(g, D, std=0.1)
    dt, z, Bm, Cm = (normal(g, B, T + S, m, dtype=t) for m in (D, D, N, N))
    A, skip = -torch.exp(normal(g, D, N)), normal(g, D)
    q = normal(g, B, T + S, H, d, dtype=t)
    k, v = normal(g, B, T + S, Hkv, d, dtype=t), normal(g, B, T + S, Hkv, d, dtype=t)
    lengths = torch.tensor(n, dtype=torch.int32, device=cuda)
    c, cs = G.causal_conv(x[:, :T], w, b, lengths=lengths)
    y, h = G.selective_scan(c, dt[:, :T], A, Bm[:, :T], Cm[:, :T], skip, z[:, :T], lengths=lengths)
    o = G.window_attention(q[:, :T], k[:, :T], v[:, :T], window, sinks, lengths)
    kc, vc = G.window_cache(B, Hkv, d, d, window, sinks, cuda)
    G.window_cache_append(k[:, :T], v[:, :T], kc, vc, None, window, sinks, lengths)
    rows, pos = torch.arange(B, device=cuda), lengths.clone()
    ys, os_ = [], []
    for s in range(S):                                # each session's own next token
        p = pos.long()
        c1 = G.causal_conv_step(x[rows, p], w, b, cs)
        ys.append(G.selective_scan_step(c1, dt[rows, p], A, Bm[rows, p], Cm[rows, p], h, skip, z[rows, p]))
        os_.append(G.window_attention_step(q[rows, p], k[rows, p], v[rows, p], kc, vc, pos, window, sinks))
        pos += 1
    done()
    for i in range(B):
        m = n[i] + S
        ci, ci_state = G.causal_conv(x[i:i + 1, :m], w, b)
        yi, hi = G.selective_scan(ci, dt[i:i + 1, :m], A, Bm[i:i + 1, :m], Cm[i:i + 1, :m], skip, z[i:i + 1, :m])
        oi = np64(G.window_attention(q[i:i + 1, :m], k[i:i + 1, :m], v[i:i + 1, :m], window, sinks))[0]
        assert torch.equal(cs[i], ci_state[0])
        got = torch.cat([y[i, :n[i]], torch.stack([a[i] for a in ys])])
        _, _, yerr, herr = M.selective_scan(np64(ci[0]), np64(dt[i, :m]), np64(A), np64(Bm[i, :m]), np64(Cm[i, :m]),
                                            np64(skip), np64(z[i, :m]))
        assert_near(np64(got), np64(yi[0]), 2 * (yerr + np.abs(np64(yi[0])) * 2.0 ** -8), "scan over a session")
        assert_near(np64(h[i]), np64(hi[0]), 2 * herr + 1e-30, "scan state over a session")
        _, mag = M.window_attention(np64(q[i, :m]), np64(k[i, :m]), np64(v[i, :m]), window, sinks)
        got = np64(torch.cat([o[i, :n[i]], torch.stack([a[i] for a in os_])]))
        assert_near(got, oi, 2 * attn_tol(oi, mag), "attention over a session")


def test_conv_feeds_the_delta_rule(cuda):
    """The short convolution in front of gdn_forward's q, k and v, as slices of one projection."""
    from oracle import gdn_reference as R
    from workloads import draw
    r = np.random.Generator(np.random.PCG64(3))
    inp = draw(r, 1, 2, 200, 32, 32, 50, "f32", 0.0, 1.0)
    g = gen(3)
    x = normal(g, 1, 200, 3 * 64)
    w = normal(g, 3 * 64, 4, std=0.5)
    c, _ = G.causal_conv(x, w)
    q, k, v = (t.reshape(1, 200, 2, 32).contiguous() for t in c.split(64, 2))
    gate, beta = torch.from_numpy(inp.gate).to(cuda), torch.from_numpy(inp.beta).to(cuda)
    out, _ = G.forward(q, k, v, gate, beta, frame_len=50, chunk_len=16)
    done()
    cr, _, _ = M.causal_conv(np64(x[0]), np64(w))
    for name, i in (("q", 0), ("k", 1), ("v", 2)):
        getattr(inp, name)[:] = cr[:, 64 * i:64 * i + 64].reshape(1, 200, 2, 32)
    ref, _ = R.token_recurrence(inp, None)
    got = np64(out)
    assert np.linalg.norm(got - ref) <= 1e-4 * np.linalg.norm(ref)


# ------------------------------------------------------------------------------------- streams, graphs, refusals

def test_captured_and_replayed_beside_eager_calls(cuda):
    """Every call captured into one graph and replayed on new inputs, eager calls on another stream between."""
    g = gen(8)
    t, B, T, D, N, H, d, window, sinks = torch.bfloat16, 2, 150, 64, 16, 4, 64, 40, 2
    p = scan_inputs(g, B, T, D, N, t)
    w = normal(g, D, 4)
    q, k, v = attn_inputs(g, B, T, T, H, H, d, d)
    kc, vc = (torch.zeros(B, window + sinks, H, d, dtype=t, device=cuda) for _ in range(2))
    pos = torch.full((B,), T, dtype=torch.int32, device=cuda)

    def calls():
        c, cs = G.causal_conv(p["x"], w)
        y, h = G.selective_scan(c, p["dt"], p["A"], p["Bm"], p["Cm"], p["D"], p["z"], p["dt_bias"], p["state"])
        o = G.window_attention(q, k, v, window, sinks)
        G.window_cache_append(k, v, kc, vc, None, window, sinks)
        c1 = G.causal_conv_step(p["x"][:, 0], w, None, cs)
        y1 = G.selective_scan_step(c1, p["dt"][:, 0], p["A"], p["Bm"][:, 0], p["Cm"][:, 0], h)
        o1 = G.window_attention_step(q[:, 0], k[:, 0], v[:, 0], kc, vc, pos, window, sinks)
        return [c, cs, y, h, o, c1, y1, o1]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        calls()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = calls()
    for seed in (1, 2):
        g2 = gen(seed)
        for x in (p["x"], p["dt"], q, k, v):
            x.copy_(normal(g2, *x.shape, dtype=t))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        kept = [a.clone() for a in got]
        kv = kc.clone(), vc.clone()
        with torch.cuda.stream(side):
            want = calls()
        done()
        assert all(torch.equal(a, b) for a, b in zip(kept, want))
        assert torch.equal(kc, kv[0]) and torch.equal(vc, kv[1])


@pytest.mark.parametrize("step", [False, True])
def test_window_attention_timeout_is_reported_and_recovers(cuda, step):
    """A wait that runs out (the bound shortened to 1 ns) is reported, and the next call is right.

    A wait that finds its copy there gives nothing to report, so the step reads 512 MB from all SMs at
    once: HBM keeps its warps waiting."""
    g = gen(12)
    if step:
        q, k, v = attn_inputs(g, 32, 1, 1, 8, 8, 128, 128)
        kc, vc = (normal(g, 32, 4010, 8, 128, dtype=torch.bfloat16) for _ in range(2))
        pos = torch.full((32,), 5000, dtype=torch.int32, device=cuda)
        call = lambda: G.window_attention_step(q[:, 0], k[:, 0], v[:, 0], kc, vc, pos, 4000, 10)
    else:
        q, k, v = attn_inputs(g, 1, 2000, 2000, 4, 2, 112, 112)
        call = lambda: G.window_attention(q, k, v, 500, 20)
    want = call()
    done()
    try:
        G.gdn_set_wait_limit_ns(1)
        call()
        assert G.gdn_get_last_device_status() == G.GDN_ERR_TIMEOUT
    finally:
        G.gdn_set_wait_limit_ns(0)
    got = call()
    done()
    assert torch.equal(got, want)


def test_python_calls_check_shapes_and_types(cuda):
    t = torch.bfloat16
    x, w = torch.zeros(2, 4, 16, dtype=t, device=cuda), torch.zeros(16, 4, device=cuda)
    for bad in (dict(weight=w.to(t)), dict(weight=w[:8]), dict(bias=torch.zeros(8, device=cuda)),
                dict(state=torch.zeros(2, 3, 16, device=cuda)), dict(lengths=torch.zeros(2, device=cuda)),
                dict(x=x.half()), dict(x=x.transpose(1, 2)), dict(weight=w.cpu()), dict(out=x[:, :2])):
        with pytest.raises(ValueError):
            G.causal_conv(**{**dict(x=x, weight=w), **bad})
    with pytest.raises(G.GdnError):
        G.causal_conv(x, torch.zeros(16, 5, device=cuda))
    with pytest.raises(G.GdnError):
        G.causal_conv(x, w, out=x)
    Bm, A = torch.zeros(2, 4, 16, dtype=t, device=cuda), torch.zeros(16, 16, device=cuda)
    for bad in (dict(dt=x.float()), dict(A=A.to(t)), dict(Bm=Bm[:, :3]), dict(Cm=Bm.cpu()), dict(z=x[:1])):
        with pytest.raises(ValueError):
            G.selective_scan(**{**dict(x=x, dt=x.clone(), A=A, Bm=Bm, Cm=Bm), **bad})
    q = torch.zeros(2, 8, 4, 32, dtype=t, device=cuda)
    for bad in (dict(k=q[:, :4]), dict(v=q.float()), dict(lengths=torch.zeros(3, dtype=torch.int32, device=cuda)),
                dict(out=q[:, :2])):
        with pytest.raises(ValueError):
            G.window_attention(**{**dict(q=q, k=q, v=q, window=4), **bad})
    for bad in (dict(window=0), dict(sinks=-1), dict(scale=-1.0), dict(out=q), dict(k=q[:, :, :3], v=q[:, :, :3])):
        with pytest.raises(G.GdnError):
            G.window_attention(**{**dict(q=q, k=q.clone(), v=q.clone(), window=4), **bad})
    kc, vc = G.window_cache(2, 4, 32, 32, 6, 2, cuda)
    pos = torch.zeros(2, dtype=torch.int32, device=cuda)
    for bad in (dict(pos=pos.long()), dict(window=7), dict(k=q[:, 0, :2]), dict(k_cache=kc[:, :4])):
        with pytest.raises(ValueError):
            G.window_attention_step(**{**dict(q=q[:, 0], k=q[:, 0], v=q[:, 0], k_cache=kc, v_cache=vc, pos=pos, window=6,
                                              sinks=2), **bad})
    done()

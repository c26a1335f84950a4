"""The sequence-mixing operators of hybrid models, as cases that can be timed and compared.

Five operators, each for a whole prompt and for the next token of a session:

* ``conv`` / ``conv_step``: a causal depthwise convolution of width 2 to 4 with SiLU, its last
  inputs carried as a state;
* ``scan`` / ``scan_step``: the selective state space scan
  h_t = exp(delta_t A) h_{t-1} + delta_t x_t B_t,  y_t = (C_t . h_t + D x_t) silu(z_t);
* ``attn``: softmax attention over a sliding window plus the first (sink) tokens, with the
  prompt's tail written into the rolling cache that the next tokens read;
* ``attn_step``: one token per session against that rolling cache, which takes the token in.

With ``own`` false, ``run`` computes them from elementary torch operations in 32 bits, rounded
once; with ``own`` true it calls the library.  Both read what ``prepare`` made.
"""

import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------------- cases

def listed():
    return [
        # the convolution in front of a 241-frame clip's mixer (31 latent frames of 880 tokens)
        {"name": "conv clip", "op": "conv", "type": "bf16", "B": 1, "T": 27280, "D": 4480, "W": 4, "ragged": False},
        # 96 sessions, one token each, float32 activations
        {"name": "conv step 96 sessions", "op": "conv_step", "type": "f32", "B": 96, "D": 2240, "W": 4},
        # a padded batch of three short prompts in the float32 mode, an odd length
        {"name": "scan padded f32", "op": "scan", "type": "f32", "B": 3, "T": 517, "D": 1128, "N": 8, "ragged": True},
        # one streaming block of 3 latent frames at the layer's width
        {"name": "scan block", "op": "scan", "type": "bf16", "B": 1, "T": 2640, "D": 2240, "N": 16, "ragged": False},
        # a 241-frame clip in one call
        {"name": "scan clip", "op": "scan", "type": "bf16", "B": 1, "T": 27280, "D": 2240, "N": 16, "ragged": False},
        # a single session's next token: latency
        {"name": "scan step 1 session", "op": "scan_step", "type": "bf16", "B": 1, "D": 2240, "N": 16},
        # a full server: 256 sessions at twice the width
        {"name": "scan step 256 sessions", "op": "scan_step", "type": "bf16", "B": 256, "D": 4480, "N": 16},
        # a padded batch of short prompts, narrow heads, a window shorter than the prompts
        {"name": "window prompt padded", "op": "attn", "B": 3, "T": 517, "Hq": 8, "Hkv": 8, "dk": 64, "dv": 64,
         "window": 130, "sinks": 4, "ragged": True},
        # one streaming block of the repository's layer, a window of one latent frame
        {"name": "window prompt block", "op": "attn", "B": 1, "T": 2640, "Hq": 20, "Hkv": 20, "dk": 112, "dv": 112,
         "window": 880, "sinks": 16, "ragged": False},
        # a clip, shared key heads, a window of one streaming block and a whole sink frame
        {"name": "window prompt clip", "op": "attn", "B": 1, "T": 27280, "Hq": 20, "Hkv": 4, "dk": 128, "dv": 128,
         "window": 2640, "sinks": 880, "ragged": False},
        # one session's next token, a short window: latency
        {"name": "window step 1 session", "op": "attn_step", "B": 1, "Hq": 20, "Hkv": 20, "dk": 112, "dv": 112,
         "window": 880, "sinks": 16, "fresh": False},
        # a full server, shared key heads, a long window, some sessions not yet at its length
        {"name": "window step 64 sessions", "op": "attn_step", "B": 64, "Hq": 32, "Hkv": 8, "dk": 128, "dv": 128,
         "window": 4096, "sinks": 64, "fresh": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["conv", "conv_step", "scan", "scan", "scan_step", "attn", "attn", "attn_step", "attn_step"])
    while True:
        c = {"op": op}
        if op in ("conv", "conv_step", "scan", "scan_step"):
            c["type"] = rng.choice(["bf16", "bf16", "f32"])
            c["D"] = 8 * _log(rng, 16, 640)
            c["B"] = _log(rng, 1, 300) if op.endswith("step") else _log(rng, 1, 12)
            if op.startswith("conv"):
                c["W"] = rng.choice([2, 3, 4])
            else:
                c["N"] = rng.choice([8, 16, 16, 32, 64])
            if not op.endswith("step"):
                c["T"] = _log(rng, 1, 27000)
                c["ragged"] = c["B"] > 1 and rng.random() < 0.5
        else:
            c["Hkv"] = rng.choice([1, 2, 4, 5, 8, 16, 20])
            c["Hq"] = c["Hkv"] * rng.choice([1, 1, 2, 3, 4, 5, 7, 8])
            c["dk"] = rng.choice([32, 64, 80, 96, 112, 128, 128])
            c["dv"] = c["dk"] if rng.random() < 0.8 else rng.choice([48, 64, 112, 128])
            c["window"] = _log(rng, 1, 6000)
            c["sinks"] = rng.choice([0, 0, 1, 4, 64, 300, 880])
            if op == "attn":
                c["B"] = _log(rng, 1, 6)
                c["T"] = _log(rng, 1, 20000)
                c["ragged"] = c["B"] > 1 and rng.random() < 0.5
            else:
                c["B"] = _log(rng, 1, 100)
                c["fresh"] = rng.random() < 0.5
        # no dearer than the largest listed case of its kind
        top = [work(x) for x in listed() if x["op"] == op]
        if op == "conv_step":
            top = [work(x) for x in listed() if x["op"] == "scan_step"]
        w = work(c)
        if w["bytes"] <= max(t["bytes"] for t in top) and w["flops"] <= max(t["flops"] for t in top):
            return c


def _pairs(T, window, sinks):
    """Visible (query, key) pairs of one sequence of T tokens: the window, and the sinks before it."""
    w = min(window, T)
    near = w * (w + 1) // 2 + (T - w) * window
    past = max(0, T - window)                     # the last `past` queries see keys 0 .. past-1 outside the window
    s = min(sinks, past)
    return near + s * (s + 1) // 2 + (past - s) * sinks


def work(case):
    op, B = case["op"], case["B"]
    if op in ("conv", "conv_step"):
        e = 2 if case["type"] == "bf16" else 4
        D, W, T = case["D"], case["W"], case.get("T", 1)
        return {"bytes": 2 * B * T * D * e + 2 * B * (W - 1) * D * e + 4 * D * (W + 1), "flops": B * T * D * (2 * W + 5)}
    if op in ("scan", "scan_step"):
        e = 2 if case["type"] == "bf16" else 4
        D, N, T = case["D"], case["N"], case.get("T", 1)
        return {"bytes": B * T * (4 * D + 2 * N) * e + 2 * 4 * B * D * N + 4 * D * (N + 2),
                "flops": B * T * D * (7 * N + 14)}
    Hq, Hkv, dk, dv = case["Hq"], case["Hkv"], case["dk"], case["dv"]
    if op == "attn":
        T = case["T"]
        kept = min(T, case["window"] + case["sinks"])
        return {"bytes": 2 * B * T * (Hq + Hkv) * (dk + dv) + 2 * B * kept * Hkv * (dk + dv),
                "flops": 2 * B * Hq * (dk + dv) * _pairs(T, case["window"], case["sinks"])}
    seen = (case["window"] + case["sinks"]) * (0.75 if case["fresh"] else 1.0)
    return {"bytes": 2 * B * Hkv * (dk + dv) * (seen + 2) + 2 * B * Hq * (dk + dv),
            "flops": 2 * B * Hq * (dk + dv) * seen}


# ------------------------------------------------------------------------------------- inputs

def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    op, B = case["op"], case["B"]

    def normal(*shape, std=1.0, to=torch.float32):
        return torch.empty(shape, dtype=torch.float32, device=dev).normal_(0.0, std, generator=g).to(to)

    def whole(lo, hi, n):
        return torch.randint(lo, hi, (n,), generator=g, device=dev, dtype=torch.int32)

    s = {"op": op}
    if op in ("conv", "conv_step"):
        t, D, W = TYPES[case["type"]], case["D"], case["W"]
        s.update(weight=normal(D, W, std=0.5), bias=normal(D, std=0.1), state=normal(B, W - 1, D, to=t))
        if op == "conv":
            # the activation is one half of a projection's output rows, as a mixer's input is
            s["x"] = normal(B, case["T"], 2 * D, to=t)[:, :, :D]
            s["lengths"] = whole(1, case["T"] + 1, B) if case["ragged"] else None
        else:
            s["x"] = normal(B, D, to=t)
        return s
    if op in ("scan", "scan_step"):
        t, D, N = TYPES[case["type"]], case["D"], case["N"]
        u = torch.rand(D, generator=g, device=dev)
        step = torch.exp(math.log(1e-3) + u * (math.log(0.1) - math.log(1e-3)))     # typical step sizes
        s["dt_bias"] = step + torch.log(-torch.expm1(-step))                        # softplus(dt_bias) = step
        s["A"] = -torch.arange(1, N + 1, device=dev, dtype=torch.float32) * torch.exp(normal(D, N, std=0.2))
        s["D"] = normal(D, std=0.5) + 1.0
        s["state"] = normal(B, D, N, std=0.3)
        lead = (B, case["T"]) if op == "scan" else (B,)
        s["x"] = torch.nn.functional.silu(normal(*lead, D)).to(t)
        s["dt"] = normal(*lead, D, std=0.7, to=t)
        s["z"] = normal(*lead, D, to=t)
        s["Bm"], s["Cm"] = normal(*lead, N, to=t), normal(*lead, N, to=t)
        if op == "scan":
            s["lengths"] = whole(1, case["T"] + 1, B) if case["ragged"] else None
        return s
    t = torch.bfloat16
    Hq, Hkv, dk, dv, window, sinks = (case[n] for n in ("Hq", "Hkv", "dk", "dv", "window", "sinks"))
    s.update(window=window, sinks=sinks)
    cap = window + sinks
    sharp = 0.5 + 2.5 * torch.rand(Hq, 1, generator=g, device=dev)                  # flat and peaked heads
    if op == "attn":
        T = case["T"]
        s["q"] = (normal(B, T, Hq, dk) * sharp).to(t)
        s["k"], s["v"] = normal(B, T, Hkv, dk, to=t), normal(B, T, Hkv, dv, to=t)
        s["lengths"] = whole(1, T + 1, B) if case["ragged"] else None
        s["k_cache"] = torch.zeros(B, cap, Hkv, dk, dtype=t, device=dev)
        s["v_cache"] = torch.zeros(B, cap, Hkv, dv, dtype=t, device=dev)
        return s
    s["q"] = (normal(B, Hq, dk) * sharp).to(t)
    s["k"], s["v"] = normal(B, Hkv, dk, to=t), normal(B, Hkv, dv, to=t)
    s["k_cache"], s["v_cache"] = normal(B, cap, Hkv, dk, to=t), normal(B, cap, Hkv, dv, to=t)
    s["pos"] = whole(cap // 2, cap, B) if case["fresh"] else whole(cap, 5 * cap, B)
    return s


# ------------------------------------------------------------------------------------- the library's calls

def _run_own(s):
    import hybrid_linear_attention_frame_b200 as G
    op = s["op"]
    if op == "conv":
        return G.causal_conv(s["x"], s["weight"], s["bias"], s["state"], lengths=s["lengths"])
    if op == "conv_step":
        return G.causal_conv_step(s["x"], s["weight"], s["bias"], s["state"]), s["state"]
    if op == "scan":
        return G.selective_scan(s["x"], s["dt"], s["A"], s["Bm"], s["Cm"], s["D"], s["z"], s["dt_bias"], s["state"],
                                lengths=s["lengths"])
    if op == "scan_step":
        y = G.selective_scan_step(s["x"], s["dt"], s["A"], s["Bm"], s["Cm"], s["state"], s["D"], s["z"], s["dt_bias"])
        return y, s["state"]
    if op == "attn":
        out = G.window_attention(s["q"], s["k"], s["v"], s["window"], s["sinks"], lengths=s["lengths"])
        G.window_cache_append(s["k"], s["v"], s["k_cache"], s["v_cache"], None, s["window"], s["sinks"],
                              lengths=s["lengths"])
        return out, s["k_cache"], s["v_cache"]
    out = G.window_attention_step(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["pos"], s["window"], s["sinks"])
    return out, s["k_cache"], s["v_cache"]


# ------------------------------------------------------------------------------------- the plain forms

def _conv(x, weight, bias, state, lengths):
    B, T, D = x.shape
    W = weight.shape[1]
    rows = torch.cat([state, x], 1)                                 # row t + W - 1 is token t
    acc = bias.expand(B, T, D)
    for j in range(W):
        acc = acc + rows[:, j:j + T].float() * weight[:, j]
    y = (acc * torch.sigmoid(acc)).to(x.dtype)
    if lengths is None:
        return y, rows[:, T:].clone()
    y = y * (torch.arange(T, device=x.device) < lengths[:, None])[:, :, None]
    at = lengths.long()[:, None] + torch.arange(W - 1, device=x.device)
    return y, torch.gather(rows, 1, at[:, :, None].expand(B, W - 1, D))


def _softplus(x):
    return torch.clamp(x, min=0) + torch.log1p(torch.exp(-x.abs()))


def _scan(x, dt, A, Bm, Cm, D, z, dt_bias, state, lengths):
    B, T, _ = x.shape
    delta = _softplus(dt.float() + dt_bias)
    if lengths is not None:                                         # a padded token leaves the state as it is
        live = (torch.arange(T, device=x.device) < lengths[:, None])[:, :, None]
        delta = delta * live
    a = torch.exp(delta[..., None] * A)
    h = (delta * x.float())[..., None] * Bm.float()[:, :, None, :]
    h[:, 0] += a[:, 0] * state
    k = 1
    while k < T:                                                    # inclusive scan of (a, h) by doubling
        h[:, k:] += a[:, k:] * h[:, :-k]
        if 2 * k < T:
            a[:, k:] = a[:, k:] * a[:, :-k]
        k *= 2
    y = (h * Cm.float()[:, :, None, :]).sum(-1) + D * x.float()
    zf = z.float()
    y = (y * zf * torch.sigmoid(zf)).to(x.dtype)
    return (y if lengths is None else y * live), h[:, -1].clone()


def _visible(pos, keys, window, sinks):
    return (keys <= pos) & ((keys > pos - window) | (keys < sinks))


def _attend(q, k, v, seen, scale):
    """q [B, t, Hq, dk], k and v [B, s, Hkv, .], seen [t, s] or [B, 1, 1, t, s]: float32 [B, t, Hq, dv]."""
    B, t, Hq, dk = q.shape
    Hkv = k.shape[2]
    qf = q.float().view(B, t, Hkv, Hq // Hkv, dk).permute(0, 2, 3, 1, 4)
    w = (qf @ k.float().permute(0, 2, 3, 1)[:, :, None]) * scale
    w = torch.exp(w.masked_fill_(~seen, -math.inf) - w.amax(-1, keepdim=True))
    o = (w @ v.float().permute(0, 2, 1, 3)[:, :, None]) / w.sum(-1, keepdim=True)
    return o.permute(0, 3, 1, 2, 4).reshape(B, t, Hq, -1)


def _attn(s):
    q, k, v, window, sinks, lengths = s["q"], s["k"], s["v"], s["window"], s["sinks"], s["lengths"]
    B, T = q.shape[:2]
    out = torch.empty(*q.shape[:3], v.shape[3], dtype=q.dtype, device=q.device)
    at = torch.arange(T, device=q.device)
    rows = 1024
    for t0 in range(0, T, rows):
        t1 = min(T, t0 + rows)
        lo = max(0, t0 - window + 1)
        keys = at[:t1] if lo <= sinks else torch.cat([at[:sinks], at[lo:t1]])
        kb, vb = (k[:, :t1], v[:, :t1]) if lo <= sinks else (k[:, keys], v[:, keys])
        seen = _visible(at[t0:t1, None], keys, window, sinks)
        out[:, t0:t1] = _attend(q[:, t0:t1], kb, vb, seen, q.shape[3] ** -0.5)
    if lengths is not None:
        out = out * (at < lengths[:, None])[:, :, None, None]
    # the rolling cache: token p in slot p while there is room, then in the window's turn; so slot c
    # ends up with the last token that has its turn, if there is one
    n = torch.full((B, 1), T, device=q.device) if lengths is None else lengths.long()[:, None]
    slot = torch.arange(window + sinks, device=q.device)
    last = torch.where(slot < sinks, slot, n - 1 - (n - 1 - slot) % window)
    held = ((last >= slot) & (last < n))[:, :, None, None]
    for cache, rows in ((s["k_cache"], k), (s["v_cache"], v)):
        got = rows[torch.arange(B, device=q.device)[:, None], last.clamp(0, T - 1)]
        cache.copy_(torch.where(held, got, cache))
    return out, s["k_cache"], s["v_cache"]


def _attn_step(s):
    q, kc, vc, window, sinks = s["q"], s["k_cache"], s["v_cache"], s["window"], s["sinks"]
    pos = s["pos"].long()
    b = torch.arange(len(pos), device=q.device)
    slot = torch.where(pos < sinks, pos, sinks + (pos - sinks) % window)
    kc[b, slot], vc[b, slot] = s["k"], s["v"]
    seen = torch.arange(kc.shape[1], device=q.device) <= pos[:, None]
    out = _attend(q[:, None], kc, vc, seen[:, None, None, None], q.shape[2] ** -0.5)
    return out[:, 0].to(q.dtype), kc, vc


def run(state):
    s = state
    if own:
        return _run_own(s)
    op = s["op"]
    if op == "conv":
        return _conv(s["x"], s["weight"], s["bias"], s["state"], s["lengths"])
    if op == "conv_step":
        y, new = _conv(s["x"][:, None], s["weight"], s["bias"], s["state"], None)
        s["state"].copy_(new)
        return y[:, 0], s["state"]
    if op in ("scan", "scan_step"):
        one = op == "scan_step"
        x, dt, z, Bm, Cm = ((s[n][:, None] if one else s[n]) for n in ("x", "dt", "z", "Bm", "Cm"))
        y, new = _scan(x, dt, s["A"], Bm, Cm, s["D"], z, s["dt_bias"], s["state"], None if one else s["lengths"])
        if one:
            s["state"].copy_(new)
            return y[:, 0], s["state"]
        return y, new
    return _attn(s) if op == "attn" else _attn_step(s)


# ------------------------------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op, B = s["op"], case["B"]
    d = {n: v.double() for n, v in s.items() if isinstance(v, torch.Tensor) and v.is_floating_point()}
    lengths = s.get("lengths")
    if op in ("conv", "conv_step"):
        x = d["x"] if op == "conv" else d["x"][:, None]
        T, W = x.shape[1], case["W"]
        rows = torch.cat([d["state"], x], 1)
        y = torch.einsum("btdw,dw->btd", rows.unfold(1, W, 1), d["weight"]) + d["bias"]
        y = y / (1 + torch.exp(-y))
        ends = [T] * B if lengths is None else lengths.tolist()
        for b, n in enumerate(ends):
            y[b, n:] = 0
        new = torch.stack([rows[b, n:n + W - 1] for b, n in enumerate(ends)])
        return (y, new) if op == "conv" else (y[:, 0], new)
    if op in ("scan", "scan_step"):
        one = op == "scan_step"
        x, dt, z, Bm, Cm = ((d[n][:, None] if one else d[n]) for n in ("x", "dt", "z", "Bm", "Cm"))
        T = x.shape[1]
        n = torch.full((B,), T, device=x.device) if lengths is None else lengths
        delta = torch.log(1 + torch.exp(dt + d["dt_bias"]))
        h, y = d["state"].clone(), torch.zeros_like(x)
        for t in range(T):                                          # the recurrence, token by token
            new = torch.exp(delta[:, t, :, None] * d["A"]) * h + (delta[:, t] * x[:, t])[:, :, None] * Bm[:, t, None, :]
            on = (t < n)[:, None, None]
            h = torch.where(on, new, h)
            y[:, t] = torch.where(on[:, :, 0], (h @ Cm[:, t, :, None])[:, :, 0] + d["D"] * x[:, t], 0.0)
        y = y * (z / (1 + torch.exp(-z)))
        return (y[:, 0], h) if one else (y, h)
    Hq, Hkv, window, sinks = case["Hq"], case["Hkv"], case["window"], case["sinks"]
    G, scale = Hq // Hkv, 1 / math.sqrt(case["dk"])
    if op == "attn_step":
        out = torch.empty(B, Hq, case["dv"], dtype=torch.float64, device="cuda")
        kc, vc = d["k_cache"], d["v_cache"]
        for b, p in enumerate(s["pos"].tolist()):
            at = p if p < sinks else sinks + (p - sinks) % window
            kc[b, at], vc[b, at] = d["k"][b], d["v"][b]
            m = min(window + sinks, p + 1)
            for h in range(Hkv):
                w = torch.softmax(d["q"][b, h * G:(h + 1) * G] @ kc[b, :m, h].T * scale, -1)
                out[b, h * G:(h + 1) * G] = w @ vc[b, :m, h]
        return out, kc, vc
    T = case["T"]
    out = torch.zeros(B, T, Hq, case["dv"], dtype=torch.float64, device="cuda")
    kc, vc = d["k_cache"], d["v_cache"]
    for b in range(B):
        n = T if lengths is None else int(lengths[b])
        for t0 in range(0, n, 512):
            t1 = min(n, t0 + 512)
            first = max(0, t0 - window + 1)
            keys = torch.tensor(sorted(set(range(min(sinks, t1))) | set(range(first, t1))), device="cuda")
            at = torch.arange(t0, t1, device="cuda")[:, None]
            hidden = (keys > at) | ((keys <= at - window) & (keys >= sinks))
            for h in range(Hkv):
                kb, vb = d["k"][b, keys, h], d["v"][b, keys, h]
                w = torch.einsum("tgd,sd->gts", d["q"][b, t0:t1, h * G:(h + 1) * G], kb) * scale
                w = torch.softmax(w.masked_fill(hidden, -math.inf), -1)
                out[b, t0:t1, h * G:(h + 1) * G] = torch.einsum("gts,sd->tgd", w, vb)
        for p in range(max(0, n - window) if sinks <= n - window else 0, n):
            at = p if p < sinks else sinks + (p - sinks) % window
            kc[b, at], vc[b, at] = d["k"][b, p], d["v"][b, p]
        for p in range(min(sinks, n)):
            kc[b, p], vc[b, p] = d["k"][b, p], d["v"][b, p]
    return out, kc, vc

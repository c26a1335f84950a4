"""Tensor-level calls of the other sequence mixers: causal convolution, selective scan, and
sliding-window attention with its rolling cache.

Each checks shapes, types and devices, allocates its outputs through PyTorch and makes one
library call on the current stream of the tensors' device; all arithmetic happens in the
library's CUDA kernels.  Activations may be slices of wider rows (contiguous in their last
dimension); padded batches take ``lengths`` (int32 [B] on the device), and rows past a
sequence's length come back as zeros, or as they were when ``out`` is given.
"""

import ctypes

from . import gdn as _gdn

_I, _L, _P, _F = ctypes.c_int, ctypes.c_longlong, ctypes.c_void_p, ctypes.c_float

_CONV = [_P, _L, _L, _P, _P, _P, _P, _P, _P] + [_I] * 5 + [_P]
_CONV_STEP = [_P, _L, _P, _P, _P, _P] + [_I] * 4 + [_P]
_SCAN = [_P, _L, _L] * 2 + [_P] + [_P, _L, _L] * 2 + [_P] + [_P, _L, _L] + [_P] * 5 + [_I] * 5 + [_P]
_SCAN_STEP = [_P, _L] * 2 + [_P] + [_P, _L] * 2 + [_P, _P, _L] + [_P] * 3 + [_I] * 4 + [_P]

_WINDOW_STEP = [_P, _L] * 3 + [_P] * 4 + [_I] * 7 + [_F, _P]

_ARGTYPES = {
    "gdn_causal_conv": _CONV, "gdn_causal_conv_f32": _CONV,
    "gdn_causal_conv_step": _CONV_STEP, "gdn_causal_conv_step_f32": _CONV_STEP,
    "gdn_selective_scan": _SCAN, "gdn_selective_scan_f32": _SCAN,
    "gdn_selective_scan_step": _SCAN_STEP, "gdn_selective_scan_step_f32": _SCAN_STEP,
    "gdn_window_attention": [_P, _L, _L, _L] * 3 + [_P, _P] + [_I] * 9 + [_F, _P],
    "gdn_window_cache_append": [_P, _L, _L] * 2 + [_P] * 4 + [_I] * 7 + [_P],
    "gdn_window_attention_step": _WINDOW_STEP, "gdn_window_attention_step_zero_idle": _WINDOW_STEP,
}

_fns = {}
_torch = None


def _fn(name):
    """The library's entry, with its argument types set (and torch at hand: callers hold tensors)."""
    global _torch
    f = _fns.get(name)
    if f is None:
        import torch
        _torch = torch
        f = getattr(_gdn.load(), name)
        f.argtypes, f.restype = _ARGTYPES[name], _I
        _fns[name] = f
    return f


def _call(name, device, *args):
    """One library call on the current stream of ``device`` (made current for it)."""
    f, cuda, index = _fn(name), _torch.cuda, device.index
    if index == cuda.current_device():
        st = f(*args, _torch._C._cuda_getCurrentRawStream(index))
    else:
        with cuda.device(index):
            st = f(*args, _torch._C._cuda_getCurrentRawStream(index))
    if st:
        raise _gdn.GdnError(st, name)


def _need(cond, what):
    if not cond:
        raise ValueError(what)


def _sizes(*n):
    """ctypes would cut a larger number to its low 32 bits."""
    _need(-2 ** 31 <= min(n) and max(n) < 2 ** 31, "a size, window or sink count exceeds 32 bits")


def _mismatch(t, name, shape, dtype, device):
    raise ValueError(f"{name}: expected {dtype} {tuple(shape)} on {device}, got {t.dtype} {tuple(t.shape)} on {t.device}")


def _rows(t, name, shape, dtype, device):
    """Pointer and strides of a tensor of this shape, type and device, contiguous in its last dimension."""
    if t.shape != shape or t.dtype is not dtype or t.device != device:
        _mismatch(t, name, shape, dtype, device)
    s = t.stride()
    if s[-1] != 1 and shape[-1] != 1:
        raise ValueError(f"{name} must be contiguous in its last dimension")
    return t.data_ptr(), s


def _whole(t, name, shape, dtype, device):
    """Pointer of a contiguous tensor of this shape, type and device; None stays None."""
    if t is None:
        return None
    if t.shape != shape or t.dtype is not dtype or t.device != device:
        _mismatch(t, name, shape, dtype, device)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _new(out, name, like, shape, dtype, lengths=None):
    """``out`` after its checks, or a new tensor on the device of ``like`` (zeros where padding stays)."""
    if out is None:
        return like.new_empty(shape, dtype=dtype) if lengths is None else like.new_zeros(shape, dtype=dtype)
    _need(out.device == like.device, f"{name} must be on {like.device}")
    _whole(out, name, shape, dtype, like.device)
    return out


def _types(t, name, entry):
    """The entry for a tensor's element type, bfloat16 or float32; its device and types."""
    _fn(entry)
    dtype, f32 = t.dtype, _torch.float32
    _need(t.is_cuda, f"{name} must be on a CUDA device")
    _need(dtype is f32 or dtype is _torch.bfloat16, f"{name} must be bfloat16 or float32, got {dtype}")
    return (entry + "_f32" if dtype is f32 else entry), t.device, dtype, f32, _torch.int32


def _bf16(t, name, entry):
    _fn(entry)
    dtype = _torch.bfloat16
    _need(t.is_cuda and t.dtype is dtype, f"{name} must be bfloat16 on a CUDA device")
    return t.device, dtype, _torch.int32


def causal_conv(x, weight, bias=None, state=None, silu=True, lengths=None, out=None, state_out=None):
    """out, state_out of the causal depthwise convolution of x [B, T, D] with weight [D, width]
    (float32, width 2 to 4); state [B, width - 1, D] holds the inputs before the call (None:
    zeros).  ``state_out`` may be ``state`` itself."""
    name, dev, ty, f32, i32 = _types(x, "x", "gdn_causal_conv")
    B, T, D = x.shape
    W = weight.shape[1]
    _sizes(B, T, D)
    xp, xs = _rows(x, "x", x.shape, ty, dev)
    wp, bp = _whole(weight, "weight", (D, W), f32, dev), _whole(bias, "bias", (D,), f32, dev)
    sp, lp = _whole(state, "state", (B, W - 1, D), ty, dev), _whole(lengths, "lengths", (B,), i32, dev)
    out = _new(out, "out", x, (B, T, D), ty, lengths)
    state_out = _new(state_out, "state_out", x, (B, W - 1, D), ty)
    _call(name, dev, xp, xs[0], xs[1], wp, bp, sp, state_out.data_ptr(), lp, out.data_ptr(), B, T, D, W, int(silu))
    return out, state_out


def causal_conv_step(x, weight, bias, state, silu=True, out=None):
    """out [B, D] for one token x [B, D]; state [B, width - 1, D] is advanced in place."""
    name, dev, ty, f32, _ = _types(x, "x", "gdn_causal_conv_step")
    B, D = x.shape
    W = weight.shape[1]
    _sizes(B, D)
    xp, xs = _rows(x, "x", x.shape, ty, dev)
    wp, bp = _whole(weight, "weight", (D, W), f32, dev), _whole(bias, "bias", (D,), f32, dev)
    sp = _whole(state, "state", (B, W - 1, D), ty, dev)
    out = _new(out, "out", x, (B, D), ty)
    _call(name, dev, xp, xs[0], wp, bp, sp, out.data_ptr(), B, D, W, int(silu))
    return out


def selective_scan(x, dt, A, Bm, Cm, D=None, z=None, dt_bias=None, state=None, dt_softplus=True, lengths=None,
                   out=None, state_out=None):
    """y [B, T, D], state_out [B, D, N] of the selective scan of x, dt, z [B, T, D] with A [D, N]
    (float32) and Bm, Cm [B, T, N]; state (float32 [B, D, N], None: zeros) may be ``state_out``."""
    name, dev, ty, f32, i32 = _types(x, "x", "gdn_selective_scan")
    B, T, E = x.shape
    N = A.shape[1]
    _sizes(B, T, E)
    xp, xs = _rows(x, "x", x.shape, ty, dev)
    dp, ds = _rows(dt, "dt", x.shape, ty, dev)
    bp, bs = _rows(Bm, "Bm", (B, T, N), ty, dev)
    cp, cs = _rows(Cm, "Cm", (B, T, N), ty, dev)
    zp, zs = (None, (0, 0)) if z is None else _rows(z, "z", x.shape, ty, dev)
    ap, kp = _whole(A, "A", (E, N), f32, dev), _whole(D, "D", (E,), f32, dev)
    tp, sp = _whole(dt_bias, "dt_bias", (E,), f32, dev), _whole(state, "state", (B, E, N), f32, dev)
    lp = _whole(lengths, "lengths", (B,), i32, dev)
    y = _new(out, "out", x, (B, T, E), ty, lengths)
    state_out = _new(state_out, "state_out", x, (B, E, N), f32)
    _call(name, dev, xp, xs[0], xs[1], dp, ds[0], ds[1], ap, bp, bs[0], bs[1], cp, cs[0], cs[1], kp, zp, zs[0], zs[1],
          tp, sp, state_out.data_ptr(), lp, y.data_ptr(), B, T, E, N, int(dt_softplus))
    return y, state_out


def selective_scan_step(x, dt, A, Bm, Cm, state, D=None, z=None, dt_bias=None, dt_softplus=True, out=None):
    """y [B, D] for one token (x, dt, z [B, D]; Bm, Cm [B, N]); state [B, D, N] advances in place."""
    name, dev, ty, f32, _ = _types(x, "x", "gdn_selective_scan_step")
    B, E = x.shape
    N = A.shape[1]
    _sizes(B, E)
    xp, xs = _rows(x, "x", x.shape, ty, dev)
    dp, ds = _rows(dt, "dt", x.shape, ty, dev)
    bp, bs = _rows(Bm, "Bm", (B, N), ty, dev)
    cp, cs = _rows(Cm, "Cm", (B, N), ty, dev)
    zp, zs = (None, (0,)) if z is None else _rows(z, "z", x.shape, ty, dev)
    ap, kp = _whole(A, "A", (E, N), f32, dev), _whole(D, "D", (E,), f32, dev)
    tp, sp = _whole(dt_bias, "dt_bias", (E,), f32, dev), _whole(state, "state", (B, E, N), f32, dev)
    y = _new(out, "out", x, (B, E), ty)
    _call(name, dev, xp, xs[0], dp, ds[0], ap, bp, bs[0], cp, cs[0], kp, zp, zs[0], tp, sp, y.data_ptr(), B, E, N,
          int(dt_softplus))
    return y


def window_attention(q, k, v, window, sinks=0, lengths=None, scale=None, out=None):
    """out [B, Tq, Hq, d_v]: softmax attention of q [B, Tq, Hq, d_k], the last Tq of the Tk tokens
    of k [B, Tk, Hkv, d_k] and v [B, Tk, Hkv, d_v], over each token's last ``window`` tokens
    (itself among them) and the first ``sinks``.  ``scale`` is 1 / sqrt(d_k) unless given."""
    dev, ty, i32 = _bf16(q, "q", "gdn_window_attention")
    B, Tq, Hq, dk = q.shape
    _, Tk, Hkv, dv = v.shape
    _sizes(B, Tk, Hq, window, sinks)
    qp, qs = _rows(q, "q", q.shape, ty, dev)
    kp, ks = _rows(k, "k", (B, Tk, Hkv, dk), ty, dev)
    vp, vs = _rows(v, "v", (B, Tk, Hkv, dv), ty, dev)
    lp = _whole(lengths, "lengths", (B,), i32, dev)
    out = _new(out, "out", q, (B, Tq, Hq, dv), ty, lengths)
    _call("gdn_window_attention", dev, qp, qs[0], qs[1], qs[2], kp, ks[0], ks[1], ks[2], vp, vs[0], vs[1], vs[2], lp,
          out.data_ptr(), B, Tq, Tk, Hq, Hkv, dk, dv, window, sinks, dk ** -0.5 if scale is None else scale)
    return out


def window_cache(B, Hkv, d_k, d_v, window, sinks=0, device="cuda"):
    """k_cache, v_cache for window_attention_step: [B, window + sinks, Hkv, d] bf16."""
    import torch
    return tuple(torch.empty((B, window + sinks, Hkv, d), dtype=torch.bfloat16, device=device) for d in (d_k, d_v))


def _token(t, name, shape, dtype, device):
    """As _rows, a token's heads contiguous."""
    p, s = _rows(t, name, shape, dtype, device)
    if s[-2] != shape[-1] and shape[-2] != 1:
        raise ValueError(f"{name}: a token's heads must be contiguous")
    return p, s


def window_cache_append(k, v, k_cache, v_cache, start, window, sinks=0, lengths=None):
    """Copy the tokens of k, v [B, T, Hkv, d] that stay visible into the rolling caches, as tokens
    start[b] .. of each session (``start`` int32 [B], None: 0)."""
    dev, ty, i32 = _bf16(k, "k", "gdn_window_cache_append")
    B, T, Hkv, dk = k.shape
    dv = v.shape[3]
    _sizes(B, T, Hkv, window, sinks)
    kp, ks = _token(k, "k", k.shape, ty, dev)
    vp, vs = _token(v, "v", (B, T, Hkv, dv), ty, dev)
    kc = _whole(k_cache, "k_cache", (B, window + sinks, Hkv, dk), ty, dev)
    vc = _whole(v_cache, "v_cache", (B, window + sinks, Hkv, dv), ty, dev)
    sp, lp = _whole(start, "start", (B,), i32, dev), _whole(lengths, "lengths", (B,), i32, dev)
    _call("gdn_window_cache_append", dev, kp, ks[0], ks[1], vp, vs[0], vs[1], kc, vc, sp, lp, B, T, Hkv, dk, dv, window,
          sinks)


def window_attention_step(q, k, v, k_cache, v_cache, pos, window, sinks=0, scale=None, out=None):
    """out [B, Hq, d_v] for one token per session: k, v [B, Hkv, d] go into the rolling caches as
    token pos[b] (int32 [B]) and q [B, Hq, d_k] attends over them.  pos[b] < 0 marks an idle
    session: its cache stays, its row of the result is zeros, or as it was when ``out`` is given."""
    name = "gdn_window_attention_step_zero_idle" if out is None else "gdn_window_attention_step"
    dev, ty, i32 = _bf16(q, "q", name)
    B, Hq, dk = q.shape
    _, Hkv, dv = v.shape
    _sizes(B, Hq, window, sinks)
    qp, qs = _token(q, "q", q.shape, ty, dev)
    kp, ks = _token(k, "k", (B, Hkv, dk), ty, dev)
    vp, vs = _token(v, "v", (B, Hkv, dv), ty, dev)
    kc = _whole(k_cache, "k_cache", (B, window + sinks, Hkv, dk), ty, dev)
    vc = _whole(v_cache, "v_cache", (B, window + sinks, Hkv, dv), ty, dev)
    pp = _whole(pos, "pos", (B,), i32, dev)
    out = _new(out, "out", q, (B, Hq, dv), ty)
    _call(name, dev, qp, qs[0], kp, ks[0], vp, vs[0], kc, vc, pp, out.data_ptr(), B, Hq, Hkv, dk,
          dv, window, sinks, dk ** -0.5 if scale is None else scale)
    return out

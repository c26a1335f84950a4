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

_ARGTYPES = {
    "gdn_causal_conv": _CONV, "gdn_causal_conv_f32": _CONV,
    "gdn_causal_conv_step": _CONV_STEP, "gdn_causal_conv_step_f32": _CONV_STEP,
    "gdn_selective_scan": _SCAN, "gdn_selective_scan_f32": _SCAN,
    "gdn_selective_scan_step": _SCAN_STEP, "gdn_selective_scan_step_f32": _SCAN_STEP,
    "gdn_window_attention": [_P, _L, _L, _L] * 3 + [_P, _P] + [_I] * 9 + [_F, _P],
    "gdn_window_cache_append": [_P, _L, _L] * 2 + [_P] * 4 + [_I] * 7 + [_P],
    "gdn_window_attention_step": [_P, _L] * 3 + [_P] * 4 + [_I] * 7 + [_F, _P],
}

_fns = {}


def _fn(name):
    f = _fns.get(name)
    if f is None:
        f = getattr(_gdn.load(), name)
        f.argtypes, f.restype = _ARGTYPES[name], _I
        _fns[name] = f
    return f


def _call(name, device, *args):
    """One library call on the current stream of ``device`` (made current for it)."""
    import torch
    index = device.index
    if index == torch.cuda.current_device():
        st = _fn(name)(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(index):
            st = _fn(name)(*args, torch._C._cuda_getCurrentRawStream(index))
    if st:
        raise _gdn.GdnError(st, name)


def _need(cond, what):
    if not cond:
        raise ValueError(what)


def _tensor(t, name, shape, dtype, device, contiguous=True):
    """``t`` has this shape, type and device, and rows contiguous in the last dimension."""
    if t.shape != shape or t.dtype is not dtype or t.device != device:
        raise ValueError(f"{name}: expected {dtype} {tuple(shape)} on {device}, "
                         f"got {t.dtype} {tuple(t.shape)} on {t.device}")
    if contiguous:
        _need(t.is_contiguous(), f"{name} must be contiguous")
    else:
        _need(t.stride(-1) == 1 or t.shape[-1] == 1, f"{name} must be contiguous in its last dimension")


def _opt(t, name, shape, dtype, device):
    if t is None:
        return None
    _tensor(t, name, shape, dtype, device)
    return t.data_ptr()


def _suffix(t, name):
    import torch
    _need(t.is_cuda, f"{name} must be on a CUDA device")
    if t.dtype is torch.bfloat16:
        return ""
    _need(t.dtype is torch.float32, f"{name} must be bfloat16 or float32, got {t.dtype}")
    return "_f32"


def _new(out, name, shape, dtype, device, lengths):
    import torch
    if out is not None:
        _tensor(out, name, shape, dtype, device)
        return out
    make = torch.empty if lengths is None else torch.zeros
    return make(shape, dtype=dtype, device=device)


def causal_conv(x, weight, bias=None, state=None, silu=True, lengths=None, out=None, state_out=None):
    """out, state_out of the causal depthwise convolution of x [B, T, D] with weight [D, width]
    (float32, width 2 to 4); state [B, width - 1, D] holds the inputs before the call (None:
    zeros).  ``state_out`` may be ``state`` itself."""
    import torch
    sfx = _suffix(x, "x")
    dev, dt = x.device, x.dtype
    B, T, D = x.shape
    W = weight.shape[1]
    _tensor(x, "x", x.shape, dt, dev, contiguous=False)
    _tensor(weight, "weight", (D, W), torch.float32, dev)
    out = _new(out, "out", (B, T, D), dt, dev, lengths)
    state_out = _new(state_out, "state_out", (B, W - 1, D), dt, dev, None)
    _call("gdn_causal_conv" + sfx, dev, x.data_ptr(), x.stride(0), x.stride(1), weight.data_ptr(),
          _opt(bias, "bias", (D,), torch.float32, dev), _opt(state, "state", (B, W - 1, D), dt, dev),
          state_out.data_ptr(), _opt(lengths, "lengths", (B,), torch.int32, dev), out.data_ptr(), B, T, D, W, int(silu))
    return out, state_out


def causal_conv_step(x, weight, bias, state, silu=True, out=None):
    """out [B, D] for one token x [B, D]; state [B, width - 1, D] is advanced in place."""
    import torch
    sfx = _suffix(x, "x")
    dev, dt = x.device, x.dtype
    B, D = x.shape
    W = weight.shape[1]
    _tensor(x, "x", x.shape, dt, dev, contiguous=False)
    _tensor(weight, "weight", (D, W), torch.float32, dev)
    _tensor(state, "state", (B, W - 1, D), dt, dev)
    out = _new(out, "out", (B, D), dt, dev, None)
    _call("gdn_causal_conv_step" + sfx, dev, x.data_ptr(), x.stride(0), weight.data_ptr(),
          _opt(bias, "bias", (D,), torch.float32, dev), state.data_ptr(), out.data_ptr(), B, D, W, int(silu))
    return out


def selective_scan(x, dt, A, Bm, Cm, D=None, z=None, dt_bias=None, state=None, dt_softplus=True, lengths=None,
                   out=None, state_out=None):
    """y [B, T, D], state_out [B, D, N] of the selective scan of x, dt, z [B, T, D] with A [D, N]
    (float32) and Bm, Cm [B, T, N]; state (float32 [B, D, N], None: zeros) may be ``state_out``."""
    import torch
    sfx = _suffix(x, "x")
    dev, ty = x.device, x.dtype
    B, T, E = x.shape
    N = A.shape[1]
    _tensor(x, "x", x.shape, ty, dev, contiguous=False)
    _tensor(dt, "dt", x.shape, ty, dev, contiguous=False)
    _tensor(A, "A", (E, N), torch.float32, dev)
    _tensor(Bm, "Bm", (B, T, N), ty, dev, contiguous=False)
    _tensor(Cm, "Cm", (B, T, N), ty, dev, contiguous=False)
    zp = (None, 0, 0)
    if z is not None:
        _tensor(z, "z", x.shape, ty, dev, contiguous=False)
        zp = (z.data_ptr(), z.stride(0), z.stride(1))
    y = _new(out, "out", (B, T, E), ty, dev, lengths)
    state_out = _new(state_out, "state_out", (B, E, N), torch.float32, dev, None)
    _call("gdn_selective_scan" + sfx, dev, x.data_ptr(), x.stride(0), x.stride(1), dt.data_ptr(), dt.stride(0),
          dt.stride(1), A.data_ptr(), Bm.data_ptr(), Bm.stride(0), Bm.stride(1), Cm.data_ptr(), Cm.stride(0),
          Cm.stride(1), _opt(D, "D", (E,), torch.float32, dev), *zp,
          _opt(dt_bias, "dt_bias", (E,), torch.float32, dev), _opt(state, "state", (B, E, N), torch.float32, dev),
          state_out.data_ptr(), _opt(lengths, "lengths", (B,), torch.int32, dev), y.data_ptr(), B, T, E, N,
          int(dt_softplus))
    return y, state_out


def selective_scan_step(x, dt, A, Bm, Cm, state, D=None, z=None, dt_bias=None, dt_softplus=True, out=None):
    """y [B, D] for one token (x, dt, z [B, D]; Bm, Cm [B, N]); state [B, D, N] advances in place."""
    import torch
    sfx = _suffix(x, "x")
    dev, ty = x.device, x.dtype
    B, E = x.shape
    N = A.shape[1]
    _tensor(x, "x", x.shape, ty, dev, contiguous=False)
    _tensor(dt, "dt", x.shape, ty, dev, contiguous=False)
    _tensor(A, "A", (E, N), torch.float32, dev)
    _tensor(Bm, "Bm", (B, N), ty, dev, contiguous=False)
    _tensor(Cm, "Cm", (B, N), ty, dev, contiguous=False)
    _tensor(state, "state", (B, E, N), torch.float32, dev)
    zp = (None, 0)
    if z is not None:
        _tensor(z, "z", x.shape, ty, dev, contiguous=False)
        zp = (z.data_ptr(), z.stride(0))
    y = _new(out, "out", (B, E), ty, dev, None)
    _call("gdn_selective_scan_step" + sfx, dev, x.data_ptr(), x.stride(0), dt.data_ptr(), dt.stride(0), A.data_ptr(),
          Bm.data_ptr(), Bm.stride(0), Cm.data_ptr(), Cm.stride(0), _opt(D, "D", (E,), torch.float32, dev), *zp,
          _opt(dt_bias, "dt_bias", (E,), torch.float32, dev), state.data_ptr(), y.data_ptr(), B, E, N,
          int(dt_softplus))
    return y


def _bf16(t, name):
    import torch
    _need(t.is_cuda and t.dtype is torch.bfloat16, f"{name} must be bfloat16 on a CUDA device")


def window_attention(q, k, v, window, sinks=0, lengths=None, scale=None, out=None):
    """out [B, Tq, Hq, d_v]: softmax attention of q [B, Tq, Hq, d_k], the last Tq of the Tk tokens
    of k [B, Tk, Hkv, d_k] and v [B, Tk, Hkv, d_v], over each token's last ``window`` tokens
    (itself among them) and the first ``sinks``.  ``scale`` is 1 / sqrt(d_k) unless given."""
    import torch
    _bf16(q, "q")
    dev, ty = q.device, q.dtype
    B, Tq, Hq, dk = q.shape
    _, Tk, Hkv, dv = v.shape
    _tensor(q, "q", q.shape, ty, dev, contiguous=False)
    _tensor(k, "k", (B, Tk, Hkv, dk), ty, dev, contiguous=False)
    _tensor(v, "v", (B, Tk, Hkv, dv), ty, dev, contiguous=False)
    out = _new(out, "out", (B, Tq, Hq, dv), ty, dev, lengths)
    _call("gdn_window_attention", dev, q.data_ptr(), q.stride(0), q.stride(1), q.stride(2), k.data_ptr(), k.stride(0),
          k.stride(1), k.stride(2), v.data_ptr(), v.stride(0), v.stride(1), v.stride(2),
          _opt(lengths, "lengths", (B,), torch.int32, dev), out.data_ptr(), B, Tq, Tk, Hq, Hkv, dk, dv, window, sinks,
          dk ** -0.5 if scale is None else scale)
    return out


def window_cache(B, Hkv, d_k, d_v, window, sinks=0, device="cuda"):
    """k_cache, v_cache for window_attention_step: [B, window + sinks, Hkv, d] bf16."""
    import torch
    return tuple(torch.empty((B, window + sinks, Hkv, d), dtype=torch.bfloat16, device=device) for d in (d_k, d_v))


def _heads_row(t, name):
    _need(t.stride(-2) == t.shape[-1] or t.shape[-2] == 1, f"{name}: a token's heads must be contiguous")


def window_cache_append(k, v, k_cache, v_cache, start, window, sinks=0, lengths=None):
    """Copy the tokens of k, v [B, T, Hkv, d] that stay visible into the rolling caches, as tokens
    start[b] .. of each session (``start`` int32 [B], None: 0)."""
    import torch
    _bf16(k, "k")
    dev, ty = k.device, k.dtype
    B, T, Hkv, dk = k.shape
    dv = v.shape[3]
    _tensor(k, "k", k.shape, ty, dev, contiguous=False)
    _tensor(v, "v", (B, T, Hkv, dv), ty, dev, contiguous=False)
    _heads_row(k, "k")
    _heads_row(v, "v")
    _tensor(k_cache, "k_cache", (B, window + sinks, Hkv, dk), ty, dev)
    _tensor(v_cache, "v_cache", (B, window + sinks, Hkv, dv), ty, dev)
    _call("gdn_window_cache_append", dev, k.data_ptr(), k.stride(0), k.stride(1), v.data_ptr(), v.stride(0),
          v.stride(1), k_cache.data_ptr(), v_cache.data_ptr(), _opt(start, "start", (B,), torch.int32, dev),
          _opt(lengths, "lengths", (B,), torch.int32, dev), B, T, Hkv, dk, dv, window, sinks)


def window_attention_step(q, k, v, k_cache, v_cache, pos, window, sinks=0, scale=None, out=None):
    """out [B, Hq, d_v] for one token per session: k, v [B, Hkv, d] go into the rolling caches as
    token pos[b] (int32 [B]; negative: an idle session) and q [B, Hq, d_k] attends over them."""
    import torch
    _bf16(q, "q")
    dev, ty = q.device, q.dtype
    B, Hq, dk = q.shape
    Hkv, dv = v.shape[1], v.shape[2]
    _tensor(q, "q", q.shape, ty, dev, contiguous=False)
    _tensor(k, "k", (B, Hkv, dk), ty, dev, contiguous=False)
    _tensor(v, "v", (B, Hkv, dv), ty, dev, contiguous=False)
    _heads_row(q, "q")
    _heads_row(k, "k")
    _heads_row(v, "v")
    _tensor(k_cache, "k_cache", (B, window + sinks, Hkv, dk), ty, dev)
    _tensor(v_cache, "v_cache", (B, window + sinks, Hkv, dv), ty, dev)
    _tensor(pos, "pos", (B,), torch.int32, dev)
    out = _new(out, "out", (B, Hq, dv), ty, dev, None)
    _call("gdn_window_attention_step", dev, q.data_ptr(), q.stride(0), k.data_ptr(), k.stride(0), v.data_ptr(),
          v.stride(0), k_cache.data_ptr(), v_cache.data_ptr(), pos.data_ptr(), out.data_ptr(), B, Hq, Hkv, dk, dv,
          window, sinks, dk ** -0.5 if scale is None else scale)
    return out

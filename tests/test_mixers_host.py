"""Refusals of the token-by-token mixers, without a GPU: the C entries check sizes, alignment,
strides and overlaps before any CUDA call (fake addresses, never dereferenced), the Python calls
check shapes, types and devices before the library is reached."""

import ctypes

import pytest
import torch

import hybrid_linear_attention_frame_b200 as G
from hybrid_linear_attention_frame_b200 import mixers

A = 1 << 24          # fake 16-byte-aligned device addresses, 16 MiB apart
INV, UNS = G.GDN_ERR_INVALID_ARG, G.GDN_ERR_UNSUPPORTED


def at(i):
    return i * A


def entry(name, base, **kw):
    args = dict(base)
    assert set(kw) <= set(args)
    args.update(kw)
    return mixers._fn(name)(*args.values(), None)


CONV = dict(x=at(1), xb=64 * 32, xr=32, weight=at(2), bias=at(3), state_in=at(4), state_out=at(5), lengths=at(6),
            out=at(7), B=2, T=64, D=32, width=4, silu=1)


@pytest.mark.parametrize("name", ["gdn_causal_conv", "gdn_causal_conv_f32"])
@pytest.mark.parametrize("kw,expect", [
    (dict(x=None), INV), (dict(weight=None), INV), (dict(out=None), INV), (dict(B=0), INV), (dict(T=-1), INV),
    (dict(D=0), INV), (dict(silu=2), INV), (dict(width=1), UNS), (dict(width=5), UNS), (dict(D=12), UNS),
    (dict(B=65536), UNS), (dict(x=at(1) + 8), INV), (dict(out=at(7) + 4), INV), (dict(state_in=at(4) + 8), INV),
    (dict(lengths=at(6) + 2), INV), (dict(weight=at(2) + 4), INV), (dict(bias=at(3) + 8), INV), (dict(xr=31), INV), (dict(xr=33), INV), (dict(xb=-64), INV),
    (dict(xr=1 << 60), INV), (dict(out=at(1) + 64), INV), (dict(out=at(4)), INV), (dict(out=at(5)), INV),
    (dict(state_out=at(1)), INV), (dict(state_out=at(4) + 16), INV), (dict(state_out=at(2)), INV),
])
def test_conv_refuses(name, kw, expect):
    assert entry(name, CONV, **kw) == expect


SCAN = dict(x=at(1), xb=64 * 32, xr=32, dt=at(2), db=64 * 32, dr=32, A=at(3), Bm=at(4), bb=64 * 16, br=16, Cm=at(5),
            cb=64 * 16, cr=16, skip=at(6), z=at(7), zb=64 * 32, zr=32, dt_bias=at(8), state_in=at(9),
            state_out=at(10), lengths=at(11), y=at(12), B=2, T=64, D=32, N=16, softplus=1)


@pytest.mark.parametrize("name", ["gdn_selective_scan", "gdn_selective_scan_f32"])
@pytest.mark.parametrize("kw,expect", [
    (dict(x=None), INV), (dict(dt=None), INV), (dict(A=None), INV), (dict(Bm=None), INV), (dict(Cm=None), INV),
    (dict(y=None), INV), (dict(B=0), INV), (dict(T=-1), INV), (dict(D=0), INV), (dict(N=0), INV),
    (dict(softplus=3), INV), (dict(N=12), UNS), (dict(N=128), UNS), (dict(D=20), UNS), (dict(B=65536), UNS),
    (dict(z=at(7) + 2), INV), (dict(Cm=at(5) + 8), INV), (dict(A=at(3) + 4), INV), (dict(br=15), INV),
    (dict(cr=18), INV), (dict(zr=16), INV), (dict(state_out=at(9) + 64), INV), (dict(state_out=at(4)), INV),
    (dict(y=at(1)), INV), (dict(y=at(7) + 32), INV), (dict(y=at(10)), INV), (dict(skip=at(6) + 1), INV),
])
def test_scan_refuses(name, kw, expect):
    assert entry(name, SCAN, **kw) == expect


ATTN = dict(q=at(1), qb=64 * 4 * 32, qr=4 * 32, qh=32, k=at(2), kb=64 * 2 * 32, kr=64, kh=32, v=at(3), vb=64 * 2 * 32,
            vr=64, vh=32, lengths=at(4), out=at(5), B=2, Tq=64, Tk=64, Hq=4, Hkv=2, dk=32, dv=32, window=8, sinks=2,
            scale=0.5)


@pytest.mark.parametrize("kw,expect", [
    (dict(q=None), INV), (dict(k=None), INV), (dict(v=None), INV), (dict(out=None), INV), (dict(B=0), INV),
    (dict(Hq=3), INV), (dict(Hkv=0), INV), (dict(Tq=-1), INV), (dict(Tq=65), INV), (dict(window=0), INV),
    (dict(sinks=-1), INV), (dict(scale=0.0), INV), (dict(scale=float("nan")), INV), (dict(scale=float("inf")), INV),
    (dict(scale=-1.0), INV), (dict(dk=24), UNS), (dict(dk=144), UNS), (dict(dv=8), UNS), (dict(B=65536), UNS),
    (dict(Tq=64, Tk=2 ** 31 - 1), UNS), (dict(q=at(1) + 8), INV), (dict(out=at(5) + 8), INV), (dict(qr=100), INV),
    (dict(kh=16), INV), (dict(vb=8), INV), (dict(kr=1 << 40), UNS), (dict(out=at(2)), INV), (dict(lengths=at(4) + 1), INV),
])
def test_window_attention_refuses(kw, expect):
    assert entry("gdn_window_attention", ATTN, **kw) == expect


APPEND = dict(k=at(1), kb=64 * 64, kr=64, v=at(2), vb=64 * 64, vr=64, k_cache=at(3), v_cache=at(4), start=at(5),
              lengths=at(6), B=2, T=64, Hkv=2, dk=32, dv=32, window=8, sinks=2)


@pytest.mark.parametrize("kw,expect", [
    (dict(k=None), INV), (dict(v_cache=None), INV), (dict(B=0), INV), (dict(T=-1), INV), (dict(window=0), INV),
    (dict(sinks=-1), INV), (dict(dk=40), UNS), (dict(window=2 ** 31 - 1, sinks=1), UNS), (dict(k=at(1) + 8), INV),
    (dict(kr=56), INV), (dict(vr=68), INV), (dict(k_cache=at(4)), INV), (dict(k_cache=at(1) + 1024), INV),
    (dict(start=at(5) + 2), INV),
])
def test_append_refuses(kw, expect):
    assert entry("gdn_window_cache_append", APPEND, **kw) == expect


STEP = dict(q=at(1), qb=128, k=at(2), kb=64, v=at(3), vb=64, k_cache=at(4), v_cache=at(5), pos=at(6), out=at(7), B=2,
            Hq=4, Hkv=2, dk=32, dv=32, window=8, sinks=2, scale=0.5)


@pytest.mark.parametrize("kw,expect", [
    (dict(q=None), INV), (dict(k_cache=None), INV), (dict(pos=None), INV), (dict(out=None), INV), (dict(Hq=5), INV),
    (dict(window=0), INV), (dict(scale=0.0), INV), (dict(dv=136), UNS), (dict(window=2 ** 31 - 1), UNS),
    (dict(qb=132), INV), (dict(kb=66), INV), (dict(out=at(4) + 64), INV), (dict(k_cache=at(5)), INV),
    (dict(pos=at(6) + 1), INV), (dict(v=at(3) + 4), INV), (dict(out=at(1)), INV),
])
def test_step_refuses(kw, expect):
    assert entry("gdn_window_attention_step", STEP, **kw) == expect


def test_step_entries_need_a_state():
    assert mixers._fn("gdn_causal_conv_step")(at(1), 32, at(2), None, None, at(3), 1, 32, 4, 1, None) == INV
    assert mixers._fn("gdn_selective_scan_step")(at(1), 32, at(2), 32, at(3), at(4), 16, at(5), 16, None, None, 0, None,
                                                 None, at(6), 1, 32, 16, 1, None) == INV


def test_python_calls_refuse_host_tensors():
    x, w = torch.zeros(1, 4, 16), torch.zeros(16, 4)
    with pytest.raises(ValueError, match="CUDA"):
        G.causal_conv(x, w)
    with pytest.raises(ValueError, match="CUDA"):
        G.selective_scan(x, x, torch.zeros(16, 8), torch.zeros(1, 4, 8), torch.zeros(1, 4, 8))
    q = torch.zeros(1, 4, 2, 16, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        G.window_attention(q, q, q, 4)
    with pytest.raises(ValueError, match="CUDA"):
        G.window_attention_step(q[:, 0], q[:, 0], q[:, 0], q, q, torch.zeros(1, dtype=torch.int32), 4)


def test_argument_lists_match_the_header():
    """Every bound entry has as many arguments as its declaration."""
    import re
    from test_abi_host import HEADER
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    for name, types in mixers._ARGTYPES.items():
        decl = re.search(name + r"\(([^)]*)\)", src).group(1).split(",")
        assert len(decl) == len(types), name
        for d, t in zip(decl, types):
            d = d.strip()
            want = (ctypes.c_void_p if "*" in d or d.startswith("cudaStream_t") else
                    ctypes.c_longlong if d.startswith("long long") else
                    ctypes.c_float if d.startswith("float") else ctypes.c_int)
            assert t is want, (name, d)


@pytest.mark.parametrize("kw,expect", [
    (dict(q=None), INV), (dict(pos=None), INV), (dict(out=at(4) + 64), INV), (dict(window=0), INV), (dict(dv=136), UNS),
])
def test_step_with_zeros_for_idle_sessions_refuses(kw, expect):
    assert entry("gdn_window_attention_step_zero_idle", STEP, **kw) == expect


@pytest.mark.parametrize("name", ["gdn_selective_scan", "gdn_selective_scan_f32"])
def test_scan_refuses_channels_that_a_rounded_up_int_cannot_count(name):
    args = dict(SCAN, B=1, T=1, D=2 ** 31 - 8, lengths=None, state_in=None, state_out=None, z=None)
    assert mixers._fn(name)(*args.values(), None) == UNS

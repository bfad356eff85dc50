"""Refusals of the layer operators, on the CPU: the C entry points reject bad
arguments before any launch (fake pointers, never dereferenced), and the
binding rejects mis-shaped tensors by name before any library call (meta
tensors)."""
import ctypes

import pytest
import torch

import gated_deltanet_amd as g
from gated_deltanet_amd import GdnError

OK, INVALID, UNSUPPORTED, MISALIGNED = 0, -1, -2, -3
A = 0x7F0000000000
STEP = 1 << 32
X, R, W, Y, O, P, S, WS = (A + i * STEP for i in range(8))
F32, BF16, F16, E4M3 = range(4)
NAN = float("nan")


@pytest.fixture(scope="module")
def lib():
    from gated_deltanet_amd import build
    import os
    if not os.path.exists(g.LIB_PATH):
        build.build(verbose=False)
    return g.load_library()


def _rc(fn, base, kw, lib):
    args = dict(base)
    args.update(kw)
    rc = fn(*args.values())
    assert (lib.gdn_last_error() != b"") == (rc != OK)
    return rc


def _norm(**kw):
    return dict(dict(x=X, residual=R, norm_w=W, eps=1e-6, r=O, y=Y, y_scale=None, rows=10, d=64,
                     it=BF16, ot=BF16, stream=None), **kw)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), INVALID), (dict(d=0), INVALID), (dict(d=32769), UNSUPPORTED),
    (dict(rows=1 << 31), INVALID), (dict(it=E4M3), UNSUPPORTED), (dict(it=7), UNSUPPORTED),
    (dict(ot=4), UNSUPPORTED), (dict(eps=-1.0), INVALID), (dict(eps=NAN), INVALID),
    (dict(x=None), INVALID), (dict(y=None), INVALID), (dict(residual=None), INVALID),
    (dict(ot=E4M3), INVALID),                      # no y_scale
    (dict(y_scale=S), INVALID),                    # y_scale without e4m3
    (dict(x=X + 8), MISALIGNED), (dict(residual=R + 2), MISALIGNED), (dict(norm_w=W + 4), MISALIGNED),
    (dict(y=Y + 8), MISALIGNED), (dict(r=O + 8), MISALIGNED),
    (dict(ot=E4M3, y_scale=S + 2), MISALIGNED),
    (dict(y=X), INVALID), (dict(y=R), INVALID), (dict(y=O), INVALID), (dict(y=W), INVALID),
    (dict(r=X + 16), INVALID), (dict(r=R + 640), INVALID),
    (dict(ot=E4M3, y_scale=Y + 16), INVALID),
])
def test_add_rmsnorm_refusals(lib, kw, code):
    assert _rc(lib.gdn_add_rmsnorm, _norm(), kw, lib) == code


def test_no_rows_need_no_tensors(lib):
    assert _rc(lib.gdn_add_rmsnorm, _norm(x=None, residual=None, r=None, y=None, rows=0), {}, lib) == OK
    assert lib.gdn_quantize_rows(None, None, None, 0, 64, BF16, None) == OK
    assert lib.gdn_linear(None, None, None, None, None, None, None, None, 0, 8, 8, 0, BF16, BF16,
                          None, 0, None) == OK


@pytest.mark.parametrize("args,code", [
    ((None, Y, S, 4, 64, BF16), INVALID), ((X, Y, None, 4, 64, BF16), INVALID),
    ((X, Y, S, 4, 64, E4M3), UNSUPPORTED), ((X, Y, S, 4, 40000, BF16), UNSUPPORTED),
    ((X, Y + 4, S, 4, 64, BF16), MISALIGNED), ((X, X + 64, S, 4, 64, BF16), INVALID),
    ((X, Y, Y + 128, 4, 64, BF16), INVALID), ((X, Y, S, -4, 64, BF16), INVALID),
])
def test_quantize_refusals(lib, args, code):
    assert lib.gdn_quantize_rows(*args, None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(dy=None), INVALID), (dict(r=None), INVALID), (dict(dx=None), INVALID),
    (dict(it=E4M3), UNSUPPORTED), (dict(gt=E4M3), UNSUPPORTED), (dict(d=32769), UNSUPPORTED),
    (dict(eps=NAN), INVALID), (dict(ws=None), INVALID), (dict(wb=16), INVALID),
    (dict(ws=WS + 16), MISALIGNED), (dict(dr=P + 8), MISALIGNED), (dict(dx=O + 2), MISALIGNED),
    (dict(dx=X), INVALID), (dict(dx=R), INVALID), (dict(dx=P + 16), INVALID),
    (dict(dw=O), INVALID), (dict(ws=O), INVALID), (dict(ws=X), INVALID),
])
def test_add_rmsnorm_bwd_refusals(lib, kw, code):
    base = dict(dy=X, r=R, dr=P, w=W, eps=1e-6, dx=O, dw=S, rows=10, d=64, it=BF16, gt=BF16,
                ws=WS, wb=1 << 20, stream=None)
    assert _rc(lib.gdn_add_rmsnorm_bwd, base, kw, lib) == code


LIN = dict(x=X, xs=None, w=W, ws_=None, bias=None, residual=R, pre=None, y=Y, M=100, N=64, K=128,
           act=0, it=BF16, ot=BF16, ws=WS, wb=1 << 30, stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), INVALID), (dict(N=0), INVALID), (dict(K=0), INVALID), (dict(M=1 << 31), INVALID),
    (dict(K=(1 << 22) + 8), INVALID), (dict(N=(1 << 22) + 8), INVALID),
    (dict(it=5), UNSUPPORTED), (dict(ot=E4M3), UNSUPPORTED), (dict(act=4), UNSUPPORTED),
    (dict(act=-1), UNSUPPORTED), (dict(x=None), INVALID), (dict(w=None), INVALID),
    (dict(y=None), INVALID), (dict(it=E4M3), INVALID), (dict(it=E4M3, xs=S), INVALID),
    (dict(xs=S, ws_=P), INVALID),
    (dict(x=X + 4), MISALIGNED), (dict(w=W + 8), MISALIGNED), (dict(bias=P + 4), MISALIGNED),
    (dict(it=E4M3, xs=S + 1, ws_=P), MISALIGNED), (dict(it=E4M3, xs=S, ws_=P + 4), MISALIGNED),
    (dict(y=X), INVALID), (dict(y=W), INVALID), (dict(y=R + 128), INVALID), (dict(pre=R), INVALID),
    (dict(pre=Y), INVALID), (dict(bias=Y + 16), INVALID), (dict(y=R, pre=R), INVALID),
    (dict(K=100, ws=None), INVALID), (dict(K=100, wb=64), INVALID),
    (dict(K=100, ws=WS + 16), MISALIGNED), (dict(K=100, ws=X), INVALID), (dict(K=100, ws=Y), INVALID),
])
def test_linear_refusals(lib, kw, code):
    assert _rc(lib.gdn_linear, LIN, kw, lib) == code


BWD = dict(dy=X, pre=P, x=R, w=W, dx=O, dw=Y, db=S, M=100, N=64, K=128, act=1, it=BF16, gt=BF16,
           ws=WS, wb=1 << 30, stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(dy=None), INVALID), (dict(pre=None), INVALID), (dict(x=None), INVALID),
    (dict(w=None), INVALID), (dict(it=E4M3), UNSUPPORTED), (dict(gt=E4M3), UNSUPPORTED),
    (dict(act=9), UNSUPPORTED), (dict(M=1 << 31), INVALID), (dict(N=0), INVALID),
    (dict(dx=O + 8), MISALIGNED), (dict(dw=Y + 8), MISALIGNED), (dict(db=S + 2), MISALIGNED),
    (dict(dx=X), INVALID), (dict(dw=W), INVALID), (dict(db=Y), INVALID), (dict(dw=O), INVALID),
    (dict(ws=None), INVALID), (dict(wb=256), INVALID), (dict(ws=WS + 32), MISALIGNED),
    (dict(ws=P), INVALID), (dict(ws=O), INVALID),
])
def test_linear_bwd_refusals(lib, kw, code):
    assert _rc(lib.gdn_linear_bwd, BWD, kw, lib) == code


def test_workspace_sizes(lib):
    assert lib.gdn_add_rmsnorm_bwd_workspace_size(0, 64) == 0
    assert lib.gdn_add_rmsnorm_bwd_workspace_size(-1, 64) == 0
    assert lib.gdn_add_rmsnorm_bwd_workspace_size(10, 1 << 20) == 0
    assert lib.gdn_linear_workspace_size(-1, 8, 8, BF16) == 0
    assert lib.gdn_linear_workspace_size(8, 8, 8, 9) == 0
    # rows that are no whole 16-byte vectors: padded copies of both operands
    assert lib.gdn_linear_workspace_size(100, 64, 100, BF16) >= (100 + 64) * 104 * 2
    assert lib.gdn_linear_bwd_workspace_size(100, 64, 128, 5, BF16, BF16) == 0
    assert lib.gdn_linear_bwd_workspace_size(100, 64, 128, 1, BF16, BF16) >= 100 * 64 * 2


# ---------------------------------------------------------------------------
# binding

bf, f32, e8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


def _t(shape, dtype=bf):
    return torch.empty(shape, dtype=dtype, device="meta")


def _raises(word, fn, *a, **kw):
    with pytest.raises(GdnError) as e:
        fn(*a, **kw)
    assert word in str(e.value), str(e.value)


def test_binding_norm_and_quantizer():
    x, w = _t((4, 8, 64)), _t((64,), f32)
    _raises("device", g.gdn_add_rmsnorm, x, w, x)
    _raises("norm_w", g.gdn_add_rmsnorm, x, _t((65,), f32))
    _raises("norm_w", g.gdn_add_rmsnorm, x, _t((64,)))
    _raises("residual", g.gdn_add_rmsnorm, x, w, _t((4, 8, 32)))
    _raises("residual", g.gdn_add_rmsnorm, x, w, _t((4, 8, 64), f32))
    _raises("r needs", g.gdn_add_rmsnorm, x, w, r=x)
    _raises("y_scale", g.gdn_add_rmsnorm, x, w, y_scale=_t((4, 8), f32))
    _raises("y_scale", g.gdn_add_rmsnorm, x, w, out_dtype=e8, y_scale=_t((32,), f32))
    _raises("y must", g.gdn_add_rmsnorm, x, w, y=_t((4, 8, 64), f32))
    _raises("dtype", g.gdn_add_rmsnorm, _t((4, 64), torch.float64))
    _raises("[..., d]", g.gdn_add_rmsnorm, _t(()))
    _raises("device", g.gdn_quantize_rows, x)
    _raises("y must", g.gdn_quantize_rows, x, y=x)
    _raises("dtype", g.gdn_quantize_rows, _t((4, 64), e8))
    _raises("contiguous", g.gdn_quantize_rows, _t((64, 4)).t())
    dy = _t((4, 8, 64), f32)
    _raises("device", g.gdn_add_rmsnorm_bwd, dy, x, w, dr=x)
    _raises("dy", g.gdn_add_rmsnorm_bwd, _t((4, 8, 63)), x, w)
    _raises("dr", g.gdn_add_rmsnorm_bwd, dy, x, w, dr=dy)
    _raises("dx", g.gdn_add_rmsnorm_bwd, dy, x, w, dx=dy)
    _raises("dnorm_w", g.gdn_add_rmsnorm_bwd, dy, x, w, dnorm_w=_t((64,)))


def test_binding_linear():
    x, w = _t((4, 8, 64)), _t((32, 64))
    _raises("device", g.gdn_linear, x, w, bias=_t((32,), f32), residual=_t((4, 8, 32)))
    _raises("w must", g.gdn_linear, x, _t((32, 65)))
    _raises("w must", g.gdn_linear, x, _t((64,)))
    _raises("w must", g.gdn_linear, x, _t((32, 64), f32))
    _raises("w must", g.gdn_linear, x, _t((0, 64)))
    _raises("bias", g.gdn_linear, x, w, bias=_t((32,)))
    _raises("residual", g.gdn_linear, x, w, residual=_t((4, 8, 64)))
    _raises("residual", g.gdn_linear, x, w, residual=_t((4, 8, 32)), out_dtype=f32)
    _raises("act", g.gdn_linear, x, w, act="tanh")
    _raises("act", g.gdn_linear, x, w, act=None)
    _raises("e4m3", g.gdn_linear, x, w, x_scale=_t((4, 8), f32), w_scale=_t((32,), f32))
    x8, w8 = _t((4, 8, 64), e8), _t((32, 64), e8)
    _raises("e4m3", g.gdn_linear, x8, w8)
    _raises("e4m3", g.gdn_linear, x8, w8, x_scale=_t((4, 8), f32))
    _raises("x_scale", g.gdn_linear, x8, w8, x_scale=_t((32,), f32), w_scale=_t((32,), f32))
    _raises("device", g.gdn_linear, x8, w8, x_scale=_t((4, 8), f32), w_scale=_t((32,), f32))
    _raises("dtype", g.gdn_linear, x, w, out_dtype=e8)
    _raises("pre", g.gdn_linear, x, w, pre=_t((4, 8, 31)))
    dy = _t((4, 8, 32), f32)
    _raises("device", g.gdn_linear_bwd, dy, x, w, pre=dy, act="silu")
    _raises("pre", g.gdn_linear_bwd, dy, x, w, act="silu")
    _raises("pre", g.gdn_linear_bwd, dy, x, w, pre=_t((4, 8, 32)), act="silu")
    _raises("dy", g.gdn_linear_bwd, _t((4, 8, 64)), x, w)
    _raises("dtype", g.gdn_linear_bwd, dy, x8, w8)
    _raises("dw", g.gdn_linear_bwd, dy, x, w, dw=_t((32, 64), f32))
    _raises("dx", g.gdn_linear_bwd, dy, x, w, dx=_t((32, 64)))
    _raises("dbias", g.gdn_linear_bwd, dy, x, w, dbias=_t((64,), f32))

"""The layer operators around the mixer (residual addition + RMSNorm, row
quantiser, matrix product with epilogue, their gradients) against plain
formulas in 64 bits.

Bounds are per element and counted from the arithmetic. u32 = 2^-24 is half a
step of fp32, U[t] that of an output type (one rounding on the way out). A sum
of R products taken in fp32 in any order is off by at most R u32 times the sum
of the products' magnitudes; the bounds allow twice that, since the matrix
cores may truncate where they align a group of products. An activation's slope
is at most 1.13 in magnitude, taken as 1.2, and its own evaluation is given
16 u32 of its argument and value.

With e4m3 inputs and a 16-bit output the 8-bit matrix instructions may be used:
of 8 products at a time each is cut off 13 bits below the largest's exponent,
so that a group's 7 smaller products are off by less than 2^-13 of the largest
each; summed over the groups that is at most 7 * 2^-13 times the sum of the
products' magnitudes.
"""
import math

import numpy as np
import pytest
import torch

import oracle
from tests.util import TOL, rel_l2

gpu = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16,
      "e4m3": torch.float8_e4m3fn}
u32 = 2.0 ** -24
U = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11, "e4m3": 2.0 ** -4}
# below the normal range a step no longer shrinks with the value
SUB = {"f32": 0.0, "bf16": 0.0, "f16": 2.0 ** -25, "e4m3": 2.0 ** -10}


def _g():
    import gated_deltanet_amd as g
    g.load_library()
    return g


def _gen(seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return gen


def _rand(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def _within(got, ref, bound, what):
    got, ref = got.double(), ref.double()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    over = (got - ref).abs() - bound
    assert torch.isfinite(got).all() or not torch.isfinite(ref).all(), what
    worst = float(over.max()) if over.numel() else -1.0
    assert worst <= 0.0, (what, "over the bound by", worst, "at", int(over.argmax()))


def _rounded(ref, err, t):
    """Bound after one rounding to t of a value that is off by at most err."""
    return err + U[t] * (ref.abs() + err) + SUB[t]


# ---------------------------------------------------------------------------
# norm


def _norm_ref(x, res, w, eps):
    r = x.double() + (res.double() if res is not None else 0.0)
    rs = 1.0 / torch.sqrt((r * r).mean(-1, keepdim=True) + eps)
    return r, rs, r * rs * (1.0 + (w.double() if w is not None else 0.0))


def _norm_err(ref, d):
    # sum of d squares (relative d u32), the root halves it, a few products
    return ref.abs() * (d / 2 + 16) * u32


WIDTHS = [1, 7, 8, 100, 128, 512, 513, 2048, 2050, 4099, 8192, 8200, 16384, 32768]


@gpu
@pytest.mark.parametrize("d", WIDTHS)
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("bf16", "e4m3"), ("f16", "f32"),
                                       ("f32", "f32"), ("f32", "e4m3"), ("f16", "f16")])
def test_add_rmsnorm(d, dtype, out):
    g = _g()
    gen = _gen(d)
    rows = 37 if d <= 8192 else 3
    x = (3.0 * _rand(gen, rows, d)).to(DT[dtype])
    res = _rand(gen, rows, d).to(DT[dtype])
    w = 0.3 * _rand(gen, d)
    for residual, weight in ((res, w), (None, None)):
        y, r, scale = g.gdn_add_rmsnorm(x, weight, residual, rms_eps=1e-6, out_dtype=DT[out])
        rr, _, yr = _norm_ref(x, residual, weight, 1e-6)
        err = _norm_err(yr, d)
        if residual is None:
            assert r is None
        else:
            _within(r, rr, _rounded(rr, u32 * rr.abs(), dtype), "r")
        if out == "e4m3":
            top = yr.abs().amax(-1, keepdim=True).clamp_min(1e-30)
            _within(scale, top[:, 0] / 448, (_norm_err(top, d) + 4 * u32 * top)[:, 0] / 448,
                    "scale")
            q = yr * 448 / top
            _within(y, q, _rounded(q, 2 * _norm_err(q, d) + 8 * u32 * q.abs(), "e4m3"), "y")
        else:
            assert scale is None
            _within(y, yr, _rounded(yr, err, out), "y")


@gpu
@pytest.mark.parametrize("rows", [0, 1, 2, 5, 1000])
def test_add_rmsnorm_rows_and_what_lies_behind_them(rows):
    """Nothing is written behind the last row, for every way rows share a workgroup."""
    g = _g()
    for d in (64, 72, 1000, 4096):
        gen = _gen(rows + d)
        x = _rand(gen, rows, d).bfloat16()
        res = _rand(gen, rows, d).bfloat16()
        back = {k: torch.full((rows * d + 4096,), 7.0, device="cuda").to(t)
                for k, t in (("y", torch.float8_e4m3fn), ("r", torch.bfloat16))}
        sc = torch.full((rows + 64,), 7.0, device="cuda")
        y, r = (back[k][:rows * d].view(rows, d) for k in ("y", "r"))
        g.gdn_add_rmsnorm(x, None, res, out_dtype=torch.float8_e4m3fn, y=y, r=r, y_scale=sc[:rows])
        y2, r2, sc2 = g.gdn_add_rmsnorm(x, None, res, out_dtype=torch.float8_e4m3fn)
        assert torch.equal(y.float(), y2.float()) and torch.equal(r, r2)
        assert torch.equal(sc[:rows], sc2)
        for t, n in ((back["y"], rows * d), (back["r"], rows * d), (sc, rows)):
            assert (t[n:].float() == 7.0).all()


@gpu
def test_add_rmsnorm_in_place_and_empty_rows():
    g = _g()
    gen = _gen(3)
    x, res = (_rand(gen, 33, 1000).bfloat16() for _ in range(2))
    x[5] = 0
    res[5] = 0
    y, r, _ = g.gdn_add_rmsnorm(x, None, res)
    assert (y[5] == 0).all() and (r[5] == 0).all()
    keep = res.clone()
    y2, r2, _ = g.gdn_add_rmsnorm(x, None, res, r=res)
    assert r2 is res and torch.equal(r, res) and torch.equal(y, y2)
    x2 = x.clone()
    y3, _, _ = g.gdn_add_rmsnorm(x2, None, keep, r=x2)
    assert torch.equal(r, x2) and torch.equal(y, y3)
    q, s = g.gdn_quantize_rows(torch.zeros(3, 100, device="cuda"))
    assert (q.float() == 0).all() and (s > 0).all() and torch.isfinite(s).all()


@gpu
@pytest.mark.parametrize("d", [64, 100, 1024, 4096, 9000])
def test_rows_with_infinities_and_nan(d):
    """A row's own values decide about its results; other rows keep theirs."""
    g = _g()
    gen = _gen(d)
    x = _rand(gen, 9, d)
    clean = x.clone()
    x[2, d // 2] = float("inf")
    x[4, d - 1] = float("nan")
    x[6, 0] = -float("inf")
    ok = [0, 1, 3, 5, 7, 8]
    for out in (torch.float32, torch.float8_e4m3fn):
        y, _, s = g.gdn_add_rmsnorm(x, out_dtype=out)
        y0, _, s0 = g.gdn_add_rmsnorm(clean, out_dtype=out)
        assert torch.equal(y.float()[ok], y0.float()[ok])
        # an infinity: mean is infinite, finite elements become 0, itself NaN
        assert torch.isnan(y.float()[4]).all()
        assert torch.isnan(y.float()[2, d // 2]) and torch.isnan(y.float()[6, 0])
        if s is not None:
            assert torch.isnan(s[[2, 4, 6]]).all() and torch.equal(s[ok], s0[ok])
        else:
            keep = torch.arange(d, device="cuda") != d // 2
            assert (y[2, keep] == 0).all()
    q, s = g.gdn_quantize_rows(x)
    q0, s0 = g.gdn_quantize_rows(clean)
    assert torch.equal(q.float()[ok], q0.float()[ok]) and torch.equal(s[ok], s0[ok])
    assert torch.isnan(s[4]) and torch.isinf(s[2]) and torch.isinf(s[6])
    assert torch.isnan(q.float()[4]).all() and torch.isnan(q.float()[2, d // 2])


@gpu
def test_quantize_rounds_to_nearest_even():
    """Every e4m3 value, every midpoint between neighbours and the values next
    to it: rows whose scale is exactly 1."""
    g = _g()
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float()
    vals = torch.unique(codes[torch.isfinite(codes)])
    mid = (vals[1:] + vals[:-1]) / 2
    x = torch.cat([vals, mid, torch.nextafter(mid, mid + 1), torch.nextafter(mid, mid - 1)]).cuda()
    q, s = g.gdn_quantize_rows(x[None])
    assert s.item() == 1.0
    assert torch.equal(q[0].float(), x.to(torch.float8_e4m3fn).float())


@gpu
@pytest.mark.parametrize("d", WIDTHS)
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_quantize_rows(d, dtype):
    g = _g()
    gen = _gen(d)
    x = (torch.exp(2.0 * _rand(gen, 21, 1)) * _rand(gen, 21, d)).to(DT[dtype])
    q, s = g.gdn_quantize_rows(x)
    top = x.double().abs().amax(-1).clamp_min(1e-30)
    _within(s, top / 448, top / 448 * 2 * u32, "scale")
    ref = x.double() * (448 / top)[:, None]
    _within(q, ref, _rounded(ref, 4 * u32 * ref.abs(), "e4m3"), "q")


def _norm_bwd_ref(dy, r, w, dr, eps):
    r, dy = r.double(), dy.double()
    d = r.shape[-1]
    rs = 1.0 / torch.sqrt((r * r).mean(-1, keepdim=True) + eps)
    g = dy * (1.0 + (w.double() if w is not None else 0.0))
    m = (g * r).mean(-1, keepdim=True)
    dx = rs * (g - r * rs * rs * m) + (dr.double() if dr is not None else 0.0)
    # magnitudes for the bounds
    mag = rs * (g.abs() + r.abs() * rs * rs * (g * r).abs().mean(-1, keepdim=True))
    return dx, (dy * r * rs).sum(0), (d + 32) * u32 * mag, (dy * r * rs).abs().sum(0)


@gpu
@pytest.mark.parametrize("rows,d", [(1, 1), (3, 7), (37, 64), (21, 513), (600, 100), (1500, 128),
                                    (70, 2048), (33, 4099), (700, 4096), (9, 8200), (3, 16384),
                                    (2, 32768), (0, 64)])
@pytest.mark.parametrize("dtype,gtype", [("bf16", "bf16"), ("f32", "f32"), ("f16", "f32")])
def test_add_rmsnorm_bwd(rows, d, dtype, gtype):
    g = _g()
    gen = _gen(rows + d)
    r = (2.0 * _rand(gen, rows, d)).to(DT[dtype])
    dy = _rand(gen, rows, d).to(DT[gtype])
    dr = _rand(gen, rows, d).to(DT[dtype])
    w = 0.3 * _rand(gen, d)
    for weight, back in ((w, dr), (None, None)):
        dx, dw = g.gdn_add_rmsnorm_bwd(dy, r, weight, dr=back)
        rx, rw, ex, mw = _norm_bwd_ref(dy, r, weight, back, 1e-6)
        _within(dx, rx, _rounded(rx, ex + 2 * u32 * rx.abs(), dtype), "dx")
        _within(dw, rw, (rows + d / 2 + 64) * u32 * mw, "dnorm_w")
    dx2, none = g.gdn_add_rmsnorm_bwd(dy, r, w, dr=dr, want_dnorm_w=False)
    keep = dr.clone()
    dx3, dw3 = g.gdn_add_rmsnorm_bwd(dy, r, w, dr=keep, dx=keep)
    assert none is None and torch.equal(dx2, dx3)


@gpu
def test_add_rmsnorm_bwd_against_differences():
    g = _g()
    gen = _gen(11)
    x, w, dy = _rand(gen, 4, 40), 0.3 * _rand(gen, 40), _rand(gen, 4, 40)
    dx, dw = g.gdn_add_rmsnorm_bwd(dy, x, w, rms_eps=0.1)

    def loss(xx, ww):
        return float((_norm_ref(xx, None, ww, 0.1)[2] * dy.double()).sum())

    h = 1e-5
    for i, j in ((0, 0), (1, 17), (3, 39)):
        e = torch.zeros(4, 40, dtype=torch.float64, device="cuda")
        e[i, j] = h
        num = (loss(x.double() + e, w) - loss(x.double() - e, w)) / (2 * h)
        assert abs(num - float(dx[i, j])) < 1e-5 * (1 + abs(num))
    for j in (0, 21):
        e = torch.zeros(40, dtype=torch.float64, device="cuda")
        e[j] = h
        num = (loss(x, w.double() + e) - loss(x, w.double() - e)) / (2 * h)
        assert abs(num - float(dw[j])) < 1e-5 * (1 + abs(num))


# ---------------------------------------------------------------------------
# matrix product


def _act_ref(u, act):
    if act == "silu":
        s = torch.sigmoid(u)
        return u * s, s * (1 + u * (1 - s))
    if act == "gelu":
        c = 0.5 * (1 + torch.erf(u / math.sqrt(2)))
        return u * c, c + u * torch.exp(-u * u / 2) / math.sqrt(2 * math.pi)
    if act == "sigmoid":
        s = torch.sigmoid(u)
        return s, s * (1 - s)
    return u, torch.ones_like(u)


def _linear_case(gen, M, N, K, dtype):
    x, w = _rand(gen, M, K), _rand(gen, N, K) / math.sqrt(K)
    if dtype != "e4m3":
        x, w = x.to(DT[dtype]), w.to(DT[dtype])
        return x, w, None, None, x.double(), w.double()
    g = _g()
    x, xs = g.gdn_quantize_rows(x)
    w, ws = g.gdn_quantize_rows(w)
    return x, w, xs, ws, x.double() * xs.double()[:, None], w.double() * ws.double()[:, None]


def _check_linear(M, N, K, dtype, out, act, bias, residual, pre, seed=0):
    g = _g()
    gen = _gen(seed + M + 3 * N + 5 * K)
    x, w, xs, ws, xd, wd = _linear_case(gen, M, N, K, dtype)
    b = _rand(gen, N) if bias else None
    res = _rand(gen, M, N).to(DT[out]) if residual else None
    y, u = g.gdn_linear(x, w, bias=b, residual=res, act=act, out_dtype=DT[out], x_scale=xs,
                        w_scale=ws, want_pre=pre)
    ur = xd @ wd.t() + (b.double() if bias else 0.0)
    mag = xd.abs() @ wd.abs().t() + (b.double().abs() if bias else 0.0)
    eu = 2 * (K + 4) * u32 * mag
    if dtype == "e4m3" and out != "f32":
        eu = eu + 7 * 2.0 ** -13 * (xd.abs() @ wd.abs().t())
    if pre:
        _within(u, ur, _rounded(ur, eu, out), "pre")
    else:
        assert u is None
    yr = _act_ref(ur, act)[0]
    ey = 1.2 * eu + 16 * u32 * (ur.abs() + yr.abs()) if act != "none" else eu
    if residual:
        yr = yr + res.double()
        ey = ey + u32 * yr.abs()
    _within(y, yr, _rounded(yr, ey, out), "y")
    if M * N > 64:
        assert rel_l2(y, yr.cpu()) <= TOL[out]


SIZES = [(1, 1, 1), (1, 16, 64), (3, 5, 7), (16, 17, 33), (1, 4096, 4096), (8, 1000, 2048),
         (17, 130, 129), (33, 64, 72), (64, 2048, 512), (65, 300, 1000), (130, 257, 136),
         (256, 256, 64), (300, 1000, 264), (1000, 48, 4096), (513, 4096, 520), (2531, 1000, 1368)]


@gpu
@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("f16", "f16"), ("f32", "f32"),
                                       ("e4m3", "bf16"), ("bf16", "f32"), ("e4m3", "f32")])
def test_linear(M, N, K, dtype, out):
    _check_linear(M, N, K, dtype, out, "none", False, False, False)
    _check_linear(M, N, K, dtype, out, "silu", True, True, True, seed=1)


# enough output for the large tiles: partial tiles, a reduction that ends inside
# a step, an odd number of steps, rows that no vector divides, a split reduction
@gpu
@pytest.mark.parametrize("M,N,K", [(2100, 2200, 328), (2100, 2201, 136), (4100, 1100, 64),
                                   (2048, 2048, 4096), (2304, 2052, 24), (1900, 2500, 1155),
                                   (4000, 4000, 328), (3900, 4001, 136), (8100, 2000, 64),
                                   (4096, 2048, 8192), (3840, 4052, 24), (4000, 4000, 1155)])
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("f16", "f32"), ("e4m3", "bf16"),
                                       ("e4m3", "f16"), ("e4m3", "f32"), ("f32", "f32")])
def test_linear_large_tiles(M, N, K, dtype, out):
    _check_linear(M, N, K, dtype, out, "none", False, True, False)
    _check_linear(M, N, K, dtype, out, "gelu", True, False, True, seed=1)
    _check_linear(M, N, K, dtype, out, "silu", True, True, False, seed=2)


@gpu
@pytest.mark.parametrize("M,N,K", [(2100, 264, 2200), (2100, 2056, 1112), (512, 2100, 2100),
                                   (4000, 264, 4000), (512, 4000, 4000), (700, 4004, 3990)])
@pytest.mark.parametrize("dtype,gtype,act", [("bf16", "bf16", "silu"), ("f16", "f16", "none"),
                                             ("bf16", "f32", "none"), ("f32", "f32", "none")])
def test_linear_bwd_large_tiles(M, N, K, dtype, gtype, act):
    _check_linear_bwd(M, N, K, dtype, gtype, act)


@gpu
@pytest.mark.parametrize("act", ["none", "silu", "gelu", "sigmoid"])
@pytest.mark.parametrize("dtype,out", [("bf16", "f16"), ("f32", "f32"), ("e4m3", "f32")])
@pytest.mark.parametrize("M,N,K", [(5, 72, 100), (200, 130, 256)])
def test_linear_activations(act, dtype, out, M, N, K):
    _check_linear(M, N, K, dtype, out, act, True, True, True)
    _check_linear(M, N, K, dtype, out, act, False, True, False)


@gpu
def test_linear_saturated_activations():
    """Far arguments: the activations reach their limits without NaN."""
    g = _g()
    u = torch.tensor([-1e4, -200.0, -88.0, -20.0, 0.0, 20.0, 88.0, 200.0, 1e4], device="cuda")
    one = torch.ones(1, 1, device="cuda")
    for act in ("silu", "gelu", "sigmoid"):
        y, _ = g.gdn_linear(one, u[:, None].contiguous(), act=act)
        ref = _act_ref(u.double(), act)[0]
        _within(y[0], ref, 32 * u32 * (u.abs().double() + 1) + SUB["f16"], act)
        dx, dw, db = g.gdn_linear_bwd(torch.ones(1, 9, device="cuda"), one, u[:, None].contiguous(),
                                      pre=u[None].contiguous(), act=act)
        _within(db, _act_ref(u.double(), act)[1], 64 * u32 * (u.abs().double() + 1), act)


@gpu
@pytest.mark.parametrize("M,N,K,dtype", [(0, 8, 8, "bf16"), (3, 5, 16, "bf16"), (40, 70, 64, "f32"),
                                         (8, 1000, 2048, "e4m3"), (200, 257, 40, "f16")])
def test_linear_writes_its_own_elements_only(M, N, K, dtype):
    g = _g()
    gen = _gen(5)
    x, w, xs, ws, _, _ = _linear_case(gen, M, N, K, dtype)
    back = torch.full((M * N + 4096,), 7.0, device="cuda", dtype=torch.bfloat16)
    y = back[:M * N].view(M, N)
    g.gdn_linear(x, w, x_scale=xs, w_scale=ws, out_dtype=torch.bfloat16, y=y)
    y2, _ = g.gdn_linear(x, w, x_scale=xs, w_scale=ws, out_dtype=torch.bfloat16)
    assert torch.equal(y, y2) and (back[M * N:] == 7.0).all()


@gpu
@pytest.mark.parametrize("M,N,K", [(4, 512, 4096), (300, 520, 256)])
def test_linear_in_place_residual(M, N, K):
    g = _g()
    gen = _gen(6)
    x, w, *_ = _linear_case(gen, M, N, K, "bf16")
    res = _rand(gen, M, N).bfloat16()
    want, _ = g.gdn_linear(x, w, residual=res, act="silu")
    y, _ = g.gdn_linear(x, w, residual=res, act="silu", y=res)
    assert y is res and torch.equal(res, want)


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32", "e4m3"])
def test_linear_nan_and_infinity_stay_in_their_row_and_column(dtype):
    g = _g()
    gen = _gen(7)
    M, N, K = 150, 140, 200
    x, w, xs, ws, _, _ = _linear_case(gen, M, N, K, dtype)
    y0, _ = g.gdn_linear(x, w, x_scale=xs, w_scale=ws, out_dtype=torch.float32)
    if dtype == "e4m3":
        xs[3], ws[5] = float("nan"), float("inf")
    else:
        x[3, 199], w[5, 0] = float("nan"), float("inf")
    y, _ = g.gdn_linear(x, w, x_scale=xs, w_scale=ws, out_dtype=torch.float32)
    assert torch.isnan(y[3]).all() and not torch.isfinite(y[:, 5]).any()
    rows = torch.arange(M, device="cuda") != 3
    cols = torch.arange(N, device="cuda") != 5
    assert torch.equal(y[rows][:, cols], y0[rows][:, cols])


def _check_linear_bwd(M, N, K, dtype, gtype, act, seed=0):
    g = _g()
    gen = _gen(seed + M + 3 * N + 5 * K)
    x, w, _, _, xd, wd = _linear_case(gen, M, N, K, dtype)
    dy = _rand(gen, M, N).to(DT[gtype])
    pre = (1.5 * _rand(gen, M, N)).to(DT[gtype]) if act != "none" else None
    dx, dw, db = g.gdn_linear_bwd(dy, x, w, pre=pre, act=act)
    du = dy.double()
    edu = torch.zeros_like(du)
    if act != "none":
        du = du * _act_ref(pre.double(), act)[1]
        edu = 32 * u32 * dy.double().abs() * (1 + pre.double().abs())
    rounded = U[dtype] if (act != "none" or gtype != dtype) else 0.0
    in_mma = edu + rounded * (du.abs() + edu) + (SUB[dtype] if rounded else 0.0)
    rx, rw = du @ wd, du.t() @ xd
    ex = in_mma @ wd.abs() + 2 * (N + 4) * u32 * (du.abs() @ wd.abs())
    ew = in_mma.t() @ xd.abs() + 2 * (M + 4) * u32 * (du.abs().t() @ xd.abs())
    _within(dx, rx, _rounded(rx, ex, dtype), "dx")
    _within(dw, rw, _rounded(rw, ew, dtype), "dw")
    _within(db, du.sum(0), (edu.abs() + (M + 4) * u32 * du.abs()).sum(0), "dbias")
    if M * N > 64 and M * K > 64 and N * K > 64:
        # the rounding of du and that of the result, each TOL at most
        assert rel_l2(dx, rx.cpu()) <= 2 * TOL[dtype] and rel_l2(dw, rw.cpu()) <= 2 * TOL[dtype]


@gpu
@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (3, 5, 7), (1, 130, 64), (16, 64, 33), (65, 17, 72),
                                   (130, 257, 136), (256, 256, 64), (300, 1000, 264),
                                   (2531, 200, 96), (5000, 64, 64), (77, 2048, 520),
                                   (1024, 512, 2048)])
@pytest.mark.parametrize("dtype,gtype,act", [("bf16", "bf16", "none"), ("bf16", "bf16", "silu"),
                                             ("f16", "f32", "gelu"), ("f32", "f32", "none"),
                                             ("f32", "f32", "sigmoid"), ("bf16", "f32", "none")])
def test_linear_bwd(M, N, K, dtype, gtype, act):
    _check_linear_bwd(M, N, K, dtype, gtype, act)


@gpu
def test_linear_bwd_parts_and_no_rows():
    g = _g()
    gen = _gen(9)
    M, N, K = 90, 130, 72
    x, w, *_ = _linear_case(gen, M, N, K, "bf16")
    dy = _rand(gen, M, N).bfloat16()
    dx, dw, db = g.gdn_linear_bwd(dy, x, w)
    for parts in ((True, False, False), (False, True, False), (False, False, True)):
        got = g.gdn_linear_bwd(dy, x, w, want_dx=parts[0], want_dw=parts[1], want_dbias=parts[2])
        for have, full, part in zip(parts, (dx, dw, db), got):
            assert (part is not None) == have and (not have or torch.equal(part, full))
    dx, dw, db = g.gdn_linear_bwd(dy[:0], x[:0], w)
    assert dx.shape == (0, K) and (dw == 0).all() and (db == 0).all()


@gpu
def test_linear_bwd_against_differences():
    g = _g()
    gen = _gen(12)
    M, N, K = 6, 9, 20
    x, w, _, _, xd, wd = _linear_case(gen, M, N, K, "f32")
    b, dy = _rand(gen, N), _rand(gen, M, N)
    for act in ("none", "silu", "gelu", "sigmoid"):
        _, pre = g.gdn_linear(x, w, bias=b, act=act, want_pre=True)
        dx, dw, db = g.gdn_linear_bwd(dy, x, w, pre=pre, act=act)

        def loss(xx, ww, bb):
            return float((_act_ref(xx @ ww.t() + bb, act)[0] * dy.double()).sum())

        h = 1e-5
        for arr, grad, which in ((xd, dx, 0), (wd, dw, 1), (b.double(), db, 2)):
            for at in (0, arr.numel() // 2, arr.numel() - 1):
                e = torch.zeros_like(arr).view(-1)
                e[at] = h
                e = e.view(arr.shape)
                args = [xd, wd, b.double()]
                hi = [a + e if i == which else a for i, a in enumerate(args)]
                lo = [a - e if i == which else a for i, a in enumerate(args)]
                num = (loss(*hi) - loss(*lo)) / (2 * h)
                assert abs(num - float(grad.reshape(-1)[at])) < 2e-5 * (1 + abs(num)), (act, which)


# ---------------------------------------------------------------------------
# as they are used


def _layer_weights(gen, D, H, d):
    hd = H * d
    return dict(wq=_rand(gen, hd, D) / math.sqrt(D), wk=_rand(gen, hd, D) / math.sqrt(D),
                wv=_rand(gen, hd, D) / math.sqrt(D), wz=_rand(gen, hd, D) / math.sqrt(D),
                wg=_rand(gen, 2 * H, D) / math.sqrt(D), wo=_rand(gen, D, hd) / math.sqrt(hd),
                norm=0.1 * _rand(gen, D), b=0.1 * _rand(gen, 2 * H))


def _softplus(x):
    return torch.nn.functional.softplus(x)


@gpu
@pytest.mark.parametrize("eight_bits", [False, True])
def test_layer_forward(eight_bits):
    """A whole layer: norm, projections, the fused mixer, output projection
    into the residual stream, against the same steps in 64 bits with the
    oracle as the mixer."""
    g = _g()
    gen = _gen(21)
    N, T, H, d, D = 2, 96, 2, 64, 320
    rows = N * T
    p = _layer_weights(gen, D, H, d)
    x, res = _rand(gen, rows, D).bfloat16(), _rand(gen, rows, D).bfloat16()
    conv = 0.5 * _rand(gen, 3, H * d, 4)
    wt = {k: v.bfloat16() for k, v in p.items() if k.startswith("w")}

    h, r, hs = g.gdn_add_rmsnorm(x, p["norm"], res,
                                 out_dtype=torch.float8_e4m3fn if eight_bits else None)
    hd = h.double() * (hs.double()[:, None] if eight_bits else 1.0)
    h16, _, _ = g.gdn_add_rmsnorm(x, p["norm"], res)
    streams, ref = [], []
    for k in ("wq", "wk", "wv", "wz"):
        if eight_bits:
            w8, s8 = g.gdn_quantize_rows(wt[k])
            s, _ = g.gdn_linear(h, w8, x_scale=hs, w_scale=s8)
            ref.append(hd @ (w8.double() * s8.double()[:, None]).t())
        else:
            s, _ = g.gdn_linear(h, wt[k])
            ref.append(hd @ wt[k].double().t())
        streams.append(s)
        assert rel_l2(s, ref[-1].cpu()) <= TOL["bf16"]
    pre, _ = g.gdn_linear(h16, wt["wg"], bias=p["b"], out_dtype=torch.float32)
    la = (-0.1 * _softplus(pre[:, :H])).contiguous()
    be = torch.sigmoid(pre[:, H:]).contiguous()
    q, k, v, z = (s.view(rows, H, d) for s in streams)
    o, _ = g.gdn_chunk_fwd_fused(q, k, v, conv, la, be, z, N=N)
    out, _ = g.gdn_linear(o.view(rows, H * d), wt["wo"], residual=r)

    cw = conv.cpu()
    qq, kk, vv = (oracle.frontend(t.cpu(), cw[i], N=N, l2=i < 2)
                  for i, t in enumerate((q, k, v)))
    yo, _ = oracle.gdn_fwd(qq, kk, vv, la.cpu(), be.cpu(), None, N=N)
    oo = oracle.output_gate(yo, z.cpu(), None)
    want = torch.from_numpy(np.asarray(oo)).reshape(rows, H * d) @ wt["wo"].double().cpu().t()
    want = want + r.double().cpu()
    # o is off by the mixer's bar and its bf16 rounding, the sum by its own
    assert rel_l2(out, want) <= 3 * TOL["bf16"]


@gpu
def test_layer_training_chain():
    """r, h = add + norm; y = silu(h w^T + b): gradients of every leaf through
    both backward calls against automatic differentiation in 64 bits."""
    g = _g()
    gen = _gen(22)
    M, D, N = 300, 520, 260
    x, res = _rand(gen, M, D), _rand(gen, M, D)
    nw, w, b = 0.2 * _rand(gen, D), _rand(gen, N, D) / math.sqrt(D), _rand(gen, N)
    dy, dr = _rand(gen, M, N), _rand(gen, M, D)
    h, r, _ = g.gdn_add_rmsnorm(x, nw, res)
    y, pre = g.gdn_linear(h, w, bias=b, act="silu", want_pre=True)
    dh, dw, db = g.gdn_linear_bwd(dy, h, w, pre=pre, act="silu")
    dx, dnw = g.gdn_add_rmsnorm_bwd(dh, r, nw, dr=dr)
    leaves = [t.double().requires_grad_() for t in (x, res, nw, w, b)]
    X, R, NW, W, B = leaves
    rr = X + R
    hh = rr * torch.rsqrt((rr * rr).mean(-1, keepdim=True) + 1e-6) * (1 + NW)
    yy = torch.nn.functional.silu(hh @ W.t() + B)
    ((yy * dy.double()).sum() + (rr * dr.double()).sum()).backward()
    assert rel_l2(y, yy.cpu().detach()) <= TOL["f32"]
    for got, leaf in ((dx, X), (dx, R), (dnw, NW), (dw, W), (db, B)):
        assert rel_l2(got, leaf.grad.cpu()) <= TOL["f32"]


def _all_ops(g, t):
    """Every operator once, small, on t's tensors; the outputs as a flat list."""
    h8, r, hs = g.gdn_add_rmsnorm(t["x"], t["nw"], t["res"], out_dtype=torch.float8_e4m3fn)
    h, _, _ = g.gdn_add_rmsnorm(t["x"], t["nw"], t["res"])
    w8, ws = g.gdn_quantize_rows(t["w"])
    y8, _ = g.gdn_linear(h8, w8, x_scale=hs, w_scale=ws, bias=t["b"])
    y, pre = g.gdn_linear(h, t["w"], bias=t["b"], act="gelu", want_pre=True)
    y1, _ = g.gdn_linear(h[:3], t["w"], residual=t["dy"][:3].contiguous())
    dh, dw, db = g.gdn_linear_bwd(t["dy"], h, t["w"], pre=pre, act="gelu")
    dx, dnw = g.gdn_add_rmsnorm_bwd(dh, r, t["nw"])
    return [h8.float(), hs, r, h, w8.float(), ws, y8, y, pre, y1, dh, dw, db, dx, dnw]


def _op_inputs(seed, M=200, D=264, N=136):
    gen = _gen(seed)
    return dict(x=_rand(gen, M, D).bfloat16(), res=_rand(gen, M, D).bfloat16(),
                nw=0.1 * _rand(gen, D), w=(_rand(gen, N, D) / 16).bfloat16(), b=_rand(gen, N),
                dy=_rand(gen, M, N).bfloat16())


@gpu
def test_operators_are_deterministic_and_follow_their_stream():
    g = _g()
    t = _op_inputs(31)
    first = _all_ops(g, t)
    again = _all_ops(g, t)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        there = _all_ops(g, t)
    torch.cuda.synchronize()
    for a, b, c in zip(first, again, there):
        assert torch.equal(a, b) and torch.equal(a, c)


@gpu
def test_operators_captured_and_replayed():
    """One graph of every operator, replayed with new inputs and eager work
    between the replays; two graphs with workspaces of their own."""
    g = _g()
    t = _op_inputs(41)
    _all_ops(g, t)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = _all_ops(g, t)
        graphs.append((graph, out))
    for seed in (42, 43, 44):
        new = _op_inputs(seed)
        for k in t:
            t[k].copy_(new[k])
        want = _all_ops(g, new)
        for graph, out in graphs:
            graph.replay()
            torch.cuda.synchronize()
            for a, b in zip(out, want):
                assert torch.equal(a, b)


@gpu
def test_refusals_on_device():
    g = _g()
    x = torch.zeros(65, device="cuda", dtype=torch.bfloat16)
    with pytest.raises(g.GdnError, match="MISALIGNED"):
        g.gdn_add_rmsnorm(x[1:].view(1, 64))
    with pytest.raises(g.GdnError, match="contiguous"):
        g.gdn_linear(torch.zeros(8, 16, device="cuda").t(), torch.zeros(4, 8, device="cuda"))
    with pytest.raises(g.GdnError, match="UNSUPPORTED"):
        g.gdn_quantize_rows(torch.zeros(1, 32769, device="cuda"))
    a = torch.zeros(16, 64, device="cuda")
    with pytest.raises(g.GdnError, match="overlaps"):
        g.gdn_linear(a, torch.zeros(64, 64, device="cuda"), y=a)
    with pytest.raises(g.GdnError, match="overlaps"):
        g.gdn_add_rmsnorm_bwd(a, a, dx=a)
    with pytest.raises(g.GdnError, match="device"):
        g.gdn_linear(a, torch.zeros(64, 64))

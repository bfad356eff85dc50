"""Cases of the layer operators around the mixer, their plain forms and their
definitions in 64 bits.

A Gated DeltaNet layer is: residual addition and RMSNorm (``gdn_add_rmsnorm``),
projections (``gdn_linear``), the mixer, the output projection with the
residual in its epilogue (``gdn_linear`` again). In 8 bits the norm writes e4m3
with one scale a row, the weights come from ``gdn_quantize_rows`` and the
product applies the scales. Training adds ``gdn_add_rmsnorm_bwd`` and
``gdn_linear_bwd``.

``run`` computes a case in elementary torch operations, or with ``own`` true by
the calls of ``gated_deltanet_amd``.
"""
import math

import torch

own = False

EPS = 1e-6
E4M3_MAX = 448.0
TINY = 1e-30  # smallest absolute maximum of a row that sets its scale

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16,
          "e4m3": torch.float8_e4m3fn}
BYTES = {"f32": 4, "bf16": 2, "f16": 2, "e4m3": 1}

# The widths are H x d of the repository's workloads (16 and 32 heads of 128)
# and small multiples of them; the rows are those of its prefill batch (4
# sequences of 4096 tokens) and of decode steps.


def _norm(name, rows, d, dtype, out, residual=True):
    return {"name": name, "op": "norm", "rows": rows, "d": d, "dtype": dtype, "out": out,
            "residual": residual}


def _norm_bwd(name, rows, d, dtype, dr=True):
    return {"name": name, "op": "norm_bwd", "rows": rows, "d": d, "dtype": dtype, "dr": dr}


def _quantize(name, rows, d, dtype):
    return {"name": name, "op": "quantize", "rows": rows, "d": d, "dtype": dtype}


def _linear(name, m, n, k, dtype, out, act="none", bias=False, residual=False, pre=False):
    return {"name": name, "op": "linear", "m": m, "n": n, "k": k, "dtype": dtype, "out": out,
            "act": act, "bias": bias, "residual": residual, "pre": pre}


def _linear_bwd(name, m, n, k, dtype, act="none", bias=True):
    return {"name": name, "op": "linear_bwd", "m": m, "n": n, "k": k, "dtype": dtype, "act": act,
            "bias": bias}


def listed():
    return [
        # a decode step of 8 sequences: the norm in front of the 8-bit projections
        _norm("norm_decode_e4m3", 8, 4096, "bf16", "e4m3"),
        # the norm in front of a mixer's prefill, residual stream kept
        _norm("norm_prefill_bf16", 16384, 2048, "bf16", "bf16"),
        # training: the norm's gradient joined with the residual stream's
        _norm_bwd("norm_bwd_bf16", 16384, 4096, "bf16"),
        # packed sequences of odd total length, a width that no vector divides
        _norm_bwd("norm_bwd_f32_ragged", 2531, 1337, "f32", dr=False),
        # a projection's weights laid out in 8 bits when a model is loaded
        _quantize("quantize_weight", 8192, 4096, "bf16"),
        # a mixer's output for a few hundred packed tokens, odd width
        _quantize("quantize_f16_ragged", 777, 4099, "f16"),
        # output projection of a decode step of 8 sequences, into the residual stream
        _linear("linear_decode_bf16", 8, 4096, 4096, "bf16", "bf16", residual=True),
        # q, k, v and z of one token from one packed 8-bit weight
        _linear("linear_decode_e4m3", 1, 16384, 4096, "e4m3", "bf16"),
        # an up-projection of the prefill batch with bias and activation
        _linear("linear_prefill_bf16", 16384, 8192, 2048, "bf16", "bf16", act="silu", bias=True),
        # output projection of the prefill batch in 8 bits, into the residual stream
        _linear("linear_prefill_e4m3", 16384, 4096, 4096, "e4m3", "bf16", residual=True),
        # training: the gradients of an up-projection with its activation
        _linear_bwd("linear_bwd_bf16", 16384, 4096, 2048, "bf16", act="silu"),
        # training in fp32 on packed sequences of odd total length
        _linear_bwd("linear_bwd_f32_ragged", 2531, 1000, 520, "f32"),
    ]


MOST_FLOPS = 2 * 16384 * 8192 * 2048
MOST_ELEMENTS = 16384 * 4096


def _log(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    """A width: mostly whole 16-byte vectors as in models, sometimes any number."""
    w = _log(rng, lo, hi)
    return w if rng.random() < 0.25 else max(16, w // 16 * 16)


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "quantize", "linear", "linear", "linear_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    while op in ("norm", "norm_bwd", "quantize"):
        rows, d = _log(rng, 1, 16384), _width(rng, 64, 16384)
        if rows * d > MOST_ELEMENTS:
            continue
        if op == "norm":
            out = rng.choice([dtype, "e4m3", "f32"])
            c = _norm("", rows, d, dtype, out, residual=rng.random() < 0.7)
        elif op == "norm_bwd":
            c = _norm_bwd("", rows, d, dtype, dr=rng.random() < 0.7)
        else:
            c = _quantize("", rows, d, dtype)
        break
    while op in ("linear", "linear_bwd"):
        m, n, k = _log(rng, 1, 16384), _width(rng, 16, 16384), _width(rng, 64, 8192)
        flops = (2 if op == "linear" else 4) * m * n * k
        # fp32 products run at a sixteenth of the 16-bit rate
        if flops * (8 if dtype == "f32" else 1) > MOST_FLOPS or m * n > 2 * MOST_ELEMENTS:
            continue
        act = rng.choice(["none", "none", "silu", "gelu", "sigmoid"])
        if op == "linear":
            if dtype != "f32" and rng.random() < 0.35:
                dtype = "e4m3"
            out = rng.choice(["f32", "bf16"]) if dtype == "e4m3" else rng.choice([dtype, dtype, "f32"])
            c = _linear("", m, n, k, dtype, out, act=act, bias=rng.random() < 0.5,
                        residual=rng.random() < 0.5, pre=rng.random() < 0.25)
        else:
            c = _linear_bwd("", m, n, k, dtype, act=act, bias=rng.random() < 0.7)
        break
    del c["name"]
    return c


# ---------------------------------------------------------------------------
# inputs


def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def _activations(gen, rows, d):
    """Hidden activations: normal, with channels of different strengths."""
    x = _randn(gen, rows, d)
    return x * torch.exp(0.5 * _randn(gen, d))


def _quantized(x):
    """x [rows, d] as a program keeps it in 8 bits: e4m3 and one scale a row."""
    scale = x.abs().amax(dim=1).clamp_min(TINY) / E4M3_MAX
    return (x / scale[:, None]).to(torch.float8_e4m3fn), scale


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    c, s = case, {"case": dict(case)}
    dt = DTYPES[c["dtype"]]
    if c["op"] in ("norm", "norm_bwd", "quantize"):
        rows, d = c["rows"], c["d"]
        s["x"] = _activations(gen, rows, d).to(dt)
        if c["op"] != "quantize":
            s["norm_w"] = 0.2 * _randn(gen, d)
        if c["op"] == "norm":
            s["residual"] = (2.0 * _randn(gen, rows, d)).to(dt) if c["residual"] else None
        if c["op"] == "norm_bwd":
            s["dy"] = (0.1 * _randn(gen, rows, d)).to(dt)
            s["dr"] = (0.1 * _randn(gen, rows, d)).to(dt) if c["dr"] else None
        return s
    m, n, k = c["m"], c["n"], c["k"]
    x, w = _activations(gen, m, k), _randn(gen, n, k) / math.sqrt(k)
    s["x_scale"] = s["w_scale"] = None
    if c["dtype"] == "e4m3":
        s["x"], s["x_scale"] = _quantized(x)
        s["w"], s["w_scale"] = _quantized(w)
    else:
        s["x"], s["w"] = x.to(dt), w.to(dt)
    del x, w
    if c["op"] == "linear":
        s["bias"] = 0.1 * _randn(gen, n) if c["bias"] else None
        s["residual"] = (2.0 * _randn(gen, m, n)).to(DTYPES[c["out"]]) if c["residual"] else None
    else:
        s["dy"] = (0.1 * _randn(gen, m, n)).to(dt)
        s["pre"] = _randn(gen, m, n).to(dt) if c["act"] != "none" else None
    return s


# ---------------------------------------------------------------------------
# plain forms: 32 bits, rounded once at the end


def _act(u, act):
    if act == "silu":
        return u * torch.sigmoid(u)
    if act == "gelu":
        return 0.5 * u * (1.0 + torch.erf(u * math.sqrt(0.5)))
    if act == "sigmoid":
        return torch.sigmoid(u)
    return u


def _act_slope(u, act):
    if act == "silu":
        p = torch.sigmoid(u)
        return p * (1.0 + u * (1.0 - p))
    if act == "gelu":
        return (0.5 * (1.0 + torch.erf(u * math.sqrt(0.5)))
                + u * torch.exp(-0.5 * u * u) * (1.0 / math.sqrt(2.0 * math.pi)))
    p = torch.sigmoid(u)
    return p * (1.0 - p)


def _plain_norm(s, c):
    r = s["x"].float()
    if s["residual"] is not None:
        r = r + s["residual"].float()
    y = r * torch.rsqrt((r * r).mean(dim=1, keepdim=True) + EPS) * (1.0 + s["norm_w"])
    out = {}
    if c["out"] == "e4m3":
        out["y"], out["y_scale"] = _quantized(y)
    else:
        out["y"] = y.to(DTYPES[c["out"]])
    if s["residual"] is not None:
        out["r"] = r.to(s["x"].dtype)
    return out


def _plain_norm_bwd(s, c):
    r, dy = s["x"].float(), s["dy"].float()
    rs = torch.rsqrt((r * r).mean(dim=1, keepdim=True) + EPS)
    n = r * rs
    g = dy * (1.0 + s["norm_w"])
    dx = rs * (g - n * (g * n).mean(dim=1, keepdim=True))
    if s["dr"] is not None:
        dx = dx + s["dr"].float()
    return {"dx": dx.to(s["x"].dtype), "dnorm_w": (dy * n).sum(dim=0)}


def _plain_quantize(s, c):
    y, scale = _quantized(s["x"].float())
    return {"y": y, "y_scale": scale}


def _plain_linear(s, c):
    u = s["x"].float() @ s["w"].float().t()
    if c["dtype"] == "e4m3":
        u = u * (s["x_scale"][:, None] * s["w_scale"])
    if s["bias"] is not None:
        u = u + s["bias"]
    y = _act(u, c["act"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    out = {"y": y.to(DTYPES[c["out"]])}
    if c["pre"]:
        out["pre"] = u.to(DTYPES[c["out"]])
    return out


def _plain_linear_bwd(s, c):
    du = s["dy"].float()
    if c["act"] != "none":
        du = du * _act_slope(s["pre"].float(), c["act"])
    out = {"dx": (du @ s["w"].float()).to(s["x"].dtype),
           "dw": (du.t() @ s["x"].float()).to(s["w"].dtype)}
    if c["bias"]:
        out["dbias"] = du.sum(dim=0)
    return out


PLAIN = {"norm": _plain_norm, "norm_bwd": _plain_norm_bwd, "quantize": _plain_quantize,
         "linear": _plain_linear, "linear_bwd": _plain_linear_bwd}


# ---------------------------------------------------------------------------
# the library's calls


def _own(s, c):
    import gated_deltanet_amd as gdn

    if c["op"] == "norm":
        y, r, y_scale = gdn.gdn_add_rmsnorm(s["x"], s["norm_w"], s["residual"], rms_eps=EPS,
                                            out_dtype=DTYPES[c["out"]])
        return {k: v for k, v in (("y", y), ("r", r), ("y_scale", y_scale)) if v is not None}
    if c["op"] == "norm_bwd":
        dx, dnorm_w = gdn.gdn_add_rmsnorm_bwd(s["dy"], s["x"], s["norm_w"], dr=s["dr"],
                                              rms_eps=EPS)
        return {"dx": dx, "dnorm_w": dnorm_w}
    if c["op"] == "quantize":
        y, y_scale = gdn.gdn_quantize_rows(s["x"])
        return {"y": y, "y_scale": y_scale}
    if c["op"] == "linear":
        y, pre = gdn.gdn_linear(s["x"], s["w"], bias=s["bias"], residual=s["residual"],
                                act=c["act"], x_scale=s["x_scale"], w_scale=s["w_scale"],
                                out_dtype=DTYPES[c["out"]], want_pre=c["pre"])
        return {"y": y, "pre": pre} if c["pre"] else {"y": y}
    dx, dw, dbias = gdn.gdn_linear_bwd(s["dy"], s["x"], s["w"], pre=s["pre"], act=c["act"],
                                       want_dbias=c["bias"])
    return {"dx": dx, "dw": dw, "dbias": dbias} if c["bias"] else {"dx": dx, "dw": dw}


def run(state):
    c = state["case"]
    if own:
        return _own(state, c)
    return PLAIN[c["op"]](state, c)


def work(case):
    c = case
    if c["op"] in ("norm", "norm_bwd", "quantize"):
        e, n = BYTES[c["dtype"]], c["rows"] * c["d"]
        if c["op"] == "norm":
            rd = n * e * (2 if c["residual"] else 1) + 4 * c["d"]
            wr = n * BYTES[c["out"]] + (n * e if c["residual"] else 0)
            wr += 4 * c["rows"] if c["out"] == "e4m3" else 0
            return {"bytes": rd + wr, "flops": 6 * n}
        if c["op"] == "norm_bwd":
            return {"bytes": n * e * (4 if c["dr"] else 3) + 8 * c["d"], "flops": 12 * n}
        return {"bytes": n * (e + 1) + 4 * c["rows"], "flops": 3 * n}
    m, n, k = c["m"], c["n"], c["k"]
    e = BYTES[c["dtype"]]
    if c["op"] == "linear":
        o = BYTES[c["out"]]
        byts = e * (m * k + n * k) + o * m * n * (1 + c["residual"] + c["pre"])
        byts += 4 * n * c["bias"] + (4 * (m + n) if c["dtype"] == "e4m3" else 0)
        return {"bytes": byts, "flops": 2 * m * n * k}
    byts = e * (2 * m * k + 2 * n * k + m * n * (2 if c["act"] != "none" else 1))
    return {"bytes": byts + 4 * n * c["bias"], "flops": 4 * m * n * k}


# ---------------------------------------------------------------------------
# the definitions in 64 bits


def _e4m3_exact(y):
    """Values before the rounding to e4m3, and the scales."""
    top = torch.maximum(y.abs().max(dim=1).values, torch.tensor(TINY, dtype=torch.float64,
                                                                device=y.device))
    return y * (E4M3_MAX / top).unsqueeze(1), top / E4M3_MAX


def exact(case, seed):
    s = prepare(case, seed)
    f = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor)}
    op = case["op"]
    if op == "quantize":
        y, scale = _e4m3_exact(f["x"])
        return {"y": y, "y_scale": scale}
    if op == "norm":
        r = f["x"] + f["residual"] if "residual" in f else f["x"]
        size = torch.sqrt(torch.linalg.vector_norm(r, dim=1).square() / r.shape[1] + EPS)
        y = torch.addcmul(r, r, f["norm_w"].expand_as(r)) / size.unsqueeze(1)
        out = {"r": r} if "residual" in f else {}
        if case["out"] == "e4m3":
            out["y"], out["y_scale"] = _e4m3_exact(y)
        else:
            out["y"] = y
        return out
    if op == "norm_bwd":
        # L = sum dy (1 + w) r / size(r): the quotient rule, row by row
        r, dy = f["x"], f["dy"]
        size = torch.sqrt(torch.linalg.vector_norm(r, dim=1).square() / r.shape[1] + EPS)
        g = dy + dy * f["norm_w"]
        along = torch.linalg.vecdot(g, r) / (r.shape[1] * size.pow(3))
        dx = g / size.unsqueeze(1) - r * along.unsqueeze(1)
        if "dr" in f:
            dx = dx + f["dr"]
        return {"dx": dx, "dnorm_w": torch.linalg.vecdot(dy, r / size.unsqueeze(1), dim=0)}
    if op == "linear":
        x, w = f["x"], f["w"]
        if "x_scale" in f:
            x, w = x * f["x_scale"].unsqueeze(1), w * f["w_scale"].unsqueeze(1)
        u = torch.nn.functional.linear(x, w, f.get("bias"))
        y = _act_exact(u, case["act"])[0]
        if "residual" in f:
            y = y + f["residual"]
        return {"y": y, "pre": u} if case["pre"] else {"y": y}
    du = f["dy"] * _act_exact(f["pre"], case["act"])[1] if "pre" in f else f["dy"]
    out = {"dx": torch.mm(du, f["w"]), "dw": torch.mm(f["x"].t(), du).t()}
    if case["bias"]:
        out["dbias"] = torch.mv(du.t(), torch.ones_like(du[:, 0]))
    return out


def _act_exact(u, act):
    """The activation and its slope, from the hyperbolic tangent and the normal
    distribution's integral."""
    half = 0.5 * (1.0 + torch.tanh(0.5 * u))
    if act == "sigmoid":
        return half, half * (1.0 - half)
    if act == "silu":
        return u * half, half + u * half * (1.0 - half)
    if act == "gelu":
        below = torch.special.ndtr(u)
        return u * below, below + u * torch.exp(-0.5 * u * u) / math.sqrt(2.0 * math.pi)
    return u, torch.ones_like(u)

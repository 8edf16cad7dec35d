"""The operators of a linear layer over block-scaled data, as cases to measure.

A linear layer here keeps its weight in microscaled 4-bit floating point (E2M1 codes, one
power-of-two scale per 32 elements: "mx", or one E4M3 scale per 16 elements and an fp32
scale per tensor: "nv"), and what its backward pass needs of the activations in 8 bits
(one power-of-two scale per 32 elements; E4M3, E5M2 or INT8 codes).

  linear             y[t, n]  = sum_k x[t, k] W[n, k]            W from 4-bit codes
  linear_grad_input  dx[t, k] = sum_n dy[t, n] W[n, k]           W from 4-bit codes
  linear_grad_weight dw[n, k] = sum_t dy[t, n] X[t, k]           X from 8-bit codes
  glu                h = a(g) u, and g, u kept as 8-bit codes
  glu_backward       du = dh a(G), dg = dh U a'(G)               G, U from 8-bit codes

with a(g) = g s(v): the logistic function s of v = g ("silu") or of
v = 2 sqrt(2 / pi) (g + 0.044715 g^3) ("gelu", its tanh form).

``run`` computes them with elementary torch operations in fp32, or (``own``) with the
library; ``exact`` computes them in fp64 from the definition.
"""

import math

import torch

own = False

DEV = "cuda"
# E2M1 values by code (sign in bit 3)
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
# 8-bit formats: largest value as f * 2^E with f in [0.5, 1); mantissa bits, smallest exponent (0: integers)
F8 = {"e4m3": (448.0, 0.875, 9, 3, -6), "e5m2": (57344.0, 0.875, 16, 2, -14), "int8_sym": (127.0, 0.9921875, 7, 0, 0)}
GELU_C = math.sqrt(2.0 / math.pi)
OUT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    return [
        # one token of one sequence through a 4096 x 4096 projection: a call that latency bounds
        {"name": "linear_decode_1", "op": "linear", "m": 1, "n": 4096, "k": 4096, "fmt": "mx", "out": "bf16"},
        # eight sequences, a token each, through the largest weight: the weight's bytes bound it
        {"name": "linear_decode_8_large", "op": "linear", "m": 8, "n": 28672, "k": 8192, "fmt": "nv", "out": "bf16"},
        # a ragged batch (chunked prompts, speculative tokens) over an odd number of outputs
        {"name": "linear_ragged_45", "op": "linear", "m": 45, "n": 11007, "k": 4128, "fmt": "mx", "out": "bf16"},
        # a prompt, or the forward pass of a training step, through an up projection
        {"name": "linear_prompt_4096", "op": "linear", "m": 4096, "n": 11008, "k": 4096, "fmt": "nv", "out": "bf16"},
        # the backward pass of the same layer
        {"name": "grad_input_4096", "op": "grad_input", "m": 4096, "n": 11008, "k": 4096, "fmt": "mx", "out": "bf16"},
        # the last, partly filled batch of a fine-tuning run, a narrow layer
        {"name": "grad_input_333", "op": "grad_input", "m": 333, "n": 4104, "k": 1056, "fmt": "nv", "out": "bf16"},
        # the weight gradient of a training step from the 8-bit copy of its input
        {"name": "grad_weight_4096", "op": "grad_weight", "m": 4096, "n": 11008, "k": 4096, "fmt": "e4m3", "out": "bf16"},
        # few tokens and a narrow layer, kept in fp32 for a master weight
        {"name": "grad_weight_1000", "op": "grad_weight", "m": 1000, "n": 1000, "k": 2080, "fmt": "int8_sym", "out": "fp32"},
        # the gated activation of a training step: forward with its 8-bit copies, then backward from them
        {"name": "glu_step_4096", "op": "glu_step", "m": 4096, "n": 11008, "fmt": "e4m3", "act": "silu"},
        # the same of a small ragged batch
        {"name": "glu_step_37", "op": "glu_step", "m": 37, "n": 1376, "fmt": "int8_sym", "act": "gelu"},
        # the backward pass alone, from copies that an earlier forward pass kept
        {"name": "glu_backward_8192", "op": "glu_backward", "m": 8192, "n": 4096, "fmt": "e5m2", "act": "gelu"},
        {"name": "glu_backward_333", "op": "glu_backward", "m": 333, "n": 11008, "fmt": "e4m3", "act": "silu"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "grad_input", "grad_weight", "glu_step", "glu_backward"])
    if op in ("glu_step", "glu_backward"):
        m, n = _log(rng, 1, 8192), 32 * _log(rng, 2, 896)
        m = max(1, min(m, 4096 * 11008 // n))
        return {"op": op, "m": m, "n": n, "fmt": rng.choice(["e4m3", "e5m2", "int8_sym"]), "act": rng.choice(["silu", "gelu"])}
    n, k = _log(rng, 64, 28672), 32 * _log(rng, 4, 344)
    if rng.random() < 0.5:
        n = max(8, n // 8 * 8)
    m = _log(rng, 1, 64) if op == "linear" and rng.random() < 0.5 else _log(rng, 16, 8192)
    m = max(1, min(m, 4096 * 11008 * 4096 // (n * k)))
    fmt = rng.choice(["e4m3", "e5m2", "int8_sym"]) if op == "grad_weight" else rng.choice(["mx", "nv"])
    return {"op": op, "m": m, "n": n, "k": k, "fmt": fmt, "out": rng.choice(["bf16", "bf16", "fp32"]) if op == "grad_weight" else "bf16"}


# ---------------------------------------------------------------------------
# Inputs: bf16 activations and gradients, codes and scales as the quantize writes them
# ---------------------------------------------------------------------------

def _activations(g, m, n, gain=0.5):
    """Student-t(3) entries with a few channels of large magnitude, as bf16."""
    x = torch.randn(m, n, device=DEV, generator=g)
    d = torch.zeros(m, n, device=DEV)
    for _ in range(3):
        d += torch.randn(m, n, device=DEV, generator=g).square_()
    x *= gain
    x /= d.div_(3.0).sqrt_()
    x.clamp_(-200.0 * gain, 200.0 * gain)
    at = torch.randint(0, n, (4,), device=DEV, generator=g)
    x[:, at] *= 8.0
    return x.to(torch.bfloat16)


def _weight(g, n, k):
    w = torch.randn(n, k, device=DEV, generator=g) * 0.02
    big = torch.rand(n, k, device=DEV, generator=g) < 0.001
    w[big] *= 8.0
    return w.to(torch.bfloat16)


def _gradient(g, m, n):
    rows = torch.exp(torch.randn(m, 1, device=DEV, generator=g) * 0.5)
    return (torch.randn(m, n, device=DEV, generator=g) * rows * 1e-3).to(torch.bfloat16)


def _mx_exponent(amax, f, e_max):
    """Smallest e with amax <= qmax 2^e, within [-127, 127], where qmax = f 2^e_max."""
    fr, ex = torch.frexp(amax)
    e = ex - e_max + (fr > f).to(ex.dtype)
    return torch.where(amax > 0, e, torch.full_like(e, -127)).clamp_(-127, 127)


def _grid8(y, fmt):
    """Values of an 8-bit format nearest to y (ties to even, saturating)."""
    qmax, _, _, mant, emin = F8[fmt]
    if fmt == "int8_sym":
        return torch.round(y).clamp_(-qmax, qmax)
    ex = torch.frexp(y.abs())[1] - 1
    step = torch.ldexp(torch.ones_like(y), ex.clamp_(min=emin) - mant)
    return (torch.round(y / step) * step).clamp_(-qmax, qmax)


def _mx8_values(x, fmt):
    """x (fp32 or fp64 [m, n]) as the values its 8-bit codes stand for, and (element values, exponents)."""
    _, f, e_max, _, _ = F8[fmt]
    b = x.reshape(x.shape[0], -1, 32)
    e = _mx_exponent(b.abs().amax(2, keepdim=True), f, e_max)
    q = _grid8(torch.ldexp(b, -e), fmt)
    return torch.ldexp(q, e).reshape(x.shape), q.reshape(x.shape), e.squeeze(2)


def _table8(fmt, dtype=torch.float32):
    """The 256 values of an 8-bit format by code (codes that stand for none: 0)."""
    c = torch.arange(256, device=DEV)
    if fmt == "int8_sym":
        return torch.where(c < 128, c, c - 256).to(dtype)
    mant = F8[fmt][3]
    bias = 7 if fmt == "e4m3" else 15
    ee, mm = (c & 127) >> mant, c & ((1 << mant) - 1)
    v = torch.where(ee > 0, torch.ldexp(1.0 + mm.double() / (1 << mant), ee - bias),
                    torch.ldexp(mm.double() / (1 << mant), torch.full_like(ee, 1 - bias)))
    v = torch.where(v > F8[fmt][0], torch.zeros_like(v), v)
    return torch.where(c < 128, v, -v).to(dtype)


def _codes8(x, fmt):
    """bf16 x -> uint8 codes [m, n] and UE8M0 scales [m, n / 32]."""
    _, q, e = _mx8_values(x.float(), fmt)
    if fmt == "int8_sym":
        codes = q.to(torch.int8).view(torch.uint8)
    else:
        mant, emin = F8[fmt][3], F8[fmt][4]
        a = q.abs()
        ex = (torch.frexp(a)[1] - 1).clamp_(min=emin)
        frac = torch.ldexp(a, mant - ex).to(torch.int32)           # includes the leading one of normal values
        codes = ((ex - emin) << mant) + frac
        codes = (codes | (torch.signbit(q).to(torch.int32) << 7)).to(torch.uint8)
    return codes, (e + 127).to(torch.uint8)


def _codes4(w, fmt):
    """bf16 w [n, k] -> packed E2M1 codes, scales and the tensor scale (nv), a few rows at a time."""
    n, k = w.shape
    block = 32 if fmt == "mx" else 16
    codes = torch.empty(n, k // 2, dtype=torch.uint8, device=DEV)
    scales = torch.empty(n, k // block, dtype=torch.uint8, device=DEV)
    ts = (w.abs().max().float() / (6.0 * 448.0)).reshape(1) if fmt == "nv" else None
    step = max(1, (1 << 25) // k)
    for r in range(0, n, step):
        b = w[r:r + step].float().reshape(-1, k // block, block)
        amax = b.abs().amax(2, keepdim=True)
        if fmt == "mx":
            e = _mx_exponent(amax, 0.75, 3)
            y = torch.ldexp(b, -e)
            scales[r:r + step] = (e + 127).to(torch.uint8).squeeze(2)
        else:
            s = _grid8((amax / 6.0 / ts).clamp_(max=448.0), "e4m3")
            d = s * ts
            y = torch.where(d > 0, b / d, torch.zeros_like(b))
            ex = (torch.frexp(s)[1] - 1).clamp_(min=-6)
            scales[r:r + step] = (((ex + 6) << 3) + torch.ldexp(s, 3 - ex).to(torch.int32)).to(torch.uint8).squeeze(2)
        a = y.abs()
        c = ((a > 0.25).byte() + (a >= 0.75).byte() + (a > 1.25).byte() + (a >= 1.75).byte() + (a > 2.5).byte()
             + (a >= 3.5).byte() + (a > 5.0).byte()) | (torch.signbit(y).byte() << 3)
        c = c.reshape(-1, k)
        codes[r:r + step] = c[:, 0::2] | (c[:, 1::2] << 4)
    return codes, scales, ts


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    op, m, n = case["op"], case["m"], case["n"]
    s = {"case": case}
    if op in ("linear", "grad_input"):
        s["codes"], s["scales"], s["ts"] = _codes4(_weight(g, n, case["k"]), case["fmt"])
        s["x"] = _activations(g, m, case["k"]) if op == "linear" else _gradient(g, m, n)
    elif op == "grad_weight":
        s["codes"], s["scales"] = _codes8(_activations(g, m, case["k"]), case["fmt"])
        s["dy"] = _gradient(g, m, n)
    else:
        # gate and up side by side, as one projection writes them
        gu = _activations(g, m, 2 * n, gain=1.0)
        if op == "glu_step":
            s["gu"] = gu
        else:
            s["g_codes"], s["g_scales"] = _codes8(gu[:, :n], case["fmt"])
            s["u_codes"], s["u_scales"] = _codes8(gu[:, n:], case["fmt"])
        s["dh"] = _gradient(g, m, n)
    return s


# ---------------------------------------------------------------------------
# Plain forms (fp32) and the definition in fp64
# ---------------------------------------------------------------------------

def _weight_values(s, dtype):
    """The values of the 4-bit weight."""
    codes, scales = s["codes"], s["scales"]
    n, k = codes.shape[0], codes.shape[1] * 2
    t = torch.tensor(E2M1 + [-v for v in E2M1], device=DEV, dtype=dtype)
    v = torch.stack((t[(codes & 15).int()], t[(codes >> 4).int()]), 2).reshape(n, -1, k // scales.shape[1])
    if s["ts"] is None:
        return torch.ldexp(v, scales.int().unsqueeze(2) - 127).reshape(n, k)
    return (v * _table8("e4m3", dtype)[scales.int()].unsqueeze(2)).reshape(n, k) * s["ts"].to(dtype)


def _values8(codes, scales, fmt, dtype):
    v = _table8(fmt, dtype)[codes.int()].reshape(codes.shape[0], -1, 32)
    return torch.ldexp(v, scales.int().unsqueeze(2) - 127).reshape(codes.shape)


def _act(g, act):
    """a(g) and a'(g)."""
    if act == "silu":
        v, dv = g, 1.0
    else:
        v, dv = 2.0 * GELU_C * (g + 0.044715 * g * g * g), 2.0 * GELU_C * (1.0 + 3.0 * 0.044715 * g * g)
    s = 1.0 / (1.0 + torch.exp(-v))
    return g * s, s + g * s * (1.0 - s) * dv


def _plain(s):
    case = s["case"]
    op = case["op"]
    f = torch.float32
    if op == "linear":
        return (s["x"].to(f) @ _weight_values(s, f).t()).to(OUT[case["out"]])
    if op == "grad_input":
        return (s["x"].to(f) @ _weight_values(s, f)).to(OUT[case["out"]])
    if op == "grad_weight":
        return (s["dy"].to(f).t() @ _values8(s["codes"], s["scales"], case["fmt"], f)).to(OUT[case["out"]])
    dh = s["dh"].to(f)
    if op == "glu_step":
        n = case["n"]
        g, u = s["gu"][:, :n].to(f), s["gu"][:, n:].to(f)
        h = (_act(g, case["act"])[0] * u).to(torch.bfloat16)
        gq, uq = _mx8_values(g, case["fmt"])[0], _mx8_values(u, case["fmt"])[0]
    else:
        gq = _values8(s["g_codes"], s["g_scales"], case["fmt"], f)
        uq = _values8(s["u_codes"], s["u_scales"], case["fmt"], f)
    a, da = _act(gq, case["act"])
    dg, du = (dh * uq * da).to(torch.bfloat16), (dh * a).to(torch.bfloat16)
    return (h, dg, du) if op == "glu_step" else (dg, du)


def _own(s):
    import block_scaled_bit_bq_b200 as bq
    case = s["case"]
    op, m, n = case["op"], case["m"], case["n"]
    if op in ("linear", "grad_input", "grad_weight"):
        q = s.get("q")
        if q is None:       # the handle of the weight (or of the kept input) that a program holds
            scheme = bq.Scheme(case["fmt"], "mx") if op == "grad_weight" else bq.Scheme("e2m1", case["fmt"])
            q = s["q"] = bq.Quantized(scheme.resolved(), m if op == "grad_weight" else n, case["k"], s["codes"],
                                      s["scales"].reshape(-1), None, s.get("ts"), None)
        if op == "linear":
            return bq.linear(s["x"], q, OUT[case["out"]])
        if op == "grad_input":
            return bq.linear_grad_input(s["x"], q, OUT[case["out"]])
        return bq.linear_grad_weight(s["dy"], q, OUT[case["out"]])
    scheme = bq.Scheme(case["fmt"], "mx")
    if op == "glu_step":
        h, kept = bq.glu(s["gu"][:, :n], s["gu"][:, n:], scheme, case["act"])
        dg, du = bq.glu_backward(s["dh"], kept)
        return h, dg, du
    kept = s.get("kept")
    if kept is None:        # the handle of the copies that the forward pass kept
        kept = s["kept"] = bq.GluCheckpoint(
            bq.Quantized(scheme.resolved(), m, n, s["g_codes"], s["g_scales"].reshape(-1), None, None, None),
            bq.Quantized(scheme.resolved(), m, n, s["u_codes"], s["u_scales"].reshape(-1), None, None, None), case["act"])
    return bq.glu_backward(s["dh"], kept)


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    op, m, n = case["op"], case["m"], case["n"]
    if op in ("glu_step", "glu_backward"):
        kept = 2 * m * n + 2 * m * n // 32
        back = kept + 6 * m * n                        # codes and scales, dh read; dg, du written
        fwd = 6 * m * n + kept                         # g, u read; h, codes and scales written
        return {"bytes": back + (fwd if op == "glu_step" else 0), "flops": (30 if op == "glu_step" else 16) * m * n}
    k = case["k"]
    ob = 2 if case["out"] == "bf16" else 4
    if op == "grad_weight":
        return {"bytes": 2 * m * n + m * k + m * k // 32 + ob * n * k, "flops": 2 * m * n * k}
    w = n * k // 2 + n * k // (32 if case["fmt"] == "mx" else 16)
    other = 2 * m * k + ob * m * n if op == "linear" else 2 * m * n + ob * m * k
    return {"bytes": w + other, "flops": 2 * m * n * k}


def exact(case, seed):
    s = prepare(case, seed)
    op, fmt = case["op"], case["fmt"]
    d = torch.float64
    if op in ("linear", "grad_input"):
        n, k, x = case["n"], case["k"], s["x"].to(d)
        out = torch.zeros(case["m"], n if op == "linear" else k, dtype=d, device=DEV)
        step = max(1, (1 << 26) // k)
        for r in range(0, n, step):                    # a band of the weight's rows at a time
            w = _weight_values({"codes": s["codes"][r:r + step], "scales": s["scales"][r:r + step], "ts": s["ts"]}, d)
            if op == "linear":
                out[:, r:r + step] = x @ w.t()
            else:
                out += x[:, r:r + step] @ w
        return out
    if op == "grad_weight":
        return s["dy"].to(d).t() @ _values8(s["codes"], s["scales"], fmt, d)
    dh, n = s["dh"].to(d), case["n"]
    h = None
    if op == "glu_step":
        g, u = s["gu"][:, :n].to(d), s["gu"][:, n:].to(d)
        v = g if case["act"] == "silu" else GELU_C * 2.0 * (g + 0.044715 * g ** 3)
        h = g * torch.special.expit(v) * u
        g, u = _mx8_values(g, fmt)[0], _mx8_values(u, fmt)[0]
    else:
        g = _values8(s["g_codes"], s["g_scales"], fmt, d)
        u = _values8(s["u_codes"], s["u_scales"], fmt, d)
    if case["act"] == "silu":
        p = torch.special.expit(g)
        slope = p * (1.0 + g * (1.0 - p))
    else:
        th = torch.tanh(GELU_C * (g + 0.044715 * g ** 3))
        p = 0.5 * (1.0 + th)
        slope = p + 0.5 * g * (1.0 - th * th) * GELU_C * (1.0 + 0.134145 * g * g)
    dg, du = dh * u * slope, dh * g * p
    return (h, dg, du) if op == "glu_step" else (dg, du)

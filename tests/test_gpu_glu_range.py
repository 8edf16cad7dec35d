"""The gated activation where values leave the ordinary range: NaN, and products that overflow."""

import numpy as np
import pytest
import torch

import oracle
import block_scaled_bit_bq_b200 as bq
from block_scaled_bit_bq_b200 import Scheme
from oracle import linear as ref

pytestmark = pytest.mark.gpu


# a NaN stays one through the forward pass, the copies and the backward pass, whatever the activation
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_nan_stays_nan(fmt, act):
    gen = torch.Generator("cuda").manual_seed(3)
    g, u, dh = (torch.randn(6, 96, device="cuda", generator=gen).to(torch.bfloat16) for _ in range(3))
    g[1, 40], g[4, 95], u[2, 7] = float("nan"), float("nan"), float("nan")
    h, kept = bq.glu(g, u, Scheme(fmt, "mx"), act)
    dg, du = bq.glu_backward(dh, kept)
    for r, c in ((1, 40), (4, 95)):
        assert torch.isnan(h[r, c]) and torch.isnan(dg[r, c]) and torch.isnan(du[r, c])
    assert torch.isnan(h[2, 7]) and torch.isnan(dg[2, 7]) and torch.isfinite(du[2, 7])


# NaN codes alone, every sign and payload of each format, in the gate's and in the up copy
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("fmt,codes", [("e4m3", (0x7F, 0xFF)), ("e5m2", (0x7D, 0x7E, 0x7F, 0xFD, 0xFE, 0xFF))])
def test_nan_codes(fmt, codes, act):
    gen = torch.Generator("cuda").manual_seed(4)
    g, u, dh = (torch.randn(2, 64, device="cuda", generator=gen).to(torch.bfloat16) for _ in range(3))
    _, kept = bq.glu(g, u, Scheme(fmt, "mx"), act)
    dg0, du0 = bq.glu_backward(dh, kept)
    for i, code in enumerate(codes):
        kept.gate.codes[0, 3 * i] = code
        kept.up.codes[1, 5 * i] = code
    dg, du = bq.glu_backward(dh, kept)
    nan_g = torch.zeros(2, 64, dtype=torch.bool, device="cuda")
    nan_u = nan_g.clone()
    nan_u[0, 0:3 * len(codes):3] = True
    nan_g[0, 0:3 * len(codes):3] = True
    nan_g[1, 0:5 * len(codes):5] = True
    assert torch.equal(torch.isnan(dg), nan_g) and torch.equal(torch.isnan(du), nan_u)
    assert torch.equal(dg[~nan_g], dg0[~nan_g]) and torch.equal(du[~nan_u], du0[~nan_u])


# dh u past fp32's range under a slope that brings it back, gates far below where the logistic
# function underflows, and small products that lose nothing on the way. Tolerances as bq.h states
# them (and test_gpu_glu.py derives them): (2^-8 + E) of the value, E = (|v| + 8) 2^-22, and 2^-126
# of the other factors; the slope is a sum of two terms with errors of their own.
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2", "int8_sym"])
def test_products_out_of_range(fmt, act):
    gates = np.array([-300.0, -120.0, -100.0, -88.0, -87.0, -60.0, -20.0, -9.0, -4.0, -1.0, 0.5, 3.0, 40.0])
    sizes = [(80, 60), (127, 100), (126, 1), (1, 126), (90, 90), (-60, 100), (100, -60), (-100, -20), (64, 64)]
    rng = np.random.default_rng(11)
    rows = [(a, b) for a in gates for b in sizes]
    g = np.repeat(np.array([a for a, _ in rows])[:, None], 64, 1) * rng.uniform(0.9, 1.1, (len(rows), 64))
    u, dh = (np.ldexp(rng.uniform(1.0, 1.9, g.shape) * rng.choice([-1.0, 1.0], g.shape),
                      np.array([b[i] for _, b in rows])[:, None]) for i in (1, 0))
    g, u, dh = (torch.from_numpy(t.astype(np.float32)).to(torch.bfloat16) for t in (g, u, dh))
    h, kept = bq.glu(g.cuda(), u.cuda(), Scheme(fmt, "mx"), act)
    dg, du = (t.float().cpu().numpy().astype(np.float64) for t in bq.glu_backward(dh.cuda(), kept))
    gv, uv = (ref.values(q.codes.cpu().numpy(), q.scales.cpu().numpy(), None, *g.shape, oracle.Scheme(fmt, "mx"))
              for q in (kept.gate, kept.up))
    d = dh.float().numpy().astype(np.float64)
    rg, ru = ref.glu_backward(d, gv, uv, act)
    c = gv if act == "silu" else np.clip(gv, -12, 12)
    k = 2 * np.sqrt(2 / np.pi)
    v, dv = (c, np.ones_like(c)) if act == "silu" else (k * (c + 0.044715 * c ** 3), k * (1 + 0.134145 * c * c))
    e, s, floor = (np.abs(v) + 8) * 2.0 ** -22, ref.logistic(v), 2.0 ** -126
    slope = e * (s + np.abs(c * dv * s)) + np.abs(c * dv * s) * 2.0 ** -22 + floor * (1 + np.abs(c * dv))
    tol_g = 2.0 ** -8 * np.abs(rg) + (1 + 2.0 ** -8) * np.abs(d * uv) * slope + floor
    tol_u = (2.0 ** -8 + e) * np.abs(ru) + floor * (1 + np.abs(d * gv))
    top = 2.0 ** 128 * (1 - 2.0 ** -9)           # what rounds to a finite bf16
    for got, want, tol in ((dg, rg, tol_g), (du, ru, tol_u)):
        fin = np.abs(want) + tol < top
        assert fin.sum() > fin.size // 2 and np.isfinite(got[fin]).all()
        bad = fin & ~(np.abs(got - want) <= tol)
        assert not bad.any(), (np.argwhere(bad)[:4], got[bad][:4], want[bad][:4], tol[bad][:4])
        over = np.abs(want) - tol > top
        assert np.array_equal(got[over], np.sign(want[over]) * np.inf)

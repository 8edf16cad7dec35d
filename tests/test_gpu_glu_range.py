"""The gated activation where values leave the ordinary range: NaN, and products that overflow."""

import pytest
import torch

import block_scaled_bit_bq_b200 as bq
from block_scaled_bit_bq_b200 import Scheme

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

"""Pins of the float64 linear layer and gated activation (no GPU).

The code values against the C oracle's dequantize, the activation against its published
values, and its derivative against central differences.
"""

import numpy as np
import pytest

import oracle
import synth
from oracle import linear as ref


@pytest.mark.parametrize("fmt,gran", [("e2m1", "mx"), ("e2m1", "nv"), ("e4m3", "mx"), ("e5m2", "mx"), ("int8_sym", "mx")])
def test_values_are_the_oracle_dequantize(fmt, gran):
    s = oracle.Scheme(fmt, gran)
    o = oracle.quantize(synth.bf16_bits(synth.weight_outliers(9, 96, seed=5)), s, stats=False)
    v = ref.values(o["codes"], o["scales"], o["tensor_scale"], 9, 96, s)
    d = oracle.dequantize(o["codes"], o["scales"], o["zps"], o["tensor_scale"], 9, 96, s).astype(np.float64)
    # MX values are exact in fp32; NV's fp32 dequantize rounds once (half a step: 2^-24)
    assert np.all(np.abs(v - d) <= (0.0 if gran == "mx" else 2.0 ** -24 * np.abs(v)))


def test_activation_values():
    # silu(1) = 1 / (1 + 1/e); gelu's tanh form at 1: 0.5 (1 + tanh(sqrt(2/pi) 1.044715))
    assert abs(ref.act(1.0, "silu")[0] - 0.7310585786300049) < 1e-15
    assert abs(ref.act(1.0, "gelu")[0] - 0.8411919906082768) < 1e-15
    for k in ("silu", "gelu"):
        assert tuple(map(float, ref.act(0.0, k))) == (0.0, 0.5)
        assert ref.act(40.0, k)[0] == 40.0 and abs(ref.act(-40.0, k)[0]) < 1e-15


@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_slope_against_differences(kind):
    g = np.linspace(-9.0, 9.0, 721)
    h = 1e-5
    d = (ref.act(g + h, kind)[0] - ref.act(g - h, kind)[0]) / (2 * h)
    # truncation h^2 |a'''| / 6 < 1e-10, rounding 10 * 2^-53 / h ~ 1e-10
    assert np.max(np.abs(ref.act(g, kind)[1] - d)) < 1e-9


@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_glu_gradient_against_differences(kind):
    rng = np.random.default_rng(3)
    g, u, dh = rng.normal(size=(3, 4, 32))
    dg, du = ref.glu_backward(dh, g, u, kind)
    h = 1e-5
    for name, at in (("g", dg), ("u", du)):
        for i in (0, 17, 99):
            e = np.zeros(128)
            e[i] = h
            e = e.reshape(4, 32)
            if name == "g":
                f = (np.sum(dh * ref.glu(g + e, u, kind)) - np.sum(dh * ref.glu(g - e, u, kind))) / (2 * h)
            else:
                f = (np.sum(dh * ref.glu(g, u + e, kind)) - np.sum(dh * ref.glu(g, u - e, kind))) / (2 * h)
            assert abs(f - at.reshape(-1)[i]) < 1e-8

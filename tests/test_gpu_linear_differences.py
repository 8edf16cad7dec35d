"""The weight gradient against differences of the forward product: one code of the weight is
changed, and the loss sum(dy * (x W^T)) changes by that step times dw there.

The layer's input is the values of its own 8-bit copy (bf16 numbers), so that forward product
and gradient are of the same function. y is off by (k / 8 + 32) 2^-23 of the sum of magnitudes,
dw by (m / 8 + 32) 2^-23 of its own (as derived in test_gpu_linear.py), NV's tensor scale and
the fp32 output round once more each (2^-23 together)."""

import numpy as np
import pytest
import torch

import oracle
import block_scaled_bit_bq_b200 as bq
from block_scaled_bit_bq_b200 import Scheme
from oracle import linear as ref

pytestmark = pytest.mark.gpu


def _f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


@pytest.mark.parametrize("gran", ["mx", "nv"])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2", "int8_sym"])
@pytest.mark.parametrize("m", [9, 40])
def test_weight_gradient_against_differences(m, fmt, gran):
    n, k = 72, 96
    gen = torch.Generator("cuda").manual_seed(12)
    kept = bq.quantize(torch.randn(m, k, device="cuda", generator=gen).to(torch.bfloat16), Scheme(fmt, "mx"), stats=False)
    w = bq.quantize(torch.randn(n, k, device="cuda", generator=gen).to(torch.bfloat16), Scheme("e2m1", gran), stats=False)
    x = bq.dequantize(kept, torch.bfloat16)
    assert torch.equal(x.float(), bq.dequantize(kept, torch.float32))
    dy = torch.randn(m, n, device="cuda", generator=gen).to(torch.bfloat16)
    dw = _f64(bq.linear_grad_weight(dy, kept))
    os_ = oracle.Scheme("e2m1", gran)
    ts = None if w.tensor_scale is None else w.tensor_scale.cpu().numpy()

    def values():
        return ref.values(w.codes.cpu().numpy(), w.scales.cpu().numpy(), ts, n, k, os_)

    v0, y0 = values(), _f64(bq.linear(x, w, torch.float32))
    rng = np.random.default_rng(13)
    told_apart = 0
    for _ in range(16):
        o, c = int(rng.integers(n)), int(rng.integers(k))
        old = int(w.codes[o, c // 2])
        w.codes[o, c // 2] = old ^ (8 << (4 * (c & 1)))          # the other sign
        v1, y1 = values(), _f64(bq.linear(x, w, torch.float32))
        w.codes[o, c // 2] = old
        step = v1[o, c] - v0[o, c]
        assert np.count_nonzero(v1 - v0) <= 1
        got, want = np.sum(_f64(dy) * (y1 - y0)), step * dw[o, c]
        a, d = np.abs(_f64(x)), np.abs(_f64(dy))
        # an output depends on its own row of W alone: the others keep their bits, and add nothing to
        # the difference or to its error
        assert np.array_equal(np.delete(y1, o, 1), np.delete(y0, o, 1))
        tol = ((k / 8 + 32 + 1) * 2.0 ** -23 * (d[:, o] @ (a @ (np.abs(v0[o]) + np.abs(v1[o]))))
               + (m / 8 + 32 + 1) * 2.0 ** -23 * abs(step) * (d[:, o] @ a[:, c]))
        assert abs(got - want) <= tol, (o, c, got, want, tol)
        told_apart += abs(want) > 8 * tol
    assert told_apart >= 4

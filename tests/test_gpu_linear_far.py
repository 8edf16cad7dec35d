"""The linear layer and the gated activation where offsets pass 32 bits: codes of more than 2^32
bytes, outputs of more than 2^32 elements. The matrices are made of random codes on the GPU;
their first and last rows are compared with float64 (tolerances as in test_gpu_linear.py and
test_gpu_glu.py)."""

import numpy as np
import pytest
import torch

import oracle
import block_scaled_bit_bq_b200 as bq
from block_scaled_bit_bq_b200 import Scheme
from oracle import linear as ref

pytestmark = pytest.mark.gpu

W4, X8 = Scheme("e2m1", "mx").resolved(), Scheme("int8_sym", "mx").resolved()


def _f64(t):
    return t.float().cpu().numpy().astype(np.float64)


def _codes(s, rows, k, gen):
    width = k // 2 if s.fmt == "e2m1" else k
    codes = torch.empty(rows, width, dtype=torch.uint8, device="cuda")
    codes.random_(0, 256, generator=gen)
    scales = torch.empty(rows * (k // 32), dtype=torch.uint8, device="cuda")
    scales.random_(118, 124, generator=gen)
    return bq.Quantized(s, rows, k, codes, scales, None, None, None)


def _values(q, a, b):
    return ref.values(q.codes[a:b].cpu().numpy(), q.scales.view(q.rows, -1)[a:b].cpu().numpy(), None, b - a, q.cols,
                      oracle.Scheme(q.scheme.fmt, "mx"))


def _near(got, a, b, steps, half):
    r = a @ b
    tol = (steps / 8 + 32) * 2.0 ** -23 * (np.abs(a) @ np.abs(b)) + half * np.abs(r) + 1e-40
    assert np.all(np.abs(_f64(got) - r) <= tol)


def test_weight_codes_past_32_bits():
    n, k = 2 ** 21 + 77, 4128
    gen = torch.Generator("cuda").manual_seed(1)
    q = _codes(W4, n, k, gen)
    assert q.codes.numel() > 2 ** 32
    for m in (3, 20):
        x = torch.randn(m, k, device="cuda", generator=gen).to(torch.bfloat16)
        y = bq.linear(x, q, torch.float32)
        for a, b in ((0, 70), (n - 70, n)):
            _near(y[:, a:b], _f64(x), _values(q, a, b).T, k, 2.0 ** -23)
    # the input gradient of outputs that touch the first and the last rows only
    dy = torch.zeros(20, n + 3, dtype=torch.bfloat16, device="cuda")[:, :n]
    dy[:, :50] = torch.randn(20, 50, device="cuda", generator=gen).to(torch.bfloat16)
    dy[:, n - 50:] = torch.randn(20, 50, device="cuda", generator=gen).to(torch.bfloat16)
    v = np.concatenate((_values(q, 0, 50), _values(q, n - 50, n)))
    d = np.concatenate((_f64(dy[:, :50]), _f64(dy[:, n - 50:])), 1)
    # sums over zeros are exact: 100 steps that add anything
    _near(bq.linear_grad_input(dy, q, torch.float32), d, v, 100, 2.0 ** -23)


def test_kept_codes_past_32_bits():
    m, k, n = 2 ** 20 + 33, 4128, 40
    gen = torch.Generator("cuda").manual_seed(2)
    q = _codes(X8, m, k, gen)
    assert q.codes.numel() > 2 ** 32
    dy = torch.zeros(m, n, dtype=torch.bfloat16, device="cuda")
    dy[:60] = torch.randn(60, n, device="cuda", generator=gen).to(torch.bfloat16)
    dy[m - 60:] = torch.randn(60, n, device="cuda", generator=gen).to(torch.bfloat16)
    v = np.concatenate((_values(q, 0, 60), _values(q, m - 60, m)))
    d = np.concatenate((_f64(dy[:60]), _f64(dy[m - 60:])))
    _near(bq.linear_grad_weight(dy, q), d.T, v, 120, 2.0 ** -23)


def test_outputs_past_32_bits():
    m, n, k = 66001, 66004, 32
    gen = torch.Generator("cuda").manual_seed(3)
    q = _codes(W4, n, k, gen)
    x = torch.randn(m, k, device="cuda", generator=gen).to(torch.bfloat16)
    y = bq.linear(x, q)
    assert y.numel() > 2 ** 32
    for a in (0, m // 2, m - 40):
        for b in (0, n - 300):
            _near(y[a:a + 40, b:b + 300], _f64(x[a:a + 40]), _values(q, b, b + 300).T, k, 2.0 ** -8)


def test_gated_activation_past_32_bits():
    rows, cols = 65537 + 8, 65536
    gen = torch.Generator("cuda").manual_seed(4)
    g = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    u = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    assert g.numel() > 2 ** 32
    h, kept = bq.glu(g, u, Scheme("e4m3", "mx"))
    dg, du = bq.glu_backward(h, kept)
    for a in (0, rows - 2):
        part = bq.glu(g[a:a + 2].clone(), u[a:a + 2].clone(), Scheme("e4m3", "mx"))
        assert torch.equal(h[a:a + 2], part[0])
        for whole, one in ((kept.gate, part[1].gate), (kept.up, part[1].up)):
            assert torch.equal(whole.codes[a:a + 2], one.codes)
            assert torch.equal(whole.scales.view(rows, -1)[a:a + 2].reshape(-1), one.scales)
        back = bq.glu_backward(h[a:a + 2].clone(), part[1])
        assert torch.equal(dg[a:a + 2], back[0]) and torch.equal(du[a:a + 2], back[1])

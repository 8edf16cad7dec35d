"""The gated activation with 8-bit copies (bq_glu, bq_glu_backward) on the GPU against the
float64 definition, and the layers' forward and backward passes together.

Copies: the codes and scales are bq_quantize's, bit for bit. Values: the logistic function
comes from an exp2 and a reciprocal of relative error at most 2^-22 each, of an argument
rounded to fp32 (|v| 2^-24 more in exp(-v)); where exp(-v) overflows it is 0 for a true value
below 2^-127. With E = (|v| + 8) 2^-22 its relative error, h and du are off by
(2^-8 + E) |ref| + 2^-126 |dh or u| |g|. The slope s + g s (1 - s) v' is a sum of terms whose
errors stay absolute: E (s + |c v' s|) + |c v' s| 2^-22 (1 - s from a rounded s), c the argument cut at 12.
"""

import numpy as np
import pytest
import torch

import oracle
import block_scaled_bit_bq_b200 as bq
from block_scaled_bit_bq_b200 import Scheme
from oracle import linear as ref

pytestmark = pytest.mark.gpu

SCHEMES = [Scheme("e4m3", "mx"), Scheme("e5m2", "mx"), Scheme("int8_sym", "mx")]
SHAPES = [(1, 32), (1, 64), (3, 96), (2, 1056), (37, 1376), (129, 512), (300, 160), (1, 11008), (700, 2048)]
TINY = 2.0 ** -126


def _bf16(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(torch.bfloat16)


def _f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _inputs(rows, cols, seed, spread=1.5):
    rng = np.random.default_rng(seed)
    g, u, dh = (rng.normal(size=(3, rows, cols)) * np.array([spread, 1.0, 0.01]).reshape(3, 1, 1))
    g[:, ::7] *= 6.0
    return _bf16(g), _bf16(u), _bf16(dh)


def _arg(g, act):
    if act == "silu":
        return g, g, np.ones_like(g)
    c = np.clip(g, -12, 12)
    k = 2 * np.sqrt(2 / np.pi)
    return c, k * (c + 0.044715 * c ** 3), k * (1 + 3 * 0.044715 * c * c)


def _check_h(h, g, u, act):
    r = ref.glu(g, u, act)
    _, v, _ = _arg(g, act)
    e = (np.abs(v) + 8) * 2.0 ** -22
    bad = ~(np.abs(_f64(h) - r) <= (2.0 ** -8 + e) * np.abs(r) + TINY * (1 + np.abs(g * u)))
    assert not bad.any(), (np.argwhere(bad)[:4], _f64(h)[bad][:4], r[bad][:4])


def _check_back(dg, du, dh, g, u, act):
    rg, ru = ref.glu_backward(dh, g, u, act)
    c, v, dv = _arg(g, act)
    e = (np.abs(v) + 8) * 2.0 ** -22
    s = ref.logistic(v)
    bad = ~(np.abs(_f64(du) - ru) <= (2.0 ** -8 + e) * np.abs(ru) + TINY * (1 + np.abs(dh * g)))
    assert not bad.any(), (np.argwhere(bad)[:4], _f64(du)[bad][:4], ru[bad][:4])
    slope = e * (s + np.abs(c * dv * s)) + np.abs(c * dv * s) * 2.0 ** -22 + TINY * (1 + np.abs(c * dv))
    bad = ~(np.abs(_f64(dg) - rg) <= 2.0 ** -8 * np.abs(rg) + (1 + 2.0 ** -8) * np.abs(dh * u) * slope + TINY)
    assert not bad.any(), (np.argwhere(bad)[:4], _f64(dg)[bad][:4], rg[bad][:4])


def _values(q):
    return ref.values(q.codes.cpu().numpy(), q.scales.cpu().numpy(), None, q.rows, q.cols,
                      oracle.Scheme(q.scheme.fmt, "mx"))


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda t: "x".join(map(str, t)))
@pytest.mark.parametrize("s", SCHEMES, ids=lambda s: s.fmt)
def test_glu_and_backward(s, shape, act):
    g, u, dh = _inputs(*shape, seed=70 + shape[1])
    h, kept = bq.glu(g.cuda(), u.cuda(), s, act)
    _check_h(h, _f64(g), _f64(u), act)
    for a, q in ((g, kept.gate), (u, kept.up)):
        want = bq.quantize(a.cuda(), s, stats=False)
        assert torch.equal(q.codes, want.codes) and torch.equal(q.scales, want.scales)
    dg, du = bq.glu_backward(dh.cuda(), kept)
    _check_back(dg, du, _f64(dh), _values(kept.gate), _values(kept.up), act)
    h2, none = bq.glu(g.cuda(), u.cuda(), None, act)
    assert none is None and torch.equal(h, h2)


# the halves of one projection's output, and one buffer for both gradients
@pytest.mark.parametrize("cols", [64, 1376])
def test_halves_of_one_tensor(cols):
    g, u, dh = _inputs(19, cols, 80)
    gu = torch.cat((g, u), 1).cuda()
    h, kept = bq.glu(gu[:, :cols], gu[:, cols:], SCHEMES[0])
    h2, kept2 = bq.glu(g.cuda(), u.cuda(), SCHEMES[0])
    assert torch.equal(h, h2) and torch.equal(kept.gate.codes, kept2.gate.codes)
    assert torch.equal(kept.up.scales, kept2.up.scales)
    buf = torch.full((24, 2 * cols), 5.0, dtype=torch.bfloat16, device="cuda")
    wide = torch.full((19, cols + 32), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, :cols] = dh.cuda()
    bq.glu_backward(wide[:, :cols], kept, out=(buf[:19, :cols], buf[:19, cols:]))
    dg, du = bq.glu_backward(dh.cuda(), kept2)
    assert torch.equal(buf[:19, :cols], dg) and torch.equal(buf[:19, cols:], du) and torch.all(buf[19:] == 5.0)
    # rows that are not a multiple of 16 elements apart, an unaligned start, transposed inputs
    odd = torch.zeros(19, 2 * cols + 9, dtype=torch.bfloat16, device="cuda")
    odd[:, 1:1 + cols], odd[:, 5 + cols:5 + 2 * cols] = g.cuda(), u.cuda()
    assert torch.equal(bq.glu(odd[:, 1:1 + cols], odd[:, 5 + cols:5 + 2 * cols])[0], h)
    assert torch.equal(bq.glu(g.cuda().t().contiguous().t(), u.cuda())[0], h)


# blocks of zeros, signed zeros, values at both ends of the range, and large arguments
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("s", SCHEMES, ids=lambda s: s.fmt)
def test_extreme_values(s, act):
    rng = np.random.default_rng(8)
    g = rng.normal(size=(64, 64)) * np.exp2(np.linspace(-110, 40, 64)).reshape(64, 1)
    u = rng.normal(size=(64, 64)) * np.exp2(np.linspace(60, -110, 64)).reshape(64, 1)
    g[3, :32], u[5] = 0.0, 0.0
    g[4, :32] = -0.0
    g, u, dh = _bf16(g), _bf16(u), _bf16(rng.normal(size=(64, 64)))
    h, kept = bq.glu(g.cuda(), u.cuda(), s, act)
    _check_h(h, _f64(g), _f64(u), act)
    for a, q in ((g, kept.gate), (u, kept.up)):
        want = bq.quantize(a.cuda(), s, stats=False)
        assert torch.equal(q.codes, want.codes) and torch.equal(q.scales, want.scales)
    dg, du = bq.glu_backward(dh.cuda(), kept)
    assert torch.isfinite(dg.float()).all() and torch.isfinite(du.float()).all()
    _check_back(dg, du, _f64(dh), _values(kept.gate), _values(kept.up), act)


def test_non_finite_values_stay_in_their_block():
    g, u, dh = _inputs(4, 128, 81)
    clean, kept_clean = bq.glu(g.cuda(), u.cuda(), SCHEMES[0])
    g[1, 40], u[2, 100] = float("nan"), float("inf")
    h, kept = bq.glu(g.cuda(), u.cuda(), SCHEMES[0])
    dg, du = bq.glu_backward(dh.cuda(), kept)
    dg0, du0 = bq.glu_backward(dh.cuda(), kept_clean)
    ok = torch.ones(4, 128, dtype=torch.bool, device="cuda")
    ok[1, 32:64], ok[2, 96:128] = False, False
    assert torch.equal(h[ok], clean[ok]) and torch.equal(dg[ok], dg0[ok]) and torch.equal(du[ok], du0[ok])


def test_empty_and_writes_stay_inside():
    e = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    h, kept = bq.glu(e, e, SCHEMES[0])
    assert h.shape == (0, 64) and bq.glu_backward(e, kept)[0].shape == (0, 64)
    g, u, dh = _inputs(3, 96, 82)
    s = SCHEMES[2].resolved()
    bufs = [torch.full((3 * 96 + 512,), 77, dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.full((9 + 55,), 77, dtype=torch.uint8, device="cuda") for _ in range(2)]
    kept = bq.GluCheckpoint(*(bq.Quantized(s, 3, 96, b[:288].view(3, 96), c[:9], None, None, None)
                              for b, c in zip(bufs, scales)), "silu")
    hb = torch.full((3 * 96 + 512,), 7.0, dtype=torch.bfloat16, device="cuda")
    bq.glu(g.cuda(), u.cuda(), s, "gelu", out=hb[:288].view(3, 96), ckpt=kept)
    _check_h(hb[:288].view(3, 96), _f64(g), _f64(u), "gelu")
    assert kept.act == "gelu" and torch.all(hb[288:] == 7.0)
    for b, c, a in zip(bufs, scales, (g, u)):
        want = bq.quantize(a.cuda(), s, stats=False)
        assert torch.equal(b[:288].view(3, 96), want.codes) and torch.equal(c[:9], want.scales)
        assert torch.all(b[288:] == 77) and torch.all(c[9:] == 77)


def test_streams_and_graphs():
    g, u, dh = (t.cuda() for t in _inputs(65, 1056, 83))
    h, kept = bq.glu(g, u, SCHEMES[0])
    want = (h, *bq.glu_backward(dh, kept))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    h2, kept2 = bq.glu(g, u, SCHEMES[0], stream=side)
    got = (h2, *bq.glu_backward(dh, kept2, stream=side))
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    gs, us = torch.zeros_like(g), torch.zeros_like(u)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h3, kept3 = bq.glu(gs, us, SCHEMES[0])
        back = bq.glu_backward(dh, kept3)
    for _ in range(2):
        gs.copy_(g)
        us.copy_(u)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, (h3, *back)))


def test_python_refusals():
    g, u, dh = (t.cuda() for t in _inputs(4, 64, 84))
    h, kept = bq.glu(g, u, SCHEMES[0])
    for call in (lambda: bq.glu(g, u[:2], SCHEMES[0]), lambda: bq.glu(g.float(), u.float(), SCHEMES[0]),
                 lambda: bq.glu(g[0], u[0], SCHEMES[0]), lambda: bq.glu(g, u.cpu(), SCHEMES[0]),
                 lambda: bq.glu(g, u, SCHEMES[1], ckpt=kept), lambda: bq.glu(g[:2], u[:2], SCHEMES[0], ckpt=kept),
                 lambda: bq.glu(g, u, ckpt=kept), lambda: bq.glu(g, u, out=torch.empty(4, 64, device="cuda")),
                 lambda: bq.glu_backward(dh[:2], kept), lambda: bq.glu_backward(dh[:, :32], kept),
                 lambda: bq.glu_backward(dh, kept, out=(torch.empty_like(dh), torch.empty_like(dh)[:2]))):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(KeyError):
        bq.glu(g, u, SCHEMES[0], "relu")
    for call in (lambda: bq.glu(g, u, Scheme("e4m3", "mx", layout="gemm")), lambda: bq.glu(g, u, Scheme("int8_sym", "row")),
                 lambda: bq.glu_backward(dh, kept, out=(dh.clone(),) * 2)):
        with pytest.raises(bq.BqError):
            call()


# The layers together: a gated block's forward pass on 4-bit weights, then every gradient
# from the 8-bit copies. Each stage's result is rounded to bf16 (2^-9 rms of a value); the
# reference rounds nothing, so a result after d stages is off by about sqrt(d) 2^-9 in norm:
# 2^-7 covers d <= 9 twice over. The reference's backward pass starts from the library's own
# copies, whose codes are checked above.
@pytest.mark.parametrize("t", [1, 6, 150])
@pytest.mark.parametrize("gran", ["mx", "nv"])
def test_block_forward_and_backward(gran, t):
    d, f = 256, 352
    rng = np.random.default_rng(9)
    ws, xs = Scheme("e2m1", gran), SCHEMES[0]
    os_ = oracle.Scheme("e2m1", gran)
    wgu, wd = _bf16(rng.normal(size=(2 * f, d)) * d ** -0.5), _bf16(rng.normal(size=(d, f)) * f ** -0.5)
    x, dy = _bf16(rng.normal(size=(t, d))).cuda(), _bf16(rng.normal(size=(t, d))).cuda()
    qgu, qd = (bq.quantize(w.cuda(), ws, stats=False) for w in (wgu, wd))
    vgu, vd = (ref.values(q.codes.cpu().numpy(), q.scales.cpu().numpy(),
                          None if q.tensor_scale is None else q.tensor_scale.cpu().numpy(), q.rows, q.cols, os_)
               for q in (qgu, qd))
    # forward
    x8 = bq.quantize(x, xs, stats=False)
    gu = bq.linear(x, qgu)
    h, kept = bq.glu(gu[:, :f], gu[:, f:], xs)
    h8 = bq.quantize(h, xs, stats=False)
    y = bq.linear(h, qd)
    # backward
    dh = bq.linear_grad_input(dy, qd)
    dwd = bq.linear_grad_weight(dy, h8)
    dgu = torch.empty(t, 2 * f, dtype=torch.bfloat16, device="cuda")
    bq.glu_backward(dh, kept, out=(dgu[:, :f], dgu[:, f:]))
    dwgu = bq.linear_grad_weight(dgu, x8)
    dx = bq.linear_grad_input(dgu, qgu)

    def near(got, want):
        assert np.linalg.norm(_f64(got) - want) <= 2.0 ** -7 * np.linalg.norm(want)

    rgu = _f64(x) @ vgu.T
    rh = ref.glu(rgu[:, :f], rgu[:, f:], "silu")
    near(gu, rgu)
    near(h, rh)
    near(y, rh @ vd.T)
    rdh = _f64(dy) @ vd
    rdgu = np.concatenate(ref.glu_backward(rdh, _values(kept.gate), _values(kept.up), "silu"), 1)
    near(dgu, rdgu)
    near(dx, rdgu @ vgu)
    near(dwd, _f64(dy).T @ _values(h8))
    near(dwgu, rdgu.T @ _values(x8))

"""The linear layer over block-scaled data (bq_linear and its two gradients) on the GPU
against float64 products of the codes' values.

Every product of a code's value (times its block scale) and a bf16 activation is exact in
fp32, so a result is off by its sum and its output rounding alone. The sums run in fp32 in
some order of at most nc / 8 + 32 additions in a row (the tensor cores add 8 or 16 products
at a time; partial sums of a split contraction are joined by fewer than 32 more), each off by
at most 2^-23 (truncation) of the sum of magnitudes so far; NV's tensor scale rounds once
more (2^-24); bf16 rounds by at most 2^-8 of the value, fp32 by 2^-24:
    |got - ref| <= ((nc / 8 + 32) 2^-23) sum |a||b| + half * |ref|.
"""

import numpy as np
import pytest
import torch

import oracle
import synth
import block_scaled_bit_bq_b200 as bq
from block_scaled_bit_bq_b200 import Scheme
from oracle import linear as ref

pytestmark = pytest.mark.gpu

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -23}
W_SCHEMES = [Scheme("e2m1", "mx"), Scheme("e2m1", "nv")]
X_SCHEMES = [Scheme("e4m3", "mx"), Scheme("e5m2", "mx"), Scheme("int8_sym", "mx")]


def _bf16(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(torch.bfloat16)


def _f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _quantized(a, s):
    """A bf16 CPU matrix quantized on the GPU, and the float64 values of its codes."""
    q = bq.quantize(a.cuda(), s, stats=False)
    rows, cols = a.shape
    sc = q.scales.cpu().numpy()
    if s.layout == "gemm":
        sc = oracle.scales_from_gemm(sc, rows, cols // (32 if s.gran == "mx" else 16))
    os_ = oracle.Scheme(s.fmt, s.gran)
    ts = None if q.tensor_scale is None else q.tensor_scale.cpu().numpy()
    return q, ref.values(q.codes.cpu().numpy(), sc, ts, rows, cols, os_)


def _weight(n, k, s, seed):
    return _quantized(synth.weight_outliers(n, k, seed=seed), s)


def _acts(m, k, seed):
    rng = np.random.default_rng(seed)
    return _bf16(rng.standard_t(3, size=(m, k)) * 0.5)


def _close(got, a, b, dtype, nc):
    """got against a @ b (float64)."""
    r = a @ b
    tol = (nc / 8 + 32) * 2.0 ** -23 * (np.abs(a) @ np.abs(b)) + HALF[dtype] * np.abs(r) + 1e-40
    assert got.dtype == dtype and tuple(got.shape) == r.shape
    bad = ~(np.abs(_f64(got) - r) <= tol)
    assert not bad.any(), (np.argwhere(bad)[:5], _f64(got)[bad][:5], r[bad][:5], tol[bad][:5])


# one token, a few, a ragged tile, several tiles; widths below, at and past the tiles' edges
SHAPES = [(1, 1, 32), (1, 128, 64), (2, 16, 128), (3, 129, 96), (5, 40, 1056), (8, 64, 4096), (9, 130, 512), (16, 257, 160),
          (17, 33, 2080), (33, 300, 320), (64, 128, 128), (65, 8, 32), (130, 384, 1056), (257, 513, 416), (513, 1000, 96),
          (48, 2049, 1024), (96, 4100, 2048), (1, 4096, 4096), (200, 96, 11008), (1000, 2200, 160)]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda t: "x".join(map(str, t)))
@pytest.mark.parametrize("s", W_SCHEMES, ids=lambda s: s.gran)
def test_linear(s, shape):
    m, n, k = shape
    q, w = _weight(n, k, s, 900 + n)
    x = _acts(m, k, 901 + m)
    for dt in (torch.bfloat16, torch.float32):
        _close(bq.linear(x.cuda(), q, dt), _f64(x), w.T, dt, k)


@pytest.mark.parametrize("shape", SHAPES, ids=lambda t: "x".join(map(str, t)))
@pytest.mark.parametrize("s", W_SCHEMES, ids=lambda s: s.gran)
def test_grad_input(s, shape):
    m, n, k = shape
    q, w = _weight(n, k, s, 920 + n)
    dy = _acts(m, n, 921 + m)
    for dt in (torch.bfloat16, torch.float32):
        _close(bq.linear_grad_input(dy.cuda(), q, dt), _f64(dy), w, dt, n)


@pytest.mark.parametrize("shape", SHAPES, ids=lambda t: "x".join(map(str, t)))
@pytest.mark.parametrize("s", X_SCHEMES, ids=lambda s: s.fmt)
def test_grad_weight(s, shape):
    m, n, k = shape
    q, xv = _quantized(_acts(m, k, 940 + m), s)
    dy = _acts(m, n, 941 + n)
    for dt in (torch.bfloat16, torch.float32):
        _close(bq.linear_grad_weight(dy.cuda(), q, dt), _f64(dy).T, xv, dt, m)


# products large enough for tiles on pairs of SMs, one to three tiles each; ragged in every
# direction (output rows, output columns, contraction length)
@pytest.mark.parametrize("s", W_SCHEMES, ids=lambda s: s.gran)
@pytest.mark.parametrize("shape", [(2560, 2048, 64), (1100, 4700, 96), (2100, 5001, 672)], ids=lambda t: "x".join(map(str, t)))
def test_linear_many_tiles(s, shape):
    m, n, k = shape
    q, w = _weight(n, k, s, 950 + n)
    x = _acts(m, k, 951 + m)
    for dt in (torch.bfloat16, torch.float32):
        _close(bq.linear(x.cuda(), q, dt), _f64(x), w.T, dt, k)


@pytest.mark.parametrize("s", W_SCHEMES, ids=lambda s: s.gran)
@pytest.mark.parametrize("shape", [(2560, 64, 2048), (1100, 201, 4640), (2100, 700, 4992)], ids=lambda t: "x".join(map(str, t)))
def test_grad_input_many_tiles(s, shape):
    m, n, k = shape
    q, w = _weight(n, k, s, 952 + n)
    dy = _acts(m, n, 953 + m)
    for dt in (torch.bfloat16, torch.float32):
        _close(bq.linear_grad_input(dy.cuda(), q, dt), _f64(dy), w, dt, n)


@pytest.mark.parametrize("s", X_SCHEMES, ids=lambda s: s.fmt)
@pytest.mark.parametrize("shape", [(64, 2560, 2048), (201, 1101, 4640), (700, 2100, 4992)], ids=lambda t: "x".join(map(str, t)))
def test_grad_weight_many_tiles(s, shape):
    m, n, k = shape
    q, xv = _quantized(_acts(m, k, 954 + m), s)
    dy = _acts(m, n, 955 + n)
    for dt in (torch.bfloat16, torch.float32):
        _close(bq.linear_grad_weight(dy.cuda(), q, dt), _f64(dy).T, xv, dt, m)


# every row and block of the scales' tiled layout: more than 128 rows, several tiles of blocks
@pytest.mark.parametrize("m", [1, 11, 40, 300])
@pytest.mark.parametrize("s", [Scheme("e2m1", "mx", layout="gemm"), Scheme("e2m1", "nv", layout="gemm")],
                         ids=lambda s: s.gran)
def test_weight_scales_in_the_gemm_layout(s, m):
    q, w = _weight(390, 640, s, 960)
    x, dy = _acts(m, 640, 961), _acts(m, 390, 962)
    _close(bq.linear(x.cuda(), q, torch.float32), _f64(x), w.T, torch.float32, 640)
    _close(bq.linear_grad_input(dy.cuda(), q, torch.float32), _f64(dy), w, torch.float32, 390)


def test_kept_input_scales_in_the_gemm_layout():
    q, xv = _quantized(_acts(200, 640, 963), Scheme("e4m3", "mx", layout="gemm"))
    dy = _acts(200, 70, 964)
    _close(bq.linear_grad_weight(dy.cuda(), q), _f64(dy).T, xv, torch.float32, 200)


# block scales over the whole exponent range: 2^-100 to 2^100 within one matrix, rows of zeros
@pytest.mark.parametrize("m", [4, 40])
@pytest.mark.parametrize("s", W_SCHEMES + X_SCHEMES, ids=lambda s: f"{s.fmt}-{s.gran}")
def test_scales_of_any_size(s, m):
    rows, k = 160, 192
    rng = np.random.default_rng(5)
    a = rng.normal(size=(rows, k))
    if s.gran == "mx":
        a *= np.ldexp(1.0, rng.integers(-100, 100, size=(rows, 1)))
    else:
        a *= np.ldexp(1.0, rng.integers(-12, 3, size=(rows, 1)))
    a[7] = 0.0
    a[:, 32:64] = 0.0
    q, v = _quantized(_bf16(a), s)
    if s in W_SCHEMES:
        x = _acts(m, k, 6)
        _close(bq.linear(x.cuda(), q, torch.float32), _f64(x), v.T, torch.float32, k)
    # the contraction runs over the rows: gradients that undo their sizes
    size = np.maximum(np.abs(v).max(1, keepdims=True), 1e-36)
    dy = _bf16(rng.normal(size=(rows, m)) / size)
    if s in W_SCHEMES:
        _close(bq.linear_grad_input(dy.t().contiguous().cuda(), q, torch.float32), _f64(dy).T, v, torch.float32, rows)
    else:
        _close(bq.linear_grad_weight(dy.cuda(), q), _f64(dy).T, v, torch.float32, rows)


def test_empty_sums_are_zero():
    q, _ = _weight(16, 64, W_SCHEMES[0], 1)
    assert bq.linear(torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"), q).shape == (0, 16)
    assert bq.linear_grad_input(torch.empty(0, 16, dtype=torch.bfloat16, device="cuda"), q).shape == (0, 64)
    e = bq.quantize(torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"), X_SCHEMES[0], stats=False)
    out = torch.full((24, 64), 7.0, device="cuda")
    bq.linear_grad_weight(torch.empty(0, 24, dtype=torch.bfloat16, device="cuda"), e, out=out)
    assert torch.count_nonzero(out) == 0
    w0 = bq.quantize(torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"), W_SCHEMES[0], stats=False)
    out = torch.full((5, 64), 7.0, device="cuda")
    bq.linear_grad_input(torch.empty(5, 0, dtype=torch.bfloat16, device="cuda"), w0, out=out)
    assert torch.count_nonzero(out) == 0


# rows apart (a slice of a wider tensor), an offset that is not aligned, odd widths
@pytest.mark.parametrize("m", [3, 70])
def test_strided_and_unaligned_operands(m):
    s = W_SCHEMES[0]
    q, w = _weight(201, 96, s, 970)
    wide = _acts(m, 400, 971).cuda()
    for x in (wide[:, 8:104], wide[:, 1:97], wide[:, ::2][:, :96], wide.t().contiguous().t()[:, :96]):
        _close(bq.linear(x, q, torch.float32), _f64(x), w.T, torch.float32, 96)
    for dy in (wide[:, 16:217], wide[:, 3:204], _acts(m, 201, 972).cuda()):
        _close(bq.linear_grad_input(dy, q, torch.float32), _f64(dy), w, torch.float32, 201)
        qx, xv = _quantized(_acts(m, 96, 973), X_SCHEMES[0])
        _close(bq.linear_grad_weight(dy, qx), _f64(dy).T, xv, torch.float32, m)


# nothing is written outside the output, nothing read from padding next to the operands
@pytest.mark.parametrize("m", [5, 37, 150])
def test_writes_stay_inside_and_padding_is_not_read(m):
    n, k = 201, 160
    q, w = _weight(n, k, W_SCHEMES[1], 980)
    pad = torch.full((m + 8, 256), float("nan"), dtype=torch.bfloat16, device="cuda")
    x = _acts(m, k, 981)
    pad[:m, :k] = x.cuda()
    for dt in (torch.bfloat16, torch.float32):
        buf = torch.full((m * n + 4096,), 3.0, dtype=dt, device="cuda")
        out = buf[:m * n].view(m, n)
        bq.linear(pad[:m, :k], q, out=out)
        _close(out, _f64(x), w.T, dt, k)
        assert torch.all(buf[m * n:] == 3.0)
    dy = _acts(m, n, 982)
    pad[:] = float("nan")
    pad[:m, :n] = dy.cuda()
    qx, xv = _quantized(_acts(m, k, 983), X_SCHEMES[0])
    for dt in (torch.bfloat16, torch.float32):
        buf = torch.full((m * k + 4096,), 3.0, dtype=dt, device="cuda")
        bq.linear_grad_input(pad[:m, :n], q, out=buf[:m * k].view(m, k))
        _close(buf[:m * k].view(m, k), _f64(dy), w, dt, n)
        assert torch.all(buf[m * k:] == 3.0)
        buf = torch.full((n * k + 4096,), 3.0, dtype=dt, device="cuda")
        bq.linear_grad_weight(pad[:m, :n], qx, out=buf[:n * k].view(n, k))
        _close(buf[:n * k].view(n, k), _f64(dy).T, xv, dt, m)
        assert torch.all(buf[n * k:] == 3.0)


@pytest.mark.parametrize("m", [6, 50])
def test_non_finite_values_stay_in_their_row(m):
    q, w = _weight(140, 96, W_SCHEMES[0], 990)
    x = _acts(m, 96, 991)
    x[2, 5], x[4, 0] = float("inf"), float("nan")
    y = bq.linear(x.cuda(), q, torch.float32).cpu()
    assert not torch.isfinite(y[4]).any() and not torch.isfinite(y[2]).all()
    keep = [i for i in range(m) if i not in (2, 4)]
    _close(y[keep], _f64(x[keep]), w.T, torch.float32, 96)


# every code, those of NaN and Inf among them; sums of few tokens, so that most stay finite
@pytest.mark.parametrize("fmt,dt", [("e4m3", torch.float8_e4m3fn), ("e5m2", torch.float8_e5m2)])
@pytest.mark.parametrize("m,n", [(3, 72), (2, 600)])
def test_grad_weight_codes_that_are_no_numbers(fmt, dt, m, n):
    k = 1024
    q, _ = _quantized(_acts(m, k, 993), Scheme(fmt, "mx"))
    q.codes.copy_(torch.from_numpy(np.random.default_rng(994).permutation(np.arange(m * k) % 256).astype(np.uint8))
                  .view(q.codes.shape))
    q.scales.fill_(125)
    dy = torch.where(_acts(m, n, 995) < 0, -1.5, 0.75).to(torch.bfloat16)
    got = bq.linear_grad_weight(dy.cuda(), q, torch.float32).cpu().double()
    want = dy.double().T @ (q.codes.cpu().view(m, k).view(dt).double() * 0.25)
    assert torch.isnan(want).any() and torch.equal(torch.isnan(got), torch.isnan(want))
    inf = torch.isinf(want)
    assert torch.equal(torch.isinf(got), inf) and torch.equal(got[inf], want[inf])
    fin = torch.isfinite(want)
    mags = dy.double().abs().T @ torch.nan_to_num(q.codes.cpu().view(m, k).view(dt).double().abs() * 0.25, 0.0, 0.0)
    assert ((got - want).abs()[fin] <= ((m / 8 + 32) * 2.0 ** -23 * mags + 2.0 ** -24 * want.abs())[fin]).all()


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_grad_weight_of_an_input_with_nan(fmt):
    m, n, k = 70, 136, 96
    x = _acts(m, k, 996)
    x[66, 40] = float("nan")
    q = bq.quantize(x.cuda(), Scheme(fmt, "mx"), stats=False)
    dw = bq.linear_grad_weight(torch.ones(m, n, dtype=torch.bfloat16, device="cuda"), q, torch.float32).cpu()
    assert torch.isnan(dw[:, 40]).all()
    assert torch.isfinite(dw[:, :32]).all() and torch.isfinite(dw[:, 64:]).all()


# the same bits from call to call, on another stream, and from a captured graph with new inputs
@pytest.mark.parametrize("m", [1, 7, 24, 300])
def test_repeats_streams_and_graphs(m):
    n, k = 520, 512
    q, w = _weight(n, k, W_SCHEMES[0], 1000)
    xs = [_acts(m, k, 1001 + i).cuda() for i in range(2)]
    dys = [_acts(m, n, 1005 + i).cuda() for i in range(2)]
    qx, _ = _quantized(_acts(m, k, 1009), X_SCHEMES[2])

    def all_three(x, dy, out=(None, None, None), stream=None):
        return (bq.linear(x, q, out=out[0], stream=stream), bq.linear_grad_input(dy, q, out=out[1], stream=stream),
                bq.linear_grad_weight(dy, qx, out=out[2], stream=stream))

    first = [all_three(x, dy) for x, dy in zip(xs, dys)]
    torch.cuda.synchronize()
    for a, b in zip(first[0], all_three(xs[0], dys[0])):
        assert torch.equal(a, b)
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        got = all_three(xs[1], dys[1], stream=stream)
        side.synchronize()
        for a, b in zip(first[1], got):
            assert torch.equal(a, b)
    x, dy = xs[0].clone(), dys[0].clone()
    outs = [torch.empty_like(t) for t in first[0]]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        all_three(x, dy, outs)
    for i in (1, 0, 1):
        x.copy_(xs[i])
        dy.copy_(dys[i])
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(first[i], outs):
            assert torch.equal(a, b)


def test_two_streams_at_once():
    q, w = _weight(1030, 1056, W_SCHEMES[1], 1020)
    streams = [torch.cuda.Stream() for _ in range(2)]
    xs = [_acts(m, 1056, 1021 + m).cuda() for m in (4, 90)]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            outs[i].append(bq.linear(xs[i], q, torch.float32, stream=s))
    torch.cuda.synchronize()
    for i in range(2):
        _close(outs[i][0], _f64(xs[i]), w.T, torch.float32, 1056)
        assert all(torch.equal(o, outs[i][0]) for o in outs[i])
    assert bq.bq_wait_timeouts() == 0


# gradients against differences of the forward product: y is linear in x and in W, so a
# difference of two products is the product of the difference, up to the two sums' roundings
def test_gradients_against_differences():
    m, n, k = 24, 72, 96
    s = X_SCHEMES[0]
    q, w = _weight(n, k, W_SCHEMES[0], 1030)
    qx, xv = _quantized(_acts(m, k, 1031), s)
    dy = _acts(m, n, 1032)
    dx = _f64(bq.linear_grad_input(dy.cuda(), q, torch.float32))
    dw = _f64(bq.linear_grad_weight(dy.cuda(), qx, torch.float32))
    rng = np.random.default_rng(4)
    x0 = _acts(m, k, 1033)
    for _ in range(8):
        t, c = rng.integers(m), rng.integers(k)
        x1 = x0.clone()
        x1[t, c] += 1.0
        step = float(x1[t, c]) - float(x0[t, c])
        y0, y1 = (_f64(bq.linear(x.cuda(), q, torch.float32)) for x in (x0, x1))
        got = np.sum(_f64(dy) * (y1 - y0))
        mag = np.abs(_f64(dy)[t]) @ (np.abs(w) @ (np.abs(_f64(x0)[t]) + np.abs(step)))
        assert abs(got - step * dx[t, c]) <= 4 * (k / 8 + n / 8 + 64) * 2.0 ** -23 * mag
        # loss sum dy (X W^T) at the kept X: its slope in W[o, c]
        o = rng.integers(n)
        assert abs(dw[o, c] - _f64(dy)[:, o] @ xv[:, c]) <= (m / 8 + 33) * 2.0 ** -23 * (np.abs(_f64(dy)[:, o]) @ np.abs(xv[:, c]))


def test_python_refusals():
    q, _ = _weight(16, 64, W_SCHEMES[0], 1040)
    x = _acts(4, 64, 1).cuda()
    qx, _ = _quantized(_acts(4, 64, 2), X_SCHEMES[0])
    for call in (lambda: bq.linear(x.float(), q), lambda: bq.linear(x[0], q), lambda: bq.linear(x[:, :32], q),
                 lambda: bq.linear(x.cpu(), q), lambda: bq.linear_grad_input(x, q), lambda: bq.linear(x, q, torch.float16),
                 lambda: bq.linear(x, q, out=torch.empty(4, 17, device="cuda")),
                 lambda: bq.linear(x, q, out=torch.empty(16, 4, device="cuda").t()),
                 lambda: bq.linear_grad_weight(x[:3], qx)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: bq.linear(x, qx), lambda: bq.linear_grad_weight(_acts(16, 8, 3).cuda(), q)):
        with pytest.raises(bq.BqError):
            call()

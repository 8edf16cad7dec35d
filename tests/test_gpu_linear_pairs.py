"""The linear layer's products that run on pairs of SMs, where one SM's tensor core reads what
the other SM copied and widened: the same bits from call to call, beside another product on a
second stream, and from a captured graph whose inputs change, checked against float64
(tolerances as in test_gpu_linear.py)."""

import numpy as np
import pytest
import torch

import oracle
import synth
import block_scaled_bit_bq_b200 as bq
from block_scaled_bit_bq_b200 import Scheme
from oracle import linear as ref

pytestmark = pytest.mark.gpu

# tokens, outputs, inputs: 64 or 72 tiles of 256 x 256 for 74 pairs of SMs, and a ragged shape of
# several tiles a pair
SHAPES = [(2304, 2048, 2048), (2605, 4801, 4128)]
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -23}


def _bf16(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(torch.bfloat16)


def _f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


class Products:
    """The three products of a layer, two sets of inputs, and their float64 references."""

    def __init__(self, shape, gran, fmt):
        m, n, k = shape
        rng = np.random.default_rng(n + k)
        w = synth.weight_outliers(n, k, seed=n)
        self.w = bq.quantize(w.cuda(), Scheme("e2m1", gran), stats=False)
        xs = [_bf16(rng.standard_t(3, size=(m, k)) * 0.5) for _ in range(2)]
        dys = [_bf16(rng.standard_t(3, size=(m, n)) * 0.5) for _ in range(2)]
        self.x, self.dy = [a.cuda() for a in xs], [a.cuda() for a in dys]
        self.kept = [bq.quantize(a, Scheme(fmt, "mx"), stats=False) for a in self.x]
        self.shape = shape

    def run(self, x, dy, kept, out=(None, None, None)):
        return (bq.linear(x, self.w, out=out[0]), bq.linear_grad_input(dy, self.w, out=out[1]),
                bq.linear_grad_weight(dy, kept, torch.bfloat16, out=out[2]))

    def check(self, i, got):
        m, n, k = self.shape
        ts = None if self.w.tensor_scale is None else self.w.tensor_scale.cpu().numpy()
        w = ref.values(self.w.codes.cpu().numpy(), self.w.scales.cpu().numpy(), ts, n, k,
                       oracle.Scheme("e2m1", self.w.scheme.gran))
        q = self.kept[i]
        xv = ref.values(q.codes.cpu().numpy(), q.scales.cpu().numpy(), None, m, k, oracle.Scheme(q.scheme.fmt, "mx"))
        x, dy = _f64(self.x[i]), _f64(self.dy[i])
        for y, a, b, nc in ((got[0], x, w.T, k), (got[1], dy, w, n), (got[2], dy.T, xv, m)):
            r = a @ b
            tol = (nc / 8 + 32) * 2.0 ** -23 * (np.abs(a) @ np.abs(b)) + HALF[y.dtype] * np.abs(r) + 1e-40
            bad = ~(np.abs(_f64(y) - r) <= tol)
            assert not bad.any(), (tuple(y.shape), np.argwhere(bad)[:5], _f64(y)[bad][:5], r[bad][:5])


@pytest.mark.parametrize("shape", SHAPES, ids=lambda t: "x".join(map(str, t)))
@pytest.mark.parametrize("gran,fmt", [("mx", "e4m3"), ("nv", "int8_sym")])
def test_repeats_streams_and_graphs(shape, gran, fmt):
    p = Products(shape, gran, fmt)
    first = [p.run(p.x[i], p.dy[i], p.kept[i]) for i in range(2)]
    torch.cuda.synchronize()
    for i in range(2):
        p.check(i, first[i])
    # from call to call, alternating, back to back
    later = [[p.run(p.x[i], p.dy[i], p.kept[i]) for i in range(2)] for _ in range(8)]
    torch.cuda.synchronize()
    for pair in later:
        for i in range(2):
            assert all(torch.equal(a, b) for a, b in zip(first[i], pair[i]))
    del later
    # beside other products on a second stream: large ones, a few tokens, a shared contraction
    side = torch.cuda.Stream()
    got, other = [], []
    few = p.x[0][:40].contiguous()
    want_few = bq.linear(few, p.w)
    torch.cuda.synchronize()
    for _ in range(6):
        got.append(p.run(p.x[0], p.dy[0], p.kept[0]))
        with torch.cuda.stream(side):
            other.append((p.run(p.x[1], p.dy[1], p.kept[1]), bq.linear(few, p.w)))
    torch.cuda.synchronize()
    for a, (b, c) in zip(got, other):
        assert all(torch.equal(u, v) for u, v in zip(first[0], a))
        assert all(torch.equal(u, v) for u, v in zip(first[1], b)) and torch.equal(c, want_few)
    del got, other
    # one graph, inputs that change between replays
    x, dy = torch.empty_like(p.x[0]), torch.empty_like(p.dy[0])
    kept = bq.Quantized(p.kept[0].scheme, *p.kept[0].codes.shape, torch.empty_like(p.kept[0].codes),
                        torch.empty_like(p.kept[0].scales), None, None, None)
    outs = [torch.empty_like(t) for t in first[0]]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p.run(x, dy, kept, outs)
    for i in (1, 0, 1, 1, 0):
        x.copy_(p.x[i])
        dy.copy_(p.dy[i])
        kept.codes.copy_(p.kept[i].codes)
        kept.scales.copy_(p.kept[i].scales)
        for t in outs:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first[i], outs))
    assert bq.bq_wait_timeouts() == 0

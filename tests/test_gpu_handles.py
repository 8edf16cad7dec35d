"""The linear layer and the gated activation refuse handles whose buffers are too short, not
contiguous or on another device (each call is refused on the host; none is launched)."""

import dataclasses

import pytest
import torch

import block_scaled_bit_bq_b200 as bq
from block_scaled_bit_bq_b200 import Scheme

pytestmark = pytest.mark.gpu


def _bad(q):
    yield dataclasses.replace(q, codes=q.codes[:-1])
    yield dataclasses.replace(q, scales=q.scales[:-1])
    yield dataclasses.replace(q, scales=q.scales.cpu())
    yield dataclasses.replace(q, codes=q.codes.t().contiguous().t())
    yield dataclasses.replace(q, rows=q.rows * 2)
    if q.tensor_scale is not None:
        yield dataclasses.replace(q, tensor_scale=q.tensor_scale.cpu())


@pytest.mark.parametrize("gran", ["mx", "nv"])
def test_linear_refuses_bad_handles(gran):
    w = bq.quantize(torch.randn(48, 64, device="cuda").to(torch.bfloat16), Scheme("e2m1", gran), stats=False)
    x = torch.randn(3, 64, device="cuda").to(torch.bfloat16)
    for bad in _bad(w):
        for call in (lambda: bq.linear(x, bad),
                     lambda: bq.linear_grad_input(torch.zeros(3, bad.rows, dtype=torch.bfloat16, device="cuda"), bad)):
            with pytest.raises(ValueError):
                call()


def test_grad_weight_refuses_bad_handles():
    q = bq.quantize(torch.randn(48, 64, device="cuda").to(torch.bfloat16), Scheme("e4m3", "mx"), stats=False)
    for bad in _bad(q):
        with pytest.raises(ValueError):
            bq.linear_grad_weight(torch.zeros(bad.rows, 16, dtype=torch.bfloat16, device="cuda"), bad)


def test_glu_refuses_bad_checkpoints():
    g, u, dh = (torch.randn(48, 64, device="cuda").to(torch.bfloat16) for _ in range(3))
    s = Scheme("e4m3", "mx").resolved()
    _, kept = bq.glu(g, u, s)
    for bad in _bad(kept.gate):
        for pair in (bq.GluCheckpoint(bad, kept.up, "silu"), bq.GluCheckpoint(kept.up, bad, "silu")):
            with pytest.raises(ValueError):
                bq.glu(g, u, s, ckpt=pair)
            with pytest.raises(ValueError):
                bq.glu_backward(dh, pair)


def test_the_other_calls_refuse_bad_handles():
    x = torch.randn(128, 256, device="cuda").to(torch.bfloat16)
    for s in (Scheme("int8_sym", "row"), Scheme("e4m3", "mx", layout="gemm"), Scheme("e2m1", "nv")):
        q = bq.quantize(x, s, stats=False)
        want = bq.dequantize(q)
        for bad in (dataclasses.replace(q, codes=q.codes[:-1]), dataclasses.replace(q, scales=q.scales[:-1]),
                    dataclasses.replace(q, scales=q.scales.cpu())):
            calls = [lambda: bq.dequantize(bad), lambda: bq.qsnr(x, bad), lambda: bq.quantize(x, s, stats=False, out=bad)]
            if s.layout == "gemm":
                calls += [lambda: bq.gemm(bad, q), lambda: bq.gemm(q, bad)]
            for call in calls:
                with pytest.raises(ValueError):
                    call()
        with pytest.raises(ValueError):
            bq.quantize(torch.cat((x, x)), s, stats=False, out=q)
        assert torch.equal(bq.dequantize(q), want)
    b = bq.quantize_batch(x.view(2, 64, 256), Scheme("e4m3", "mx"), stats=False)
    with pytest.raises(ValueError):
        bq.quantize_batch(x.view(4, 32, 256).repeat(2, 1, 1), b.scheme, stats=False, out=b)

"""The linear layer's bounded waits, made to run out without faulting the GPU.

bq_debug_skip_linear_copy makes one CTA of the next product skip the copies of its first
stage, so the barrier that its MMAs wait for is never completed: a flag that nothing sets. The
waits give up after about a second, the CTA (a pair: both) stops, waits for its other copies
in flight and ends, and bq_wait_timeouts counts it. The other CTAs' tiles are right, the
skipped one's are not written, and the next call is exact again."""

import time

import pytest
import torch

import synth
import block_scaled_bit_bq_b200 as bq
from block_scaled_bit_bq_b200 import Scheme

pytestmark = pytest.mark.gpu

# tokens, outputs, inputs of the forward product: a CTA a tile (several tiles, none shared), a
# contraction shared by a cluster, tiles on pairs (of either CTA)
CASES = [("alone", (300, 16500, 512), 0, 1), ("alone-last", (300, 16500, 512), 100, 1), ("shared", (40, 300, 4096), 1, 1),
         ("pair-first", (2304, 2048, 512), 0, 2), ("pair-second", (2304, 2048, 512), 7, 2)]


@pytest.mark.parametrize("shape,cta,count", [c[1:] for c in CASES], ids=[c[0] for c in CASES])
def test_wait_runs_out_and_the_next_call_is_exact(shape, cta, count):
    m, n, k = shape
    w = bq.quantize(synth.weight_outliers(n, k, seed=n).cuda(), Scheme("e2m1", "mx"), stats=False)
    gen = torch.Generator("cuda").manual_seed(6)
    x = torch.randn(m, k, device="cuda", generator=gen).to(torch.bfloat16)
    want = bq.linear(x, w)
    torch.cuda.synchronize()
    bq.bq_wait_timeouts(reset=True)
    out = torch.full_like(want, 12345.0)
    bq.bq_debug_skip_linear_copy(cta)
    t0 = time.time()
    bq.linear(x, w, out=out)
    torch.cuda.synchronize()
    dt = time.time() - t0
    assert 1.0 <= dt < 20.0, dt
    assert bq.bq_wait_timeouts() == count
    if shape[0] != 40:
        left = out == 12345.0
        assert left.any() and not left.all() and torch.equal(out[~left], want[~left])
    # one-shot: the next call runs normally, on the same memory
    bq.linear(x, w, out=out)
    assert torch.equal(out, want) and bq.bq_wait_timeouts() == count
    bq.bq_wait_timeouts(reset=True)
    assert bq.bq_wait_timeouts() == 0


def test_gradients_give_up_too():
    m, n, k = 2304, 512, 2048
    gen = torch.Generator("cuda").manual_seed(7)
    w = bq.quantize(synth.weight_outliers(n, k, seed=n).cuda(), Scheme("e2m1", "nv"), stats=False)
    dy = torch.randn(m, n, device="cuda", generator=gen).to(torch.bfloat16)
    q = bq.quantize(torch.randn(m, k, device="cuda", generator=gen).to(torch.bfloat16), Scheme("e4m3", "mx"), stats=False)
    for call, ctas in ((lambda: bq.linear_grad_input(dy, w), 2), (lambda: bq.linear_grad_weight(dy, q), 1)):
        want = call()
        torch.cuda.synchronize()
        bq.bq_wait_timeouts(reset=True)
        bq.bq_debug_skip_linear_copy(3)
        call()
        assert bq.bq_wait_timeouts() == ctas
        assert torch.equal(call(), want) and bq.bq_wait_timeouts(reset=True) == ctas


def test_refusal():
    with pytest.raises(bq.BqError):
        bq.bq_debug_skip_linear_copy(-1)

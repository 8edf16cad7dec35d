"""The longest contraction that the linear layer takes: one tile of 2^31 - 64 steps, shared by
eight SMs. Each of them has about four million parts of some 0.28 us, so the accumulator comes
later (after 1.15 s) than any single wait may last (about 1.06 s): the wait for it has to go by
whether stages get done. The matrix is random codes; all but some outputs' gradients are
zero, so that few rows count (tolerance as in test_gpu_linear.py; sums over zeros are exact)."""

import numpy as np
import pytest
import torch

import oracle
import block_scaled_bit_bq_b200 as bq
from block_scaled_bit_bq_b200 import Scheme
from oracle import linear as ref

pytestmark = pytest.mark.gpu


def test_grad_input_of_two_billion_outputs():
    n, k = 2 ** 31 - 64, 32
    gen = torch.Generator("cuda").manual_seed(5)
    codes = torch.empty(n, k // 2, dtype=torch.uint8, device="cuda").random_(0, 256, generator=gen)
    scales = torch.empty(n, dtype=torch.uint8, device="cuda").random_(118, 124, generator=gen)
    q = bq.Quantized(Scheme("e2m1", "mx").resolved(), n, k, codes, scales, None, None, None)
    dy = torch.zeros(1, n, dtype=torch.bfloat16, device="cuda")
    at = [(0, 60), (n // 3, n // 3 + 60), (n // 2 - 30, n // 2 + 30), (n - 700, n - 640), (n - 60, n)]
    for a, b in at:
        dy[0, a:b] = torch.randn(b - a, device="cuda", generator=gen).to(torch.bfloat16)
    bq.bq_wait_timeouts(reset=True)
    dx = bq.linear_grad_input(dy, q, torch.float32)
    assert bq.bq_wait_timeouts() == 0
    v = np.concatenate([ref.values(codes[a:b].cpu().numpy(), scales[a:b].cpu().numpy(), None, b - a, k, oracle.Scheme("e2m1", "mx"))
                        for a, b in at])
    d = np.concatenate([dy[:, a:b].float().cpu().numpy().astype(np.float64) for a, b in at], 1)
    want = d @ v
    tol = (d.size / 8 + 32) * 2.0 ** -23 * (np.abs(d) @ np.abs(v)) + 2.0 ** -23 * np.abs(want)
    assert np.all(np.abs(dx.cpu().numpy() - want) <= tol)

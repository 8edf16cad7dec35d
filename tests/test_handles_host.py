"""Handles (Quantized) whose buffers do not hold what their scheme and shape say are refused
before any launch (no GPU)."""

import dataclasses

import pytest
import torch

import block_scaled_bit_bq_b200 as bq
from block_scaled_bit_bq_b200 import Scheme

CPU = torch.device("cpu")
SCHEMES = [Scheme("e2m1", "mx"), Scheme("e2m1", "nv"), Scheme("e4m3", "mx"), Scheme("int8_sym", "mx"),
           Scheme("e2m1", "mx", layout="gemm"), Scheme("e2m1", "nv", layout="gemm"), Scheme("e4m3", "mx", layout="gemm")]


def _handle(s, rows=130, cols=256):
    return bq.alloc_outputs(s, rows, cols, CPU, stats=False)


@pytest.mark.parametrize("s", SCHEMES, ids=lambda s: f"{s.fmt}-{s.gran}-{s.layout}")
def test_what_quantize_allocates_passes(s):
    for rows, cols in ((130, 256), (1, 128), (0, 128), (128, 512)):
        bq._handle(_handle(s, rows, cols), CPU)
    # an unresolved scheme, flat codes, signed bytes and a longer buffer are as good
    q = _handle(s)
    q.scheme, q.codes, q.scales = s, q.codes.reshape(-1).view(torch.int8), torch.cat((q.scales, q.scales))
    bq._handle(q, CPU)


@pytest.mark.parametrize("s", SCHEMES, ids=lambda s: f"{s.fmt}-{s.gran}-{s.layout}")
def test_short_or_strange_buffers_are_refused(s):
    q = _handle(s)
    bad = [{"codes": q.codes[:-1]}, {"codes": q.codes[:, :-1]}, {"codes": q.codes.float()}, {"scales": q.scales[:-1]},
           {"codes": q.codes.t().contiguous().t()}, {"scales": torch.cat((q.scales, q.scales))[::2]},
           {"scales": q.scales.float()}, {"rows": q.rows + 128}, {"cols": q.cols + 128}]
    if s.gran == "nv":
        bad += [{"tensor_scale": q.tensor_scale.double()}, {"tensor_scale": q.tensor_scale[:0]}]
    for change in bad:
        with pytest.raises(ValueError):
            bq._handle(dataclasses.replace(q, **change), CPU)
    with pytest.raises(ValueError):
        bq._handle(q, torch.device("cuda", 0))

"""Handles (Quantized) whose buffers do not hold what their scheme and shape say are refused
before any launch (no GPU)."""

import copy
import dataclasses
import io
import pickle

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


# the calls that take any scheme: every refusal comes before the library is called
ANY = [Scheme("int8_sym", "row"), Scheme("uint4_asym", "group", 128, "fp16"), Scheme("e4m3", "tensor"), Scheme("int8_asym", "tile2d"),
       Scheme("e2m1", "nv"), Scheme("e4m3", "mx", layout="gemm")]


class _Elsewhere:
    """A tensor that says it is on a CUDA device (there is none here)."""

    def __init__(self, t):
        self.t = t

    device = torch.device("cuda", 0)

    def __getattr__(self, name):
        return getattr(self.t, name)


def _on_cuda(q):
    return dataclasses.replace(q, **{n: _Elsewhere(getattr(q, n)) for n in ("codes", "scales", "zero_points", "tensor_scale")
                                     if getattr(q, n, None) is not None})


@pytest.mark.parametrize("s", ANY, ids=lambda s: f"{s.fmt}-{s.gran}")
def test_buffers_of_any_scheme(s):
    dev = _Elsewhere.device
    q = bq.alloc_outputs(s, 130, 256, CPU, stats=False)
    bq._buffers(_on_cuda(q), dev, 130, 256)
    for n in ("codes", "scales", "zero_points", "tensor_scale"):
        t = getattr(q, n)
        if t is None:
            continue
        for short in (t.reshape(-1)[:-1], t.reshape(-1, 1).expand(-1, 2)):
            with pytest.raises(ValueError):
                bq._buffers(_on_cuda(dataclasses.replace(q, **{n: short})), dev, 130, 256)
        with pytest.raises(ValueError):
            bq._buffers(dataclasses.replace(_on_cuda(q), **{n: t}), dev, 130, 256)
    with pytest.raises(ValueError):
        bq._buffers(_on_cuda(q), dev, 386, 256)
    b = bq.alloc_batch_outputs(s, 3, 130, 256, CPU, stats=False) if s.gran in ("group", "mx") else None
    if b is not None:
        bq._buffers(_on_cuda(b), dev, 130, 256, 3)
        with pytest.raises(ValueError):
            bq._buffers(_on_cuda(b), dev, 130, 256, 5)


def test_calls_refuse_cpu_handles():
    q = bq.alloc_outputs(Scheme("e4m3", "mx"), 4, 64, CPU, stats=False)
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    for call in (lambda: bq.dequantize(q), lambda: bq.dequantize_rt(q), lambda: bq.qsnr(x, q), lambda: bq.gemm(q, q)):
        with pytest.raises(ValueError):
            call()


# a handle that has been through a call is saved and loaded as before it
def test_saved_handles_hold_no_cached_forms():
    q = _handle(SCHEMES[1], 4, 64)
    for s in (q.scheme, SCHEMES[1]):
        bq._c_scheme(s)
        bq._resolved(s)
    assert set(pickle.loads(pickle.dumps(q.scheme)).__dict__) == {f.name for f in dataclasses.fields(Scheme)}
    f = io.BytesIO()
    torch.save(q, f)
    f.seek(0)
    with torch.serialization.safe_globals([bq.Quantized, bq.Scheme]):
        r = torch.load(f, weights_only=True)
    assert r.scheme == q.scheme and torch.equal(r.codes, q.codes) and copy.deepcopy(q).scheme == q.scheme

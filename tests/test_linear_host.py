"""Host-side checks of the linear layer's and the gated activation's entry points (no GPU):
every refusal happens before any launch, with the status that bq.h names."""

import ctypes

import pytest
import torch

import block_scaled_bit_bq_b200 as bq
from block_scaled_bit_bq_b200 import Scheme

FAKE = 1 << 40          # never dereferenced: every call below fails its host checks or is empty
MX4, NV4, MX8 = Scheme("e2m1", "mx"), Scheme("e2m1", "nv"), Scheme("e4m3", "mx")
INVALID, UNSUPPORTED, SHAPE, ALIGN = 1, 2, 3, 4


def _lin(op="forward", scheme=MX4, m=4, n=16, k=64, ld=None, x=FAKE, dt=0, codes=FAKE, scales=FAKE, ts=FAKE, out=FAKE,
         out_dt=0):
    L, sc = bq.lib(), scheme.c()
    if ld is None:
        ld = k if op == "forward" else -(-max(n, 1) // 8) * 8
    if op == "weight":
        return L.bq_linear_grad_weight(x, dt, ld, codes, scales, m, n, k, ctypes.byref(sc), out, out_dt, None)
    f = L.bq_linear if op == "forward" else L.bq_linear_grad_input
    return f(x, dt, ld, codes, scales, ts, m, n, k, ctypes.byref(sc), out, out_dt, None)


OPS = [("forward", MX4), ("forward", NV4), ("input", MX4), ("input", NV4), ("weight", MX8)]


@pytest.mark.parametrize("op,s", OPS, ids=str)
def test_linear_refusals(op, s):
    def q(**kw):
        return _lin(op, **{"scheme": s, **kw})
    # schemes: only 4-bit MX / NV weights, only 8-bit MX inputs, no rotation
    for bad in [Scheme("int4_sym", "nv"), Scheme("e2m3", "mx"), Scheme("int8_sym", "row"), Scheme("e4m3", "tensor"),
                Scheme("e2m1", "mx", hadamard=True), Scheme("e4m3", "mx", hadamard=True),
                MX8 if op != "weight" else MX4]:
        assert q(scheme=bad) == UNSUPPORTED, bad
    assert q(dt=2) == UNSUPPORTED and q(out_dt=1) == UNSUPPORTED and q(out_dt=3) == UNSUPPORTED
    # shapes
    assert q(m=-1) == SHAPE and q(n=-1) == SHAPE and q(k=0) == SHAPE and q(k=48) == SHAPE
    assert q(ld=8) == SHAPE and q(ld=68) == SHAPE and q(ld=1 << 31) == SHAPE
    assert q(m=1 << 31) == SHAPE and q(n=1 << 31) == SHAPE
    assert q(m=1 << 30, n=128, ld=128) == SHAPE                  # m * n or m * k past 2^36
    # pointers and alignment
    assert q(x=None) == INVALID and q(codes=None) == INVALID and q(scales=None) == INVALID and q(out=None) == INVALID
    assert q(x=FAKE + 8) == ALIGN and q(codes=FAKE + 16) == ALIGN and q(scales=FAKE + 2) == ALIGN
    assert q(out=FAKE + 8) == ALIGN
    if s is NV4:
        assert q(ts=None) == INVALID and q(ts=FAKE + 2) == ALIGN


def test_linear_null_scheme():
    L = bq.lib()
    assert L.bq_linear(FAKE, 0, 64, FAKE, FAKE, None, 4, 16, 64, None, FAKE, 0, None) == INVALID
    assert L.bq_linear_grad_weight(FAKE, 0, 16, FAKE, FAKE, 4, 16, 64, None, FAKE, 0, None) == INVALID


def test_linear_empty_outputs_are_no_ops():
    assert _lin("forward", m=0, x=None, out=None) == 0
    assert _lin("forward", n=0, out=None) == 0
    assert _lin("input", m=0, x=None, out=None) == 0
    assert _lin("weight", scheme=MX8, n=0, out=None) == 0


def _glu(scheme=MX8, rows=4, cols=64, ldg=None, ldu=None, dt=0, act=0, gate=FAKE, up=FAKE, out=FAKE, gc=FAKE, gs=FAKE,
         uc=FAKE, us=FAKE):
    sc = None if scheme is None else ctypes.byref(scheme.c())
    return bq.lib().bq_glu(gate, cols if ldg is None else ldg, up, cols if ldu is None else ldu, dt, rows, cols, act,
                           out, sc, gc, gs, uc, us, None)


def _back(scheme=MX8, rows=4, cols=64, ldh=None, ldg=None, ldu=None, dt=0, act=0, dh=FAKE, gc=FAKE, gs=FAKE, uc=FAKE,
          us=FAKE, dg=FAKE, du=2 * FAKE):
    sc = None if scheme is None else ctypes.byref(scheme.c())
    lds = [cols if v is None else v for v in (ldh, ldg, ldu)]
    return bq.lib().bq_glu_backward(dh, lds[0], dt, gc, gs, uc, us, sc, rows, cols, act, dg, lds[1], du, lds[2], None)


@pytest.mark.parametrize("f", [_glu, _back], ids=["forward", "backward"])
def test_glu_refusals(f):
    for bad in [MX4, NV4, Scheme("e2m3", "mx"), Scheme("int8_sym", "row"), Scheme("e4m3", "mx", hadamard=True),
                Scheme("e4m3", "group", 32)]:
        assert f(scheme=bad) == UNSUPPORTED, bad
    assert f(scheme=Scheme("e4m3", "mx", layout="gemm"), cols=128) == UNSUPPORTED
    assert f(dt=2) == UNSUPPORTED
    assert f(act=2) == INVALID and f(act=-1) == INVALID
    assert f(rows=-1) == SHAPE and f(cols=48) == SHAPE and f(cols=0) == SHAPE
    assert f(rows=1 << 30, cols=128) == SHAPE
    assert f(ldg=48) == SHAPE and f(ldg=72) == SHAPE and f(ldu=72) == SHAPE and f(ldu=1 << 31) == SHAPE
    assert f(gc=None) == INVALID and f(gs=None) == INVALID and f(uc=None) == INVALID and f(us=None) == INVALID
    assert f(gc=FAKE + 16) == ALIGN and f(uc=FAKE + 16) == ALIGN and f(gs=FAKE + 2) == ALIGN and f(us=FAKE + 1) == ALIGN
    assert f(rows=0) == 0


def test_glu_forward_refusals():
    assert _glu(gate=None) == INVALID and _glu(up=None) == INVALID and _glu(out=None) == INVALID
    assert _glu(gate=FAKE + 16) == ALIGN and _glu(up=FAKE + 16) == ALIGN and _glu(out=FAKE + 16) == ALIGN
    # without a scheme there is nowhere to keep copies
    for name in ("gc", "gs", "uc", "us"):
        kw = {"gc": None, "gs": None, "uc": None, "us": None, name: FAKE}
        assert _glu(scheme=None, **kw) == INVALID


def test_glu_backward_refusals():
    assert _back(scheme=None) == INVALID
    assert _back(dh=None) == INVALID and _back(dg=None) == INVALID and _back(du=None) == INVALID
    assert _back(dg=FAKE, du=FAKE) == INVALID
    assert _back(dh=FAKE + 16) == ALIGN and _back(dg=FAKE + 16) == ALIGN and _back(du=2 * FAKE + 16) == ALIGN
    assert _back(ldh=72) == SHAPE


def test_python_checks_on_cpu_tensors():
    q = bq.Quantized(MX4.resolved(), 16, 64, torch.zeros(16, 32, dtype=torch.uint8), torch.zeros(32, dtype=torch.uint8),
                     None, None, None)
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    for call in (lambda: bq.linear(x, q), lambda: bq.linear_grad_input(x, q), lambda: bq.linear_grad_weight(x, q),
                 lambda: bq.glu(x, x), lambda: bq.glu(x, x[:2]),
                 lambda: bq.glu_backward(x, bq.GluCheckpoint(q, q, "silu"))):
        with pytest.raises(ValueError):
            call()

"""Refusals of the operators around the sparse FFN, without a GPU: the C ABI
rejects bad arguments before it touches CUDA, the classes reject tensors of a
wrong type, shape, layout or place before they call it."""
from __future__ import annotations

import ctypes

import pytest
import torch

from activation_sparse_gated_relu_b200 import binding as B
from activation_sparse_gated_relu_b200 import Fp8Linear, GroupedLinear, RmsNorm, layer, quantize_blocks, quantize_rows
from activation_sparse_gated_relu_b200.build import build

P = 0x7F0000000000        # 16-byte aligned, never dereferenced by validation
BAD, UNSUP = B.SFFN_ERR_INVALID_ARG, B.SFFN_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    build()
    return B.load_library()


def _norm_desc(**kw):
    d = B.sffn_rmsnorm_desc(d=256, eps=1e-6, weight=P, weight_dtype=B.SFFN_BF16, x_dtype=B.SFFN_FP32,
                            residual_dtype=B.SFFN_BF16, y_dtype=B.SFFN_BF16)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


@pytest.mark.parametrize("desc,call,want", [
    (dict(d=0), {}, BAD), (dict(d=-8), {}, BAD), (dict(d=12), {}, UNSUP), (dict(d=16392), {}, UNSUP),
    (dict(eps=-1.0), {}, BAD), (dict(eps=float("nan")), {}, BAD), (dict(eps=float("inf")), {}, BAD),
    (dict(weight=None), {}, BAD), (dict(weight=P + 8), {}, BAD), (dict(weight_dtype=2), {}, BAD),
    (dict(x_dtype=2), {}, BAD), (dict(residual_dtype=2), {}, BAD), (dict(y_dtype=3), {}, BAD), (dict(y_dtype=-1), {}, BAD),
    ({}, dict(T=-1), BAD), ({}, dict(T=(1 << 24) + 1), BAD), ({}, dict(x=None), BAD), ({}, dict(x=P + 4), BAD),
    ({}, dict(y=None), BAD), ({}, dict(y=P + 2), BAD), ({}, dict(res=P + 2), BAD), ({}, dict(res=None), BAD),
    ({}, dict(sout=None), BAD), ({}, dict(sout=P + 8), BAD), ({}, dict(scale=P), BAD), (dict(y_dtype=2), {}, BAD),
])
def test_rmsnorm_forward_refuses(lib, desc, call, want):
    a = dict(x=P, res=P, T=4, sout=P, y=P, scale=None)
    a.update(call)
    d = _norm_desc(**desc)
    assert lib.sffn_rmsnorm_forward(ctypes.byref(d), a["x"], a["res"], a["T"], a["sout"], a["y"], a["scale"], None) == want


def test_rmsnorm_without_rows_or_descriptor(lib):
    d = _norm_desc()
    assert lib.sffn_rmsnorm_forward(ctypes.byref(d), None, None, 0, None, None, None, None) == B.SFFN_OK
    assert lib.sffn_rmsnorm_forward(None, P, None, 1, None, P, None, None) == BAD


@pytest.mark.parametrize("desc,call", [
    (dict(y_dtype=2), {}), ({}, dict(dy=None)), ({}, dict(s=None)), ({}, dict(dx=None)), ({}, dict(dw=None)),
    ({}, dict(dw=P + 4)), ({}, dict(ds=P + 2)), ({}, dict(work=None)), ({}, dict(bytes=0)), ({}, dict(T=-2)),
])
def test_rmsnorm_backward_refuses(lib, desc, call):
    a = dict(dy=P, s=P, ds=None, T=4, dx=P, dw=P, work=P, bytes=1 << 30)
    a.update(call)
    d = _norm_desc(**desc)
    assert lib.sffn_rmsnorm_backward(ctypes.byref(d), a["dy"], a["s"], a["ds"], a["T"], a["dx"], a["dw"], a["work"],
                                     a["bytes"], None) == BAD


def test_rmsnorm_workspace(lib):
    n = ctypes.c_size_t()
    assert lib.sffn_rmsnorm_workspace_bytes(4096, 0, ctypes.byref(n)) == B.SFFN_OK and n.value == 0
    last = 0
    for T in (1, 7, 296, 5000, 1 << 24):
        assert lib.sffn_rmsnorm_workspace_bytes(4096, T, ctypes.byref(n)) == B.SFFN_OK
        assert n.value >= last and n.value <= 64 << 20
        last = n.value
    assert lib.sffn_rmsnorm_workspace_bytes(4100, 1, ctypes.byref(n)) == UNSUP
    assert lib.sffn_rmsnorm_workspace_bytes(0, 1, ctypes.byref(n)) == BAD
    assert lib.sffn_rmsnorm_workspace_bytes(64, 1, None) == BAD


@pytest.mark.parametrize("args,want", [
    ((None, 0, 4, 64, P, P), BAD), ((P + 1, 0, 4, 64, P, P), BAD), ((P, 2, 4, 64, P, P), BAD), ((P, 0, -1, 64, P, P), BAD),
    ((P, 0, 4, 0, P, P), BAD), ((P, 0, 4, 60, P, P), UNSUP), ((P, 0, 4, 64, None, P), BAD), ((P, 0, 4, 64, P, P + 4), BAD),
])
def test_quantisers_refuse(lib, args, want):
    assert lib.sffn_quantize_rows(*args, None) == want
    if args[2] != -1:
        assert lib.sffn_quantize_blocks(*args, None) == want


@pytest.mark.parametrize("kw,want", [
    (dict(d_in=0), BAD), (dict(d_out=-8), BAD), (dict(d_in=24), UNSUP), (dict(d_out=12), UNSUP), (dict(d_in=(1 << 20) + 16), UNSUP),
    (dict(Wq=None), BAD), (dict(Wq=P + 8), BAD), (dict(Ws=None), BAD), (dict(Ws=P + 4), BAD),
])
def test_qlinear_create_refuses(lib, kw, want):
    d = B.sffn_qlinear_desc(d_in=256, d_out=128, Wq=P, Ws=P)
    for k, v in kw.items():
        setattr(d, k, v)
    h = ctypes.c_void_p()
    assert lib.sffn_qlinear_create(ctypes.byref(d), None, ctypes.byref(h)) == want and not h.value
    assert lib.sffn_qlinear_create(None, None, ctypes.byref(h)) == BAD
    assert lib.sffn_qlinear_create(ctypes.byref(d), None, None) == BAD


@pytest.mark.parametrize("kw,want", [
    (dict(n_experts=0), BAD), (dict(n_experts=1025), UNSUP), (dict(d_in=0), BAD), (dict(d_in=12), UNSUP), (dict(d_out=12), UNSUP),
    (dict(d_out=(1 << 20) + 8), UNSUP), (dict(W=None), BAD), (dict(W=P + 8), BAD),
])
def test_grouped_create_refuses(lib, kw, want):
    d = B.sffn_grouped_desc(n_experts=4, d_in=256, d_out=128, W=P)
    for k, v in kw.items():
        setattr(d, k, v)
    h = ctypes.c_void_p()
    assert lib.sffn_grouped_create(ctypes.byref(d), None, ctypes.byref(h)) == want and not h.value


def test_calls_without_a_handle(lib):
    assert lib.sffn_qlinear_forward(None, P, P, 1, P, 0, None) == BAD
    assert lib.sffn_qlinear_quantize_forward(None, P, 0, 1, P, 0, P, 1 << 20, None) == BAD
    assert lib.sffn_qlinear_read_status(None, None) == BAD
    assert lib.sffn_qlinear_destroy(None) == B.SFFN_OK
    assert lib.sffn_grouped_forward(None, P, P, 1, P, 0, None) == BAD
    assert lib.sffn_grouped_backward_input(None, P, P, 1, P, 0, None) == BAD
    assert lib.sffn_grouped_backward_weight(None, P, P, P, 1, P, 0, None) == BAD
    assert lib.sffn_grouped_read_status(None, None) == BAD
    assert lib.sffn_grouped_destroy(None) == B.SFFN_OK


def test_no_device_is_an_error(lib):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    h = ctypes.c_void_p()
    d = B.sffn_qlinear_desc(d_in=256, d_out=128, Wq=P, Ws=P)
    assert lib.sffn_qlinear_create(ctypes.byref(d), None, ctypes.byref(h)) == B.SFFN_ERR_NO_DEVICE
    g = B.sffn_grouped_desc(n_experts=4, d_in=256, d_out=128, W=P)
    assert lib.sffn_grouped_create(ctypes.byref(g), None, ctypes.byref(h)) == B.SFFN_ERR_NO_DEVICE


def test_classes_refuse_host_tensors():
    w = torch.ones(64)
    with pytest.raises(ValueError, match="CUDA"):
        RmsNorm(w)
    with pytest.raises(ValueError, match="\\[d\\]"):
        RmsNorm(torch.ones(2, 64))
    with pytest.raises(TypeError, match="weight"):
        RmsNorm(torch.ones(64, dtype=torch.float16))
    with pytest.raises(ValueError, match="CUDA"):
        quantize_rows(torch.ones(2, 64))
    with pytest.raises(TypeError, match="x must be"):
        quantize_rows(torch.ones(2, 64, dtype=torch.float64))
    with pytest.raises(ValueError, match="CUDA"):
        quantize_blocks(torch.ones(2, 64))
    with pytest.raises(ValueError, match="CUDA"):
        Fp8Linear(torch.ones(8, 128).to(torch.float8_e4m3fn), torch.ones(1, 1))
    with pytest.raises(TypeError, match="Wq"):
        Fp8Linear(torch.ones(8, 128), torch.ones(1, 1))
    with pytest.raises(ValueError, match="n_experts"):
        GroupedLinear(torch.ones(8, 128))
    with pytest.raises(ValueError, match="CUDA"):
        GroupedLinear(torch.ones(2, 8, 128, dtype=torch.bfloat16))


def test_checks_name_what_is_wrong():
    t = torch.ones(4, 64)
    for bad, kind, text in ((t.t(), ValueError, "shape"), (t.double(), TypeError, "float64"), (None, TypeError, "Tensor"),
                            (t, ValueError, "CUDA")):
        with pytest.raises(kind, match=text):
            layer._check(bad, "x", (torch.float32,), (4, 64), None)
    with pytest.raises(ValueError, match="overlap"):
        layer._apart(t, "y", t[1:])
    layer._apart(t[:2], "y", t[2:])
    layer._apart_or_in_place(t, "y", t, None)
    with pytest.raises(ValueError, match="overlap"):
        layer._apart_or_in_place(t[1:], "y", t)
    with pytest.raises(ValueError, match="out must be"):
        layer._out_type("fp16")

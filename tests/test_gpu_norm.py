"""The RMS norm with the residual's addition, its 8-bit output and its gradient,
and the quantisers, against plain forms in 64 bits.

Bounds.  A row's sum of squares adds each square at most 32 times in a thread,
5 times in a warp and 16 times over warps, after one rounding of s and one of
the square: at most 56 fp32 roundings, halved by the root, plus 4 U for the
root (2 ulp), the division and eps.  With the rounding of s and two products y
is off by less than REL = 40 U relative, and by half a step of its type."""
from __future__ import annotations

import pytest
import torch

from activation_sparse_gated_relu_b200 import RmsNorm, quantize_blocks, quantize_rows
from layer_util import HALF, U, check_codes, groups, randn, within

pytestmark = pytest.mark.gpu

REL = 40 * U
BF, F32 = torch.bfloat16, torch.float32


def ref_forward(x, res, w, eps):
    s = x.double() + (res.double() if res is not None else 0)
    return s * torch.rsqrt((s * s).mean(1, keepdim=True) + eps) * w.double(), s


def case(T, d, xt, rt, wt=BF, seed=0):
    x = randn(seed, T, d, dtype=xt, scale=0.5)
    res = None if rt is None else randn(seed + 1, T, d, dtype=rt, scale=2.0)
    w = (1 + 0.2 * randn(seed + 2, d)).to(wt)
    return x, res, w


SHAPES = [(1, 8), (1, 4096), (3, 128), (5, 136), (7, 256), (2, 1032), (9, 2048), (130, 512), (13, 4104), (4, 8192),
          (3, 16384), (2, 12296), (600, 264)]


@pytest.mark.parametrize("T,d", SHAPES)
@pytest.mark.parametrize("xt,rt", [(F32, BF), (BF, None), (BF, F32), (F32, None), (BF, BF), (F32, F32)])
def test_forward_bf16_and_fp32(T, d, xt, rt):
    x, res, w = case(T, d, xt, rt)
    op = RmsNorm(w, 1e-6)
    ref, s = ref_forward(x, res, w, 1e-6)
    for out, t in (("bf16", BF), ("fp32", F32)):
        y, got_s = op(x, res, out=out)
        assert y.dtype is t
        within(y, ref, ref.abs() * (REL + HALF[t]) + 1e-38, f"y {out}")
        if res is None:
            assert got_s is x
        else:
            assert got_s.dtype is rt
            assert torch.equal(got_s, (x.float() + res.float()).to(rt))   # one fp32 sum, one rounding


@pytest.mark.parametrize("T,d", SHAPES)
@pytest.mark.parametrize("xt,rt,wt", [(F32, BF, BF), (BF, None, F32), (BF, F32, BF)])
def test_forward_8_bits(T, d, xt, rt, wt):
    x, res, w = case(T, d, xt, rt, wt, seed=10)
    q, scale, s = RmsNorm(w, 1e-5).forward_fp8(x, res)
    ref, _ = ref_forward(x, res, w, 1e-5)
    assert q.dtype is torch.float8_e4m3fn and scale.shape == (T, groups(d))
    check_codes(q, scale, ref, REL)
    if res is not None:
        assert torch.equal(s, (x.float() + res.float()).to(rt))


def test_rows_keep_to_themselves():
    # a NaN or an infinity reaches its own row only; a row of zeros gives zeros and codes 0
    x, res, w = case(6, 264, F32, BF)
    want_y, _ = RmsNorm(w)(x, res)
    want_q, want_c, _ = RmsNorm(w).forward_fp8(x, res)
    x[1, 5] = float("nan")
    x[3, 263] = float("inf")
    x[4], res[4] = 0.0, 0.0
    y, _ = RmsNorm(w)(x, res)
    q, c, _ = RmsNorm(w).forward_fp8(x, res)
    keep = [0, 2, 5]
    assert torch.equal(y[keep], want_y[keep]) and torch.equal(c[keep], want_c[keep])
    assert torch.equal(q.view(torch.uint8)[keep], want_q.view(torch.uint8)[keep])
    assert torch.isnan(y[1]).all()
    assert torch.isnan(y[3, 263]) and (y[3, :263] == 0).all()      # s / inf
    assert (y[4] == 0).all() and (q[4].float() == 0).all() and torch.isfinite(c[4]).all()
    z, _ = RmsNorm(w, 0.0)(x, res)
    assert torch.isnan(z[4]).all()                                  # 0 / 0, as the formula says


def test_extreme_magnitudes_and_groups_of_zeros():
    x = torch.zeros(3, 512, device="cuda")
    x[0, :4] = torch.tensor([1e15, -1e15, 1.0, 1e-30])
    x[1, 300] = 1e-25
    x[2, 511] = -3.0
    w = torch.ones(512, device="cuda")
    ref, _ = ref_forward(x, None, w, 1e-6)
    y, _ = RmsNorm(w)(x, out="fp32")
    within(y, ref, ref.abs() * REL + 1e-38)
    check_codes(*RmsNorm(w).forward_fp8(x)[:2], ref, REL)


def test_in_place_residual_and_given_outputs():
    x, res, w = case(70, 2056, F32, BF)
    op = RmsNorm(w)
    want_y, want_s = op(x, res)
    y = torch.empty_like(want_y)
    got_y, got_s = op(x, res, y=y, residual_out=res)
    assert got_y is y and got_s is res
    assert torch.equal(y, want_y) and torch.equal(res, want_s)
    xb = want_y.clone()
    want, _ = op(xb)
    op(xb, y=xb)
    assert torch.equal(xb, want)


def test_no_rows():
    w = torch.ones(64, device="cuda")
    op = RmsNorm(w)
    x = torch.empty(0, 64, device="cuda")
    y, s = op(x, x)
    assert y.shape == (0, 64) and s.shape == (0, 64)
    q, c, _ = op.forward_fp8(x)
    assert q.shape == (0, 64) and c.shape == (0, 1)
    g = op.backward(x, x)
    assert g["dx"].shape == (0, 64) and (g["dweight"] == 0).all()


def ref_backward(dy, s, ds, w, eps):
    dy, s, w = dy.double(), s.double(), w.double()
    d = s.shape[1]
    rstd = torch.rsqrt((s * s).mean(1, keepdim=True) + eps)
    g = dy * w
    a = (g * s).sum(1, keepdim=True)
    dx = rstd * g - s * a * rstd ** 3 / d
    if ds is not None:
        dx = dx + ds.double()
    return dx, (dy * s * rstd).sum(0), rstd, g


@pytest.mark.parametrize("T,d", SHAPES + [(1000, 256), (1500, 4096)])
@pytest.mark.parametrize("st,yt,with_ds", [(BF, BF, True), (F32, BF, False), (BF, F32, False), (F32, F32, True)])
def test_backward(T, d, st, yt, with_ds):
    s = randn(20, T, d, dtype=st, scale=1.5)
    dy = randn(21, T, d, dtype=yt, scale=0.1)
    ds = randn(22, T, d, dtype=st, scale=0.1) if with_ds else None
    w = (1 + 0.2 * randn(23, d)).to(BF)
    dx, dw, rstd, g = ref_backward(dy, s, ds, w, 1e-6)
    got = RmsNorm(w, 1e-6).backward(dy, s, ds)
    assert got["dx"].dtype is st and got["dweight"].dtype is F32
    # a = sum g s is off by at most 56 U of sum |g s|; rstd^3 by three times its own error
    size = rstd * g.abs() + s.double().abs() * rstd ** 3 / d * (g * s.double()).abs().sum(1, keepdim=True)
    tol = dx.abs() * HALF[st] + 160 * U * size
    if ds is not None:
        tol = tol + 4 * U * ds.double().abs()
    within(got["dx"], dx, tol, "dx")
    # a column adds its rows one after another: at most T/8 + T/8 + 16 additions on any path for these T
    # (8 rows side by side or 296 CTAs, then eight sums side by side), each product off by REL
    n = T / 8 + 400
    within(got["dweight"], dw, (n * U + REL) * (dy.double() * s.double() * rstd).abs().sum(0) + 1e-38, "dweight")


def test_backward_against_differences():
    # the 64-bit formula against central differences of the 64-bit forward: L = sum(y·dy) + sum(s·ds)
    T, d, eps, h = 3, 24, 1e-6, 1e-5
    s, dy, ds = (randn(i, T, d).double() for i in (30, 31, 32))
    w = 1 + 0.2 * randn(33, d).double()

    def loss(s, w):
        y, _ = ref_forward(s, None, w, eps)
        return (y * dy).sum() + (s * ds).sum()

    dx, dw, _, _ = ref_backward(dy, s, ds, w, eps)
    for i in range(T):
        for j in range(0, d, 5):
            e = torch.zeros_like(s)
            e[i, j] = h
            assert abs((loss(s + e, w) - loss(s - e, w)) / (2 * h) - dx[i, j]) < 1e-7
    for j in range(0, d, 5):
        e = torch.zeros_like(w)
        e[j] = h
        assert abs((loss(s, w + e) - loss(s, w - e)) / (2 * h) - dw[j]) < 1e-7


def test_backward_is_deterministic_and_in_place():
    s, dy, ds = (randn(i, 700, 1032, dtype=BF) for i in (40, 41, 42))
    op = RmsNorm(torch.ones(1032, device="cuda"))
    want = op.backward(dy, s, ds)
    for _ in range(3):
        again = op.backward(dy, s, ds)
        assert torch.equal(want["dx"], again["dx"]) and torch.equal(want["dweight"], again["dweight"])
    dw = torch.full((1032,), float("nan"), device="cuda")
    got = op.backward(dy, s, ds, dx=ds, dweight=dw)
    assert got["dx"] is ds and got["dweight"] is dw
    assert torch.equal(ds, want["dx"]) and torch.equal(dw, want["dweight"])


def test_graph_replay_and_two_streams():
    x, res, w = case(33, 2048, F32, BF)
    op = RmsNorm(w)
    s0, dy = randn(50, 33, 2048, dtype=BF), randn(51, 33, 2048, dtype=BF)
    g = torch.cuda.CUDAGraph()
    op(x, res), op.backward(dy, s0)
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        y, s = op(x, res)
        grad = op.backward(dy, s0)
    x.copy_(randn(52, 33, 2048))
    dy.copy_(randn(53, 33, 2048))
    g.replay()
    torch.cuda.synchronize()
    want_y, want_s = op(x, res)
    want = op.backward(dy, s0)
    assert torch.equal(y, want_y) and torch.equal(s, want_s)
    assert torch.equal(grad["dx"], want["dx"]) and torch.equal(grad["dweight"], want["dweight"])
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = []
    for i in range(20):
        st = (a, b)[i & 1]
        outs.append(op.backward(dy, s0, stream=st.cuda_stream))
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o["dx"], want["dx"]) and torch.equal(o["dweight"], want["dweight"])


@pytest.mark.parametrize("T,d", [(1, 8), (3, 128), (17, 136), (5, 4096), (300, 264), (2, 14336)])
@pytest.mark.parametrize("dt", [BF, F32])
def test_quantize_rows(T, d, dt):
    x = randn(60, T, d, dtype=dt, scale=3.0)
    x[0, :8] = 0
    check_codes(*quantize_rows(x), x.double(), 0.0)


@pytest.mark.parametrize("n,k", [(1, 8), (128, 128), (130, 264), (256, 1000), (8, 4096), (1000, 72)])
@pytest.mark.parametrize("dt", [BF, F32])
def test_quantize_blocks(n, k, dt):
    W = randn(61, n, k, dtype=dt, scale=0.02)
    q, c = quantize_blocks(W)
    assert c.shape == (groups(n), groups(k))
    for b in range(groups(n)):
        rows = W[b * 128:(b + 1) * 128].double()
        flat = torch.zeros(rows.shape[0], groups(k) * 128, dtype=torch.float64, device="cuda")
        flat[:, :k] = rows
        m = flat.view(rows.shape[0], -1, 128).abs().amax((0, 2)).clamp_min(1e-30)
        within(c[b], m / 448, m / 448 * 2 * U)
        v = rows * 448 / m.repeat_interleave(128)[:k]
        half = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 4)
        within(q[b * 128:(b + 1) * 128].float(), v, half + v.abs() * 3 * U)


def test_quantize_nan_stays_in_its_element():
    x = randn(62, 2, 256, dtype=F32)
    want_q, want_c = quantize_rows(x)
    x[1, 200] = float("nan")
    q, c = quantize_rows(x)
    assert torch.isnan(q[1, 200].float()) and torch.isfinite(c).all()
    assert torch.equal(q[0].view(torch.uint8), want_q[0].view(torch.uint8))
    assert torch.equal(q[1, :128].view(torch.uint8), want_q[1, :128].view(torch.uint8))


@pytest.mark.parametrize("T", [1, 3, 13])
@pytest.mark.parametrize("d", [8, 256, 264, 512, 1024, 1032])
@pytest.mark.parametrize("st,yt,with_ds", [(BF, BF, True), (F32, BF, False), (BF, F32, False), (F32, F32, True)])
def test_backward_without_eps(T, d, st, yt, with_ds):
    # up to 1024 columns a CTA has 2, 4 or 8 rows' threads, some of them past the last row here: what
    # they hold (zeros, whose norm is 0) reaches no sum.  Bounds as in test_backward.
    s = randn(70, T, d, dtype=st, scale=1.5)
    dy = randn(71, T, d, dtype=yt, scale=0.1)
    ds = randn(72, T, d, dtype=st, scale=0.1) if with_ds else None
    w = (1 + 0.2 * randn(73, d)).to(BF)
    dx, dw, rstd, g = ref_backward(dy, s, ds, w, 0.0)
    got = RmsNorm(w, 0.0).backward(dy, s, ds)
    size = rstd * g.abs() + s.double().abs() * rstd ** 3 / d * (g * s.double()).abs().sum(1, keepdim=True)
    tol = dx.abs() * HALF[st] + 160 * U * size
    if ds is not None:
        tol = tol + 4 * U * ds.double().abs()
    within(got["dx"], dx, tol, "dx")
    within(got["dweight"], dw, ((T / 8 + 400) * U + REL) * (dy.double() * s.double() * rstd).abs().sum(0) + 1e-38, "dweight")


def test_a_norm_in_place_gives_no_sum():
    # without a residual the sum is x itself; where y replaces x, x holds it no longer
    x, _, w = case(5, 264, BF, None, seed=80)
    op = RmsNorm(w)
    want, s = op(x)
    assert s is x
    other = torch.empty_like(x)
    assert op(x, y=other)[1] is x and torch.equal(other, want)
    for y in (x.clone(), x.clone()):
        got, s = op(y, y=y.view(5, 264))
        assert s is None and torch.equal(y, want) and got.data_ptr() == y.data_ptr()
    r = randn(81, 5, 264, dtype=BF)
    want, want_s = op(x, r)
    xb = x.clone()
    got, s = op(xb, r, y=xb)
    assert torch.equal(got, want) and torch.equal(s, want_s)


@pytest.mark.parametrize("T,d", [(1500, 4104), (1500, 8192), (700, 12296), (700, 16384)])
@pytest.mark.parametrize("st", [BF, F32])
@pytest.mark.parametrize("yt", [BF, F32])
@pytest.mark.parametrize("with_ds", [False, True])
def test_backward_with_several_rows_per_cta(T, d, st, yt, with_ds):
    test_backward(T, d, st, yt, with_ds)

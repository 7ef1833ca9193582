"""The 8-bit linear layer against plain products in 64 bits.

Bounds.  Products of two codes are exact in fp32 (4 + 4 significant bits) and
a 128-wide block's sum is off by less than 128 U of the sum of magnitudes; one
product of the scales, one with the block's sum and one addition per block
follow: (128 + kb + 8) U · sum |x||w|, and half a step of y's type.  On inputs
whose sums are exact in fp32 (small whole codes, scales powers of two) y has
to be the exact value, rounded once."""
from __future__ import annotations

import pytest
import torch

from activation_sparse_gated_relu_b200 import SFFN_OK, Fp8Linear, quantize_blocks, quantize_rows
from layer_util import HALF, U, gen, groups, ints, randn, spread_cols, within

pytestmark = pytest.mark.gpu

BF, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


def values(q, scale):
    return q.double() * spread_cols(scale.double(), q.shape[1])


def weights(Wq, Ws):
    n, k = Wq.shape
    return Wq.double() * spread_cols(Ws.double().repeat_interleave(128, 0)[:n], k)


def check(op, xq, xs, out="bf16"):
    y = op.forward(xq, xs, out=out)
    torch.cuda.synchronize()
    assert op.read_status() == SFFN_OK
    x, w = values(xq, xs), weights(op.Wq, op.Ws)
    ref = x @ w.t()
    size = x.abs() @ w.abs().t()
    within(y, ref, ref.abs() * HALF[y.dtype] + (128 + groups(op.d_in) + 8) * U * size + 1e-38, f"y {out}")
    return y


SHAPES = [(1, 16, 8), (1, 128, 128), (2, 144, 136), (7, 256, 1000), (8, 4096, 512), (13, 1040, 264), (16, 512, 256),
          (17, 400, 128), (33, 2048, 384), (64, 272, 520), (65, 256, 256), (100, 1024, 1032), (128, 4096, 256),
          (129, 144, 8), (257, 640, 392), (333, 2048, 512), (520, 512, 1544), (1000, 1168, 640),
          (3, 4096, 9728), (20, 4096, 9728), (40, 4096, 9728), (70, 4224, 9728), (2, 14336, 264)]


@pytest.mark.parametrize("T,k,n", SHAPES)
@pytest.mark.parametrize("out", ["bf16", "fp32"])
def test_random_codes(T, k, n, out):
    op = Fp8Linear.from_weight(randn(1, n, k, dtype=BF, scale=k ** -0.5))
    check(op, *quantize_rows(randn(2, T, k, dtype=BF)), out=out)


@pytest.mark.parametrize("T,k,n", SHAPES)
def test_exact_sums(T, k, n):
    # codes in -3..3 and scales 2^-2..2^2: every partial sum is a multiple of 2^-4 below 9 · 16 · 14336 < 2^21,
    # 25 bits at most with sums that stay far below that bound: fp32 holds all of them exactly and any order of additions
    # gives the same sum
    xq, Wq = ints(3, T, k, lim=3, dtype=F32).to(F8), ints(4, n, k, lim=3, dtype=F32).to(F8)
    xs = torch.exp2(torch.randint(-2, 3, (T, groups(k)), generator=gen(5)).float()).cuda()
    Ws = torch.exp2(torch.randint(-2, 3, (groups(n), groups(k)), generator=gen(6)).float()).cuda()
    op = Fp8Linear(Wq, Ws)
    ref = values(xq, xs) @ weights(Wq, Ws).t()
    assert torch.equal(op.forward(xq, xs, out="fp32"), ref.float())
    assert torch.equal(op.forward(xq, xs), ref.float().to(BF))
    assert op.read_status() == SFFN_OK


@pytest.mark.parametrize("T", [1, 13, 200])
@pytest.mark.parametrize("dt", [BF, F32])
def test_unquantised_input(T, dt):
    op = Fp8Linear.from_weight(randn(7, 384, 528, dtype=BF))
    x = randn(8, T, 528, dtype=dt)
    assert torch.equal(op(x), op(*quantize_rows(x)))


@pytest.mark.parametrize("T", [3, 40, 300])
def test_rows_keep_to_themselves(T):
    op = Fp8Linear.from_weight(randn(9, 264, 400, dtype=BF))
    xq, xs = quantize_rows(randn(10, T, 400, dtype=BF))
    want = op(xq, xs)
    q = xq.clone()
    q.view(torch.uint8)[T // 2, 17] = 0x7F                # NaN
    y = op(q, xs)
    keep = [t for t in range(T) if t != T // 2]
    assert torch.equal(y[keep], want[keep]) and torch.isnan(y[T // 2]).all()
    c = xs.clone()
    c[T // 2, 1] = float("inf")
    y = op(xq, c)
    assert torch.equal(y[keep], want[keep]) and not torch.isfinite(y[T // 2]).any()


def test_nothing_is_written_behind_y():
    op = Fp8Linear.from_weight(randn(11, 200, 272, dtype=BF))
    for T in (1, 9, 130):
        xq, xs = quantize_rows(randn(12, T, 272, dtype=BF))
        buf = torch.full((T + 8, 200), 7.0, dtype=BF, device="cuda")
        op(xq, xs, y=buf[:T])
        assert (buf[T:] == 7).all()
        assert torch.equal(buf[:T], op(xq, xs))


def test_no_rows():
    op = Fp8Linear.from_weight(randn(13, 64, 128, dtype=BF))
    assert op(torch.empty(0, 128, dtype=BF, device="cuda")).shape == (0, 64)


def test_graph_replay_and_overlapping_calls():
    op = Fp8Linear.from_weight(randn(14, 1024, 2048, dtype=BF, scale=0.02))
    for T in (4, 150):
        x = randn(15, T, 2048, dtype=BF)
        want = op(x)
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            y = op(x)
        x.copy_(randn(16, T, 2048, dtype=BF))
        g.replay()
        torch.cuda.synchronize()
        want2 = op(x)
        assert torch.equal(y, want2) and not torch.equal(want, want2)
        a, b = torch.cuda.Stream(), torch.cuda.Stream()
        torch.cuda.synchronize()
        outs = [op(x, stream=(a, b)[i & 1].cuda_stream) for i in range(20)]
        torch.cuda.synchronize()
        assert all(torch.equal(o, want2) for o in outs)
    assert op.read_status() == SFFN_OK


def test_weight_blocks_of_zeros_and_large_scales():
    W = randn(17, 304, 512, dtype=BF)
    W[:128, 128:256] = 0
    op = Fp8Linear.from_weight(W)
    assert torch.isfinite(op.Ws).all()
    xq, xs = quantize_rows(randn(18, 5, 512, dtype=BF))
    check(op, xq, xs, "fp32")
    check(Fp8Linear(op.Wq, op.Ws * 2.0 ** 60), xq, xs * 2.0 ** -70, "fp32")


# long k and few tiles of 128 x 128: 3, 1, 1, 18, 26, 63 and 112 of them, k cut in up to eight parts, also uneven ones
LONG = [(33, 4096, 264), (128, 4112, 128), (100, 14336, 8), (300, 4240, 648), (200, 4240, 1544), (257, 6160, 2568),
        (448, 6160, 3584)]


@pytest.mark.parametrize("T,k,n", LONG)
@pytest.mark.parametrize("out", ["bf16", "fp32"])
def test_long_inner_sizes(T, k, n, out):
    test_random_codes(T, k, n, out)
    test_exact_sums(T, k, n)


@pytest.mark.parametrize("T,k,n", LONG[:5])
def test_long_inner_sizes_leave_what_lies_behind_y(T, k, n):
    op = Fp8Linear.from_weight(randn(20, n, k, dtype=BF, scale=k ** -0.5))
    xq, xs = quantize_rows(randn(21, T, k, dtype=BF))
    for dt, out in ((BF, "bf16"), (F32, "fp32")):
        buf = torch.full((T + 3, n), 7.0, dtype=dt, device="cuda")
        y = op.forward(xq, xs, out=out)
        assert torch.equal(op.forward(xq, xs, out=out, y=buf[:T]), y)
        assert (buf[T:] == 7).all()
        assert all(torch.equal(op.forward(xq, xs, out=out), y) for _ in range(5))

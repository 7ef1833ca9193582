"""The experts' grouped products, forward and both gradients, against plain
products in 64 bits.

Bounds.  Sums over K terms are fp32: off by less than (K + 64) U · sum |a||b|
whatever their order, plus half a step of the output's type.  On small whole
numbers, whose sums fp32 holds exactly, the outputs have to be the exact
values, rounded once."""
from __future__ import annotations

import pytest
import torch

from activation_sparse_gated_relu_b200 import SFFN_ERR_DEVICE, SFFN_OK, GroupedLinear
from layer_util import HALF, U, ints, randn, within

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def layout(counts, lead=0):
    off = [lead]
    for c in counts:
        off.append(off[-1] + c)
    return off, torch.tensor(off, dtype=torch.int32, device="cuda")


# counts per expert, rows before the first and behind the last group, d_in, d_out
CASES = [
    ([1], 0, 0, 8, 8),
    ([0], 0, 3, 64, 64),
    ([5, 0, 3], 0, 0, 64, 128),
    ([1, 1, 1, 1], 0, 4, 72, 136),
    ([16, 17, 0, 15], 2, 5, 128, 264),
    ([33, 0, 0, 64, 1], 0, 0, 200, 256),
    ([130, 7], 1, 0, 512, 384),
    ([127, 128, 129], 0, 9, 136, 136),
    ([255, 0, 257], 3, 1, 320, 520),
    ([600], 0, 0, 264, 1032),
    ([0, 0, 300, 0], 0, 20, 1024, 128),
    ([2] * 40 + [0] * 24, 0, 0, 256, 256),
    ([70, 3, 0, 900, 1], 7, 11, 648, 776),
]


@pytest.mark.parametrize("counts,lead,tail,k,n", CASES)
@pytest.mark.parametrize("out", ["bf16", "fp32"])
def test_forward_and_gradients(counts, lead, tail, k, n, out):
    E, t = len(counts), BF if out == "bf16" else F32
    off, offsets = layout(counts, lead)
    R = off[-1] + tail
    x, dy, W = randn(1, R, k, dtype=BF), randn(2, R, n, dtype=BF), randn(3, E, n, k, dtype=BF, scale=k ** -0.5)
    op = GroupedLinear(W)
    y = torch.full((R, n), 7.0, dtype=t, device="cuda")
    dx = torch.full((R, k), 7.0, dtype=t, device="cuda")
    dW = torch.full((E, n, k), float("nan"), dtype=t, device="cuda")
    op.forward(x, offsets, out=out, y=y)
    op.backward(x, dy, offsets, out=out, dx=dx, dW=dW)
    torch.cuda.synchronize()
    assert op.read_status() == SFFN_OK
    for rows in (slice(0, lead), slice(off[-1], R)):
        assert (y[rows] == 7).all() and (dx[rows] == 7).all()
    for e in range(E):
        r = slice(off[e], off[e + 1])
        xe, de, we = x[r].double(), dy[r].double(), W[e].double()
        for got, a, b, K in ((y[r], xe, we.t(), k), (dx[r], de, we, n), (dW[e], de.t(), xe, counts[e])):
            ref = a @ b
            within(got, ref, ref.abs() * HALF[t] + (K + 64) * U * (a.abs() @ b.abs()) + 1e-38, f"expert {e}")


@pytest.mark.parametrize("counts,lead,tail,k,n", CASES)
def test_exact_sums(counts, lead, tail, k, n):
    # values in -4..4: sums below 16 · 1032 < 2^24 in magnitude
    E = len(counts)
    off, offsets = layout(counts, lead)
    R = off[-1] + tail
    x, dy, W = ints(4, R, k), ints(5, R, n), ints(6, E, n, k)
    op = GroupedLinear(W)
    y = op.forward(x, offsets, out="fp32")
    g = op.backward(x, dy, offsets, out="fp32")
    yb = op.forward(x, offsets)
    for e in range(E):
        r = slice(off[e], off[e + 1])
        ref = (x[r].double() @ W[e].double().t()).float()
        assert torch.equal(y[r], ref) and torch.equal(yb[r], ref.to(BF))
        assert torch.equal(g["dx"][r], (dy[r].double() @ W[e].double()).float())
        assert torch.equal(g["dW"][e], (dy[r].double().t() @ x[r].double()).float())
    assert op.read_status() == SFFN_OK


def test_values_outside_a_group_never_reach_it():
    # rows of other experts, rows in no group and the weights of other experts hold NaN and infinities
    counts, k, n = [20, 0, 150, 3], 136, 264
    off, offsets = layout(counts, 5)
    R = off[-1] + 6
    x, dy, W = ints(7, R, k), ints(8, R, n), ints(9, 4, n, k)
    good = GroupedLinear(W)
    y, g = good(x, offsets), good.backward(x, dy, offsets)
    for e in (0, 2, 3):
        bx, bd, bw = x.clone(), dy.clone(), W.clone()
        mine = slice(off[e], off[e + 1])
        other = torch.ones(R, dtype=torch.bool, device="cuda")
        other[mine] = False
        bx[other], bd[other] = float("nan"), float("inf")
        for f in range(4):
            if f != e:
                bw[f] = float("inf")
        op = GroupedLinear(bw)
        y2, g2 = op(bx, offsets), op.backward(bx, bd, offsets)
        assert torch.equal(y2[mine], y[mine])
        assert torch.equal(g2["dx"][mine], g["dx"][mine])
        assert torch.equal(g2["dW"][e], g["dW"][e])
        assert (g2["dW"][1] == 0).all()


def test_offsets_out_of_range_are_reported_and_clamped():
    op = GroupedLinear(ints(10, 3, 64, 64))
    x, dy = ints(11, 40, 64), ints(12, 40, 64)
    good = torch.tensor([0, 10, 20, 40], dtype=torch.int32, device="cuda")
    for bad in ([0, 10, 20, 41], [-5, 10, 20, 40], [0, 30, 20, 40], [0, 2 ** 31 - 1, 20, 40], [-2 ** 31, 5, 5, 2 ** 30]):
        off = torch.tensor(bad, dtype=torch.int32, device="cuda")
        for call in (lambda: op.forward(x, off), lambda: op.backward(x, dy, off)):
            call()
            assert op.read_status() == SFFN_ERR_DEVICE
            assert op.read_status() == SFFN_OK
    op.forward(x, good), op.backward(x, dy, good)
    assert op.read_status() == SFFN_OK


def test_no_rows_and_many_experts():
    op = GroupedLinear(ints(13, 1024, 16, 16))
    off = torch.zeros(1025, dtype=torch.int32, device="cuda")
    x = torch.empty(0, 16, dtype=BF, device="cuda")
    assert op(x, off).shape == (0, 16)
    g = op.backward(x, x, off)
    assert g["dx"].shape == (0, 16) and (g["dW"] == 0).all()
    counts = [(i * 7) % 3 for i in range(1024)]
    o, offsets = layout(counts)
    x = ints(14, o[-1], 16)
    y = op(x, offsets, out="fp32")
    e = torch.repeat_interleave(torch.arange(1024), torch.tensor(counts)).cuda()
    assert torch.equal(y, torch.einsum("rk,rnk->rn", x.double(), op.W[e].double()).float())
    g = op.backward(x, x, offsets)
    dW = torch.zeros(1024, 16, 16, dtype=torch.float64, device="cuda")
    dW.index_add_(0, e, torch.einsum("rn,rk->rnk", x.double(), x.double()))
    assert torch.equal(g["dW"], dW.float())


def test_weights_may_change_between_calls():
    W = ints(15, 2, 128, 64)
    op = GroupedLinear(W)
    off, offsets = layout([9, 4])
    x = ints(16, 13, 64)
    op(x, offsets)
    W.copy_(ints(17, 2, 128, 64))
    assert torch.equal(op(x, offsets, out="fp32")[9:], (x[9:].double() @ W[1].double().t()).float())


def test_graph_replay_with_new_offsets_and_overlapping_calls():
    E, k, n, R = 4, 256, 512, 300
    W, x, dy = ints(18, E, n, k), ints(19, R, k), ints(20, R, n)
    op = GroupedLinear(W)
    _, a = layout([100, 0, 150, 50])
    _, b = layout([3, 250, 0, 47])
    off = a.clone()
    torch.cuda.synchronize()
    op(x, off), op.backward(x, dy, off)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        y = op(x, off)
        grad = op.backward(x, dy, off)
    for o in (b, a):
        off.copy_(o)
        g.replay()
        torch.cuda.synchronize()
        want = op.backward(x, dy, o)
        assert torch.equal(y, op(x, o)) and torch.equal(grad["dx"], want["dx"]) and torch.equal(grad["dW"], want["dW"])
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = [op.backward(x, dy, a, stream=(s, t)[i & 1].cuda_stream) for i in range(12)]
    torch.cuda.synchronize()
    want = op.backward(x, dy, a)
    assert all(torch.equal(v["dx"], want["dx"]) and torch.equal(v["dW"], want["dW"]) for v in outs)
    assert op.read_status() == SFFN_OK


def test_gradients_against_differences():
    # the 64-bit formulas against differences of L = sum(y·dy), y = W[e(r)] x[r] (linear: any step is exact to rounding)
    counts, k, n = [3, 0, 2], 8, 16
    off, _ = layout(counts)
    x, dy, W = randn(21, 5, k).double(), randn(22, 5, n).double(), randn(23, 3, n, k).double()
    e = torch.tensor([0, 0, 0, 2, 2], device="cuda")

    def loss(x, W):
        return (torch.einsum("rk,rnk->rn", x, W[e]) * dy).sum()

    dx = torch.einsum("rn,rnk->rk", dy, W[e])
    dW = torch.stack([dy[off[i]:off[i + 1]].t() @ x[off[i]:off[i + 1]] for i in range(3)])
    for r, c in ((0, 0), (3, 7)):
        h = torch.zeros_like(x)
        h[r, c] = 0.5
        assert abs(loss(x + h, W) - loss(x - h, W) - dx[r, c]) < 1e-12
    for i, o, c in ((0, 3, 2), (1, 0, 0), (2, 15, 7)):
        h = torch.zeros_like(W)
        h[i, o, c] = 0.5
        assert abs(loss(x, W + h) - loss(x, W - h) - dW[i, o, c]) < 1e-12


def test_offsets_that_run_back_and_forth_count_no_row_twice():
    # the first group has all rows, so the others, whatever they ask for, have none
    op = GroupedLinear(ints(30, 64, 64, 64))
    x, dy = ints(31, 40, 64), ints(32, 40, 64)
    off = torch.tensor([0, 40] * 32 + [40], dtype=torch.int32, device="cuda")
    y, g = op(x, off), op.backward(x, dy, off)
    assert op.read_status() == SFFN_ERR_DEVICE
    assert torch.equal(y, (x.float() @ op.W[0].float().t()).to(BF))
    assert torch.equal(g["dx"], (dy.float() @ op.W[0].float()).to(BF))
    assert torch.equal(g["dW"][0], dy.float().t() @ x.float()) and (g["dW"][1:] == 0).all()


# few rows and a long inner size, whose parts the CTAs of a cluster take: forward in the first four, both in the
# fifth, the input gradient in the last two; odd part lengths, short last blocks, groups of 32 and 33 rows
FEW = [
    ([1, 0, 1, 1], 0, 5, 3472, 920),
    ([3], 2, 1, 2056, 136),
    ([0, 2, 0, 33, 1], 1, 0, 4104, 264),
    ([0] * 60 + [1, 0, 1, 0], 0, 0, 6152, 1032),
    ([20, 3], 0, 2, 2056, 2120),
    ([2, 0, 5], 0, 0, 264, 4104),
    ([7], 0, 0, 128, 14336),
]


@pytest.mark.parametrize("counts,lead,tail,k,n", FEW)
@pytest.mark.parametrize("out", ["bf16", "fp32"])
def test_few_rows_and_long_sums(counts, lead, tail, k, n, out):
    test_forward_and_gradients(counts, lead, tail, k, n, out)


@pytest.mark.parametrize("counts,lead,tail,k,n", FEW[:5])
def test_few_rows_are_exact_and_alike(counts, lead, tail, k, n):
    # whole numbers up to 4: sums below 16 · 6152 < 2^24, exact in fp32
    off, offsets = layout(counts, lead)
    R = off[-1] + tail
    x, W = ints(40, R, k), ints(41, len(counts), n, k)
    x[off[-1]:] = float("nan")
    x[:lead] = float("nan")
    op = GroupedLinear(W)
    ref = torch.cat([x[off[e]:off[e + 1]].double() @ W[e].double().t() for e in range(len(counts))])
    rows = slice(lead, off[-1])
    for _ in range(5):
        assert torch.equal(op.forward(x, offsets, out="fp32")[rows], ref.float())
        assert torch.equal(op.forward(x, offsets)[rows], ref.float().to(BF))
    assert op.read_status() == SFFN_OK
    # offsets that name other groups, or none, than the call before
    none = torch.full_like(offsets, lead)
    y = torch.full((R, n), 7.0, dtype=BF, device="cuda")
    op.forward(x, none, y=y)
    assert (y == 7).all() and op.read_status() == SFFN_OK


def _half_step(ref, eps_bits=8):
    """Half of bf16's step in each value's own binade."""
    return torch.exp2(torch.floor(torch.log2(ref.abs())) - eps_bits)


@pytest.mark.parametrize("what", ["y", "dx", "dW"])
def test_long_sums_into_bf16(what):
    """Sums of 2^20 positive terms, rounded to bf16 once.  The tensor core adds 16 terms at a time to a sum of 24 bits
    and drops what lies below, less than 2^-22 of the sum (its own last bit and the terms'); runs of 16384 terms are 1024
    such steps, 2^-12 at most, and 64 runs added in fp32 at most 64 U more.  Columns of different sizes, so that the
    sums lie all over a binade."""
    K = 1 << 20
    size = torch.linspace(1, 2, 64, device="cuda")
    a = (1 + torch.rand(K, 64, generator=torch.Generator("cuda").manual_seed(50), device="cuda")) * size
    b = 1 + torch.rand(K, 24, generator=torch.Generator("cuda").manual_seed(51), device="cuda")
    a, b = a.to(BF), b.to(BF)
    if what == "dW":
        op = GroupedLinear(torch.zeros(1, 24, 64, dtype=BF, device="cuda"))
        dW = torch.empty(1, 24, 64, dtype=BF, device="cuda")
        op.backward(a, b, torch.tensor([0, K], dtype=torch.int32, device="cuda"), dW=dW)
        got = dW[0]
    else:
        off = torch.tensor([0, 24], dtype=torch.int32, device="cuda")
        if what == "y":
            op = GroupedLinear(a.t().contiguous()[None])
            got = op.forward(b.t().contiguous(), off)
        else:
            op = GroupedLinear(a[None])
            got = op.backward(torch.zeros(24, 64, dtype=BF, device="cuda"), b.t().contiguous(), off)["dx"]
    ref = b.double().t() @ a.double()
    within(got, ref, _half_step(ref) + ref * (2.0 ** -12 + 64 * U), what)
    assert op.read_status() == SFFN_OK


def test_gradients_of_the_operator_against_differences():
    # whole numbers up to 4: L = sum(y·dy) is exact, and linear in x and in W, so that a difference over a step of 2
    # is the gradient's very value
    counts, k, n = [3, 0, 2], 16, 24
    off, offsets = layout(counts, 1)
    R = off[-1] + 2
    x, dy, W = ints(60, R, k), ints(61, R, n), ints(62, 3, n, k)
    mine = slice(off[0], off[-1])
    got = GroupedLinear(W).backward(x, dy, offsets, out="fp32")

    def loss(x, W):
        y = GroupedLinear(W).forward(x, offsets, out="fp32")
        return (y[mine].double() * dy[mine].double()).sum().item()

    for r, c in ((1, 0), (3, 15), (4, 7), (5, 9)):
        up, down = x.clone(), x.clone()
        up[r, c] += 1
        down[r, c] -= 1
        assert (loss(up, W) - loss(down, W)) / 2 == got["dx"][r, c].item()
    for e, o, c in ((0, 3, 2), (0, 23, 15), (1, 0, 0), (2, 15, 7)):
        up, down = W.clone(), W.clone()
        up[e, o, c] += 1
        down[e, o, c] -= 1
        assert (loss(x, up) - loss(x, down)) / 2 == got["dW"][e, o, c].item()

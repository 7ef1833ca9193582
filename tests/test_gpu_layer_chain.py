"""The operators around the sparse FFN as a layer uses them: FFN output and
residual through the norm into the 8-bit linear; the mixture's routing into the
experts' dense products, forward and backward.  Each stage is checked against
its formula in 64 bits on the values that the stage before it gave, with the
bounds of that operator's own tests.  Also what the classes refuse on a GPU."""
from __future__ import annotations

import pytest
import torch

from activation_sparse_gated_relu_b200 import (SFFN_OK, Fp8Linear, GroupedLinear, MoeFFN, RmsNorm, SparseFFN,
                                               quantize_blocks, quantize_rows)
from layer_util import HALF, U, check_codes, groups, ints, randn, spread_cols, within

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("T", [1, 8, 40])
def test_ffn_norm_linear(T):
    d, F = 512, 1024
    ffn = SparseFFN(randn(1, F, d, dtype=BF, scale=d ** -0.5), randn(2, F, d, dtype=BF, scale=F ** -0.5),
                    W_gate=randn(3, F, d, dtype=BF, scale=d ** -0.5), bias=randn(4, F, scale=0.1), max_tokens=T)
    n1, n2 = RmsNorm(torch.ones(d, device="cuda", dtype=BF)), RmsNorm((1 + 0.1 * randn(5, d)).to(BF))
    lin = Fp8Linear.from_weight(randn(6, 768, d, dtype=BF, scale=d ** -0.5))
    h = randn(7, T, d, dtype=BF)
    x, _ = n1(h)
    y = ffn(x)
    q, scale, s = n2.forward_fp8(y, h)
    out = lin(q, scale)
    torch.cuda.synchronize()
    assert ffn.read_status() == SFFN_OK and lin.read_status() == SFFN_OK
    assert y.abs().max() > 0
    v = y.double() + h.double()
    v = v * torch.rsqrt((v * v).mean(1, keepdim=True) + 1e-6) * n2.weight.double()
    check_codes(q, scale, v, 40 * U)
    xv = q.double() * spread_cols(scale.double(), d)
    wv = lin.Wq.double() * spread_cols(lin.Ws.double().repeat_interleave(128, 0), d)
    ref = xv @ wv.t()
    within(out, ref, ref.abs() * HALF[BF] + (136 + groups(d)) * U * (xv.abs() @ wv.abs().t()))


def test_mixture_routing_into_grouped_products():
    T, d, F, E, k = 24, 256, 512, 4, 2
    ex = [dict(A=randn(10 + e, d, 64, dtype=BF, scale=d ** -0.5), B=randn(20 + e, 64, F, dtype=BF, scale=0.125),
               W_up=randn(30 + e, F, d, dtype=BF, scale=d ** -0.5), W_down=randn(40 + e, F, d, dtype=BF, scale=F ** -0.5),
               bias=None) for e in range(E)]
    moe = MoeFFN(randn(50, E, d, dtype=BF), ex, k, max_tokens=T)
    x = randn(51, T, d, dtype=BF)
    sparse = moe(x)
    torch.cuda.synchronize()
    assert moe.read_status() == SFFN_OK
    route = moe.routing(T)
    sel = route["sel"].long()
    order = sel.flatten().argsort(stable=True)
    offsets = torch.searchsorted(sel.flatten()[order], torch.arange(E + 1, device="cuda")).int()
    xs = x[order // k]
    stack = lambda key: torch.stack([e[key] for e in ex])  # noqa: E731
    gate_w = torch.stack([(e["A"].double() @ e["B"].double()).t() for e in ex]).to(BF).contiguous()
    up, gate = GroupedLinear(stack("W_up")), GroupedLinear(gate_w)
    down = GroupedLinear(stack("W_down").transpose(1, 2).contiguous())
    u, g = up(xs, offsets), gate(xs, offsets)
    h = (g.relu() * u).contiguous()
    y = down(h, offsets, out="fp32")
    out = torch.zeros(T, d, device="cuda").index_add_(0, order // k, y * route["w"].flatten()[order][:, None])
    # both ways compute the same mixture; the sparse one rounds z, the dense one u, g, h and the gate's weight, each
    # to bf16: at most 8 roundings of 2^-8 relative to sums of magnitudes on the way, far below this band
    assert (out - sparse).norm() <= 8 * 2 ** -8 * sparse.norm()
    e = sel.flatten()[order]
    dy = randn(52, T * k, d, dtype=BF)
    gd = down.backward(h, dy, offsets)
    gu = up.backward(xs, (gd["dx"] * g.relu()).contiguous(), offsets)
    for got, a, w in ((y, h, down.W), (u, xs, up.W)):
        ref = torch.einsum("rk,rnk->rn", a.double(), w[e].double())
        size = torch.einsum("rk,rnk->rn", a.double().abs(), w[e].double().abs())
        within(got, ref, ref.abs() * HALF[got.dtype] + (F + 64) * U * size)
    for i in range(E):
        m = e == i
        ref = dy[m].double().t() @ h[m].double()
        within(gd["dW"][i], ref, (T * k + 64) * U * (dy[m].double().abs().t() @ h[m].double().abs()) + ref.abs() * U + 1e-38)
        du = (gd["dx"] * g.relu())[m].double()
        ref = du @ up.W[i].double()
        within(gu["dx"][m], ref, ref.abs() * HALF[BF] + (F + 64) * U * (du.abs() @ up.W[i].double().abs()) + 1e-38)
    for op in (up, gate, down):
        assert op.read_status() == SFFN_OK


def test_classes_refuse():
    op = RmsNorm(torch.ones(256, device="cuda"))
    x = randn(60, 4, 256)
    for bad, kind in ((x[:, :128], ValueError), (randn(0, 4, 512)[:, ::2], ValueError), (x.half(), TypeError),
                      (x.cpu(), ValueError), (randn(0, 4 * 256 + 1)[1:].view(4, 256), ValueError), (x[0], ValueError)):
        with pytest.raises(kind):
            op(bad)
        with pytest.raises(kind):
            op(x, bad)
        with pytest.raises(kind):
            op.backward(x, bad)
    with pytest.raises(ValueError):
        op(x, residual_out=x)
    with pytest.raises(ValueError, match="overlap"):
        buf = randn(61, 5, 256, dtype=BF)
        op(buf[:4], y=buf[1:])
    with pytest.raises(TypeError):
        op(x, y=torch.empty(4, 256, device="cuda"))
    with pytest.raises(ValueError):
        RmsNorm(torch.ones(256, device="cuda"), eps=-1.0)
    with pytest.raises(RuntimeError):
        RmsNorm(torch.ones(250, device="cuda"))
    lin = Fp8Linear.from_weight(randn(62, 128, 256, dtype=BF))
    q, c = quantize_rows(x)
    with pytest.raises(TypeError):
        lin(q)
    with pytest.raises(TypeError):
        lin(x, c)
    with pytest.raises(ValueError):
        lin(q, c[:, :1].contiguous())
    with pytest.raises(ValueError):
        lin(q, c, out="fp64")
    with pytest.raises(ValueError):
        lin(randn(0, 4, 128))
    sq = Fp8Linear.from_weight(randn(63, 256, 256, dtype=BF))
    both = torch.empty(4, 512, dtype=torch.uint8, device="cuda")
    with pytest.raises(ValueError, match="overlap"):
        sq(both.view(-1)[:1024].view(torch.float8_e4m3fn).view(4, 256), c, y=both.view(BF).view(4, 256))
    grp = GroupedLinear(randn(64, 2, 128, 128, dtype=BF))
    xb, off = randn(65, 6, 128, dtype=BF), torch.tensor([0, 2, 6], dtype=torch.int32, device="cuda")
    for bad in (off.long(), off.cpu(), off[:2], [0, 2, 6]):
        with pytest.raises(ValueError, match="offsets"):
            grp(xb, bad)
    with pytest.raises(TypeError):
        grp(xb.float(), off)
    with pytest.raises(ValueError, match="overlap"):
        grp(xb, off, y=xb)
    with pytest.raises(ValueError):
        grp.backward(xb, xb[:4], off)
    with pytest.raises(RuntimeError):
        GroupedLinear(randn(66, 2, 12, 128, dtype=BF))


def test_quantisers_refuse_overlapping_outputs():
    x = torch.zeros(64, 256, dtype=torch.bfloat16, device="cuda")
    bytes_ = x.view(torch.uint8).flatten()
    over = bytes_[:64 * 256].view(torch.float8_e4m3fn).view(64, 256)
    codes = torch.zeros(64, 256, dtype=torch.float8_e4m3fn, device="cuda")
    inside = codes.view(torch.uint8).flatten()
    with pytest.raises(ValueError, match="overlap"):
        quantize_rows(x, codes=over)
    with pytest.raises(ValueError, match="overlap"):
        quantize_rows(x, codes=codes, scale=inside[:64 * 8].view(torch.float32).view(64, 2))
    with pytest.raises(ValueError, match="overlap"):
        quantize_rows(x, scale=bytes_[:64 * 8].view(torch.float32).view(64, 2))
    with pytest.raises(ValueError, match="overlap"):
        quantize_blocks(x, codes=over)
    with pytest.raises(ValueError, match="overlap"):
        quantize_blocks(x, codes=codes, scale=inside[:8].view(torch.float32).view(1, 2))


def test_a_replaced_weight_is_noticed():
    x = torch.zeros(4, 256, dtype=torch.bfloat16, device="cuda")
    norm = RmsNorm(torch.ones(256, dtype=torch.bfloat16, device="cuda"))
    lin = Fp8Linear.from_weight(torch.ones(64, 256, dtype=torch.bfloat16, device="cuda"))
    experts = GroupedLinear(torch.ones(2, 64, 256, dtype=torch.bfloat16, device="cuda"))
    off = torch.tensor([0, 2, 4], dtype=torch.int32, device="cuda")
    norm.forward(x), lin(x), experts(x, off)
    for owner, name in ((norm, "weight"), (lin, "Wq"), (experts, "W")):
        t = getattr(owner, name)
        t.data = t.clone()
    for call in (lambda: norm.forward(x), lambda: norm.backward(x, x), lambda: lin(x), lambda: experts(x, off),
                 lambda: experts.backward(x, x[:, :64].contiguous(), off)):
        with pytest.raises(ValueError, match="replaced"):
            call()


def test_offsets_past_32_bits():
    # 2^31 + 2^21 elements of 16 bits: the last rows against the same call on those rows alone (bit for bit, a row
    # depends on no other), products of small whole numbers against their exact sums
    free, _ = torch.cuda.mem_get_info()
    if free < 40 << 30:
        pytest.skip("needs 40 GB")
    T, d, last = 262400, 8192, slice(262400 - 130, 262400)
    x = torch.empty(T, d, dtype=BF, device="cuda").fill_(0.5)
    x[last] = randn(50, 130, d, dtype=BF)
    norm = RmsNorm(randn(51, d, dtype=BF))
    y, s = norm.forward(x, x)
    y1, s1 = norm.forward(x[last].contiguous(), x[last].contiguous())
    assert torch.equal(y[last], y1) and torch.equal(s[last], s1)
    dx = norm.backward(y, s)["dx"]
    assert torch.equal(dx[last], norm.backward(y1, s1)["dx"])
    del s, dx
    q, scale = quantize_rows(y)
    q1, scale1 = quantize_rows(y1)
    assert torch.equal(q[last].view(torch.uint8), q1.view(torch.uint8)) and torch.equal(scale[last], scale1)
    del q, y
    W = ints(52, d, 64, lim=3)
    small = ints(53, T, 64, lim=3)
    ref = (small[last].float() @ W.float().t()).to(BF)     # below 9 · 64: exact in fp32
    lin = Fp8Linear(W.to(torch.float8_e4m3fn), torch.ones(groups(d), 1, device="cuda"))
    out = lin(small.to(torch.float8_e4m3fn), torch.ones(T, 1, device="cuda"))
    assert torch.equal(out[last], ref) and lin.read_status() == SFFN_OK
    op = GroupedLinear(torch.stack([-W, W]))
    off = torch.tensor([0, 1000, T], dtype=torch.int32, device="cuda")
    op.forward(small, off, y=out.zero_())
    assert torch.equal(out[last], ref) and op.read_status() == SFFN_OK
    dx = op.backward(small, x, off)["dx"]
    within(dx[last], x[last].double() @ W.double(), (x[last].double() @ W.double()).abs() * HALF[BF]
           + (d + 64) * U * (x[last].double().abs() @ W.double().abs()), "dx")

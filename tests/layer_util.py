"""Plain 64-bit forms of the operators around the sparse FFN, and the error
bounds that their tests use.  One rounding to a type is off by at most half a
step, eps(type) / 2 relative to the value: HALF."""
from __future__ import annotations

import torch

GROUP = 128
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
U = 2.0 ** -24            # one fp32 rounding


def gen(seed: int) -> torch.Generator:
    return torch.Generator().manual_seed(seed)


def randn(seed: int, *shape, dtype=torch.float32, scale: float = 1.0):
    return (torch.randn(*shape, generator=gen(seed)) * scale).to(dtype).cuda()


def ints(seed: int, *shape, lim: int = 4, dtype=torch.bfloat16):
    return torch.randint(-lim, lim + 1, shape, generator=gen(seed)).to(dtype).cuda()


def within(got, ref, tol, what: str = "") -> None:
    got, ref, tol = got.double(), ref.double(), tol.double()
    assert got.shape == ref.shape
    assert torch.isfinite(got).all(), f"{what}: not finite"
    over = (got - ref).abs() > tol
    if over.any():
        i = tuple(over.nonzero()[0].tolist())
        raise AssertionError(f"{what}: {int(over.sum())} of {over.numel()} outside, first at {i}: "
                             f"{got[i].item():.9g} against {ref[i].item():.9g}, tolerance {tol[i].item():.3g}")


def groups(d: int) -> int:
    return -(-d // GROUP)


def spread_cols(scale, d: int):
    """A scale per group as one per column."""
    return scale.repeat_interleave(GROUP, 1)[:, :d]


def check_codes(q, scale, v, rel: float, what: str = "") -> None:
    """e4m3 codes and scales against the values v (64 bits) they stand for, each
    v known to the kernel up to a relative error `rel`.

    scale = m / 448 with m the group's amax: relative error rel + 2 U (the
    clamp is exact; a division and a rounding).  code = nearest of c = v·448/m:
    c is off by 2 rel + 3 U relative, so |code - c| <= half the step of c's
    binade (2^-9 below 2^-6) plus that, the saturation at 448 included."""
    T, d = v.shape
    pad = torch.zeros(T, groups(d) * GROUP, dtype=torch.float64, device=v.device)
    pad[:, :d] = v
    m = pad.view(T, -1, GROUP).abs().amax(2).clamp_min(1e-30)
    within(scale, m / 448, (m / 448) * (rel + 2 * U), what + " scale")
    c = v * 448 / spread_cols(m, d)
    e = torch.floor(torch.log2(c.abs().clamp_min(2.0 ** -6)))
    half = torch.exp2(e - 4)
    within(q.float(), c, half + c.abs() * (2 * rel + 3 * U), what + " codes")

"""Timed cases of the layer operators around the sparse FFN: RMS norm, the 8-bit linear and the experts' grouped products.

Three operators, each beside the framework's own of its kind:

* ``RmsNorm``: s = residual + x, y = s / sqrt(mean(s^2) + eps) * weight, with y in bf16, fp32 or as e4m3 codes with an
  fp32 scale for each 128 columns of a row; and its gradient.  It takes the FFN's fp32 output as x and gives the next
  layer's operand.
* ``Fp8Linear``: y = x W^T with both operands in e4m3, x with a scale for each (row, 128 columns), W with one for each
  128 x 128 block.
* ``GroupedLinear``: y[r] = W[e(r)] x[r] for rows sorted by expert with ragged (also empty) groups; dx and dW.

``run`` with ``own`` false is the plain form in elementary torch operations, with ``own`` true the framework's call on
the same state.
"""
import math

import torch

own = False

G = 128          # columns that share a scale, and the side of a weight block that shares one
E4M3_MAX = 448.0
TINY = 1e-30     # least amax of a group: an all-zero group gets codes 0 and a finite scale

_DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # decode step of the 4096-wide layer: the FFN's fp32 output joins the residual and becomes the next linear's
        # 8-bit operand; a few microseconds, so launch and host time count
        {"name": "norm decode to 8 bits", "kind": "norm", "tokens": 8, "d": 4096, "x": "fp32", "residual": "bf16", "out": "fp8"},
        # prefill of the 2048-wide layer: fp32 FFN output, bf16 residual stream and bf16 operand
        {"name": "norm prefill", "kind": "norm", "tokens": 4096, "d": 2048, "x": "fp32", "residual": "bf16", "out": "bf16"},
        # training step of the 4096-wide layer, an odd number of rows, with the gradient that comes down the residual
        {"name": "norm backward", "kind": "norm_bwd", "tokens": 8191, "d": 4096, "s": "bf16", "ds": True},
        # one token through the up projection: every weight is read once for one row
        {"name": "linear 8-bit one token", "kind": "linear", "tokens": 1, "d_in": 4096, "d_out": 14336, "x": "fp8"},
        # a ragged decode batch through the down projection, from bf16 activations (quantised within the call)
        {"name": "linear 8-bit decode bf16 in", "kind": "linear", "tokens": 13, "d_in": 14336, "d_out": 4096, "x": "bf16"},
        # a short prompt chunk of the 2048-wide layer
        {"name": "linear 8-bit chunk", "kind": "linear", "tokens": 333, "d_in": 2048, "d_out": 8192, "x": "fp8"},
        # prefill of the 4096-wide layer
        {"name": "linear 8-bit prefill", "kind": "linear", "tokens": 4096, "d_in": 4096, "d_out": 14336, "x": "fp8"},
        # decode of 8 tokens with the top 2 of 8 experts, in a buffer padded to 24 rows
        {"name": "experts decode", "kind": "grouped", "rows": 16, "pad": 8, "experts": 8, "empty": 1, "d_in": 4096, "d_out": 14336, "out": "bf16"},
        # many small experts, a few rows each
        {"name": "experts many small", "kind": "grouped", "rows": 1000, "pad": 0, "experts": 64, "empty": 3, "d_in": 1024, "d_out": 2048, "out": "bf16"},
        # prefill of 4096 tokens with the top 2 of 8 experts
        {"name": "experts prefill", "kind": "grouped", "rows": 8192, "pad": 0, "experts": 8, "empty": 0, "d_in": 2048, "d_out": 8192, "out": "bf16"},
        # gradients of many small experts, two without any row
        {"name": "experts backward small", "kind": "grouped_bwd", "rows": 1531, "experts": 32, "empty": 2, "d_in": 1024, "d_out": 1024},
        # gradients of the prefill-sized training step
        {"name": "experts backward", "kind": "grouped_bwd", "rows": 8192, "experts": 8, "empty": 0, "d_in": 2048, "d_out": 8192},
    ]


def _spread(rng, lo, hi, step=1):
    """A multiple of step in lo .. hi, even over its logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return int(min(hi, max(lo, round(v / step) * step)))


def draw(rng):
    kind = rng.choice(["norm", "norm_bwd", "linear", "grouped", "grouped_bwd"])
    if kind == "norm":
        return {"kind": kind, "tokens": _spread(rng, 1, 8192), "d": _spread(rng, 256, 8192, 8), "x": rng.choice(["fp32", "bf16"]),
                "residual": rng.choice(["none", "bf16", "fp32"]), "out": rng.choice(["bf16", "fp32", "fp8"])}
    if kind == "norm_bwd":
        return {"kind": kind, "tokens": _spread(rng, 1, 8192), "d": _spread(rng, 256, 8192, 8), "s": rng.choice(["bf16", "fp32"]),
                "ds": rng.random() < 0.5}
    if kind == "linear":
        return {"kind": kind, "tokens": _spread(rng, 1, 4096), "d_in": _spread(rng, 512, 8192, 16), "d_out": _spread(rng, 512, 8192, 8),
                "x": rng.choice(["fp8", "fp8", "bf16"])}
    experts = _spread(rng, 2, 64)
    d_in, d_out = _spread(rng, 512, 4096, 8), _spread(rng, 512, 8192, 8)
    while experts * d_in * d_out > 8 * 4096 * 14336:
        experts //= 2
    c = {"kind": kind, "rows": _spread(rng, 1 if kind == "grouped" else 16, 8192), "experts": experts, "empty": rng.randrange(0, 1 + experts // 4),
         "d_in": d_in, "d_out": d_out}
    while c["rows"] * d_in * d_out > 8192 * 2048 * 8192:
        c["rows"] //= 2
    if kind == "grouped":
        c.update(pad=rng.choice([0, 0, 5, 64]), out="bf16")
    return c


# ------------------------------------------------------------------------------------------------------------ inputs
def _counts(rows, experts, empty):
    """Rows of each used expert: shares that fall off like 1 / (rank + 2), as a router's do, whole numbers that add up."""
    used = max(1, min(experts - empty, rows))
    share = [1.0 / (i + 2) for i in range(used)]
    n = [1 + int((rows - used) * s / sum(share)) for s in share]
    n[0] += rows - sum(n)
    return n + [0] * (experts - used)


def _quant_rows(v):
    """e4m3 codes and scales of v's rows, one scale for each G columns (the last group may be short)."""
    v = v.float()
    at = torch.arange(v.shape[1], device=v.device) // G
    amax = torch.zeros(v.shape[0], int(at[-1]) + 1, device=v.device).scatter_reduce_(1, at.expand(v.shape), v.abs(), "amax")
    amax = amax.clamp_min(TINY)
    q = (v * (E4M3_MAX / amax)[:, at]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return q, amax / E4M3_MAX


def _quant_blocks(w):
    """e4m3 codes and scales of w, one scale for each G x G block."""
    n, k = -(-w.shape[0] // G), -(-w.shape[1] // G)
    full = torch.zeros(n * G, k * G, device=w.device)
    full[: w.shape[0], : w.shape[1]] = w.float()
    b = full.view(n, G, k, G)
    amax = b.abs().amax((1, 3)).clamp_min(TINY)
    q = (b * (E4M3_MAX / amax)[:, None, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return q.view(n * G, k * G)[: w.shape[0], : w.shape[1]].contiguous(), amax / E4M3_MAX


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
    kind = case["kind"]
    st = {"case": dict(case)}
    if kind in ("norm", "norm_bwd"):
        T, d = case["tokens"], case["d"]
        channel = 1 + 15 * (torch.rand(d, generator=g, device="cuda") < 0.01)  # a few strong channels, as hidden states have
        st["weight"] = (1 + 0.2 * rand(d)).bfloat16()
        st["eps"] = 1e-6
        if kind == "norm":
            st["x"] = (rand(T, d) * 0.3).to(_DT[case["x"]])
            st["residual"] = None if case["residual"] == "none" else (rand(T, d) * channel).to(_DT[case["residual"]])
        else:
            st["s"] = (rand(T, d) * channel).to(_DT[case["s"]])
            st["dy"] = (rand(T, d) * 1e-2).bfloat16()
            st["ds"] = (rand(T, d) * 1e-2).to(_DT[case["s"]]) if case["ds"] else None
        if own:
            from activation_sparse_gated_relu_b200 import RmsNorm
            st["op"] = RmsNorm(st["weight"], st["eps"])
    elif kind == "linear":
        T, k, n = case["tokens"], case["d_in"], case["d_out"]
        channel = 1 + 15 * (torch.rand(k, generator=g, device="cuda") < 0.01)
        st["wq"], st["ws"] = _quant_blocks(rand(n, k) * k ** -0.5)
        x = (rand(T, k) * channel).bfloat16()
        if case["x"] == "fp8":
            st["xq"], st["xs"] = _quant_rows(x)
        else:
            st["x"] = x
        if own:
            from activation_sparse_gated_relu_b200 import Fp8Linear
            st["op"] = Fp8Linear(st["wq"], st["ws"])
    else:
        R, E, k, n = case["rows"], case["experts"], case["d_in"], case["d_out"]
        counts = _counts(R, E, case["empty"])
        order = torch.randperm(E, generator=torch.Generator().manual_seed(seed)).tolist()
        counts = [counts[i] for i in order]
        st["ends"] = [sum(counts[:i]) for i in range(E + 1)]  # the plain form's loop bounds, on the host
        st["offsets"] = torch.tensor(st["ends"], dtype=torch.int32, device="cuda")
        st["W"] = (rand(E, n, k) * k ** -0.5).bfloat16()
        rows = R + case.get("pad", 0)
        st["x"] = rand(rows, k).bfloat16()
        if kind == "grouped":
            st["y"] = torch.zeros(rows, n, dtype=_DT[case["out"]], device="cuda")  # rows behind the last group stay as they are
        else:
            st["dy"] = (rand(rows, n) * 1e-2).bfloat16()
        if own:
            from activation_sparse_gated_relu_b200 import GroupedLinear
            st["op"] = GroupedLinear(st["W"])
    return st


# ---------------------------------------------------------------------------------------------------------- one pass
def run(st):
    return _own(st) if own else _plain(st)


def _own(st):
    case, op = st["case"], st["op"]
    kind = case["kind"]
    if kind == "norm" and case["out"] == "fp8":
        q, scale, s = op.forward_fp8(st["x"], st["residual"])
        return {"q": q, "scale": scale, "s": s if st["residual"] is not None else None}
    if kind == "norm":
        y, s = op.forward(st["x"], st["residual"], out=case["out"])
        return {"y": y, "s": s if st["residual"] is not None else None}
    if kind == "norm_bwd":
        return op.backward(st["dy"], st["s"], st["ds"])
    if kind == "linear":
        return op.forward(st["xq"], st["xs"]) if "xq" in st else op.forward(st["x"])
    if kind == "grouped":
        return op.forward(st["x"], st["offsets"], y=st["y"])
    return op.backward(st["x"], st["dy"], st["offsets"])


def _plain(st):
    case = st["case"]
    kind = case["kind"]
    if kind == "norm":
        s = st["x"].float()
        if st["residual"] is not None:
            s = s + st["residual"].float()
        y = s * torch.rsqrt(s.square().mean(1, keepdim=True) + st["eps"]) * st["weight"].float()
        s = s.to(st["residual"].dtype) if st["residual"] is not None else None
        if case["out"] == "fp8":
            q, scale = _quant_rows(y)
            return {"q": q, "scale": scale, "s": s}
        return {"y": y.to(_DT[case["out"]]), "s": s}
    if kind == "norm_bwd":
        s, dy = st["s"].float(), st["dy"].float()
        r = torch.rsqrt(s.square().mean(1, keepdim=True) + st["eps"])
        hat, gy = s * r, dy * st["weight"].float()
        dx = r * (gy - hat * (gy * hat).mean(1, keepdim=True))
        if st["ds"] is not None:
            dx = dx + st["ds"].float()
        return {"dx": dx.to(st["s"].dtype), "dweight": (dy * hat).sum(0)}
    if kind == "linear":
        xq, xs = (st["xq"], st["xs"]) if "xq" in st else _quant_rows(st["x"])
        col = torch.arange(case["d_in"], device=xq.device) // G
        row = torch.arange(case["d_out"], device=xq.device) // G
        x = xq.float() * xs[:, col]
        w = st["wq"].float() * st["ws"][row][:, col]
        return (x @ w.t()).bfloat16()
    ends = st["ends"]
    if kind == "grouped":
        for e in range(case["experts"]):  # ragged groups: one product each
            a, b = ends[e], ends[e + 1]
            if b > a:
                st["y"][a:b] = (st["x"][a:b].float() @ st["W"][e].float().t()).to(st["y"].dtype)
        return st["y"]
    dx = torch.empty_like(st["x"])
    dW = torch.zeros(st["W"].shape, dtype=torch.float32, device=dx.device)
    for e in range(case["experts"]):
        a, b = ends[e], ends[e + 1]
        if b > a:
            dy = st["dy"][a:b].float()
            dx[a:b] = (dy @ st["W"][e].float()).to(dx.dtype)
            dW[e] = dy.t() @ st["x"][a:b].float()
    return {"dx": dx, "dW": dW}


# -------------------------------------------------------------------------------------------------------------- work
def work(case):
    kind = case["kind"]
    size = {"none": 0, "bf16": 2, "fp32": 4, "fp8": 1}
    if kind == "norm":
        T, d = case["tokens"], case["d"]
        scales = 4 * T * -(-d // G) if case["out"] == "fp8" else 0
        return {"bytes": T * d * (size[case["x"]] + 2 * size[case["residual"]] + size[case["out"]]) + scales + 2 * d, "flops": 6 * T * d}
    if kind == "norm_bwd":
        T, d = case["tokens"], case["d"]
        return {"bytes": T * d * (2 + (3 if case["ds"] else 2) * size[case["s"]]) + 6 * d, "flops": 13 * T * d}
    if kind == "linear":
        T, k, n = case["tokens"], case["d_in"], case["d_out"]
        x = T * k * (1 if case["x"] == "fp8" else 2) + (4 * T * -(-k // G) if case["x"] == "fp8" else 0)
        return {"bytes": n * k + 4 * -(-n // G) * -(-k // G) + x + 2 * T * n, "flops": 2 * T * n * k}
    R, E, k, n = case["rows"], case["experts"], case["d_in"], case["d_out"]
    used = max(1, min(E - case["empty"], R))
    if kind == "grouped":
        return {"bytes": 2 * used * n * k + 2 * R * k + size[case["out"]] * R * n, "flops": 2 * R * n * k}
    return {"bytes": 2 * used * n * k + 4 * E * n * k + 2 * R * (2 * k + n), "flops": 4 * R * n * k}


# ------------------------------------------------------------------------------------------------- values in 64 bits
def _e4m3(v):
    """v rounded to the nearest e4m3 value (ties to the even code), by the format's definition: 3 fraction bits, exponents from
    2^-6, 448 the largest."""
    e = torch.frexp(v.abs().clamp_min(2.0 ** -6))[1].double() - 1
    step = torch.exp2(e - 3)
    return (torch.round(v / step) * step).clamp(-448.0, 448.0)


def _exact_codes(v):
    """Codes' values and scales of v [rows][cols] in float64, group by group."""
    q, scale = torch.empty_like(v), []
    for a in range(0, v.shape[1], G):
        m = v[:, a:a + G].abs().max(1, keepdim=True).values.clamp_min(TINY)
        q[:, a:a + G] = _e4m3(v[:, a:a + G] * 448.0 / m)
        scale.append(m / 448.0)
    return q, torch.cat(scale, 1)


def exact(case, seed):
    st = prepare(case, seed)
    kind = case["kind"]
    if kind == "norm":
        s = st["x"].double()
        if st["residual"] is not None:
            s = s + st["residual"].double()
        norm = torch.linalg.vector_norm(s, dim=1, keepdim=True)
        y = s / torch.sqrt(norm ** 2 / case["d"] + st["eps"]) * st["weight"].double()
        s = s if st["residual"] is not None else None
        if case["out"] == "fp8":
            q, scale = _exact_codes(y)
            return {"q": q, "scale": scale, "s": s}
        return {"y": y, "s": s}
    if kind == "norm_bwd":
        # s / rho with rho = sqrt(mean(s^2) + eps): d(s_j / rho) / d s_i = delta_ij / rho - s_i s_j / (d rho^3)
        s, dy, w = st["s"].double(), st["dy"].double(), st["weight"].double()
        rho = torch.sqrt(torch.linalg.vector_norm(s, dim=1) ** 2 / case["d"] + st["eps"])
        along = torch.einsum("td,td,d->t", s, dy, w)
        dx = dy * w / rho[:, None] - s * (along / (case["d"] * rho ** 3))[:, None]
        if st["ds"] is not None:
            dx = dx + st["ds"].double()
        return {"dx": dx, "dweight": torch.einsum("td,td,t->d", dy, s, 1 / rho)}
    if kind == "linear":
        if "xq" in st:
            xq, xs = st["xq"].double(), st["xs"].double()
        else:
            xq, xs = _exact_codes(st["x"].double())
        y = torch.zeros(case["tokens"], case["d_out"], dtype=torch.float64, device="cuda")
        rows = st["ws"].double().repeat_interleave(G, 0)[: case["d_out"]]
        for b, a in enumerate(range(0, case["d_in"], G)):
            y += (xq[:, a:a + G] @ st["wq"][:, a:a + G].double().t()) * xs[:, b:b + 1] * rows[:, b]
        return y
    at = torch.arange(st["x"].shape[0], device="cuda")
    if kind == "grouped":
        y = torch.zeros(st["y"].shape, dtype=torch.float64, device="cuda")
        for e in range(case["experts"]):
            mine = ((at >= st["offsets"][e]) & (at < st["offsets"][e + 1])).nonzero()[:, 0]
            y[mine] = torch.einsum("rk,nk->rn", st["x"][mine].double(), st["W"][e].double())
        return y
    dx = torch.zeros(st["x"].shape, dtype=torch.float64, device="cuda")
    dW = torch.zeros(st["W"].shape, dtype=torch.float64, device="cuda")
    for e in range(case["experts"]):
        mine = ((at >= st["offsets"][e]) & (at < st["offsets"][e + 1])).nonzero()[:, 0]
        dx[mine] = torch.einsum("rn,nk->rk", st["dy"][mine].double(), st["W"][e].double())
        dW[e] = torch.einsum("rn,rk->nk", st["dy"][mine].double(), st["x"][mine].double())
    return {"dx": dx, "dW": dW}

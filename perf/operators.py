"""The feed-forward operators on this framework's 16-bit types, as cases to be measured.

``linear``  Y = act(X W + b) + R, with its gradients, and
``gated``   H = act(X Wg) * (X Wu), with its gradients:

the two halves of a transformer's feed-forward block. Rows are tokens: one to a few dozen while
answers are generated, hundreds to thousands for prompts and training. ``wt`` cases keep the
weights as (outputs x inputs), the other common order.

With ``own`` false every operator is computed in plain float32 torch operations; with ``own``
true through the package's entry points.
"""
from __future__ import annotations

import math

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
_ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh"]
# The most work of one pass, in units of rows * inputs * outputs * products (forward linear: 1,
# its gradients: 2, forward gated: 2, its gradients: 4): that of the largest listed case.
_MOST = 4 * 4096 * 4096 * 4096


def _linear(name, rows, k, n, dtype="bf16", act="none", bias=False, residual=False, save=False,
            wt=False):
    return {"name": name, "op": "linear", "rows": rows, "k": k, "n": n, "dtype": dtype, "act": act,
            "bias": bias, "residual": residual, "save": save, "wt": wt}


def _linear_bwd(name, rows, k, n, dtype="bf16", act="none", bias=False, wt=False):
    return {"name": name, "op": "linear_bwd", "rows": rows, "k": k, "n": n, "dtype": dtype,
            "act": act, "bias": bias, "wt": wt}


def _gated(name, rows, k, n, dtype="bf16", act="silu", save=False, wt=False):
    return {"name": name, "op": "gated", "rows": rows, "k": k, "n": n, "dtype": dtype, "act": act,
            "save": save, "wt": wt}


def _gated_bwd(name, rows, k, n, dtype="bf16", act="silu", wt=False):
    return {"name": name, "op": "gated_bwd", "rows": rows, "k": k, "n": n, "dtype": dtype,
            "act": act, "wt": wt}


def listed():
    return [
        # One token through the first half of a small model's block: a call of a few microseconds.
        _linear("linear 1x1024x4096", 1, 1024, 4096, act="gelu_tanh", bias=True),
        # Eight answers at once through the block's second half, added onto the block's input.
        _linear("linear 8x8192x4096", 8, 8192, 4096, residual=True, wt=True),
        # A prompt whose three sizes are odd (no row starts on a 16-byte boundary).
        _linear("linear 1000x997x1003 f16", 1000, 997, 1003, dtype="f16", act="relu", bias=True,
                residual=True),
        # A batch of prompts; every part of the epilogue at once.
        _linear("linear 2048x2048x2048", 2048, 2048, 2048, act="gelu", bias=True, residual=True),
        # A training step's forward pass, which keeps the pre-activations for the backward pass.
        _linear("linear 4096x4096x4096 save", 4096, 4096, 4096, act="gelu_tanh", bias=True, save=True),
        # Its gradients.
        _linear_bwd("linear bwd 4096x4096x4096", 4096, 4096, 4096, act="gelu_tanh", bias=True),
        # Gradients at odd sizes.
        _linear_bwd("linear bwd 1000x997x1003 f16", 1000, 997, 1003, dtype="f16", act="gelu", bias=True),
        # One token through the gated half of a block.
        _gated("gated 1x4096x8192", 1, 4096, 8192),
        # A few dozen answers at once, weights as (outputs x inputs).
        _gated("gated 48x2048x6144 f16", 48, 2048, 6144, dtype="f16", wt=True),
        # A long prompt: the largest forward pass.
        _gated("gated 4096x4096x8192", 4096, 4096, 8192),
        # Training: the gradients of a gated half, the largest call here.
        _gated_bwd("gated bwd 4096x4096x4096", 4096, 4096, 4096),
        # A short fine-tuning batch whose row count is odd.
        _gated_bwd("gated bwd 333x1024x2800 f16", 333, 1024, 2800, dtype="f16", act="gelu_tanh", wt=True),
    ]


def _products(op):
    return {"linear": 1, "linear_bwd": 2, "gated": 2, "gated_bwd": 4}[op]


def draw(rng):
    op = rng.choice(["linear", "linear_bwd", "gated", "gated_bwd"])
    case = {"op": op, "dtype": rng.choice(["bf16", "f16"])}

    def size(lo, hi):
        v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
        step = rng.choice([64, 64, 8, 1])
        return min(max(v // step * step, lo), hi)

    case["k"], case["n"] = size(256, 8192), size(256, 8192)
    top = min(4096, _MOST // (_products(op) * case["k"] * case["n"]))
    # Training batches are not a handful of rows; what is generated one token at a time is.
    low = 32 if op.endswith("_bwd") else 1
    case["rows"] = max(low, min(top, int(round(math.exp(rng.uniform(math.log(low), math.log(max(top, low + 1))))))))
    case["wt"] = rng.random() < 0.5
    if op.startswith("linear"):
        case["act"] = rng.choice(_ACTS)
        case["bias"] = rng.random() < 0.6
        if op == "linear":
            case["residual"] = rng.random() < 0.5
    else:
        case["act"] = rng.choice(["silu", "silu", "gelu", "gelu_tanh", "relu"])
    if op in ("linear", "gated"):
        case["save"] = case["rows"] >= 128 and rng.random() < 0.4
    return case


def prepare(case, seed):
    """The tensors in a program's hands: normal values as they stand after a norm layer, weights
    of variance 1 / inputs, and for the gradients the pre-activations as the forward pass left
    them, rounded to the case's type."""
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    dtype, m, k, n = _DTYPES[case["dtype"]], case["rows"], case["k"], case["n"]

    def normal(rows, cols, scale=1.0):
        return (torch.randn(rows, cols, generator=gen, device="cuda") * scale).to(dtype)

    def weight():
        return normal(n, k, k ** -0.5).t() if case["wt"] else normal(k, n, k ** -0.5)

    s = {"op": case["op"], "act": case["act"], "x": normal(m, k)}
    if case["op"].startswith("linear"):
        s["w"] = weight()
        bias = normal(1, n, 0.5).view(n) if case["bias"] else None
        if case["op"] == "linear":
            s["bias"] = bias
            s["residual"] = normal(m, n) if case["residual"] else None
            s["save"] = case["save"]
        else:
            s["db"] = case["bias"]
            s["dy"] = normal(m, n)
            z = s["x"].float() @ s["w"].float()
            s["z"] = (z if bias is None else z + bias.float()).to(dtype)
    else:
        s["w_gate"], s["w_up"] = weight(), weight()
        if case["op"] == "gated":
            s["save"] = case["save"]
        else:
            s["dh"] = normal(m, n)
            s["g"] = (s["x"].float() @ s["w_gate"].float()).to(dtype)
            s["u"] = (s["x"].float() @ s["w_up"].float()).to(dtype)
    return s


_C, _A = math.sqrt(2.0 / math.pi), 0.044715


def _act(z, act):
    if act == "relu":
        return torch.where(z < 0, torch.zeros_like(z), z)
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(_C * (z + _A * z * z * z)))
    return z


def _act_grad(z, act):
    if act == "relu":
        return torch.where(z <= 0, torch.zeros_like(z), torch.ones_like(z))
    if act == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s * (1 + z * (1 - s))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        t = torch.tanh(_C * (z + _A * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * _C * (1 + 3 * _A * z * z)
    return torch.ones_like(z)


def _run_own(s):
    import roofline_driven_tiling_gb300 as t2s
    x, act = s["x"], s["act"]
    if s["op"] == "linear":
        if not s["save"]:
            return {"y": t2s.linear(x, s["w"], s["bias"], s["residual"], act=act)}
        z = torch.empty(x.shape[0], s["w"].shape[1], dtype=x.dtype, device=x.device)
        return {"y": t2s.linear(x, s["w"], s["bias"], s["residual"], act=act, preact=z), "z": z}
    if s["op"] == "linear_bwd":
        dx, dw, db = t2s.linear_backward(s["dy"], x, s["w"], s["z"], act=act, db=None if s["db"] else False)
        return {"dx": dx, "dw": dw, "db": db} if s["db"] else {"dx": dx, "dw": dw}
    if s["op"] == "gated":
        if not s["save"]:
            return {"h": t2s.gated_linear(x, s["w_gate"], s["w_up"], act=act)}
        g = torch.empty(x.shape[0], s["w_up"].shape[1], dtype=x.dtype, device=x.device)
        u = torch.empty_like(g)
        return {"h": t2s.gated_linear(x, s["w_gate"], s["w_up"], act=act, preact=(g, u)), "g": g, "u": u}
    dx, dw_gate, dw_up = t2s.gated_linear_backward(s["dh"], x, s["w_gate"], s["w_up"], (s["g"], s["u"]), act=act)
    return {"dx": dx, "dw_gate": dw_gate, "dw_up": dw_up}


def run(state):
    if own:
        return _run_own(state)
    s, act, dtype = state, state["act"], state["x"].dtype
    x = s["x"].float()
    if s["op"] == "linear":
        z = x @ s["w"].float()
        if s["bias"] is not None:
            z = z + s["bias"].float()
        y = _act(z, act)
        if s["residual"] is not None:
            y = y + s["residual"].float()
        return {"y": y.to(dtype), "z": z.to(dtype)} if s["save"] else {"y": y.to(dtype)}
    if s["op"] == "linear_bwd":
        dz = s["dy"].float() * _act_grad(s["z"].float(), act)
        out = {"dx": (dz @ s["w"].float().t()).to(dtype), "dw": (x.t() @ dz).to(dtype)}
        if s["db"]:
            out["db"] = dz.sum(0).to(dtype)
        return out
    if s["op"] == "gated":
        g, u = x @ s["w_gate"].float(), x @ s["w_up"].float()
        h = (_act(g, act) * u).to(dtype)
        return {"h": h, "g": g.to(dtype), "u": u.to(dtype)} if s["save"] else {"h": h}
    dh, g, u = s["dh"].float(), s["g"].float(), s["u"].float()
    dg, du = dh * u * _act_grad(g, act), dh * _act(g, act)
    return {"dx": (dg @ s["w_gate"].float().t() + du @ s["w_up"].float().t()).to(dtype),
            "dw_gate": (x.t() @ dg).to(dtype), "dw_up": (x.t() @ du).to(dtype)}


def work(case):
    m, k, n = case["rows"], case["k"], case["n"]
    flops = 2 * m * n * k * _products(case["op"])
    if case["op"] == "linear":
        values = m * k + k * n + m * n * (1 + case["residual"] + case["save"]) + n * case["bias"]
    elif case["op"] == "linear_bwd":
        values = m * n * (1 if case["act"] == "none" else 2) + 2 * m * k + 2 * k * n + n * case["bias"]
    elif case["op"] == "gated":
        values = m * k + 2 * k * n + m * n * (3 if case["save"] else 1)
    else:
        values = 3 * m * n + 2 * m * k + 4 * k * n
    return {"bytes": 2 * values, "flops": flops}


def _value_and_slope(z, act):
    """act(z) and act'(z) in float64 from their definitions: relu max(z, 0), silu z s(z) with the
    logistic s, gelu z P(z) with the normal distribution P, gelu_tanh z s(2 c (z + a z^3))."""
    if act == "none":
        return z, torch.ones_like(z)
    if act == "relu":
        return z.clamp(min=0), (z > 0).double()
    if act == "silu":
        s = torch.sigmoid(z)
        return z * s, s + z * s * torch.sigmoid(-z)
    if act == "gelu":
        p = torch.special.ndtr(z)
        return z * p, p + z * torch.exp(-z.square() / 2) * (2 * math.pi) ** -0.5
    v = 2 * _C * (z + _A * z ** 3)
    s = torch.sigmoid(v)
    return z * s, s + z * s * torch.sigmoid(-v) * 2 * _C * (1 + 3 * _A * z.square())


def exact(case, seed):
    """run()'s outputs from the definitions in float64."""
    s = prepare(case, seed)
    d = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor)}
    if s["op"] == "linear":
        z = torch.matmul(d["x"], d["w"])
        z += d["bias"] if "bias" in d else 0.0
        y = _value_and_slope(z, s["act"])[0] + (d["residual"] if "residual" in d else 0.0)
        return {"y": y, "z": z} if s["save"] else {"y": y}
    if s["op"] == "linear_bwd":
        dz = _value_and_slope(d["z"], s["act"])[1].mul(d["dy"])
        out = {"dx": torch.einsum("mn,kn->mk", dz, d["w"]), "dw": torch.einsum("mk,mn->kn", d["x"], dz)}
        return dict(out, db=torch.einsum("mn->n", dz)) if s["db"] else out
    if s["op"] == "gated":
        g, u = torch.matmul(d["x"], d["w_gate"]), torch.matmul(d["x"], d["w_up"])
        h = _value_and_slope(g, s["act"])[0].mul(u)
        return {"h": h, "g": g, "u": u} if s["save"] else {"h": h}
    value, slope = _value_and_slope(d["g"], s["act"])
    dg, du = slope.mul(d["u"]).mul(d["dh"]), value.mul(d["dh"])
    dx = torch.einsum("mn,kn->mk", dg, d["w_gate"])
    dx += torch.einsum("mn,kn->mk", du, d["w_up"])
    return {"dx": dx, "dw_gate": torch.einsum("mk,mn->kn", d["x"], dg),
            "dw_up": torch.einsum("mk,mn->kn", d["x"], du)}

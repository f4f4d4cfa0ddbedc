"""The operators around a feed-forward block's products, as cases to be measured.

``fp8``       C = A B of 8-bit floating-point operands with a float32 scale for each block of 128
              values of the sum (of each row, or of 128 rows),
``quantize``  the 8-bit operands and their scales from 16-bit tensors, along rows, columns or both,
``norm``      r = scale * x + gate * dropout(post_norm(h)),  y = norm(r): what stands between two
              blocks of a transformer, and
``norm_bwd``  its gradients,
``dropout``   dropout from a counter-based generator, whose mask is never stored.

Rows are tokens: one to a few dozen while answers are generated, hundreds to thousands for
prompts and training.

With ``own`` false every operator is computed in plain torch operations; with ``own`` true
through the package's entry points.
"""
from __future__ import annotations

import math

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
_EPS = 1e-6
# The most work of one product: rows * inputs * outputs of the largest listed case.
_MOST = 4096 * 4096 * 4096
# The most values of one call of the other operators.
_MOST_VALUES = 16384 * 4096


def _fp8(name, m, k, n, out="bf16", square=True, a="e4m3", b="e4m3"):
    return {"name": name, "op": "fp8", "m": m, "k": k, "n": n, "out": out, "square": square, "a": a, "b": b}


def _quantize(name, rows, cols, dtype="bf16", f8="e4m3", along="rows", square=False):
    return {"name": name, "op": "quantize", "rows": rows, "cols": cols, "dtype": dtype, "f8": f8, "along": along,
            "square": square}


def _norm(name, rows, cols, op="norm", dtype="bf16", norm="rms", bias=False, h=True, post="none", gates=1, scale=1.0,
          p=0.0):
    return {"name": name, "op": op, "rows": rows, "cols": cols, "dtype": dtype, "norm": norm, "bias": bias, "h": h,
            "post": post, "gates": gates, "scale": scale, "p": p}


def _dropout(name, rows, cols, dtype="bf16", p=0.1, residual=False):
    return {"name": name, "op": "dropout", "rows": rows, "cols": cols, "dtype": dtype, "p": p, "residual": residual}


def listed():
    return [
        # One token through a block's first half, weights in 8 bits with a scale for each 128 x 128.
        _fp8("fp8 1x4096x8192", 1, 4096, 8192),
        # A prompt whose three sizes are odd.
        _fp8("fp8 1000x997x1003 f16", 1000, 997, 1003, out="f16"),
        # A batch of prompts.
        _fp8("fp8 4096x4096x4096", 4096, 4096, 4096),
        # A weight's gradient summed over 8192 tokens: every row of both operands has scales of its
        # own, the outputs' gradients have the wider exponent, and the result is for a float32 weight.
        _fp8("fp8 grad 4096x8192x2048", 4096, 8192, 2048, out="f32", square=False, b="e5m2"),
        # A short batch's activations before a product.
        _quantize("quantize 333x2800 f16", 333, 2800, dtype="f16"),
        # Gradients of a training step's activations: along rows for the inputs' gradient, along
        # columns for the weight's.
        _quantize("quantize 4096x8192 both", 4096, 8192, f8="e5m2", along="both"),
        # One token between two blocks.
        _norm("norm 1x4096", 1, 4096),
        # Prompts between two blocks, with a norm after the block too and a gate for every channel.
        _norm("norm 8192x4096 post", 8192, 4096, post="rms", scale=0.5),
        # A training step's gradients, with dropout.
        _norm("norm bwd 8192x2048", 8192, 2048, op="norm_bwd", p=0.1),
        # Gradients at odd sizes: layer norms before and after, gates of each of four samples.
        _norm("norm bwd 1300x1003 f16", 1300, 1003, op="norm_bwd", dtype="f16", norm="layer", bias=True, post="layer",
              gates=4, p=0.25),
        # A small batch's activations at odd sizes, added onto the residual stream.
        _dropout("dropout 777x1003 f16", 777, 1003, dtype="f16", residual=True),
        # A long training batch's activations.
        _dropout("dropout 16384x4096", 16384, 4096),
    ]


def draw(rng):
    op = rng.choice(["fp8", "fp8", "quantize", "norm", "norm_bwd", "dropout"])

    def size(lo, hi):
        v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
        step = rng.choice([64, 64, 8, 1])
        return min(max(v // step * step, lo), hi)

    def rows(low, top):
        return max(low, min(top, int(round(math.exp(rng.uniform(math.log(low), math.log(max(top, low + 1))))))))

    if op == "fp8":
        k, n = size(128, 8192), size(128, 8192)
        if rng.random() < 0.3:  # a weight's gradient
            return {"op": op, "m": rows(128, min(8192, _MOST // (k * n))), "k": k, "n": n, "square": False,
                    "out": rng.choice(["bf16", "f16", "f32"]), "a": "e4m3", "b": "e5m2"}
        return {"op": op, "m": rows(1, min(8192, _MOST // (k * n))), "k": k, "n": n, "square": True,
                "out": rng.choice(["bf16", "f16"]), "a": rng.choice(["e4m3", "e4m3", "e5m2"]), "b": "e4m3"}
    case = {"op": op, "dtype": rng.choice(["bf16", "f16"])}
    case["cols"] = size(64, 8192)
    top = min(16384, _MOST_VALUES // case["cols"])
    if op == "quantize":
        case["along"] = rng.choice(["rows", "columns", "both"])
        case["rows"] = rows(1, top // 2)
        case["f8"], case["square"] = rng.choice(["e4m3", "e5m2"]), rng.random() < 0.3
    elif op == "dropout":
        case["rows"], case["p"], case["residual"] = rows(1, top), rng.choice([0.05, 0.1, 0.3, 0.5]), rng.random() < 0.5
    else:
        low = 32 if op == "norm_bwd" else 1
        case["rows"] = rows(low, top // 2)
        case["norm"], case["bias"] = rng.choice(["rms", "layer"]), rng.random() < 0.4
        case["h"] = rng.random() < 0.85
        case["post"] = rng.choice(["none", "rms", "layer"]) if case["h"] else "none"
        case["gates"] = rng.choice([0, 1, 1, 4]) if case["h"] else 0
        if case["gates"] == 4:
            case["rows"] = max(4, case["rows"] // 4 * 4)
        case["scale"] = rng.choice([1.0, 0.5]) if case["h"] else 1.0
        case["p"] = rng.choice([0.0, 0.1]) if case["h"] else 0.0
    return case


def _blocks(n):
    return -(-n // 128)


def _scales(amax, f8):
    """The power of two that takes the largest magnitude of a block just under the type's largest value."""
    mantissa, exponent = torch.frexp(amax)  # 448 = 0.875 * 2^9, 57344 = 0.875 * 2^16
    exponent = exponent - (9 if f8 == torch.float8_e4m3fn else 16) + (mantissa > 0.875).int()
    return torch.where(amax == 0, torch.full_like(amax, 2.0 ** -126),
                       torch.ldexp(torch.ones_like(amax), exponent).clamp(min=2.0 ** -126))


def _quantized(x, f8, square):
    """x's values in 8 bits and the scales of blocks of 128 of each row, or of 128 x 128."""
    m, k = x.shape
    kb, mb = _blocks(k), _blocks(m)
    wide = torch.zeros(mb * 128 if square else m, kb * 128, device=x.device)
    wide[:m, :k] = x.float()
    if square:
        scale = _scales(wide.view(mb, 128, kb, 128).abs().amax((1, 3)), f8)
        full = scale.repeat_interleave(128, 0).repeat_interleave(128, 1)
    else:
        scale = _scales(wide.view(m, kb, 128).abs().amax(2), f8)
        full = scale.repeat_interleave(128, 1)
    most = 448.0 if f8 == torch.float8_e4m3fn else 57344.0
    return (wide / full)[:m, :k].clamp(-most, most).to(f8), scale


def prepare(case, seed):
    """The tensors in a program's hands: normal values as they stand after a norm layer with a few
    large channels, weights of variance 1 / inputs, and 8-bit operands as they are kept."""
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    op = case["op"]

    def normal(rows, cols, scale=1.0):
        return torch.randn(rows, cols, generator=gen, device="cuda") * scale

    def channels(rows, cols):
        return normal(rows, cols) * torch.exp(0.5 * normal(1, cols))

    if op == "fp8":
        m, k, n = case["m"], case["k"], case["n"]

        def operand(rows, f8, square, scale):
            q, s = _quantized(channels(rows, k) * scale, f8, square)
            kept = torch.zeros(rows, -(-k // 16) * 16, dtype=torch.uint8, device="cuda")
            kept[:, :k] = q.view(torch.uint8)  # rows that start on 16-byte boundaries
            return kept.view(f8)[:, :k], s if square else s.t().contiguous().t()

        a, sa = operand(m, _F8[case["a"]], False, 1.0)
        b, sb = operand(n, _F8[case["b"]], case["square"], k ** -0.5)
        return {"op": op, "a": a, "sa": sa, "b": b.t(), "sb": sb.t(), "out": _DTYPES[case["out"]]}
    rows, cols, dtype = case["rows"], case["cols"], _DTYPES[case["dtype"]]
    if op == "quantize":
        return {"op": op, "x": channels(rows, cols).to(dtype), "f8": _F8[case["f8"]], "along": case["along"],
                "square": case["square"]}
    if op == "dropout":
        return {"op": op, "x": normal(rows, cols).to(dtype), "p": case["p"], "seed": int(seed), "sequence": 3,
                "residual": normal(rows, cols).to(dtype) if case["residual"] else None}

    def vector(mean, scale):
        return (mean + normal(1, cols, scale)).view(cols).to(dtype)

    s = {"op": op, "norm": case["norm"], "scale": case["scale"], "post": case["post"], "p": case["p"],
         "seed": int(seed), "sequence": 3, "x": channels(rows, cols).to(dtype), "weight": vector(1.0, 0.2)}
    s["h"] = channels(rows, cols).to(dtype) if case["h"] else None
    s["bias"] = vector(0.0, 0.2) if case["bias"] else None
    s["post_weight"] = vector(1.0, 0.2) if case["post"] != "none" else None
    s["post_bias"] = vector(0.0, 0.2) if case["post"] != "none" and case["bias"] else None
    gates = case["gates"]
    s["gate"] = None if not gates else vector(0.5, 0.2) if gates == 1 else normal(gates, cols, 0.5).to(dtype)
    if op == "norm_bwd":
        s["dy"], s["dr"] = normal(rows, cols).to(dtype), normal(rows, cols).to(dtype)
        s["r"] = _stream(s).to(dtype)  # what the forward pass left
        del s["x"]
    return s


_GAMMA, _M1, _M2 = (v - 2 ** 64 for v in (0x9E3779B97F4A7C15, 0xBF58476D1CE4E5B9, 0x94D049BB133111EB))


def _mix(z):
    """The output function of SplitMix64 on int64 tensors (products modulo 2^64, logical shifts)."""
    z = (z ^ ((z >> 30) & (2 ** 34 - 1))) * _M1
    z = (z ^ ((z >> 27) & (2 ** 37 - 1))) * _M2
    return z ^ ((z >> 31) & (2 ** 33 - 1))


def _keep(rows, cols, p, seed, sequence, device):
    """Where dropout keeps a value, and the factor of the values that stay: 16 bits a value, four
    values to one output of the generator, each row from an output of its own on."""
    least = int(p * 65536 + 0.5)
    groups = -(-cols // 4)
    start = (seed + (sequence + 1) * _GAMMA + 2 ** 63) % 2 ** 64 - 2 ** 63  # as a signed number
    key = _mix(torch.full((), start, dtype=torch.int64, device=device))
    z = _mix(key + (torch.arange(rows * groups, device=device) + 1) * _GAMMA)
    parts = torch.stack([(z >> 16 * j) & 0xffff for j in range(4)], 1).view(rows, 4 * groups)
    return parts[:, :cols] >= least, 65536.0 / (65536 - least) if least < 65536 else 0.0


def _normed(x, kind):
    """(x - mean) / deviation of every row ("layer"), x / root mean square ("rms"), and 1 / the latter."""
    if kind == "layer":
        x = x - x.mean(1, keepdim=True)
    inverse = 1 / torch.sqrt(x.square().mean(1, keepdim=True) + _EPS)
    return x * inverse, inverse


def _per_row(gate, rows):
    return gate if gate.dim() == 1 else gate.repeat_interleave(rows // gate.shape[0], 0)


def _branch(s):
    """What the block's output adds to the residual stream before its gate, and where it was kept."""
    h = s["h"].float()
    n = h if s["post"] == "none" else _normed(h, s["post"])[0] * s["post_weight"].float()
    if s["post_bias"] is not None:
        n = n + s["post_bias"].float()
    if s["p"] == 0:
        return n, None, 1.0
    keep, factor = _keep(*n.shape, s["p"], s["seed"], s["sequence"], n.device)
    return torch.where(keep, n * factor, torch.zeros_like(n)), keep, factor


def _stream(s):
    if s["h"] is None:
        return s["x"].float()
    n = _branch(s)[0]
    if s["gate"] is not None:
        n = n * _per_row(s["gate"].float(), n.shape[0])
    return s["scale"] * s["x"].float() + n


def _norm_gradient(g, xh, inverse, kind):
    g_xh = (g * xh).mean(1, keepdim=True)
    if kind == "layer":
        g = g - g.mean(1, keepdim=True)
    return inverse * (g - xh * g_xh)


def _run_norm_bwd(s):
    dtype, dy, out = s["r"].dtype, s["dy"].float(), {}
    xh, inverse = _normed(s["r"].float(), s["norm"])
    out["dweight"] = (dy * xh).sum(0)
    if s["bias"] is not None:
        out["dbias"] = dy.sum(0)
    d = s["dr"].float() + _norm_gradient(dy * s["weight"].float(), xh, inverse, s["norm"])
    out["dx"] = s["scale"] * d
    if s["h"] is not None:
        n, keep, factor = _branch(s)
        if s["gate"] is not None:
            dn, gate = d * n, s["gate"].float()
            out["dgate"] = dn.sum(0) if gate.dim() == 1 else dn.view(gate.shape[0], -1, dn.shape[1]).sum(1)
            d = d * _per_row(gate, d.shape[0])
        if keep is not None:
            d = torch.where(keep, d * factor, torch.zeros_like(d))
        if s["post"] != "none":
            hh, inverse = _normed(s["h"].float(), s["post"])
            out["dpost_weight"] = (d * hh).sum(0)
            if s["post_bias"] is not None:
                out["dpost_bias"] = d.sum(0)
            d = _norm_gradient(d * s["post_weight"].float(), hh, inverse, s["post"])
        out["dh"] = d
    return {k: v.to(dtype) for k, v in out.items()}


def _run_own(s):
    import roofline_driven_tiling_gb300 as t2s
    op = s["op"]
    if op == "fp8":
        return {"c": t2s.gemm_fp8(s["a"], s["sa"], s["b"], s["sb"], dtype=s["out"])}
    if op == "quantize":
        got = t2s.quantize_fp8(s["x"], dtype=s["f8"], along=s["along"], square=s["square"])
        return dict(zip(["q", "scale", "qt", "scale_t"], got))
    if op == "dropout":
        return {"y": t2s.dropout(s["x"], s["p"], s["seed"], s["sequence"], residual=s["residual"])}
    how = {k: s[k] for k in ("norm", "scale", "gate", "post_weight", "post_bias", "p", "seed", "sequence")}
    how["post_norm"], how["eps"] = s["post"], _EPS
    if op == "norm":
        r, y = t2s.residual_norm(s["x"], s["h"], s["weight"], s["bias"], **how)
        return {"r": r, "y": y} if s["h"] is not None else {"y": y}
    g = t2s.residual_norm_backward(s["dy"], s["dr"], s["r"], s["h"], s["weight"], s["bias"], **how)
    return {k: v for k, v in g._asdict().items() if v is not None}


def run(state):
    if own:
        return _run_own(state)
    s, op = state, state["op"]
    if op == "fp8":
        def values(q, scale):
            full = scale.repeat_interleave(128, 1)[:, :q.shape[1]]
            if scale.shape[0] != q.shape[0]:
                full = full.repeat_interleave(128, 0)[:q.shape[0]]
            return q.float() * full
        return {"c": (values(s["a"], s["sa"]) @ values(s["b"].t(), s["sb"].t()).t()).to(s["out"])}
    if op == "quantize":
        out = {}
        if s["along"] != "columns":
            out["q"], out["scale"] = _quantized(s["x"], s["f8"], s["square"])
        if s["along"] != "rows":
            out["qt"], out["scale_t"] = _quantized(s["x"].t(), s["f8"], s["square"])
        # The first two results are what the call was asked for.
        return out if s["along"] != "columns" else {"q": out["qt"], "scale": out["scale_t"]}
    dtype = s["r"].dtype if op == "norm_bwd" else s["x"].dtype
    if op == "dropout":
        x = s["x"].float()
        keep, factor = _keep(*x.shape, s["p"], s["seed"], s["sequence"], x.device)
        y = torch.where(keep, x * factor, torch.zeros_like(x))
        return {"y": (y if s["residual"] is None else y + s["residual"].float()).to(dtype)}
    if op == "norm_bwd":
        return _run_norm_bwd(s)
    r = _stream(s).to(dtype)
    y = _normed(r.float(), s["norm"])[0] * s["weight"].float()
    y = (y if s["bias"] is None else y + s["bias"].float()).to(dtype)
    return {"r": r, "y": y} if s["h"] is not None else {"y": y}


def work(case):
    op = case["op"]
    if op == "fp8":
        m, k, n = case["m"], case["k"], case["n"]
        scales = 4 * _blocks(k) * (m + (_blocks(n) if case["square"] else n))
        return {"bytes": (m + n) * k + scales + m * n * (4 if case["out"] == "f32" else 2), "flops": 2 * m * n * k}
    rows, cols = case["rows"], case["cols"]
    values = rows * cols
    if op == "quantize":
        return {"bytes": values * (4 if case["along"] == "both" else 3), "flops": 3 * values}
    if op == "dropout":
        return {"bytes": 2 * values * (3 if case["residual"] else 2), "flops": 2 * values}
    if op == "norm":
        return {"bytes": 2 * values * (4 if case["h"] else 2), "flops": 6 * values}
    return {"bytes": 2 * values * (6 if case["h"] else 4), "flops": 12 * values}


def _exact_keep(rows, cols, case, seed):
    """The factor of every value (0 where it is dropped), the generator's outputs in Python's whole numbers'
    halves: 32-bit parts of 64-bit products, so that nothing wraps."""
    low = 2 ** 32 - 1
    dev = "cuda"

    def times(z, c):  # (high, low) halves times a constant, modulo 2^64
        zh, zl = z
        ch, cl = c >> 32, c & low
        a, b = cl >> 16, cl & 0xffff
        # zl * cl in 16-bit steps of the constant: each product is below 2^48.
        first, second = zl * b, zl * a
        total = first + ((second & 0xffff) << 16)
        carry = (second >> 16) + (total >> 32)
        mixed = ((zh * a & 0xffff) << 16) + zh * b + ((zl * (ch >> 16) & 0xffff) << 16) + zl * (ch & 0xffff)
        return (carry + mixed) & low, total & low

    def shifted(z, n):  # z ^ (z >> n), 0 < n < 32
        return z[0] ^ (z[0] >> n), z[1] ^ ((z[1] >> n) | ((z[0] << (32 - n)) & low))

    def plus(z, c):
        t = z[1] + (c & low)
        return (z[0] + (c >> 32) + (t >> 32)) & low, t & low

    def mix(z):
        return shifted(times(shifted(times(shifted(z, 30), 0xBF58476D1CE4E5B9), 27), 0x94D049BB133111EB), 31)

    gamma, groups = 0x9E3779B97F4A7C15, (cols + 3) // 4
    start = (int(seed) + 4 * gamma) % 2 ** 64  # sequence 3
    kh, kl = mix((torch.full((), start >> 32, device=dev), torch.full((), start & low, device=dev)))
    at = torch.arange(1, rows * groups + 1, device=dev)
    z = mix(plus(times((at >> 32, at & low), gamma), int(kh) << 32 | int(kl)))
    parts = torch.stack([z[1] & 0xffff, z[1] >> 16, z[0] & 0xffff, z[0] >> 16], -1).reshape(rows, -1)[:, :cols]
    least = math.floor(case["p"] * 65536 + 0.5)
    return torch.where(parts < least, 0.0, 65536.0 / max(65536 - least, 1)).double()


def _exact_statistics(v, kind):
    """The deviations from the rows' mean (0 for "rms") and 1 / their root mean square, in float64."""
    mu = torch.einsum("ij->i", v)[:, None] / v.shape[1] if kind == "layer" else 0.0
    c = v - mu
    return c, torch.rsqrt(torch.einsum("ij,ij->i", c, c)[:, None] / v.shape[1] + _EPS)


def _exact_parts(s, case, seed, d):
    """Factor of dropout, the post norm's value, deviations and scale, and the gate of every row."""
    h = d["h"]
    rows, cols = h.shape
    factor = _exact_keep(rows, cols, case, seed) if case["p"] else torch.ones_like(h)
    c, inv = (h, None) if case["post"] == "none" else _exact_statistics(h, case["post"])
    n = c if inv is None else torch.addcmul(d.get("post_bias", torch.zeros(cols, device=h.device).double()),
                                            c * inv, d["post_weight"])
    gate = d.get("gate", torch.ones(cols, device=h.device).double()).reshape(-1, 1, cols)
    return factor, n, c, inv, gate.expand(-1, rows // gate.shape[0], -1).reshape(-1, cols)


def exact(case, seed):
    """run()'s outputs from the definitions in float64."""
    s = prepare(case, seed)
    op, d = s["op"], {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor)}
    if op == "fp8":
        m, n, k = d["a"].shape[0], d["b"].shape[1], d["a"].shape[1]
        c = torch.zeros(m, n, dtype=torch.float64, device="cuda")
        for i in range(_blocks(k)):
            at = slice(128 * i, min(128 * i + 128, k))
            sb = d["sb"][i] if d["sb"].shape[1] == n else d["sb"][i].repeat_interleave(128)[:n]
            c += torch.einsum("mk,kn->mn", d["a"][:, at] * d["sa"][:, i:i + 1], d["b"][at] * sb)
        return {"c": c}
    if op == "quantize":
        most, power = (448.0, 8) if s["f8"] == torch.float8_e4m3fn else (57344.0, 15)

        def quantized(x):
            q, scales = torch.zeros_like(x), []
            for j in range(0, x.shape[1], 128):
                part = x[:, j:j + 128].abs().amax(1)
                if s["square"]:
                    part = torch.stack([p.max() for p in part.split(128)])
                # The least power of two with amax / scale <= the largest value.
                e = torch.log2(part / 1.75).sub(power).ceil()
                e = torch.where(part > most * torch.exp2(e), e + 1, e)
                e = torch.where(part <= most * torch.exp2(e - 1), e - 1, e).clamp(min=-126)
                scales.append(torch.exp2(e))
                full = scales[-1].repeat_interleave(128)[:x.shape[0]] if s["square"] else scales[-1]
                q[:, j:j + 128] = x[:, j:j + 128] / full[:, None]
            # To the nearest of the type's values, ties to even: three or two fraction bits, and a
            # fixed step below the smallest normal number.
            bits, least = (3, -6) if s["f8"] == torch.float8_e4m3fn else (2, -14)
            step = torch.exp2(torch.frexp(q)[1].double().sub(1).clamp(min=least) - bits)
            return torch.round(q / step) * step, torch.stack(scales, 1)

        got = []
        if s["along"] != "columns":
            got += quantized(d["x"])
        if s["along"] != "rows":
            got += quantized(d["x"].t().contiguous())
        return dict(zip(["q", "scale", "qt", "scale_t"], got))
    if op == "dropout":
        y = d["x"] * _exact_keep(*d["x"].shape, case, seed)
        return {"y": y + d["residual"] if "residual" in d else y}
    if op == "norm":
        r = d["x"]
        if "h" in d:
            factor, n, _, _, gate = _exact_parts(s, case, seed, d)
            r = torch.addcmul(r * case["scale"], factor * n, gate)
        kept = r.to(s["x"].dtype).double()
        c, inv = _exact_statistics(kept, case["norm"])
        y = c * inv * d["weight"] + d.get("bias", 0.0)
        return {"r": r, "y": y} if "h" in d else {"y": y}
    out, cols = {}, d["r"].shape[1]
    c, inv = _exact_statistics(d["r"], case["norm"])
    out["dweight"] = torch.einsum("ij,ij,ik->j", d["dy"], c, inv)
    if "bias" in d:
        out["dbias"] = torch.einsum("ij->j", d["dy"])

    def through(g, c, inv, kind):  # the gradient of c * inv with respect to the row
        g = g - (torch.einsum("ij->i", g)[:, None] / cols if kind == "layer" else 0.0)
        return inv * g - inv ** 3 * c * (torch.einsum("ij,ij->i", g, c)[:, None] / cols)

    total = d["dr"] + through(d["dy"] * d["weight"], c, inv, case["norm"])
    out["dx"] = total * case["scale"]
    if "h" in d:
        factor, n, c, inv, gate = _exact_parts(s, case, seed, d)
        if "gate" in d:
            shape = (d["gate"].shape[0] if d["gate"].dim() == 2 else 1, -1, cols)
            out["dgate"] = torch.einsum("gij,gij->gj", total.view(shape), (factor * n).view(shape)).view(d["gate"].shape)
        g = total * gate * factor
        if inv is not None:
            out["dpost_weight"] = torch.einsum("ij,ij,ik->j", g, c, inv)
            if "post_bias" in d:
                out["dpost_bias"] = torch.einsum("ij->j", g)
            g = through(g * d["post_weight"], c, inv, case["post"])
        out["dh"] = g
    return out

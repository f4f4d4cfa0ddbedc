"""residual_norm, its gradients and dropout's mask from their definitions in float64, with bounds on FP32 arithmetic."""
from __future__ import annotations

import numpy as np
import torch

from roofline_driven_tiling_gb300 import inputs

GAMMA = 0x9E3779B97F4A7C15


def factors(rows, cols, p, seed, sequence):
    """0 where a value is dropped, else 1 / the probability of staying (float64, CPU): 16 bits of SplitMix64
    output row * ceil(cols / 4) + col / 4 of the key, which is output `sequence` of the seed."""
    dropped, groups = int(p * 65536 + 0.5), -(-cols // 4)
    key = int(inputs.splitmix64(seed % 2 ** 64, 1, start=sequence % 2 ** 64)[0]) if sequence % 2 ** 64 < 2 ** 62 else None
    if key is None:  # beyond the generator's counter: its definition in Python's integers
        key = mix((seed + (sequence + 1) * GAMMA) % 2 ** 64)
    u = inputs.splitmix64(key, rows * groups)
    parts = np.stack([(u >> np.uint64(16 * j)) & np.uint64(0xffff) for j in range(4)], 1).reshape(rows, 4 * groups)[:, :cols]
    stays = 65536.0 / (65536 - dropped) if dropped < 65536 else 0.0
    return torch.from_numpy(np.where(parts < dropped, 0.0, stays))


def mix(z):
    z = (z ^ (z >> 30)) * 0xBF58476D1CE4E5B9 % 2 ** 64
    z = (z ^ (z >> 27)) * 0x94D049BB133111EB % 2 ** 64
    return z ^ (z >> 31)


def normed(x, kind, eps):
    """Deviations over their scale, and 1 / the scale."""
    if kind == "none":
        return x, torch.ones(x.shape[0], 1, dtype=x.dtype, device=x.device)
    c = x - x.mean(1, keepdim=True) if kind == "layer" else x
    inv = 1 / torch.sqrt(c.square().mean(1, keepdim=True) + eps)
    return c * inv, inv


def per_row(gate, rows):
    if gate is None:
        return 1.0
    return gate if gate.dim() == 1 else gate.repeat_interleave(rows // gate.shape[0], 0)


class Case:
    """Parameters in float64; absent ones None. `keep`: factors() or None."""

    def __init__(self, norm="rms", post_norm="none", eps=1e-6, scale=1.0, keep=None, **tensors):
        self.norm, self.post, self.eps, self.scale, self.keep = norm, post_norm, eps, scale, keep
        for name in ("weight", "bias", "gate", "post_weight", "post_bias"):
            t = tensors.pop(name, None)
            setattr(self, name, None if t is None else t.double())
        assert not tensors

    def branch(self, h):
        n = normed(h, self.post, self.eps)[0]
        if self.post_weight is not None:
            n = n * self.post_weight
        if self.post_bias is not None:
            n = n + self.post_bias
        return n if self.keep is None else n * self.keep

    def stream(self, x, h):
        return self.scale * x + per_row(self.gate, x.shape[0]) * self.branch(h)

    def y(self, r):
        y = normed(r, self.norm, self.eps)[0]
        if self.weight is not None:
            y = y * self.weight
        return y if self.bias is None else y + self.bias

    def gradients(self, dy, dr, r, h):
        """All seven by their formulas, as a dict, with the sums' terms' magnitudes under "|name|"."""
        out, rows = {}, r.shape[0]

        def through(g, v, kind):
            vh, inv = normed(v, kind, self.eps)
            mean = g.mean(1, keepdim=True) if kind == "layer" else 0.0
            return g if kind == "none" else inv * (g - mean - vh * (g * vh).mean(1, keepdim=True))

        def total(name, terms, groups=1):
            out[name] = terms.view(groups, -1, terms.shape[1]).sum(1)
            out["|%s|" % name] = terms.abs().view(groups, -1, terms.shape[1]).sum(1)

        d = torch.zeros_like(r) if dr is None else dr
        if dy is not None:
            xh = normed(r, self.norm, self.eps)[0]
            total("dweight", dy * xh)
            total("dbias", dy)
            d = d + through(dy if self.weight is None else dy * self.weight, r, self.norm)
        out["d"], out["dx"] = d, self.scale * d
        if h is None:
            return out
        total("dgate", d * self.branch(h), 1 if self.gate is None or self.gate.dim() == 1 else self.gate.shape[0])
        dn = d * per_row(self.gate, rows)
        dn = dn if self.keep is None else dn * self.keep
        if self.post != "none":
            total("dpost_weight", dn * normed(h, self.post, self.eps)[0])
            total("dpost_bias", dn)
        out["dn"] = dn
        out["dh"] = through(dn if self.post_weight is None else dn * self.post_weight, h, self.post)
        return out


# Bounds. A sum of n values in any of the kernels' orders passes at most n / 32 + 16 additions, so E(n) =
# (n / 32 + 32) 2^-23 bounds its error relative to its sum of magnitudes, with the roundings of the few
# operations and the reciprocal root around it.
def E(n):
    return (n / 32 + 32) * 2.0 ** -23


def normed_error(v, kind, eps):
    """Of a normed value: its own rounding, that of the scale, and of the mean before it is taken off."""
    vh, inv = normed(v, kind, eps)
    e = E(v.shape[1]) * vh.abs()
    return e + E(v.shape[1]) * inv * v.abs().mean(1, keepdim=True) if kind == "layer" else e


def through_error(g, v, kind, eps):
    """Of a norm's gradient for g exact in FP32."""
    if kind == "none":
        return 2.0 ** -22 * g.abs()
    vh, inv = normed(v, kind, eps)
    worse = 1 + (inv * v.abs().mean(1, keepdim=True) if kind == "layer" else 0.0)
    means = g.abs().mean(1, keepdim=True) + (vh.abs() + 1) * (g * vh).abs().mean(1, keepdim=True)
    return 4 * E(v.shape[1]) * worse * inv * (g.abs() + means)

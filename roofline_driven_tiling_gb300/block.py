"""A transformer's feed-forward block on the package's operators: y = x + act(x Wg) * (x Wu) Wd.

    python -m roofline_driven_tiling_gb300.block [--width 1024] [--hidden 4096] [--rows 2048] [--steps 20]

trains the block for some steps towards the outputs of another one (float32 master weights,
16-bit weights and activations), then answers single rows from a captured graph, and prints the
losses and the times of a training step and of a single row.
"""
from __future__ import annotations

import argparse

import torch

from .feed_forward import gated_linear, gated_linear_backward, linear, linear_backward


class FeedForwardBlock:
    """The block's three weights (inputs x outputs), its forward and backward pass."""

    def __init__(self, width: int, hidden: int, dtype=torch.bfloat16, act: str = "silu", seed: int = 0):
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def weight(k, n):
            return torch.randn(k, n, generator=gen, device="cuda") * k ** -0.5

        self.act = act
        self.master = [weight(width, hidden), weight(width, hidden), weight(hidden, width)]
        self.weights = [w.to(dtype) for w in self.master]
        self.kept = None

    def forward(self, x, keep: bool = False):
        """The block's output; with ``keep`` what ``backward`` needs stays in the block."""
        gate, up, down = self.weights
        preact = None
        if keep:
            preact = tuple(torch.empty(x.shape[0], gate.shape[1], dtype=x.dtype, device=x.device) for _ in range(2))
        h = gated_linear(x, gate, up, act=self.act, preact=preact)
        if keep:
            self.kept = (x, h, preact)
        return linear(h, down, residual=x)

    def backward(self, dy):
        """dx and the gradients of the three weights for the last kept forward pass."""
        gate, up, down = self.weights
        x, h, preact = self.kept
        dh, d_down, _ = linear_backward(dy, h, down)
        dx, d_gate, d_up = gated_linear_backward(dh, x, gate, up, preact, act=self.act)
        return dx.add_(dy), [d_gate, d_up, d_down]

    def step(self, gradients, rate: float):
        for master, weight, gradient in zip(self.master, self.weights, gradients):
            master.add_(gradient.float(), alpha=-rate)
            weight.copy_(master)


def train(block, x, target, steps: int, rate: float):
    """Gradient descent on the mean square of (output - target); the losses of all steps."""
    losses = []
    for _ in range(steps):
        y = block.forward(x, keep=True)
        error = y.float() - target.float()
        losses.append(float(error.square().mean()))
        # The gradient of the sum over the row's values, averaged over the rows.
        _, gradients = block.backward(error.to(x.dtype))
        block.step(gradients, rate / x.shape[0])
    return losses


def single_row(block, width: int, dtype):
    """A captured graph of the block on one row, with its input and output."""
    x = torch.zeros(1, width, dtype=dtype, device="cuda")
    block.forward(x)  # loads the kernels outside the capture
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = block.forward(x)
    return graph, x, y


def _microseconds(run, count: int) -> float:
    run()
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    torch.cuda.synchronize()
    begin.record()
    for _ in range(count):
        run()
    end.record()
    torch.cuda.synchronize()
    return begin.elapsed_time(end) / count * 1e3


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--width", type=int, default=1024)
    ap.add_argument("--hidden", type=int, default=4096)
    ap.add_argument("--rows", type=int, default=2048)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--rate", type=float, default=0.2)
    a = ap.parse_args()
    dtype = torch.bfloat16
    block, teacher = FeedForwardBlock(a.width, a.hidden, dtype), FeedForwardBlock(a.width, a.hidden, dtype, seed=1)
    gen = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(a.rows, a.width, generator=gen, device="cuda").to(dtype)
    target = teacher.forward(x)
    losses = train(block, x, target, a.steps, a.rate)
    print("loss %.4f -> %.4f in %d steps" % (losses[0], losses[-1], a.steps))

    def pass_of_both():
        block.backward(block.forward(x, keep=True))

    print("forward and backward, %d rows: %.1f us" % (a.rows, _microseconds(pass_of_both, 50)))
    graph, _, _ = single_row(block, a.width, dtype)
    print("one row from a graph: %.1f us" % _microseconds(graph.replay, 200))


if __name__ == "__main__":
    main()

"""A mixture-of-experts feed-forward layer on the grouped and 4-bit products: trained
for some steps, then served in microscaled 4 bits.

    python examples/expert_layer.py [--tokens 4096] [--experts 8] [--top 2] [--steps 20]

The router's choice stays on the device: tokens are sorted by expert, and the group
offsets go to the products as they are, with no synchronisation in a step. The layer
learns to reproduce a fixed random layer of the same shape (synthetic data), with
fp32 master weights that the weight gradients are taken against in fp32.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import tiled_dense_gemm_bias_amd as gba  # noqa: E402


def route(scores, top):
    """(order, offsets, gates): rows of the sorted copies, their groups, their weights.

    scores [T, E]; each token goes to its `top` best experts with softmax weights.
    Row r of the sorted copies is token order[r] // top."""
    T, E = scores.shape
    best, expert = scores.topk(top, dim=1)
    gates = best.float().softmax(dim=1).reshape(-1)
    expert, order = expert.reshape(-1).sort(stable=True)
    offsets = torch.searchsorted(expert, torch.arange(E + 1, device=scores.device)).to(torch.int32)
    return order, offsets, gates[order]


class ExpertLayer:
    """y[t] = sum over t's experts e of gate * (gelu(x[t] W1_e^T + b1_e) W2_e^T)."""

    def __init__(self, experts, width, hidden, dtype=torch.bfloat16, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def init(*shape, scale):
            return torch.randn(shape, generator=g, device="cuda") * scale
        self.dtype = dtype
        self.master = [init(experts, hidden, width, scale=width ** -0.5), init(experts, hidden, scale=0.1),
                       init(experts, width, hidden, scale=hidden ** -0.5)]
        self.grads = [torch.empty_like(m) for m in self.master]
        self.workspace = torch.empty(8 << 20, dtype=torch.uint8, device="cuda")
        self.cast()

    def cast(self):
        self.w1, self.b1, self.w2 = (m.to(self.dtype) for m in self.master)

    def new(self, rows, cols):
        return torch.empty(rows, cols, dtype=self.dtype, device="cuda")

    def forward(self, x, offsets):
        """Rows sorted by expert -> (y, what the backward pass needs)."""
        rows, hidden = x.shape[0], self.w1.shape[1]
        h, z, y = self.new(rows, hidden), self.new(rows, hidden), self.new(*x.shape)
        gba.grouped_gemm_bias_act(x, offsets, self.w1, self.b1, h, "gelu", transpose_b=True, preact=z,
                                  workspace=self.workspace)
        gba.grouped_gemm_bias_act(h, offsets, self.w2, None, y, "none", transpose_b=True, workspace=self.workspace)
        return y, (x, z, h)

    def backward(self, dy, offsets, saved):
        """Fills self.grads (fp32) and returns dx."""
        x, z, h = saved
        dz, dx = self.new(*z.shape), self.new(*x.shape)
        gba.grouped_gemm_wgrad(h, dy, offsets, self.grads[2], None, transpose_b=True, workspace=self.workspace)
        gba.grouped_gemm_act_grad(dy, offsets, self.w2, z, dz, "gelu", transpose_b=True, workspace=self.workspace)
        gba.grouped_gemm_wgrad(x, dz, offsets, self.grads[0], self.grads[1], transpose_b=True, workspace=self.workspace)
        gba.grouped_gemm_act_grad(dz, offsets, self.w1, None, dx, "none", transpose_b=True, workspace=self.workspace)
        return dx

    def step(self, rate):
        for m, g in zip(self.master, self.grads):
            m.add_(g, alpha=-rate)
        self.cast()


class Served4Bit:
    """The layer with both weights quantised once; activations are quantised as they come."""

    def __init__(self, layer):
        self.layer, self.weights = layer, []
        for w in (layer.w1, layer.w2):
            E, N, K = w.shape
            self.weights.append(quantised(w.reshape(E * N, K), (E, N, K // 2)))

    def forward(self, x, offsets):
        layer = self.layer
        h, y = layer.new(x.shape[0], layer.w1.shape[1]), layer.new(*x.shape)
        for a, (codes, scales), bias, out, act in ((x, self.weights[0], layer.b1, h, "gelu"),
                                                   (h, self.weights[1], None, y, "none")):
            gba.grouped_gemm_bias_act_mx4(*quantised(a), offsets, codes, scales, bias, out, act,
                                          workspace=layer.workspace)
        return y


def quantised(x, shape=None):
    codes = torch.empty(x.shape[0], x.shape[1] // 2, dtype=torch.uint8, device=x.device)
    scales = torch.empty(gba.mx4_scales_shape(*x.shape), dtype=torch.uint8, device=x.device)
    gba.mx4_quantize(x, codes, scales)
    return (codes if shape is None else codes.view(shape)), scales


def combine(y, order, gates, tokens, top):
    """Sums each token's expert outputs by its gates."""
    out = torch.zeros(tokens, y.shape[1], device=y.device)
    return out.index_add_(0, order // top, y.float() * gates[:, None])


def run(tokens=4096, experts=8, top=2, width=512, hidden=1024, steps=20, seed=1):
    """Trains and serves; returns (losses: squared error of a token, relative error of the 4-bit outputs)."""
    rate = 32.0 / hidden   # the largest curvature is that of W2 along the mean of h, in proportion to its length
    g = torch.Generator(device="cuda").manual_seed(seed)
    teacher, layer = (ExpertLayer(experts, width, hidden, seed=s) for s in (seed + 1, seed + 2))
    router = torch.randn(width, experts, generator=g, device="cuda")
    losses = []
    for _ in range(steps):
        x = torch.randn(tokens, width, generator=g, device="cuda").to(layer.dtype)
        order, offsets, gates = route(x.float() @ router, top)
        rows = x[order // top]
        goal = combine(teacher.forward(rows, offsets)[0], order, gates, tokens, top)
        y, saved = layer.forward(rows, offsets)
        off = combine(y, order, gates, tokens, top) - goal
        losses.append(off.square().sum(1).mean())
        # d(loss) of each sorted row: its token's, times its gate
        dy = (off[order // top] * (gates[:, None] * (2.0 / tokens))).to(layer.dtype)
        layer.backward(dy, offsets, saved)
        layer.step(rate)
    y = combine(layer.forward(rows, offsets)[0], order, gates, tokens, top)
    y4 = combine(Served4Bit(layer).forward(rows, offsets), order, gates, tokens, top)
    return [v.item() for v in losses], ((y4 - y).norm() / y.norm()).item()


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    for name, value in (("tokens", 4096), ("experts", 8), ("top", 2), ("width", 512), ("hidden", 1024), ("steps", 20)):
        p.add_argument("--" + name, type=int, default=value)
    losses, error = run(**vars(p.parse_args()))
    for i, loss in enumerate(losses):
        print("step %3d  loss %.5f" % (i, loss))
    print("4-bit outputs: relative error %.3f" % error)


if __name__ == "__main__":
    main()

"""A mixture-of-experts feed-forward layer on the routing and grouped products: trained
for some steps, router and all, then served in microscaled 4 bits and in 8-bit floats.

    python examples/expert_layer.py [--tokens 4096] [--experts 8] [--top 2] [--steps 20]

The router's choice stays on the device: tokens are sorted by expert, and the group
offsets go to the products as they are, with no synchronisation in a step. The layer
learns to reproduce a fixed random layer of the same shape (synthetic data), from that
layer's router, with fp32 master weights that the weight gradients are taken against in fp32.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import tiled_dense_gemm_bias_amd as gba  # noqa: E402


class Routing:
    """Where a batch's tokens go: each to its `top` best experts by logits [T, E] (fp32), with softmax weights."""

    def __init__(self, logits, top):
        T, E = logits.shape
        i32 = dict(dtype=torch.int32, device=logits.device)
        self.logits, self.indices, self.rows = logits, torch.empty(T, top, **i32), torch.empty(T, top, **i32)
        self.weights, self.offsets = torch.empty(T, top, device=logits.device), torch.empty(E + 1, **i32)
        workspace = torch.empty(gba.moe_sort_workspace(T, E, top), dtype=torch.uint8, device=logits.device)
        gba.moe_route(logits, self.indices, self.weights, offsets=self.offsets, rows=self.rows, workspace=workspace)

    def dispatch(self, x):
        """A row of each token for each of its experts, sorted by expert."""
        return gba.moe_dispatch(x, self.rows, x.new_empty(self.rows.numel(), x.shape[1]))

    def combine(self, y, weighted=True):
        """Each token's sum over its rows, in fp32; without weights, what dispatch's gradient is."""
        out = y.new_empty(self.rows.shape[0], y.shape[1], dtype=torch.float32)
        return gba.moe_combine(y, self.rows, self.weights if weighted else None, out)

    def backward(self, dout, y):
        """(dy, dlogits) of combine(y), for its gradient dout (fp32)."""
        dy, dweights, dlogits = torch.empty_like(y), torch.empty_like(self.weights), torch.empty_like(self.logits)
        gba.moe_combine_grad(dout, y, self.rows, self.weights, dy, dweights)
        return dy, gba.moe_route_grad(self.logits, self.indices, dweights, dlogits)


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


class Served8Bit:
    """The layer with both weights in 8-bit floats, a scale for each 128 x 128 block; activations are quantised as they
    come, a token's straight to its experts' rows."""

    def __init__(self, layer):
        self.layer, self.weights = layer, []
        for w in (layer.w1, layer.w2):
            codes = torch.empty(w.shape, dtype=torch.float8_e4m3fn, device=w.device)
            scales = torch.empty(gba.fp8_weight_scales_shape(*w.shape), device=w.device)
            self.weights.append(gba.fp8_quantize_weights(w, codes, scales))

    @staticmethod
    def quantised(x, rows=None):
        R = x.shape[0] if rows is None else rows.numel()
        codes = torch.empty(R, x.shape[1], dtype=torch.float8_e4m3fn, device=x.device)
        return gba.fp8_quantize(x, codes, torch.empty(gba.fp8_scales_shape(R, x.shape[1]), device=x.device), rows=rows)

    def forward(self, x, to):
        """Tokens and their routing -> the experts' rows."""
        layer, R = self.layer, to.rows.numel()
        h, y = layer.new(R, layer.w1.shape[1]), layer.new(R, x.shape[1])
        gba.grouped_gemm_bias_act_fp8_block(*self.quantised(x, to.rows), to.offsets, *self.weights[0], layer.b1, h, "gelu",
                                            workspace=layer.workspace)
        return gba.grouped_gemm_bias_act_fp8_block(*self.quantised(h), to.offsets, *self.weights[1], None, y, "none",
                                                   workspace=layer.workspace)


def quantised(x, shape=None):
    codes = torch.empty(x.shape[0], x.shape[1] // 2, dtype=torch.uint8, device=x.device)
    scales = torch.empty(gba.mx4_scales_shape(*x.shape), dtype=torch.uint8, device=x.device)
    gba.mx4_quantize(x, codes, scales)
    return (codes if shape is None else codes.view(shape)), scales


def gradients(layer, router, x, goal, top):
    """(loss: squared error of a token, d router) with the layer's in layer.grads. router [E, width] fp32."""
    to = Routing(x.float() @ router.T, top)
    y, saved = layer.forward(to.dispatch(x), to.offsets)
    off = to.combine(y) - goal
    dy, dlogits = to.backward(off * (2.0 / x.shape[0]), y)
    layer.backward(dy, to.offsets, saved)
    return off.square().sum(1).mean(), dlogits.T @ x.float()


def train(tokens, experts, top, width, hidden, steps, seed):
    """(losses, layer, router, the last tokens)"""
    rate = 32.0 / hidden   # the largest curvature is that of W2 along the mean of h, in proportion to its length
    g = torch.Generator(device="cuda").manual_seed(seed)
    teacher, layer = (ExpertLayer(experts, width, hidden, seed=s) for s in (seed + 1, seed + 2))
    goal_router = torch.randn(experts, width, generator=g, device="cuda")
    router, losses = goal_router.clone(), []
    for _ in range(steps):
        x = torch.randn(tokens, width, generator=g, device="cuda").to(layer.dtype)
        to = Routing(x.float() @ goal_router.T, top)
        goal = to.combine(teacher.forward(to.dispatch(x), to.offsets)[0])
        loss, drouter = gradients(layer, router, x, goal, top)
        losses.append(loss)
        layer.step(rate)
        router.add_(drouter, alpha=-rate / width)   # (the logits grow with the width)
    return losses, layer, router, x


def served_errors(layer, router, x, top):
    """Relative errors of the layer's outputs for x in 4 and in 8 bits."""
    to = Routing(x.float() @ router.T, top)
    rows = to.dispatch(x)
    y, *served = (to.combine(r) for r in (layer.forward(rows, to.offsets)[0], Served4Bit(layer).forward(rows, to.offsets),
                                          Served8Bit(layer).forward(x, to)))
    return [((s - y).norm() / y.norm()).item() for s in served]


def run(tokens=4096, experts=8, top=2, width=512, hidden=1024, steps=20, seed=1):
    """Trains and serves; returns (losses: squared error of a token, relative error of the 4-bit outputs)."""
    losses, layer, router, x = train(tokens, experts, top, width, hidden, steps, seed)
    return [v.item() for v in losses], served_errors(layer, router, x, top)[0]


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    for name, value in (("tokens", 4096), ("experts", 8), ("top", 2), ("width", 512), ("hidden", 1024), ("steps", 20)):
        p.add_argument("--" + name, type=int, default=value)
    p.add_argument("--seed", type=int, default=1)
    args = p.parse_args()
    losses, layer, router, x = train(**vars(args))
    for i, loss in enumerate(losses):
        print("step %3d  loss %.5f" % (i, loss.item()))
    for bits, error in zip((4, 8), served_errors(layer, router, x, args.top)):
        print("%d-bit outputs: relative error %.3f" % (bits, error))


if __name__ == "__main__":
    main()

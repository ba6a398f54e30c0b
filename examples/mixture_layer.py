"""A mixture-of-experts feed-forward layer with 4-bit microscaled weights, as a serving
program runs it: weights quantized once, then for each batch the router's product, the
choice of experts, the plan of the batch's rows and the experts' products.

    python examples/mixture_layer.py

prints, for a prefill batch and for one decode token, how far the layer is from the same
layer in plain fp32 arithmetic over the quantized values, and its time.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))

import dense_sparse_bit_amd as mq  # noqa: E402


class MixtureLayer:
    """y = sum over the k chosen experts e of weight_e * down_e(silu(gate_e x) * (up_e x))."""

    def __init__(self, w_router, w_gate, w_up, w_down, k: int):
        """w_router [E, D], w_gate and w_up [E, I, D], w_down [E, D, I]."""
        self.k, self.experts = k, w_router.shape[0]
        self.router = mq.mx_quantize(w_router)
        self.gate, self.up, self.down = (mq.mx_quantize(w) for w in (w_gate, w_up, w_down))

    def __call__(self, x):
        logits = mq.mx_linear(x, self.router, out_dtype=torch.float32)
        ids, weights = mq.route(logits, self.k)
        plan = mq.expert_plan(ids, self.experts)
        return mq.mx_experts(x, self.gate, self.up, self.down, plan, weights)

    def plain(self, x):
        """The same in fp32 over the quantized values, token by token and slot by slot."""
        read = lambda a: mq.mx_dequantize(a)
        q = lambda v: read(mq.mx_quantize(v))
        logits = q(x) @ read(self.router).t()
        score, ids = torch.softmax(logits, 1).topk(self.k, 1)
        score = score / score.sum(1, keepdim=True)
        y = torch.zeros(x.shape, device=x.device)
        gate, up, down, xq = read(self.gate), read(self.up), read(self.down), q(x)
        for j in range(self.k):
            for e in ids[:, j].unique().tolist():
                t = torch.nonzero(ids[:, j] == e).flatten()
                g, u = xq[t] @ gate[e].t(), xq[t] @ up[e].t()
                h = (g / (1 + torch.exp(-g)) * u).to(torch.bfloat16)
                y[t] += score[t, j][:, None] * (q(h) @ down[e].t())
        return y


def make(D: int, I: int, E: int, k: int, seed: int = 0) -> MixtureLayer:
    g = torch.Generator(device="cuda").manual_seed(seed)
    draw = lambda *shape: torch.randn(*shape, generator=g, device="cuda") / shape[-1] ** 0.5
    return MixtureLayer(draw(E, D), draw(E, I, D), draw(E, I, D), draw(E, D, I), k)


def main(D: int = 1024, I: int = 512, E: int = 16, k: int = 4):
    layer = make(D, I, E, k)
    errors = []
    for tokens in (300, 1):
        x = torch.randn(tokens, D, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)).to(torch.bfloat16)
        y, want = layer(x), layer.plain(x)
        errors.append(float((y.float() - want).norm() / want.norm()))
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        start.record()
        for _ in range(20):
            layer(x)
        end.record()
        end.synchronize()
        print(f"{tokens} tokens: relative error {errors[-1]:.2e}, {start.elapsed_time(end) / 20 * 1e3:.0f} us")
    return errors


if __name__ == "__main__":
    main()

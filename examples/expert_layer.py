"""The feed-forward half of a decoder layer made of experts, on block-scaled FP8 weights.

    python examples/expert_layer.py [--tokens 300] [--experts 16]

A layer of 16 experts of 1024 x (2 x 768), three for each token, and a shared one:

  route      scores of the experts, the best three of two groups, pairs sorted by expert;
  products   quantize the tokens, every pair's first product with its expert's weight, gate
             and quantize, second product;
  sum        each token's weighted sum of its experts' rows, plus the shared expert's.

The experts' part is computed a second way, expert by expert with the dense product on the
gathered rows, and compared: the same blocks added in the same order, so the same numbers up to
the rounding of a sum of three.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import scaled_gemm_amd as sg  # noqa: E402

HIDDEN, WIDTH, TOP_K, GROUPS, TOP_GROUPS = 1024, 768, 3, 4, 2


class ExpertLayer:
    """Router, experts and a shared expert with FP8 weights."""

    def __init__(self, experts, seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)

        def weights(*shape):
            w = torch.randn(shape, device="cuda", generator=g) * shape[-2] ** -0.5
            return w.bfloat16()

        self.router = weights(HIDDEN, experts)
        self.bias = 0.01 * torch.randn(experts, device="cuda", generator=g)
        up, down = weights(experts, HIDDEN, 2 * WIDTH), weights(experts, WIDTH, HIDDEN)
        self.up, self.down = sg.quant_weight_block(up), sg.quant_weight_block(down)
        self.each = [(sg.quant_weight_block(u), sg.quant_weight_block(d)) for u, d in zip(up, down)]
        self.shared = (sg.quant_weight_block(weights(HIDDEN, 2 * WIDTH)),
                       sg.quant_weight_block(weights(WIDTH, HIDDEN)))

    def route(self, x):
        return sg.route_experts(x @ self.router, TOP_K, scoring="sigmoid", bias=self.bias,
                                groups=GROUPS, top_groups=TOP_GROUPS)

    def experts(self, x, routing):
        qx, sx = sg.quant_act_block(x)
        h = sg.gemm_experts(qx, sx, self.up, routing, gather=True)
        y = sg.gemm_experts(*sg.quant_act_block(h, gate=True), self.down, routing)
        return sg.combine_experts(y, routing)

    def feed_forward(self, x, up, down):
        h = sg.linear_block(x, up)
        return sg.gemm_block(*sg.quant_act_block(h, gate=True), down)

    def __call__(self, x):
        return x + self.experts(x, self.route(x)) + self.feed_forward(x, *self.shared)

    def experts_one_by_one(self, x, routing):
        """The experts' part by dense products, in fp32 sums."""
        out = torch.zeros(x.shape, device="cuda")
        for e, (up, down) in enumerate(self.each):
            t, k = (routing.ids == e).nonzero(as_tuple=True)
            if t.numel():
                y = self.feed_forward(x[t], up, down)
                out.index_add_(0, t, y.float() * routing.weights[t, k, None])
        return out


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--tokens", type=int, default=300)
    ap.add_argument("--experts", type=int, default=16)
    args = ap.parse_args(argv)
    layer = ExpertLayer(args.experts)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    worst = 0.0
    for tokens in (args.tokens, 1):                    # a prompt's tokens, a decoded one
        x = torch.randn((tokens, HIDDEN), device="cuda", generator=g).bfloat16()
        r = layer.route(x)
        a, b = layer.experts(x, r).float(), layer.experts_one_by_one(x, r)
        worst = max(worst, ((a - b).norm() / b.norm()).item())
        y = layer(x)
        load = r.offsets.diff()
        print(f"{tokens} tokens: rows an expert {load.min().item()}..{load.max().item()}, output "
              f"{tuple(y.shape)}, one by one differs by {worst:.2e}")
    return worst


if __name__ == "__main__":
    main()

"""A feed-forward layer of experts in microscaled 4-bit floats.

    python examples/mx4_experts.py [--tokens 64] [--experts 16] [--choices 4]

A router picks a few experts for each token.  ``sort_by_expert`` puts the
(token, choice) pairs in the experts' order, ``MX4Experts`` multiplies each
expert's rows by its weights (the tokens are quantised once, each expert takes
its rows from there), and ``ExpertOrder.combine`` adds a token's results with the
router's weights.  The experts are frozen: the router's gradient comes from
``combine_backward``, and is what a fine-tuning step would use.  Weights are
random: the example shows the calls, not a trained model.
"""

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import popcount_convolution_amd as pca  # noqa: E402


def mx4_experts(weights: torch.Tensor) -> pca.MX4Experts:
    """A layer from float weights ``[experts, out, in]`` on the GPU: quantised by
    rows, without the padding that quantised rows have."""
    experts, n, k = weights.shape
    q = pca.mx4_quantize(weights)
    return pca.MX4Experts(experts=experts, in_features=k, out_features=n, codes=q.codes[..., :-(-k // 2)].contiguous(),
                          scales=q.scales[..., :-(-k // 32)].contiguous())


class ExpertLayer:
    def __init__(self, width: int, hidden: int, experts: int, choices: int, seed: int = 0, dtype=torch.bfloat16):
        g = torch.Generator(device="cuda").manual_seed(seed)
        normal = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
        self.router = normal(experts, width) * width ** -0.5
        self.up = mx4_experts(normal(experts, 2 * hidden, width) * width ** -0.5)
        self.down = mx4_experts(normal(experts, width, hidden) * hidden ** -0.5)
        self.experts, self.choices, self.hidden, self.dtype = experts, choices, hidden, dtype

    def route(self, x):
        """(ids, weights) ``[tokens, choices]`` of rows x."""
        logits = x.float() @ self.router.t()
        top = torch.topk(logits, self.choices, dim=1)
        return top.indices, torch.softmax(top.values, 1)

    def forward(self, x):
        """Rows ``[tokens, width]`` -> the same, and what the gradient needs."""
        ids, weights = self.route(x)
        order = pca.sort_by_expert(ids, self.experts)
        both = self.up.forward(x, order)
        h = torch.nn.functional.silu(both[:, :self.hidden]) * both[:, self.hidden:]
        rows = self.down.forward(h, order, in_order=True)
        return order.combine(rows, weights), (x, ids, weights, order, rows)

    def router_gradient(self, dy, saved):
        """Gradient of the router's weights for the gradient dy of the result."""
        x, ids, weights, order, rows = saved
        _, d_weights = order.combine_backward(dy, rows, weights)
        d_logits = weights * (d_weights - (weights * d_weights).sum(1, keepdim=True))
        grad = torch.zeros_like(self.router)
        for j in range(self.choices):
            grad.index_add_(0, ids[:, j], d_logits[:, j:j + 1] * x.float())
        return grad


def main():
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--tokens", type=int, default=64)
    p.add_argument("--width", type=int, default=1024)
    p.add_argument("--hidden", type=int, default=704)
    p.add_argument("--experts", type=int, default=16)
    p.add_argument("--choices", type=int, default=4)
    a = p.parse_args()
    layer = ExpertLayer(a.width, a.hidden, a.experts, a.choices)
    x = torch.randn((a.tokens, a.width), device="cuda").to(layer.dtype)
    y, saved = layer.forward(x)
    grad = layer.router_gradient(torch.ones_like(y), saved)
    counts = (saved[3].offsets[1:] - saved[3].offsets[:-1]).tolist()
    print(f"{a.tokens} tokens, {a.choices} of {a.experts} experts each: rows an expert {min(counts)} to {max(counts)}, "
          f"result rms {y.float().square().mean().sqrt().item():.3f}, router gradient rms {grad.square().mean().sqrt().item():.2e}")


if __name__ == "__main__":
    main()

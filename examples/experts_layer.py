"""A layer of experts in 8 bits, trained and then decoded with, by the package's entry points.

    python examples/experts_layer.py [tokens] [width] [hidden] [experts] [choices] [steps]

Each step routes the tokens, quantises the rows that each expert gets, multiplies them by the
experts' weights, adds the results up for each token, and goes the same way back: gradients of
the rows, of the experts' weights (each over its own tokens) and of the router.  Activations
and weights are e4m3, gradients e5m2, every product sums in fp32; the weights themselves and
their updates stay in fp32.  The layer learns to imitate a fixed one of the same shape.
"""
import sys
from pathlib import Path

import torch

sys.path.insert(0, str(Path(__file__).resolve().parent.parent))
import dense_gemm_05_gb300 as g  # noqa: E402

E5M2 = torch.float8_e5m2


class Experts:
    """y = sum over a token's choices j of weight_j * W2[e_j] relu(W1[e_j] x)."""

    def __init__(self, width, hidden, experts, choices, device="cuda", seed=0):
        r = torch.Generator().manual_seed(seed)
        self.choices = choices
        self.router = (torch.randn((experts, width), generator=r) / width ** 0.5).to(device)
        self.up = (torch.randn((experts, hidden, width), generator=r) / width ** 0.5).to(device)
        self.down = (torch.randn((experts, width, hidden), generator=r) / hidden ** 0.5).to(device)
        self.lay_out()

    def lay_out(self):
        """The weights' codes, once for each change of them: as they are and transposed."""
        self.up8, self.down8 = g.quantize_fp8_tiles(self.up), g.quantize_fp8_tiles(self.down)
        self.up8t = g.quantize_fp8_tiles(self.up, transpose=True)
        self.down8t = g.quantize_fp8_tiles(self.down, transpose=True)

    def forward(self, x):
        """x [T, width] (bfloat16) -> y (float32), and what the way back needs."""
        logits = x.float() @ self.router.t()
        way = g.route(logits, self.choices)
        h = g.matmul_fp8(*g.quantize_fp8_rows(x, rows=way.tokens), *self.up8, offsets=way.offsets)
        h = torch.relu(h)
        rows = g.matmul_fp8(*g.quantize_fp8_rows(h), *self.down8, offsets=way.offsets)
        y = g.combine(rows, way.slots, way.weights, out_dtype=torch.float32)
        return y, (x, logits, way, h, rows)

    def backward(self, dy, saved):
        """dx (float32) and the gradients of router, up and down."""
        x, logits, way, h, rows = saved
        drows, dweights = g.combine_backward(dy.to(rows.dtype), rows, way.slots, way.weights)
        dh = g.matmul_fp8(*g.quantize_fp8_rows(drows, dtype=E5M2), *self.down8t, offsets=way.offsets)
        dh = dh * (h > 0)
        ddown = g.matmul_fp8_depth(*g.quantize_fp8_columns(drows, offsets=way.offsets, dtype=E5M2),
                                   *g.quantize_fp8_columns(h, offsets=way.offsets), way.offsets)
        dup = g.matmul_fp8_depth(*g.quantize_fp8_columns(dh, offsets=way.offsets, dtype=E5M2),
                                 *g.quantize_fp8_columns(x, rows=way.tokens, offsets=way.offsets),
                                 way.offsets)
        dx = g.matmul_fp8(*g.quantize_fp8_rows(dh, dtype=E5M2), *self.up8t, offsets=way.offsets)
        dx = g.combine(dx, way.slots, out_dtype=torch.float32)
        dlogits = g.route_backward(dweights, logits, way.ids)
        return dx + dlogits @ self.router, (dlogits.t() @ x.float(), dup, ddown)


def train(tokens=512, width=256, hidden=512, experts=16, choices=4, steps=30, rate=0.04):
    """Mean squared errors, one for each step."""
    layer, goal = Experts(width, hidden, experts, choices), Experts(width, hidden, experts, choices, seed=1)
    goal.router.copy_(layer.router)
    errors = []
    for step in range(steps):
        r = torch.Generator().manual_seed(100 + step)
        x = torch.randn((tokens, width), generator=r).to("cuda", torch.bfloat16)
        y, saved = layer.forward(x)
        off = y - goal.forward(x)[0]
        errors.append(float((off * off).mean()))
        _, (drouter, dup, ddown) = layer.backward(off, saved)
        scale = rate * experts / (tokens * choices)
        layer.router -= scale / 10 * drouter
        layer.up -= scale * dup
        layer.down -= scale * ddown
        layer.lay_out()
    return layer, errors


def decode(layer, tokens=8, steps=4):
    """Steps of a few tokens each, captured once into a graph and replayed."""
    width = layer.router.size(1)
    x = torch.zeros((tokens, width), device="cuda", dtype=torch.bfloat16)
    layer.forward(x)                                  # the library and its kernels are loaded
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, _ = layer.forward(x)
    x.copy_(torch.randn((tokens, width), generator=torch.Generator().manual_seed(0)))
    out = []
    for _ in range(steps):
        graph.replay()
        out.append(y.clone())
        x.copy_(y)                                    # the next step's input is this one's result
    return out


if __name__ == "__main__":
    sizes = [int(a) for a in sys.argv[1:]]
    layer, errors = train(*sizes)
    print("mean squared error: first step %.4f, last step %.4f" % (errors[0], errors[-1]))
    print("decoded", [list(o.shape) for o in decode(layer)])

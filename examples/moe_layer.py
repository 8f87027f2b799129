"""An expert layer in MXFP8 on one MI355X, forward and backward.

    python examples/moe_layer.py [--tokens T] [--hidden H] [--inner F] [--experts E] [--top-k K]

Tokens are routed to their top-k experts and sorted by expert; their rows go
through a gated (SiLU) product and a second one, by expert and in MXFP8, and
come back weighted, on top of the residual stream.  The backward pass gives
the gradients of the tokens, the routing weights and both weight tensors.
Prints the time of a prompt step, a training step and a decoding step.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import mxfp8_block_scaled_mxgemm_amd as mx  # noqa: E402


class ExpertLayer:
    """w1 [E, 2 F, H] (gate rows, then up rows) and w2 [E, H, F], held in MXFP8
    both ways: along their inner axis for the forward products and transposed
    for the gradients."""

    def __init__(self, w1, w2, precision="exact"):
        self.precision = precision
        self.E, self.F, self.H = w1.shape[0], w1.shape[1] // 2, w1.shape[2]
        self.w1, self.w1t = self._both(w1)
        self.w2, self.w2t = self._both(w2)

    @staticmethod
    def _both(w):
        parts = [mx.epilogue_backward(x, bias=False)[:2] for x in w]
        return tuple(tuple(torch.stack([p[way][i] for p in parts]) for i in (0, 1)) for way in (0, 1))

    def forward(self, x, ids, weights):
        """Serving: the hidden rows stay in MXFP8 between the products."""
        sort = mx.sort_tokens(ids, self.E)
        rows = mx.dispatch_tokens_mx(x, sort)
        hidden = mx.linear(*rows, *self.w1, act="silu", gated=True, offsets=sort.offsets, out_dtype="e4m3",
                           precision=self.precision)
        out = mx.linear(*hidden, *self.w2, offsets=sort.offsets, precision=self.precision)
        return mx.combine_tokens(out, sort, weights, residual=x)

    def train_step(self, x, ids, weights, d_y):
        """Forward and backward: (y, (d_x, d_weights, d_w1, d_w2))."""
        sort = mx.sort_tokens(ids, self.E)
        rows = mx.dispatch_tokens(x, sort)
        (a, a_s), (at, at_s), _ = mx.epilogue_backward(rows, sort=sort, bias=False)
        h, z = mx.linear(a, a_s, *self.w1, act="silu", gated=True, offsets=sort.offsets, preact=True,
                         precision=self.precision)
        (b, b_s), (bt, bt_s), _ = mx.epilogue_backward(h, sort=sort, bias=False)
        out = mx.linear(b, b_s, *self.w2, offsets=sort.offsets, precision=self.precision)
        y = mx.combine_tokens(out, sort, weights, residual=x)

        d_out, d_weights = mx.combine_tokens_backward(d_y, out, sort, weights)
        g2 = mx.linear_backward(d_out, None, bt, bt_s, *self.w2t, sort=sort, bias=False, precision=self.precision)
        g1 = mx.linear_backward(g2.d_a, z, at, at_s, *self.w1t, act="silu", gated=True, sort=sort, bias=False,
                                precision=self.precision)
        d_x = d_y + mx.dispatch_tokens_backward(g1.d_a, sort)       # the residual stream's share
        return y, (d_x, d_weights, g1.d_w, g2.d_w)


def route(logits, k):
    """Top-k experts of each token and their weights."""
    top, ids = logits.topk(k, dim=1)
    return ids.to(torch.int32), torch.softmax(top.float(), dim=1)


def timed(f, n=20):
    f()
    torch.cuda.synchronize()
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(n):
        f()
    end.record()
    torch.cuda.synchronize()
    return start.elapsed_time(end) / n


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("tokens", 4096), ("hidden", 2048), ("inner", 1024), ("experts", 32), ("top-k", 4)):
        ap.add_argument(f"--{name}", type=int, default=value)
    ap.add_argument("--precision", choices=("exact", "native"), default="exact")
    a = ap.parse_args()
    g = torch.Generator(device="cuda").manual_seed(0)
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    layer = ExpertLayer((randn(a.experts, 2 * a.inner, a.hidden) * a.hidden ** -0.5).bfloat16(),
                        (randn(a.experts, a.hidden, a.inner) * a.inner ** -0.5).bfloat16(), a.precision)
    x, d_y = randn(a.tokens, a.hidden).bfloat16(), randn(a.tokens, a.hidden).bfloat16()
    ids, weights = route(randn(a.tokens, a.experts), a.top_k)
    few = min(8, a.tokens)
    one, one_ids, one_w = x[:few].contiguous(), ids[:few].contiguous(), weights[:few].contiguous()
    print(f"{a.tokens} tokens, {a.experts} experts, top {a.top_k}, {a.hidden} -> {a.inner}: "
          f"forward {timed(lambda: layer.forward(x, ids, weights)):.3f} ms, "
          f"training step {timed(lambda: layer.train_step(x, ids, weights, d_y)):.3f} ms, "
          f"{few} tokens {timed(lambda: layer.forward(one, one_ids, one_w)):.3f} ms")


if __name__ == "__main__":
    main()

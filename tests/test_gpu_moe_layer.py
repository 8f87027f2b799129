"""The expert layer of examples/moe_layer.py, forward and backward, against
float64 autograd on the CPU with unquantised operands: what differs is the
MXFP8 rounding of the operands (3 mantissa bits: at most 2^-4 / sqrt(3) = 3.6%
of a value, root mean square).  An output passes through two products of two
such operands each (with a slope of at most 1.1 in between): sqrt(4) * 3.6% *
1.1 < 8%; a gradient through four products: sqrt(8) * 3.6% * 1.1 < 12%, and the
gated pair doubles one of them."""
import importlib.util
import os

import pytest
import torch

from gpu_common import say, torch_cuda

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("moe_layer", os.path.join(ROOT, "examples", "moe_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _reference(x, ids, weights, w1, w2, d_y):
    x, weights, w1, w2 = (t.double().requires_grad_() for t in (x, weights, w1, w2))
    F = w1.shape[1] // 2
    y = x.clone()
    for e in range(w1.shape[0]):
        t, j = (ids == e).nonzero(as_tuple=True)
        if len(t):
            z = x[t] @ w1[e].t()
            h = torch.nn.functional.silu(z[:, :F]) * z[:, F:]
            y = y.index_add(0, t, weights[t, j].unsqueeze(1) * (h @ w2[e].t()))
    y.backward(d_y.double())
    return y.detach(), (x.grad, weights.grad, w1.grad, w2.grad)


def _off(got, ref):
    return float((got.double().cpu() - ref).norm() / ref.norm())


@pytest.mark.parametrize("precision", ["exact", "native"])
@pytest.mark.parametrize("T,k,E,H,F,drop", [(1, 2, 4, 128, 128, 0.0), (37, 2, 6, 256, 128, 0.1),
                                            (300, 3, 8, 384, 256, 0.05), (700, 2, 3, 256, 384, 0.0)])
def test_layer(example, T, k, E, H, F, drop, precision):
    torch_cuda()
    say(f"layer T={T} k={k} E={E} H={H} F={F} drop={drop} {precision}")
    g = torch.Generator().manual_seed(T)
    randn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    w1, w2 = (randn(E, 2 * F, H) * H ** -0.5).bfloat16(), (randn(E, H, F) * F ** -0.5).bfloat16()
    x, d_y = randn(T, H).bfloat16(), randn(T, H).bfloat16()
    ids, weights = example.route(randn(T, E), k)
    ids[torch.rand(T, k, generator=g) < drop] = -1
    layer = example.ExpertLayer(w1.cuda(), w2.cuda(), precision)
    y, grads = layer.train_step(x.cuda(), ids.cuda(), weights.cuda(), d_y.cuda())
    served = layer.forward(x.cuda(), ids.cuda(), weights.cuda())
    ref, ref_grads = _reference(x, ids, weights, w1, w2, d_y)
    assert _off(y, ref) < 0.08 and _off(served, ref) < 0.08
    for name, got, want in zip(("d_x", "d_weights", "d_w1", "d_w2"), grads, ref_grads):
        assert got.shape == want.shape and _off(got, want) < 0.16, name
    # experts without tokens have no gradient, dropped choices none either
    assert all(not bool(grads[2][e].any()) for e in range(E) if not bool((ids == e).any()))
    assert not bool(grads[1].cpu()[ids < 0].any())

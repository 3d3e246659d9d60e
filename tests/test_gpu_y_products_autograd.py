"""The 16-bit products and their gradients as an autograd function, written as the README shows it."""
import pytest
import torch

from test_gpu_y_products import _cuda, gen, normal, offsets_of, product_bound, spans  # noqa: F401
from weight_only_bit_route_b200 import moe

pytestmark = pytest.mark.gpu


class ExpertsProduct(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, off, ws):
        ctx.save_for_backward(x, w, off)
        ctx.ws = ws
        return moe.grouped_mm(x, w, off, ws)

    @staticmethod
    def backward(ctx, dy):
        x, w, off = ctx.saved_tensors
        dy = dy.contiguous()
        return moe.grouped_mm_dgrad(dy, w, off, ctx.ws), moe.grouped_mm_wgrad(dy, x, off, ctx.ws), None, None


@pytest.mark.parametrize("counts,K,N", [([5, 0, 60, 1], 136, 72), ([700, 0, 129, 300], 512, 520)])
def test_backward_of_the_function(counts, K, N):
    """d sum(c y) / dx and / dw against the formulas, for a cotangent that arrives transposed and for one that is shared
    by every row (a broadcast, of stride 0)."""
    g = gen(40)
    rows, E = sum(counts), len(counts)
    off, ws = offsets_of(counts), moe.control_block()
    for c in (normal(g, N, rows).t(), normal(g, 1, N).expand(rows, N)):
        x, w = normal(g, rows, K).requires_grad_(), normal(g, E, N, K, std=0.1).requires_grad_()
        ExpertsProduct.apply(x, w, off, ws).backward(c)
        assert moe.read_status(ws) == 0
        for e, a, b in spans(counts):
            ce, xe, we = c[a:b].double(), x[a:b].detach().double(), w[e].detach().double()
            for got, p, q, terms in ((x.grad[a:b], ce, we, N), (w.grad[e], ce.T, xe, b - a)):
                ref = p @ q
                assert ((got.double() - ref).abs() <= product_bound(p.abs() @ q.abs(), terms, ref, got.dtype)).all(), e


def test_no_history_is_recorded_outside_it():
    g = gen(41)
    x, w = normal(g, 8, 64).requires_grad_(), normal(g, 2, 32, 64).requires_grad_()
    y = moe.grouped_mm(x, w, offsets_of([3, 5]), moe.control_block())
    assert not y.requires_grad and y.grad_fn is None

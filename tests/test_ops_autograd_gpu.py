"""The operators beside torch's automatic differentiation: they record nothing, and say so."""
import warnings

import pytest
import torch

from ops_util import offsets_of, randn
from sparse_moe_router_amd import ops

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def calls():
    x, w, off, n = randn(1, 12, 64).cuda(), randn(2, 2, 32, 64).cuda(), offsets_of([5, 7]).cuda(), randn(3, 64).cuda()
    return {"grouped_matmul": (lambda t: ops.grouped_matmul(x, t, off), w),
            "quantize_i8": (lambda t: ops.quantize_i8(t), x), "block_norm": (lambda t: ops.block_norm(x, t, 1e-6), n),
            "block_merge": (lambda t: ops.block_merge(x, t, n, 1e-6, next_weight=n), x.clone())}


@pytest.mark.parametrize("name", ["grouped_matmul", "quantize_i8", "block_norm", "block_merge"])
def test_a_gradient_that_is_not_recorded_is_said(name):
    f, t = calls()[name]
    t.requires_grad_()
    with pytest.warns(UserWarning, match="requires a gradient") as seen:
        res = f(t)
    assert len(seen) == 1 and seen[0].filename == __file__
    assert not any(r.requires_grad for r in (res if isinstance(res, tuple) else (res,)))
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        with torch.no_grad():
            f(t)
        with pytest.raises(UserWarning):
            f(t)
        t.requires_grad_(False)
        f(t)


def test_inside_an_autograd_function():
    """As the gradient calls are meant to be used: no warning, and the gradients arrive."""

    class Product(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, w, off):
            ctx.save_for_backward(x, w, off)
            return ops.grouped_matmul(x, w, off)

        @staticmethod
        def backward(ctx, dy):
            x, w, off = ctx.saved_tensors
            return ops.grouped_matmul_grad_input(dy, w, off), ops.grouped_matmul_grad_weight(x, dy, off, out_dtype=BF16), None

    x, w = randn(1, 12, 64).cuda().requires_grad_(), randn(2, 2, 32, 64).cuda().requires_grad_()
    off, dy = offsets_of([5, 7]).cuda(), randn(3, 12, 32).cuda()
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        Product.apply(x, w, off).backward(dy)
        with torch.no_grad():
            assert torch.equal(x.grad, ops.grouped_matmul_grad_input(dy, w, off))
            assert torch.equal(w.grad, ops.grouped_matmul_grad_weight(x, dy, off, out_dtype=BF16))

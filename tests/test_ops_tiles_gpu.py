"""The matrix-matrix kernels of the products where rows, strides or indexes go wrong: every call here is
large enough for them (few rows take the matrix-vector kernel)."""
import pytest
import torch

from ops_util import offsets_of, randn
from sparse_moe_router_amd import ops

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def codes(seed, *shape):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(-127, 128, shape, generator=g, dtype=torch.int8)


def scales(seed, *shape):
    g = torch.Generator().manual_seed(seed)
    return torch.rand(shape, generator=g) * 0.01 + 1e-3


@pytest.mark.parametrize("kind", ["bf16", "int8 tokens", "int8 codes"])
def test_no_rows_of_x(kind):
    """A permutation that no row of x backs: rows of zeros in every tile height and every step of the
    reduction, and weight gradients of zeros."""
    counts, N, K = [300, 90, 200, 150], 1024, 1040
    R, E, off = sum(counts), len(counts), offsets_of(counts).cuda()
    perm = torch.arange(R, dtype=torch.int32, device="cuda")
    y = torch.full((R, N), 7.0, device="cuda")
    if kind == "bf16":
        x = torch.empty(0, K, dtype=BF16, device="cuda")
        ops.grouped_matmul(x, randn(1, E, N, K).cuda(), off, perm=perm, top_k=2, out=y)
        dw = ops.grouped_matmul_grad_weight(x, randn(2, R, N).cuda(), off, perm=perm, top_k=2)
        assert dw.shape == (E, N, K) and (dw == 0).all()
    else:
        tokens = kind == "int8 tokens"
        x = torch.empty(0, K, dtype=BF16 if tokens else torch.int8, device="cuda")
        ops.grouped_matmul_i8(x, codes(1, E, N, K).cuda(), scales(2, E, N).cuda(), off, perm=perm, top_k=2, out=y,
                              x_scale=None if tokens else torch.empty(0, device="cuda"))
    assert (y == 0).all()


def test_out_of_fewer_rows_than_x_is_refused():
    """A product of x's rows has a row for each of them."""
    x, w, off = randn(1, 12, 64).cuda(), randn(2, 2, 32, 64).cuda(), offsets_of([5, 7]).cuda()
    out = torch.empty(11, 32, dtype=BF16, device="cuda")
    with pytest.raises(ValueError, match="out"):
        ops.grouped_matmul(x, w, off, out=out)
    with pytest.raises(ValueError, match="out"):
        ops.grouped_matmul_i8(x, codes(3, 2, 32, 64).cuda(), scales(4, 2, 32).cuda(), off, out=out)

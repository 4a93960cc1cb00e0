"""Offsets past 32 bits in the training operators: matrices whose rows lie far apart, tensors and buffers of more than
2^31 elements, each against the same call on small contiguous ones."""
import pytest
import torch

from ops_util import randn
from sparse_moe_router_amd import ops

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
R, LD = 70000, 1 << 15  # 4.6 GB of bf16


def far(t, fill=0.0):
    """t in columns 8.. of a matrix with rows LD apart."""
    wide = torch.full((t.shape[0], LD), fill, dtype=t.dtype, device="cuda")
    v = wide[:, 8:8 + t.shape[1]]
    v.copy_(t)
    return v


def test_gated_products():
    x, w, dy, wd = randn(1, R, 16).cuda(), randn(2, 1, 32, 16).cuda(), randn(3, R, 8).cuda(), randn(4, 1, 8, 16).cuda()
    h, gu = ops.gated_matmul(x, w, None, save=True)
    fx, fh, fg = far(x), far(torch.zeros_like(h)), far(torch.zeros_like(gu))
    ops.gated_matmul(fx, w, None, save=True, out=fh, gate_up=fg)
    assert torch.equal(fh, h) and torch.equal(fg, gu)
    perm = torch.randperm(R, generator=torch.Generator().manual_seed(5)).to(torch.int32).cuda()
    assert torch.equal(ops.gated_matmul(fx, w, None, perm=perm), ops.gated_matmul(x, w, None, perm=perm))
    want = ops.gated_matmul_grad(dy, wd, gu, None)
    del fx, fh
    got = ops.gated_matmul_grad(far(dy), wd, fg, None)
    assert all(torch.equal(got[k], want[k]) for k in want)
    a, b = (ops.feed_forward_grad(v, x, w, wd, g, None, dw_dtype=F32) for v, g in ((dy, gu), (far(dy), fg)))
    assert all(torch.equal(a[k], b[k]) for k in a)


def test_combine():
    T, k, H = R // 2, 2, 24
    y, d, w = randn(1, R, H).cuda(), randn(2, T, H).cuda(), torch.rand(T, k, device="cuda")
    perm = torch.randperm(R, generator=torch.Generator().manual_seed(5)).to(torch.int32).cuda()
    inv = ops.invert_permutation(perm)
    want = ops.combine(y, inv, k, weight=w, add=d)
    fy = far(y)
    out = far(torch.zeros_like(want))
    assert torch.equal(ops.combine(fy, inv, k, weight=w, add=d, out=out), want)
    a = ops.combine_grad(d, y, perm, inv, w)
    dy = far(torch.zeros_like(y))
    b = ops.combine_grad(d, fy, perm, inv, w, dy=dy)
    assert torch.equal(dy, a["y"]) and torch.equal(b["weight"], a["weight"])


def test_cross_entropy():
    x, w = randn(1, R, 16).cuda(), randn(2, 40, 16).cuda()
    t = torch.randint(-1, 40, (R,), generator=torch.Generator().manual_seed(3)).cuda()
    dl = torch.rand(R, device="cuda")
    fx = far(x)
    (a, la), (b, lb) = ops.cross_entropy(x, w, t), ops.cross_entropy(fx, w, t)
    assert torch.equal(a, b) and torch.equal(la, lb)
    g, h = ops.cross_entropy_grad(dl, x, w, t, la), ops.cross_entropy_grad(dl, fx, w, t, la)
    assert torch.equal(g["x"], h["x"]) and torch.equal(g["w"], h["w"])
    # logits of more than 2^31 elements, which are never there: 70000 x 32800
    w = randn(4, 32800, 16).cuda()
    t = torch.randint(0, 32800, (R,), generator=torch.Generator().manual_seed(6)).cuda()
    loss, lse = ops.cross_entropy(x, w, t)
    g = ops.cross_entropy_grad(dl, x, w, t, lse, dx_dtype=F32, dw_dtype=None)
    for i in (0, R - 100):  # rows at both ends, alone
        s = slice(i, i + 100)
        z = x[s].double() @ w.double().t()
        want = torch.logsumexp(z, 1)
        assert ((lse[s] - want).abs() <= 1e-5 * want.abs()).all()
        p = torch.softmax(z, 1)
        p[torch.arange(100), t[s]] -= 1
        dx = dl[s, None] * (p @ w.double())
        assert (g["x"][s] - dx).norm() <= 2 ** -8 * dx.norm()


def test_clipping():
    n = (1 << 31) + 1001
    t = torch.zeros(n, dtype=BF16, device="cuda")
    t[5], t[1 << 30], t[n - 1], t[n - 40000] = 3.0, 4.0, 12.0, 84.0
    assert ops.grad_norm([t]).item() == 85.0
    assert ops.clip_grads([t[1:]], 42.5, eps=1e-30).item() == 85.0
    assert t[5] == 1.5 and t[1 << 30] == 2.0 and t[n - 1] == 6.0 and t[n - 40000] == 42.0
    assert t.count_nonzero() == 4

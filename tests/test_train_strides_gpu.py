"""The C entry points whose gradients may have rows further apart than they are wide, which the Python calls do not
use: the same bits as contiguous ones and nothing written between the rows.  Gathered rows of x that lie past 32 bits,
and none at all, in the backward pass of a feed-forward block."""
import ctypes

import pytest
import torch

from ops_util import offsets_of, randn
from sparse_moe_router_amd import ops

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
MARK = 7.0


def mat(t):
    return ops.MoeMat(t.data_ptr(), t.stride(0))


def ptr(t):
    return None if t is None else t.data_ptr()


def stream():
    return torch.cuda.current_stream().cuda_stream


def padded(rows, cols, dtype):
    """A matrix in columns 16.. of a wider one: (all of it, the matrix)."""
    a = torch.full((rows, cols + 40), MARK, dtype=dtype, device="cuda")
    return a, a[:, 16:16 + cols]


def untouched(a, cols):
    return bool((a[:, :16] == MARK).all() and (a[:, 16 + cols:] == MARK).all())


@pytest.mark.parametrize("dw", [BF16, F32])
@pytest.mark.parametrize("counts,I,K,H", [([4, 0, 5], 72, 136, 88), ([32], 40, 264, 72), ([70, 0, 130], 72, 264, 88),
                                          ([300, 40, 0, 200], 136, 520, 72), ([2100], 72, 136, 88)], ids=lambda v: str(v)[:16])
def test_feed_forward_gradient(counts, I, K, H, dw):
    R, E, k = sum(counts), len(counts), 2
    T = (R + k - 1) // k
    perm = torch.randperm(T * k, generator=torch.Generator().manual_seed(1))[:R].to(torch.int32).cuda()
    dy, x, gu, dn, pre = (v.cuda() for v in (randn(1, R, H), randn(2, T, K), randn(3, E, 2 * I, K, scale=0.2),
                                             randn(4, E, H, I, scale=0.2), randn(5, R, 2 * I)))
    off = offsets_of(counts).cuda()
    want = ops.feed_forward_grad(dy, x, gu, dn, pre, off, perm=perm, top_k=k, dw_dtype=dw)
    d = ops.MoeFeedForward(R, T, K, H, E, I, K, H, k, off.data_ptr(), perm.data_ptr())
    wk = torch.empty(ops.lib().moe_feed_forward_grad_workspace_size(ctypes.byref(d)), dtype=torch.uint8, device="cuda")
    a, dx = padded(R, K, BF16)
    dgu, dd = torch.empty(E, 2 * I, K, dtype=dw, device="cuda"), torch.empty(E, H, I, dtype=dw, device="cuda")
    st = ops.lib().moe_feed_forward_grad(ctypes.byref(d), ptr(dy), ptr(x), ptr(gu), ptr(dn), mat(pre), mat(dx), ptr(dgu),
                                         ptr(dd), int(dw == F32), ptr(wk), wk.numel(), stream())
    assert st == 0
    assert torch.equal(dx, want["x"]) and torch.equal(dgu, want["w_gate_up"]) and torch.equal(dd, want["w_down"])
    assert untouched(a, K)


@pytest.mark.parametrize("dx_type", [BF16, F32])
@pytest.mark.parametrize("T,V,H", [(300, 200, 72), (100, 200, 1032), (40, 120, 264), (2100, 1300, 2056),  # one slice
                                   (999, 9001, 520), (300, 20001, 72), (60, 5000, 264)])  # several
def test_cross_entropy_gradient(T, V, H, dx_type):
    x, w = randn(1, T, H).cuda(), randn(2, V, H, scale=2.0 / H ** 0.5).cuda()
    t = torch.randint(-1, V, (T,), generator=torch.Generator().manual_seed(3)).cuda()
    dl = (torch.rand(T, generator=torch.Generator().manual_seed(4)) - 0.2).cuda()
    lse = ops.cross_entropy(x, w, t)[1]
    want = ops.cross_entropy_grad(dl, x, w, t, lse, dx_dtype=dx_type, dw_dtype=F32)
    d = ops.MoeLoss(T, H, V, H, -100)
    wk = torch.empty(ops.lib().moe_cross_entropy_grad_workspace_size(ctypes.byref(d)), dtype=torch.uint8, device="cuda")
    for dw in (torch.empty(V, H, dtype=F32, device="cuda"), None):
        a, dx = padded(T, H, dx_type)
        st = ops.lib().moe_cross_entropy_grad(ctypes.byref(d), ptr(dl), ptr(x), ptr(w), ptr(t), ptr(lse), mat(dx),
                                              int(dx_type == F32), ptr(dw), 1, ptr(wk), wk.numel(), stream())
        assert st == 0
        assert torch.equal(dx, want["x"]) and (dw is None or torch.equal(dw, want["w"]))
        assert untouched(a, H)


@pytest.mark.parametrize("R", [9, 70000])
def test_feed_forward_gradient_of_rows_past_32_bits(R):
    """R grouped rows of 70000 tokens 2^15 elements apart (4.6 GB), gathered."""
    T, LD, I, K, H = 70000, 1 << 15, 16, 16, 8
    x, gu, dn = randn(1, T, K).cuda(), randn(2, 1, 2 * I, K).cuda(), randn(3, 1, H, I).cuda()
    dy, pre = randn(4, R, H).cuda(), randn(5, R, 2 * I).cuda()
    perm = torch.randperm(T, generator=torch.Generator().manual_seed(5))[:R].to(torch.int32).cuda()
    perm[0], perm[R // 2] = T - 1, -1
    want = ops.feed_forward_grad(dy, x, gu, dn, pre, None, perm=perm)
    wide = torch.full((T, LD), float("nan"), dtype=BF16, device="cuda")
    wide[:, 8:8 + K] = x
    got = ops.feed_forward_grad(dy, wide[:, 8:8 + K], gu, dn, pre, None, perm=perm)
    assert all(torch.equal(got[n], want[n]) for n in want)


@pytest.mark.parametrize("counts", [[3, 0, 2], [100, 0, 300]])
def test_no_row_of_x_at_all(counts):
    """Every entry of the permutation then stands for a row of zeros."""
    R, E, I, K, H = sum(counts), len(counts), 72, 136, 88
    off = offsets_of(counts).cuda()
    gu, dn = randn(3, E, 2 * I, K, scale=0.2).cuda(), randn(4, E, H, I, scale=0.2).cuda()
    perm = torch.arange(R, dtype=torch.int32, device="cuda")
    none, zeros = torch.empty(0, K, dtype=BF16, device="cuda"), torch.zeros(R, K, dtype=BF16, device="cuda")
    h, pre = ops.gated_matmul(none, gu, off, perm=perm, save=True)
    assert not h.any() and not pre.any()
    dy, pre = randn(1, R, H).cuda(), randn(5, R, 2 * I).cuda()
    a = ops.feed_forward_grad(dy, none, gu, dn, pre, off, perm=perm)
    b = ops.feed_forward_grad(dy, zeros, gu, dn, pre, off, perm=perm)
    assert all(torch.equal(a[n], b[n]) for n in a) and not a["w_gate_up"].any() and a["w_down"].any()

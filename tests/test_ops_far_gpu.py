"""Offsets past 32 bits: far rows of x, weights and results of more than 2^31 elements or 2^32 bytes."""
import pytest
import torch

from ops_util import EPS32, F8, close, eps_of, merge_ref, randn, rms, rms_grad, sum_terms
from sparse_moe_router_amd import ops

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("few", [True, False])
def test_rows_gathered_from_far_apart(few):
    """x of 2.2 GB (more than the range of one buffer descriptor), of which a permutation takes rows
    from both ends."""
    K, N, M = 2048, 72, 540_000
    R = 12 if few else 700
    src = torch.cat([torch.arange(R // 2), M - 1 - torch.arange(R - R // 2)])
    src = src[torch.randperm(R, generator=torch.Generator().manual_seed(1))]
    rows = randn(1, R, K)
    x = torch.zeros(M, K, dtype=BF16, device="cuda")
    x[src.cuda()] = rows.cuda()
    perm = src.to(torch.int32)
    perm[3] = -1
    rows[3] = 0
    off = torch.tensor([0, R // 3, R], dtype=torch.int32)
    w, dy = randn(2, 2, N, K), randn(3, R, N)
    y = ops.grouped_matmul(x, w.cuda(), off.cuda(), perm=perm.cuda())
    dw = ops.grouped_matmul_grad_weight(x, dy.cuda(), off.cuda(), perm=perm.cuda())
    for e in range(2):
        a, b = int(off[e]), int(off[e + 1])
        r, we, d = rows[a:b].to(F8), w[e].to(F8).t(), dy[a:b].to(F8).t()
        want = r @ we
        close(y[a:b], want, 2 * EPS32 * K * (r.abs() @ we.abs()) + eps_of(BF16) * want.abs(), "y")
        want = d @ r
        close(dw[e], want, 2 * EPS32 * (b - a) * (d.abs() @ r.abs()) + EPS32 * want.abs(), "dw")


def test_codes_gathered_from_far_apart():
    K, N, M, R = 2048, 40, 1_100_000, 600
    src = torch.cat([torch.arange(R // 2), M - 1 - torch.arange(R // 2)])
    g = torch.Generator().manual_seed(1)
    q = torch.randint(-127, 128, (R, K), generator=g, dtype=torch.int8)
    x = torch.zeros(M, K, dtype=torch.int8, device="cuda")
    x[src.cuda()] = q.cuda()
    xs, w, ws = torch.rand(M, device="cuda"), torch.randint(-127, 128, (N, K), generator=g, dtype=torch.int8), \
        torch.rand(N, generator=g)
    y = ops.grouped_matmul_i8(x, w.cuda().unsqueeze(0), ws.cuda().unsqueeze(0), None, perm=src.to(torch.int32).cuda(),
                              x_scale=xs, out_dtype=F32)
    want = (q.to(F8) @ w.to(F8).t()) * (xs.cpu()[src].to(F8)[:, None] * ws.to(F8))
    close(y, want, 6 * EPS32 * want.abs())


def test_weights_of_more_than_2_31_elements():
    """E N K = 2.2e9: the forward product by rows and by tiles, and the rows' gradient, whose reduction
    runs over N = 2^20."""
    E, N, K = 2, 1 << 20, 1032
    w = torch.empty(E, N, K, dtype=BF16, device="cuda")
    w.normal_(0, 1, generator=torch.Generator(device="cuda").manual_seed(1))
    cols = torch.tensor([0, 1, 255, 256, 524287, N - 9, N - 1])
    wc = w[:, cols.cuda()].cpu().to(F8)
    for R, off in ((5, [0, 2, 5]), (300, [0, 7, 300])):
        x = randn(2, R, K)
        y = ops.grouped_matmul(x.cuda(), w, torch.tensor(off, dtype=torch.int32).cuda())
        for e in range(E):
            r = x[off[e]:off[e + 1]].to(F8)
            want = r @ wc[e].t()
            close(y[off[e]:off[e + 1]][:, cols.cuda()], want,
                  2 * EPS32 * K * (r.abs() @ wc[e].t().abs()) + eps_of(BF16) * want.abs(), "y")
    R, off = 40, [0, 7, 40]
    dy = torch.zeros(R, N, dtype=BF16)
    dy[:, cols] = randn(3, R, len(cols))
    dx = ops.grouped_matmul_grad_input(dy.cuda(), w, torch.tensor(off, dtype=torch.int32).cuda(), out_dtype=F32)
    for e in range(E):
        d = dy[off[e]:off[e + 1]][:, cols].to(F8)
        want = d @ wc[e]
        # all but seven terms of a sum are exact zeros
        close(dx[off[e]:off[e + 1]], want, 2 * EPS32 * len(cols) * (d.abs() @ wc[e].abs()) + EPS32 * want.abs(), "dx")


def test_results_past_32_bits():
    """y of 2.3e9 elements (4.6 GB) and a weight gradient of the same size."""
    R, N, K = 70_000, 32_768, 8
    x, w = randn(1, R, K), randn(2, N, K)
    y = ops.grouped_matmul(x.cuda(), w.cuda().unsqueeze(0), None)
    rows, cols = torch.tensor([0, 255, 256, R // 2, R - 1]), torch.tensor([0, 8, 511, N - 1])
    want = x[rows].to(F8) @ w[cols].to(F8).t()
    mag = x[rows].to(F8).abs() @ w[cols].to(F8).t().abs()
    close(y[rows.cuda()][:, cols.cuda()], want, 2 * EPS32 * K * mag + eps_of(BF16) * want.abs(), "y")
    del y
    E, N, K, R = 64, 2048, 16384, 128
    x, dy = randn(3, R, K), randn(4, R, N)
    off = torch.arange(0, 2 * E + 1, 2, dtype=torch.int32)
    dw = ops.grouped_matmul_grad_weight(x.cuda(), dy.cuda(), off.cuda(), out_dtype=BF16)
    for e in (0, 1, 40, E - 1):
        d, r = dy[2 * e:2 * e + 2].to(F8).t(), x[2 * e:2 * e + 2].to(F8)
        want = d @ r
        close(dw[e], want, 2 * EPS32 * 2 * (d.abs() @ r.abs()) + eps_of(BF16) * want.abs(), f"dw {e}")


def test_norms_past_32_bits():
    M, H = 1_100_000, 2048
    x = torch.empty(M, H, dtype=BF16, device="cuda").normal_(0, 1, generator=torch.Generator(device="cuda").manual_seed(1))
    w = (randn(2, H, scale=0.1) + 1).cuda()
    h = ops.block_norm(x, w, 1e-6)
    out = ops.block_merge(x, h, w, 1e-6, scale=0.5)
    rows = torch.tensor([0, 1, 524_287, 524_288, 1_048_575, 1_048_576, M - 1]).cuda()
    # (a call of these rows alone sums in another order: the row's threads go by the number of rows)
    xr, hr, wr = (t.cpu().to(F8) for t in (x[rows], h[rows], w))
    want = rms(xr, wr, 1e-6)
    close(h[rows], want, (sum_terms(H) * EPS32 + eps_of(BF16)) * want.abs(), "h")
    want = merge_ref(xr, hr, wr, 1e-6, None, 0.5)
    close(out[rows], want, sum_terms(H) * EPS32 * (want - xr).abs() + (EPS32 + eps_of(BF16)) * want.abs(), "out")
    del out
    g = ops.block_norm_grad(h, x, w, 1e-6)
    dv, mag, _ = rms_grad(hr, xr, wr, 1e-6)
    close(g["x"][rows], dv, 3 * sum_terms(H) * EPS32 * mag + eps_of(BF16) * dv.abs(), "dx")

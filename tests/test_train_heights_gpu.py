"""Row tiles of every height: low ones, where all tiles run at a time, and 256 rows with shorter last ones, where
they do not; of one group and of several, gathered or not, for each product that they serve."""
import pytest
import torch

import train_util as U
from ops_util import EPS32, F8, close, eps_of, grad_input_ref, grouped_ref, offsets_of, randn, source_rows, take
from sparse_moe_router_amd import ops

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
COUNTS = [200, 100, 150, 0, 300, 20, 64, 65, 1, 511] * 3  # 30 groups, 4233 rows: 96, 63 and 46 tiles of 64, 128 and 256
# columns: of 256 each 2, 4 and 6 panels: tiles of 64, 128 and 256 rows
WIDTHS = [512, 1000, 1504]
# rows of one group and columns: heights of 64, 128, 192 and 256 rows, evenly shared
ONE = [(65, 40), (300, 4000), (300, 20008), (300, 32008), (570, 16008), (100, 40008), (160, 40008), (250, 40008),
       (300, 33008), (700, 30008)]


def gathered(rows, gather):
    if not gather:
        return rows, None, 1
    tokens = (rows + 2) // 3
    return tokens, torch.randperm(tokens * 3, generator=torch.Generator().manual_seed(7))[:rows].to(torch.int32), 3


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("N", WIDTHS)
def test_grouped(N, gather):
    R, E, K = sum(COUNTS), len(COUNTS), 72
    T, perm, k = gathered(R, gather)
    off, x, w = offsets_of(COUNTS), randn(1, T, K), randn(2, E, N, K)
    y, tol = grouped_ref(take(x, source_rows(R, perm, k, T)), w, off)
    got = ops.grouped_matmul(x.cuda(), w.cuda(), off.cuda(), perm=None if perm is None else perm.cuda(), top_k=k)
    close(got, y, tol + eps_of(BF16) * (y.abs() + tol))
    if gather:
        return
    dy, w = randn(3, R, K), randn(4, E, K, N)
    y, tol = grad_input_ref(dy, w, off)
    close(ops.grouped_matmul_grad_input(dy.cuda(), w.cuda(), off.cuda(), out_dtype=F32), y, tol + EPS32 * (y.abs() + tol))


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("N", WIDTHS)
def test_grouped_i8(N, gather):
    R, E, K = sum(COUNTS), len(COUNTS), 80
    T, perm, k = gathered(R, gather)
    g = torch.Generator().manual_seed(5)
    x, w = (torch.randint(-127, 128, s, generator=g, dtype=torch.int8) for s in ((T, K), (E, N, K)))
    xs, ws = torch.rand(T, generator=g) + 0.1, torch.rand(E, N, generator=g) + 0.1
    off, src = offsets_of(COUNTS), source_rows(R, perm, k, T)
    y = torch.cat([(x.to(F8)[src[a:b]] @ w[e].to(F8).t()) * (xs.to(F8)[src[a:b], None] * ws[e].to(F8))
                   for e, (a, b) in enumerate(zip(off[:-1].tolist(), off[1:].tolist()))])
    got = ops.grouped_matmul_i8(x.cuda(), w.cuda(), ws.cuda(), off.cuda(), perm=None if perm is None else perm.cuda(), top_k=k,
                                x_scale=xs.cuda(), out_dtype=F32)
    close(got, y, 5 * EPS32 * y.abs())  # the sum is exact; its conversion, two scales and two products round


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("I", [256, 500 // 8 * 8, 760])  # 128 columns a panel
def test_gated(I, gather):
    R, E, K = sum(COUNTS), len(COUNTS), 72
    T, perm, k = gathered(R, gather)
    off, x, w = offsets_of(COUNTS), randn(1, T, K), randn(2, E, 2 * I, K, scale=1.5 / K ** 0.5)
    (h, th), (pre, tp) = U.gated_ref(take(x, source_rows(R, perm, k, T)), w, off)
    a, b = ops.gated_matmul(x.cuda(), w.cuda(), off.cuda(), perm=None if perm is None else perm.cuda(), top_k=k, save=True)
    close(a, h, th, "h")
    close(b, pre, tp, "gate_up")


@pytest.mark.parametrize("I", WIDTHS)
def test_gated_gradient(I):
    R, E, H = sum(COUNTS), len(COUNTS), 40
    off, dy, wd, pre = offsets_of(COUNTS), randn(1, R, H), randn(2, E, H, I, scale=0.2), randn(3, R, 2 * I)
    (d, td), (h, th) = U.gated_grad_ref(dy, wd, pre, off)
    g = ops.gated_matmul_grad(dy.cuda(), wd.cuda(), pre.cuda(), off.cuda())
    close(g["gate_up"], d, td)
    close(g["h"], h, th)


@pytest.mark.parametrize("R,N", ONE)
def test_one_group(R, N):
    K = 24
    x, w = randn(1, R, K), randn(2, 1, N, K)
    y, tol = grouped_ref(x.to(F8), w, [0, R])
    close(ops.grouped_matmul(x.cuda(), w.cuda(), None), y, tol + eps_of(BF16) * (y.abs() + tol))
    close(ops.grouped_matmul(x.cuda(), w.cuda(), offsets_of([R]).cuda()), y, tol + eps_of(BF16) * (y.abs() + tol))


@pytest.mark.parametrize("R", [90, 300, 700, 1000, 1100])  # 64 panels: 128, 128, 192, 256 rows, evenly shared, and 256 + rest
def test_one_group_rows_gradient(R):
    N, K = 16, 16384
    dy, w = randn(1, R, N), randn(2, 1, N, K)
    y, tol = grad_input_ref(dy, w, [0, R])
    close(ops.grouped_matmul_grad_input(dy.cuda(), w.cuda(), None), y, tol + eps_of(BF16) * (y.abs() + tol))


@pytest.mark.parametrize("T,V", [(100, 40001), (160, 40001), (250, 40007), (300, 33003), (300, 20003), (570, 16001), (200, 2801),
                                 (64, 4096), (64, 4097)])
def test_loss(T, V):
    H = 24
    x, w = randn(1, T, H), randn(2, V, H, scale=2.0 / H ** 0.5)
    t = torch.randint(0, V, (T,), generator=torch.Generator().manual_seed(3))
    t[0], t[1], t[2] = V - 1, -100, 0
    loss, tol, lse, tl, *_ = U.loss_ref(x, w, t)
    dl = torch.rand(T, generator=torch.Generator().manual_seed(9)) - 0.2
    c = [v.cuda() for v in (dl, x, w, t)]
    a, b = ops.cross_entropy(*c[1:])
    close(a, loss, tol, "loss")
    close(b, lse, tl, "lse")
    (dx, tx), (dw, tw) = U.loss_grad_ref(dl, x, w, t)
    g = ops.cross_entropy_grad(*c, b, dx_dtype=F32, dw_dtype=F32)
    close(g["x"], dx, tx + EPS32 * dx.abs(), "x")
    close(g["w"], dw, tw + EPS32 * dw.abs(), "w")

"""Gated products and their backward pass against 64 bits: both kernels, every tile height, odd sizes,
strided rows, empty groups, rows behind the last group, entries of the permutation that are out of range."""
import pytest
import torch

import train_util as U
from ops_util import F8, close, eps_of, grad_input_ref, grad_weight_ref, grouped_ref, offsets_of, randn, source_rows, take
from sparse_moe_router_amd import ops

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32

# counts of the groups, features, K
FORWARD = [
    ([1], 8, 8), ([1], 512, 2048), ([0, 3, 0, 1], 24, 72), ([5] * 16, 40, 136),  # few rows
    ([256], 128, 64), ([257, 0, 64, 65, 1], 136, 200), ([130, 193, 700], 264, 1032), ([33] * 40, 64, 128),
    ([0] * 7 + [300], 1000, 88), ([90] * 70, 128, 64), ([512, 511], 120, 16),
]


def inputs(counts, I, K, gather, seed=0):
    R, E = sum(counts), len(counts)
    k = 3 if gather else 1
    T = (R + k - 1) // k if gather else R
    perm = torch.randperm(T * k, generator=torch.Generator().manual_seed(seed))[:R].to(torch.int32) if gather else None
    return randn(seed + 1, T, K), randn(seed + 2, E, 2 * I, K, scale=1.5 / K ** 0.5), offsets_of(counts), perm, k


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("counts,I,K", FORWARD, ids=lambda v: str(v)[:24])
def test_forward(counts, I, K, gather):
    x, w, off, perm, k = inputs(counts, I, K, gather)
    rows = take(x, source_rows(sum(counts), perm, k, x.shape[0]))
    (h, th), (pre, tp) = U.gated_ref(rows, w, off)
    args = (x.cuda(), w.cuda(), off.cuda())
    kw = dict(perm=None if perm is None else perm.cuda(), top_k=k)
    got = ops.gated_matmul(*args, **kw)
    close(got, h, th, "h")
    h2, p2 = ops.gated_matmul(*args, save=True, **kw)
    close(p2, pre, tp, "gate_up")
    assert torch.equal(h2, got), "keeping the products changes nothing"
    assert torch.equal(ops.gated_matmul(*args, **kw), got), "the same bits again"


@pytest.mark.parametrize("rows", [3, 300])
def test_strided_rows_and_given_outputs(rows):
    I, K = 72, 136
    wide = randn(5, rows, K + 64).cuda()
    x, w = wide[:, 32:32 + K], randn(6, 1, 2 * I, K, scale=0.1)
    out = torch.full((rows, I + 24), 7.0, dtype=BF16, device="cuda")
    pre = torch.full((rows, 2 * I + 8), 7.0, dtype=BF16, device="cuda")
    (h, th), (p, tp) = U.gated_ref(x.cpu().to(F8), w, offsets_of([rows]))
    a, b = ops.gated_matmul(x, w.cuda(), None, save=True, out=out[:, 8:8 + I], gate_up=pre[:, :2 * I])
    close(a, h, th)
    close(b, p, tp)
    assert (out[:, :8] == 7).all() and (out[:, 8 + I:] == 7).all() and (pre[:, 2 * I:] == 7).all()


@pytest.mark.parametrize("rows,E", [(7, 3), (400, 3)])
def test_rows_behind_the_last_group_and_bad_permutations(rows, E):
    I, K, k = 64, 128, 2
    counts = [rows // 4, 0, rows // 3]
    end = sum(counts)
    x, w = randn(1, rows, K), randn(2, E, 2 * I, K, scale=0.1)
    perm = torch.randint(0, rows * k, (rows,), generator=torch.Generator().manual_seed(3)).to(torch.int32)
    perm[0], perm[1] = -1, rows * k  # rows of zeros
    off = offsets_of(counts)
    out = torch.full((rows, I), 5.0, dtype=BF16, device="cuda")
    pre = torch.full((rows, 2 * I), 5.0, dtype=BF16, device="cuda")
    ops.gated_matmul(x.cuda(), w.cuda(), off.cuda(), perm=perm.cuda(), top_k=k, save=True, out=out, gate_up=pre)
    (h, th), (p, tp) = U.gated_ref(take(x, source_rows(rows, perm, k, rows)), w, off)
    close(out[:end], h[:end], th[:end])
    close(pre[:end], p[:end], tp[:end])
    assert not out[:2].any() and (out[end:] == 5).all() and (pre[end:] == 5).all()
    # the gradient leaves them too
    dy, wd = randn(4, rows, 72), randn(5, E, 72, I, scale=0.1)
    gu = randn(6, rows, 2 * I)
    gu[end:] = float("nan")
    g = ops.gated_matmul_grad(dy.cuda(), wd.cuda(), gu.cuda(), off.cuda())
    (d, td), (h, th) = U.gated_grad_ref(dy, wd, gu, off)
    close(g["gate_up"][:end], d[:end], td[:end])
    close(g["h"][:end], h[:end], th[:end])


def test_offsets_out_of_range_stay_in_bounds():
    x, w = randn(1, 40, 64).cuda(), randn(2, 3, 32, 64, scale=0.1).cuda()
    for o in ([-5, 10, 1000, 20], [0, 40, 30, 90], [50, 60, 70, 80]):
        ops.gated_matmul(x, w, torch.tensor(o, dtype=torch.int32, device="cuda"))
        ops.gated_matmul_grad(x, randn(3, 3, 64, 16, scale=0.1).cuda(), randn(4, 40, 32).cuda(),
                              torch.tensor(o, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()


@pytest.mark.parametrize("counts,N,I", [([1], 8, 8), ([3, 0, 61], 72, 40), ([200, 70], 136, 264), ([256, 1, 500], 64, 128),
                                        ([130] * 66, 32, 16), ([0, 0], 16, 16)], ids=lambda v: str(v)[:24])
def test_gradient(counts, N, I):
    R, E = sum(counts), len(counts)
    dy, w, off = randn(1, R, N), randn(2, E, N, I, scale=0.2), offsets_of(counts)
    gu = randn(3, R, 2 * I, scale=2.0)
    if R > 2:
        gu[1, :I] = torch.linspace(-90, 90, I).to(BF16)  # far on both sides
        gu[2] = 0
    (d, td), (h, th) = U.gated_grad_ref(dy, w, gu, off)
    g = ops.gated_matmul_grad(dy.cuda(), w.cuda(), gu.cuda(), off.cuda())
    close(g["gate_up"], d, td, "gate_up")
    close(g["h"], h, th, "h")


def test_infinities_and_nan_stay_in_their_rows():
    x, w = randn(1, 300, 64), randn(2, 1, 64, 64, scale=0.2)
    x[7, 3], x[201, 5] = float("nan"), float("inf")
    clean = torch.ones(300, dtype=torch.bool)
    clean[7] = clean[201] = False
    for rows in (10, 300):
        h = ops.gated_matmul(x[:rows].cuda(), w.cuda(), None).cpu()
        c = clean[:rows]
        assert torch.isnan(h[7]).all() and torch.isfinite(h[c]).all()
        if rows > 201:
            assert not torch.isfinite(h[201]).all()


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("dw", [BF16, F32])
@pytest.mark.parametrize("counts,I,K,H", [([70, 0, 261, 5, 1], 72, 136, 136), ([3001], 40, 72, 24), ([1500, 0, 700], 264, 40, 72),
                                          ([520] * 20, 16, 264, 8), ([9000], 8, 8, 264)], ids=lambda v: str(v)[:24])
def test_block_and_its_gradients(gather, dw, counts, I, K, H):
    """Each kernel of the block against 64 bits on the values that the kernels before it stored; few experts with
    long groups, whose weight gradients are summed in parts, among them."""
    x, w, off, perm, k = inputs(counts, I, K, gather)
    R, E = sum(counts), len(counts)
    wd, dy = randn(8, E, H, I, scale=0.1), randn(9, R, H)
    ffn = ops.MoeFeedForward(R, x.shape[0], K, H, E, I, K, H, k, 1 << 20, 1 << 24 if gather else None)
    parts = ops.lib().moe_feed_forward_grad_workspace_size(ffn) - sum((n + 255) // 256 * 256 for n in (R * 4 * I, R * 2 * I))
    assert (parts > 0) == (R >= 512 * E)
    c = lambda t: None if t is None else t.cuda()
    y, gu = ops.feed_forward(c(x), c(w), c(wd), c(off), perm=c(perm), top_k=k, save=True)
    assert torch.equal(y, ops.feed_forward(c(x), c(w), c(wd), c(off), perm=c(perm), top_k=k))
    h = ops.gated_matmul(c(x), c(w), c(off), perm=c(perm), top_k=k).cpu().to(F8)
    want, t = grouped_ref(h, wd, off)
    close(y, want, t + eps_of(BF16) * want.abs())
    g = ops.feed_forward_grad(c(dy), c(x), c(w), c(wd), gu, c(off), perm=c(perm), top_k=k, dw_dtype=dw)
    m = ops.gated_matmul_grad(c(dy), c(wd), gu, c(off))
    d, h = m["gate_up"].cpu(), m["h"].cpu()
    dx, t = grad_input_ref(d, w, off)
    close(g["x"], dx, t + eps_of(BF16) * dx.abs(), "x")
    rows = take(x, source_rows(R, perm, k, x.shape[0]))
    for name, a, b in (("w_gate_up", rows, d), ("w_down", h.to(F8), dy)):
        v, t = grad_weight_ref(a, b, off)
        assert g[name].dtype == dw
        close(g[name], v, t + eps_of(dw) * v.abs(), name)


def test_refuses():
    x, w, o = randn(1, 8, 64).cuda(), randn(2, 2, 64, 64).cuda(), offsets_of([4, 4]).cuda()
    with pytest.raises(ValueError, match="two matrices"):
        ops.gated_matmul(x, w[:, :63].contiguous(), o)
    with pytest.raises(ValueError, match="contiguous"):
        ops.gated_matmul(x, w[:, :32], o)
    with pytest.raises(ValueError, match="save"):
        ops.gated_matmul(x, w, o, gate_up=torch.empty(8, 64, dtype=BF16, device="cuda"))
    with pytest.raises(ValueError, match="gate_up"):
        ops.gated_matmul_grad(x, w, torch.empty(8, 64, dtype=BF16, device="cuda"), o)
    with pytest.raises(ValueError, match="offsets"):
        ops.gated_matmul(x, w, None)
    with pytest.raises(TypeError):
        ops.gated_matmul(x, w, o, out=torch.empty(8, 32, device="cuda"))
    with pytest.raises(ops.MoeError):
        ops.gated_matmul(x, randn(2, 2, 24, 64).cuda(), o)  # 12 features
    with pytest.raises(ops.MoeError):
        ops.gated_matmul(x, w, o, out=x[:, :32])
    with pytest.warns(UserWarning, match="requires a gradient"):
        ops.gated_matmul(x.clone().requires_grad_(), w, o)

"""Cross entropy against a vocabulary and its gradients, against 64 bits: every tile height, vocabularies that
end inside a tile and a chunk, several pieces and slices, targets at the borders and none."""
import pytest
import torch

import train_util as U
from ops_util import EPS32, F8, close, eps_of, randn
from sparse_moe_router_amd import ops

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
SHAPES = [(1, 1, 8), (1, 300, 64), (3, 7, 16), (64, 257, 72), (65, 1000, 136), (129, 4099, 64), (200, 255, 264),
          (300, 513, 128), (257, 2049, 1032), (5, 70001, 16), (3001, 300, 264), (700, 4099, 16),
          # by tiles of every height
          (1, 11500, 16), (60, 11300, 8), (100, 6001, 24), (180, 4099, 72), (300, 2500, 40)]


def inputs(T, V, H, scale=2.0, seed=0):
    x, w = randn(seed, T, H), randn(seed + 1, V, H, scale=scale / H ** 0.5)
    t = torch.randint(0, V, (T,), generator=torch.Generator().manual_seed(seed + 2))
    t[0] = V - 1
    if T > 2:
        t[1], t[2] = 0, -100
    if T > 20:
        t[10], t[11], t[12] = V, -1, 1 << 40
    return x, w, t


@pytest.mark.parametrize("T,V,H", SHAPES)
def test_loss(T, V, H):
    x, w, t = inputs(T, V, H)
    loss, tol, lse, tl, *_ = U.loss_ref(x, w, t)
    a, b = ops.cross_entropy(x.cuda(), w.cuda(), t.cuda())
    close(a, loss, tol, "loss")
    close(b, lse, tl, "lse")
    c, d = ops.cross_entropy(x.cuda(), w.cuda(), t.cuda())
    assert torch.equal(a, c) and torch.equal(b, d)


@pytest.mark.parametrize("T,V,H", SHAPES)
def test_gradients(T, V, H):
    x, w, t = inputs(T, V, H)
    dl = torch.rand(T, generator=torch.Generator().manual_seed(9)) - 0.2
    (dx, tx), (dw, tw) = U.loss_grad_ref(dl, x, w, t)
    c = [v.cuda() for v in (dl, x, w, t)]
    lse = ops.cross_entropy(*c[1:])[1]
    for dt in (BF16, F32):
        g = ops.cross_entropy_grad(*c, lse, dx_dtype=dt, dw_dtype=dt)
        close(g["x"], dx, tx + eps_of(dt) * (dx.abs() + tx), "x")
        close(g["w"], dw, tw + eps_of(dt) * (dw.abs() + tw), "w")
    # one of the two alone
    a, b = (ops.cross_entropy_grad(*c, lse, dx_dtype=p, dw_dtype=q) for p, q in ((F32, None), (None, F32)))
    assert list(a) == ["x"] and list(b) == ["w"] and torch.equal(a["x"], g["x"]) and torch.equal(b["w"], g["w"])


def test_several_pieces():
    """Tokens enough that the vocabulary takes several pieces, the last one short."""
    T, V, H = 40000, 4099, 16
    x, w, t = inputs(T, V, H)
    assert ops.lib().moe_cross_entropy_grad_workspace_size(ops.MoeLoss(T, H, V, H, -100)) < T * V * 2
    dl = torch.rand(T, generator=torch.Generator().manual_seed(9)) / T
    c = [v.cuda() for v in (dl, x, w, t)]  # the reference too: 64 bits of 40000 x 4099 logits
    loss, lse = ops.cross_entropy(*c[1:])
    ref = U.loss_ref(*c[1:])
    close(loss, ref[0].cpu(), ref[1].cpu())
    del ref
    (dx, tx), (dw, tw) = ((v.cpu() for v in p) for p in U.loss_grad_ref(*c))
    g = ops.cross_entropy_grad(*c, lse, dx_dtype=F32, dw_dtype=F32)
    close(g["x"], dx, tx + EPS32 * dx.abs(), "x")
    close(g["w"], dw, tw + EPS32 * dw.abs(), "w")


@pytest.mark.parametrize("c", [1 / 999, 1.0039, -3e-5])
def test_a_common_weight_is_not_rounded(c):
    """A d_loss that all tokens share (a mean's 1 / n) scales the gradients: nothing but fp32 products of the
    results is rounded by it, though bf16 holds none of these values."""
    T, V, H = 300, 513, 128
    x, w, t = (v.cuda() for v in inputs(T, V, H))
    lse = ops.cross_entropy(x, w, t)[1]
    one, other = (ops.cross_entropy_grad(torch.full((T,), v, device="cuda"), x, w, t, lse, dx_dtype=F32, dw_dtype=F32)
                  for v in (1.0, c))
    c32 = torch.tensor(c, dtype=F32).to(F8)
    for k in ("x", "w"):
        want = one[k].cpu().to(F8) * c32
        close(other[k], want, 2 * EPS32 * want.abs(), k)


@pytest.mark.parametrize("ignore", [-100, 3, 0])
def test_ignored_tokens(ignore):
    """Tokens without a target have no part, whatever their logits are."""
    x, w, t = inputs(80, 300, 64)
    t[5:9] = ignore
    x[6] = float("nan")
    valid = (t >= 0) & (t < 300) & (t != ignore)
    loss, lse = ops.cross_entropy(x.cuda(), w.cuda(), t.cuda(), ignore_index=ignore)
    assert not loss.cpu()[~valid].any() and torch.isfinite(loss).all()
    clean = x.clone()
    clean[6] = 0
    ref = U.loss_ref(clean, w, t, ignore)
    close(loss, ref[0], ref[1])
    x[6] = 0  # 0 x NaN of its row would reach dw through the product itself
    lse[6] = float("nan")
    dl = torch.ones(80)
    g = ops.cross_entropy_grad(dl.cuda(), x.cuda(), w.cuda(), t.cuda(), lse, ignore_index=ignore, dx_dtype=F32, dw_dtype=F32)
    (dx, tx), (dw, tw) = U.loss_grad_ref(dl, x, w, t, ignore)
    close(g["x"], dx, tx + EPS32 * dx.abs())
    close(g["w"], dw, tw + EPS32 * dw.abs())
    assert not g["x"].cpu()[~valid].any()


def test_sharp_and_far_logits():
    """One logit far above the others, logits of some hundreds, and equal ones."""
    T, V, H = 70, 1000, 64
    x, w, t = inputs(T, V, H, scale=40.0)
    x[1] = 0
    w[17] = 0
    loss, tol, lse, tl, *_ = U.loss_ref(x, w, t)
    a, b = ops.cross_entropy(x.cuda(), w.cuda(), t.cuda())
    close(a, loss, tol)
    close(b, lse, tl)
    assert lse.max() > 80
    dl = torch.ones(T)
    (dx, tx), (dw, tw) = U.loss_grad_ref(dl, x, w, t)
    g = ops.cross_entropy_grad(dl.cuda(), x.cuda(), w.cuda(), t.cuda(), b, dx_dtype=F32, dw_dtype=F32)
    close(g["x"], dx, tx + EPS32 * dx.abs())
    close(g["w"], dw, tw + EPS32 * dw.abs())


def test_rows_with_nan_and_infinity_stay_apart():
    x, w, t = inputs(300, 700, 64)
    x[20] = float("nan")
    x[290, 3] = float("inf")
    loss, lse = (v.cpu() for v in ops.cross_entropy(x.cuda(), w.cuda(), t.cuda()))
    rest = torch.ones(300, dtype=torch.bool)
    rest[20] = rest[290] = False
    assert torch.isnan(lse[20]) and not torch.isfinite(lse[290]) and torch.isfinite(lse[rest]).all()
    ref = U.loss_ref(x[rest], w, t[rest])
    close(loss[rest], ref[0], ref[1])


def test_strided_rows():
    x, w, t = inputs(100, 300, 64)
    wide = torch.zeros(100, 128, dtype=BF16, device="cuda")
    wide[:, 32:96] = x.cuda()
    s = wide[:, 32:96]
    a, b = ops.cross_entropy(x.cuda(), w.cuda(), t.cuda()), ops.cross_entropy(s, w.cuda(), t.cuda())
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    dl = torch.ones(100, device="cuda")
    g, h = (ops.cross_entropy_grad(dl, v, w.cuda(), t.cuda(), a[1]) for v in (x.cuda(), s))
    assert torch.equal(g["x"], h["x"]) and torch.equal(g["w"], h["w"])


def test_no_tokens():
    w = randn(1, 300, 64).cuda()
    x, t, f = torch.empty(0, 64, dtype=BF16, device="cuda"), torch.empty(0, dtype=torch.int64, device="cuda"), \
        torch.empty(0, device="cuda")
    loss, lse = ops.cross_entropy(x, w, t)
    assert loss.shape == lse.shape == (0,)
    g = ops.cross_entropy_grad(f, x, w, t, f)
    assert g["x"].shape == (0, 64) and g["w"].shape == (300, 64) and not g["w"].any()


def test_refuses():
    x, w, t = (v.cuda() for v in inputs(10, 300, 64))
    f = torch.ones(10, device="cuda")
    for call in (lambda: ops.cross_entropy(x, w, t[:9]), lambda: ops.cross_entropy(x[:, :56], w, t),
                 lambda: ops.cross_entropy(x, w[:, :56], t), lambda: ops.cross_entropy(x, w.t(), t),
                 lambda: ops.cross_entropy_grad(f[:9], x, w, t, f), lambda: ops.cross_entropy_grad(f, x, w, t, f[:, None])):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: ops.cross_entropy(x.float(), w, t), lambda: ops.cross_entropy(x, w, t.int()),
                 lambda: ops.cross_entropy(x, w, t, ignore_index=1.5),
                 lambda: ops.cross_entropy_grad(f.double(), x, w, t, f)):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: ops.cross_entropy(x[:, :60].contiguous(), w[:, :60].contiguous(), t),
                 lambda: ops.cross_entropy(x, w[:0], t), lambda: ops.cross_entropy_grad(f, x, w, t, f, dx_dtype=None, dw_dtype=None),
                 lambda: ops.cross_entropy(x, w, t, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(ops.MoeError):
            call()
    with pytest.warns(UserWarning, match="requires a gradient"):
        ops.cross_entropy(x.clone().requires_grad_(), w, t)


@pytest.mark.parametrize("T,V,H,least", [(999, 9001, 520, 9), (300, 20001, 72, 16), (2100, 1300, 2056, 1)])
def test_slices_of_the_rows_gradient(T, V, H, least):
    """Few and many slices of dx (the workspace holds them), with and without dw."""
    x, w, t = inputs(T, V, H)
    assert ops.lib().moe_cross_entropy_grad_workspace_size(ops.MoeLoss(T, H, V, H, -100)) >= T * V * 2 + least * T * H * 4
    dl = torch.rand(T, generator=torch.Generator().manual_seed(9)) - 0.2
    c = [v.cuda() for v in (dl, x, w, t)]
    (dx, tx), (dw, tw) = ((v.cpu() for v in p) for p in U.loss_grad_ref(*c))
    lse = ops.cross_entropy(*c[1:])[1]
    for g in (ops.cross_entropy_grad(*c, lse, dx_dtype=F32, dw_dtype=F32),
              ops.cross_entropy_grad(*c, lse, dx_dtype=F32, dw_dtype=None),
              ops.cross_entropy_grad(*c, lse, dx_dtype=None, dw_dtype=F32)):
        if "x" in g:
            close(g["x"], dx, tx + EPS32 * dx.abs(), "x")
        if "w" in g:
            close(g["w"], dw, tw + EPS32 * dw.abs(), "w")

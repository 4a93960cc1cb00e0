"""The plain forms of the training operators against differences and automatic differentiation (CPU)."""
import torch

import train_util as U
from ops_util import F8, offsets_of, randn


def differences(f, x, eps=1e-6):
    g = torch.zeros_like(x)
    flat, out = x.view(-1), g.view(-1)
    for i in range(flat.numel()):
        v = flat[i].item()
        flat[i] = v + eps
        a = f()
        flat[i] = v - eps
        out[i] = (a - f()) / (2 * eps)
        flat[i] = v
    return g


def test_gated_gradient_is_the_derivative():
    off = offsets_of([2, 0, 3])
    g = torch.Generator().manual_seed(0)
    pre = torch.randn(5, 8, generator=g, dtype=F8)
    w, dy = torch.randn(3, 6, 4, generator=g, dtype=F8), torch.randn(5, 6, generator=g, dtype=F8)
    (d, _), (h, _) = U.gated_grad_ref(dy, w, pre, off)

    def total():
        t = 0.0
        for e in range(3):
            a, b = int(off[e]), int(off[e + 1])
            t += ((U.silu(pre[a:b, :4]) * pre[a:b, 4:]) @ w[e].t() * dy[a:b]).sum().item()
        return t
    assert torch.allclose(d, differences(total, pre), atol=1e-7)
    assert torch.allclose(h, U.silu(pre[:, :4]) * pre[:, 4:])


def test_loss_gradient_is_the_derivative():
    g = torch.Generator().manual_seed(1)
    x, w = torch.randn(6, 8, generator=g, dtype=F8), torch.randn(11, 8, generator=g, dtype=F8)
    t = torch.tensor([0, 10, 5, -100, 11, 3])
    dl = torch.randn(6, generator=g, dtype=F8)
    (dx, _), (dw, _) = U.loss_grad_ref(dl, x, w, t, ignore=3)
    total = lambda: (U.loss_ref(x, w, t, ignore=3)[0] * dl).sum().item()
    assert torch.allclose(dx, differences(total, x), atol=1e-7)
    assert torch.allclose(dw, differences(total, w), atol=1e-7)
    loss, valid = U.loss_ref(x, w, t, ignore=3)[0], torch.tensor([1, 1, 1, 0, 0, 0]).bool()
    want = torch.nn.functional.cross_entropy(x @ w.t(), torch.where(valid, t, -100), reduction="none")
    assert torch.allclose(loss, want) and not loss[~valid].any()


def test_combine_is_a_weighted_sum():
    perm = torch.tensor([4, 1, 7, 0, 9, 3], dtype=torch.int32)  # 4 tokens x 2, one entry out of range
    inv = U.invert_ref(perm, 8, 6)
    assert inv.tolist() == [3, 1, -1, 5, 0, -1, -1, 2]
    assert U.invert_ref(torch.tensor([2, 2, 0]), 3, 2).tolist() == [-1, -1, 0]
    y, w = randn(0, 6, 8), torch.rand(4, 2)
    out, _ = U.combine_ref(y, inv, 2, w)
    want = torch.zeros(4, 8, dtype=F8)
    for p, a in enumerate(perm.tolist()):
        if a < 8:
            want[a // 2] += w.view(-1)[a].double() * y[p].double()
    assert torch.allclose(out, want)

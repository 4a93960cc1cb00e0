"""Tokens without a target whose rows hold NaN and infinities: their loss is 0, they have no part in any gradient and
the other tokens' values are as if the rows were zeros.  Sizes on both sides of the rule of the logits' kernel and of
the number of tokens up to which every workgroup finds the largest d_loss itself (2048), d_loss alike and not."""
import pytest
import torch

import train_util as U
from ops_util import EPS32, close, randn
from sparse_moe_router_amd import ops

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("mean", [False, True])
@pytest.mark.parametrize("T,V,H", [(80, 300, 64), (300, 1003, 136), (700, 2500, 72), (2100, 70, 64), (2500, 1009, 64)])
def test_rows_of_ignored_tokens(T, V, H, mean):
    x, w = randn(1, T, H), randn(2, V, H, scale=2.0 / H ** 0.5)
    t = torch.randint(0, V, (T,), generator=torch.Generator().manual_seed(3))
    bad = [0, 5, 63, 64, T // 2, T - 1]
    for i, r in enumerate(bad):
        t[r] = (-100, V, -1)[i % 3]  # the ignored index, and targets outside of the vocabulary
        x[r] = float("nan")
    x[bad[1]], x[bad[2], 3], x[bad[3], 1] = float("inf"), float("-inf"), float("inf")
    clean = x.clone()
    clean[bad] = 0
    dl = torch.full((T,), 1.0 / T) if mean else torch.rand(T, generator=torch.Generator().manual_seed(4)) - 0.3
    dl[bad[0]], dl[bad[1]] = float("nan"), float("inf")  # of no token that counts
    c = [v.cuda() for v in (dl, x, w, t)]
    loss, lse = ops.cross_entropy(*c[1:])
    ref = U.loss_ref(clean, w, t)
    close(loss, ref[0], ref[1])
    rest = ref[6]
    assert not loss.cpu()[bad].any() and not torch.isfinite(lse.cpu()[bad]).any()
    close(lse.cpu()[rest], ref[2][rest], ref[3][rest])
    dl[bad] = 0
    (dx, tx), (dw, tw) = U.loss_grad_ref(dl, clean, w, t)
    for kw in (dict(dx_dtype=F32, dw_dtype=F32), dict(dx_dtype=F32, dw_dtype=None), dict(dx_dtype=None, dw_dtype=F32)):
        g = ops.cross_entropy_grad(*c, lse, **kw)
        if "x" in g:
            close(g["x"], dx, tx + EPS32 * dx.abs(), "x")
            assert not g["x"].cpu()[bad].any()
        if "w" in g:
            close(g["w"], dw, tw + EPS32 * dw.abs(), "w")

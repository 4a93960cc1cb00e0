"""The sum over a token's grouped rows, its gradients and the inverse permutation, against 64 bits."""
import pytest
import torch

import train_util as U
from ops_util import EPS32, F8, close, eps_of, offsets_of, randn
from sparse_moe_router_amd import ops

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def permutation(n, seed=0):
    return torch.randperm(n, generator=torch.Generator().manual_seed(seed)).to(torch.int32)


def weights(T, k, seed=1):
    return torch.rand(T, k, generator=torch.Generator().manual_seed(seed)) - 0.3


@pytest.mark.parametrize("n", [1, 7, 256, 5000, 100003])
def test_inverse(n):
    perm = permutation(n)
    inv = ops.invert_permutation(perm.cuda()).cpu()
    want = torch.empty(n, dtype=torch.int32)
    want[perm.long()] = torch.arange(n, dtype=torch.int32)
    assert torch.equal(inv, want)


def test_inverse_of_what_is_no_permutation():
    perm = torch.tensor([5, 5, -1, 2, 12, 0, 2, 7, 1], dtype=torch.int32)
    for off in (None, offsets_of([2, 0, 5]), offsets_of([0, 0]), torch.tensor([0, 99], dtype=torch.int32),
                torch.tensor([0, -3], dtype=torch.int32)):
        end = len(perm) if off is None else max(0, min(int(off[-1]), len(perm)))
        for n in (8, 3, 20):
            out = torch.full((n,), 77, dtype=torch.int32, device="cuda")
            got = ops.invert_permutation(perm.cuda(), n, None if off is None else off.cuda(), out=out)
            assert got is out and torch.equal(out.cpu(), U.invert_ref(perm, n, end)), (off, n)
    assert ops.invert_permutation(perm.cuda(), 0).numel() == 0
    assert (ops.invert_permutation(perm[:0].cuda(), 4) == -1).all()


SHAPES = [(1, 1, 8), (1, 8, 2048), (5, 3, 64), (33, 8, 2056), (100, 32, 72), (257, 2, 4096), (64, 9, 16384), (1000, 6, 128)]


@pytest.mark.parametrize("T,k,H", SHAPES)
@pytest.mark.parametrize("out", [BF16, F32])
def test_combine(T, k, H, out):
    perm = permutation(T * k)
    inv, y, w = U.invert_ref(perm, T * k, T * k), randn(2, T * k, H), weights(T, k)
    add = randn(3, T, H, dtype=out)
    for weight, a in ((w, None), (None, None), (w, add), (None, add)):
        want, t = U.combine_ref(y, inv, k, weight, a)
        got = ops.combine(y.cuda(), inv.cuda(), k, weight=None if weight is None else weight.cuda(),
                          add=None if a is None else a.cuda(), out_dtype=out)
        close(got, want, t + eps_of(out) * (want.abs() + t))


@pytest.mark.parametrize("T,k,H", SHAPES)
def test_gradients(T, k, H):
    perm = permutation(T * k)
    inv, y, w, d = U.invert_ref(perm, T * k, T * k), randn(2, T * k, H), weights(T, k), randn(4, T, H)
    p = perm.long()
    g = ops.combine_grad(d.cuda(), y.cuda(), perm.cuda(), inv.cuda(), w.cuda())
    dy = d.to(F8)[p // k] * w.to(F8).view(-1)[p][:, None]
    close(g["y"], dy, (eps_of(BF16) + 2 * EPS32) * dy.abs())
    terms = y.to(F8)[inv.long()].view(T, k, H) * d.to(F8)[:, None, :]
    close(g["weight"], terms.sum(2), U.dot_terms(H) * EPS32 * terms.abs().sum(2))
    # without weights: copies of d_out, no gradient of weights
    g = ops.combine_grad(d.cuda(), None, perm.cuda(), inv.cuda(), top_k=k)
    assert list(g) == ["y"] and torch.equal(g["y"].cpu(), d[p // k])


def test_assignments_without_rows_and_rows_without_assignments():
    """Dropped assignments, rows behind the last group, entries out of range, an assignment named twice; NaN in
    every place that counts for nothing."""
    T, k, H, rows = 40, 4, 136, 130
    perm = permutation(T * k)[:rows]
    perm[3], perm[50], perm[60] = -7, T * k, perm[61]
    off = offsets_of([30, 0, 71])
    end = 101
    inv = U.invert_ref(perm, T * k, end)
    assert torch.equal(ops.invert_permutation(perm.cuda(), T * k, off.cuda()).cpu(), inv)
    y, w, d = randn(2, rows, H), weights(T, k), randn(4, T, H)
    named = torch.zeros(rows, dtype=torch.bool)
    named[inv[inv >= 0].long()] = True
    y[~named] = float("nan")
    w.view(-1)[inv < 0] = float("nan")
    want, t = U.combine_ref(y, inv, k, w)
    got = ops.combine(y.cuda(), inv.cuda(), k, weight=w.cuda())
    close(got, want, t + eps_of(BF16) * (want.abs() + t))
    dy = torch.full((rows, H), 9.0, dtype=BF16, device="cuda")
    g = ops.combine_grad(d.cuda(), y.cuda(), perm.cuda(), inv.cuda(), w.cuda(), offsets=off.cuda(), dy=dy)
    assert g["y"] is dy and (dy[end:] == 9).all() and not dy[:end].cpu()[~named[:end]].any()
    p = perm.long().clamp(0, T * k - 1)
    ref = d.to(F8)[p // k] * w.to(F8).view(-1)[p][:, None]
    close(dy.cpu()[named], ref[named], (eps_of(BF16) + 2 * EPS32) * ref[named].abs())
    terms = torch.where((inv >= 0).view(T, k, 1), y.to(F8)[inv.long().clamp(min=0)].view(T, k, H),
                        torch.zeros((), dtype=F8)) * d.to(F8)[:, None, :]
    close(g["weight"], terms.sum(2), U.dot_terms(H) * EPS32 * terms.abs().sum(2))


def test_inverse_that_does_not_fit_stays_in_bounds():
    T, k, H = 20, 2, 64
    inv = torch.tensor([-5, 1 << 30, 40, 39] * 10, dtype=torch.int32)
    y, w, d = randn(1, 40, H).cuda(), weights(T, k).cuda(), randn(2, T, H).cuda()
    want, t = U.combine_ref(y.cpu(), torch.where(inv < 40, inv, -1), k, w.cpu())
    close(ops.combine(y, inv.cuda(), k, weight=w), want, t + eps_of(BF16) * (want.abs() + t))
    g = ops.combine_grad(d, y, permutation(40).cuda(), inv.cuda(), w)
    torch.cuda.synchronize()
    assert torch.isfinite(g["weight"]).all()


def test_strided_and_given():
    T, k, H = 30, 4, 256
    wide, perm = randn(1, T * k, H + 64).cuda(), permutation(T * k)
    inv, w = U.invert_ref(perm, T * k, T * k), weights(T, k)
    y = wide[:, 64:]
    out = torch.full((T, H + 8), 3.0, device="cuda")
    want, t = U.combine_ref(y.cpu(), inv, k, w)
    close(ops.combine(y, inv.cuda(), k, weight=w.cuda(), out=out[:, :H]), want, t + eps_of(F32) * (want.abs() + t))
    assert (out[:, H:] == 3).all()
    dout = randn(2, T, H + 32).cuda()[:, 32:]
    dy = torch.full((T * k, H + 8), 3.0, dtype=BF16, device="cuda")
    ops.combine_grad(dout, y, perm.cuda(), inv.cuda(), w.cuda(), dy=dy[:, 8:])
    ref = dout.cpu().to(F8)[perm.long() // k] * w.to(F8).view(-1)[perm.long()][:, None]
    close(dy[:, 8:], ref, (eps_of(BF16) + 2 * EPS32) * ref.abs())
    assert (dy[:, :8] == 3).all()


def test_nothing():
    y, inv = torch.empty(0, 64, dtype=BF16, device="cuda"), torch.empty(0, dtype=torch.int32, device="cuda")
    assert ops.combine(y, inv, 4).shape == (0, 64)
    none = torch.full((6,), -1, dtype=torch.int32, device="cuda")
    add = randn(1, 3, 64).cuda()
    assert not ops.combine(y, none, 2).any() and torch.equal(ops.combine(y, none, 2, add=add), add)
    g = ops.combine_grad(add, y, inv, none, torch.ones(3, 2, device="cuda"))
    assert g["y"].shape == (0, 64) and not g["weight"].any()


def test_refuses():
    y, inv, w = randn(1, 8, 64).cuda(), permutation(8).cuda(), torch.ones(4, 2, device="cuda")
    for call in (lambda: ops.combine(y, inv, 3), lambda: ops.combine(y, inv, 0), lambda: ops.combine(y, inv, 2, weight=w.t()),
                 lambda: ops.combine(y, inv, 2, weight=w[:3]), lambda: ops.combine(y, inv, 2, add=y),
                 lambda: ops.combine_grad(y[:4], None, inv, inv), lambda: ops.combine_grad(y[:4], None, inv, inv, w),
                 lambda: ops.combine_grad(y[:3], y, inv, inv, w[:3]), lambda: ops.combine_grad(y, y, inv, inv, w),
                 lambda: ops.combine_grad(y[:4], y, inv, inv, w, top_k=4), lambda: ops.invert_permutation(inv, -1),
                 lambda: ops.invert_permutation(inv, offsets=inv[:1])):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        ops.combine(y, inv.long(), 2)
    with pytest.raises(TypeError):
        ops.combine(y, inv, 2, out_dtype=torch.float16)
    with pytest.raises(ops.MoeError):
        ops.combine(y, inv, 2, out=y[:4])

"""The training operators' C entry points refuse bad arguments with the documented status before launching
anything, and the binding refuses tensors the kernels cannot take (CPU only: no call here reaches a launch)."""
import ctypes
import math

import pytest
import torch

from sparse_moe_router_amd import ops

OK, INVALID, SHAPE, WS, MISALIGNED = 0, 1, 2, 3, 4
FAKE = 0x7F0000000000  # never dereferenced: every call below fails its checks first, or has nothing to do
GAP = 1 << 32


def at(i):
    return FAKE + i * GAP


def mat(i, ld=128):
    return ops.MoeMat(None if i is None else at(i), ld)


def groups(rows=100, x_rows=50, ldx=64, ldy=128, E=4, N=128, K=64, top_k=2, offsets=at(10), perm=at(11)):
    return ops.MoeGroups(rows, x_rows, ldx, ldy, E, N, K, top_k, offsets, perm)


def gated(g, x=at(0), w=at(1), h=at(2), gu=mat(3, 256)):
    return ops.lib().moe_gated_matmul(None if g is None else ctypes.byref(g), x, w, h, gu, None)


def ggrad(g, dy=at(0), w=at(1), gu=mat(3), d=mat(4), h=at(2)):
    return ops.lib().moe_gated_matmul_grad(None if g is None else ctypes.byref(g), dy, w, gu, d, h, None)


@pytest.mark.parametrize("call", [gated, ggrad])
def test_gated_products_refuse(call):
    assert call(None) == INVALID
    assert call(groups(rows=-1)) == INVALID and call(groups(x_rows=-1)) == INVALID
    for bad in (dict(rows=1 << 31), dict(N=12, ldy=16), dict(N=0), dict(K=60), dict(K=16392, ldx=16392), dict(E=0),
                dict(E=1025), dict(top_k=0), dict(top_k=33), dict(ldx=(1 << 20) + 8)):
        assert call(groups(**bad)) == SHAPE, bad
    assert call(groups(ldx=56)) == INVALID and call(groups(ldy=120)) == INVALID
    assert call(groups(ldx=68)) == MISALIGNED and call(groups(ldy=132)) == MISALIGNED
    assert call(groups(offsets=None)) == INVALID and call(groups(offsets=at(10) + 2)) == MISALIGNED
    assert call(groups(rows=(1 << 31) - 1, x_rows=1 << 29, N=1 << 20, ldy=1 << 20, K=16384, ldx=16384, E=1024)) == SHAPE
    assert call(groups(rows=0)) == OK
    assert call(groups(), gu=ops.MoeMat(at(3) + 8, 256)) == MISALIGNED
    assert call(groups(), gu=mat(3, 260)) == MISALIGNED
    assert call(groups(), gu=mat(3, 120)) == INVALID
    assert call(groups(), gu=mat(3, (1 << 31) + 8)) == SHAPE
    assert call(groups(), h=at(10)) == INVALID and call(groups(), gu=mat(2, 256)) == INVALID


def test_gated_products_refuse_pointers():
    g = groups()
    for n in ("x", "w", "h"):
        assert gated(g, **{n: None}) == INVALID, n
        assert gated(g, **{n: at(5) + 8}) == MISALIGNED, n
    assert gated(g, h=at(0)) == INVALID and gated(g, h=at(1)) == INVALID and gated(g, gu=mat(0, 256)) == INVALID
    assert gated(g, gu=ops.MoeMat(at(1) + 4 * 128 * 64 * 4 - 256, 256)) == INVALID  # the end of both matrices
    assert gated(groups(perm=None, x_rows=99)) == INVALID
    assert gated(groups(x_rows=1 << 30)) == SHAPE
    for n in ("dy", "w", "h"):
        assert ggrad(g, **{n: None}) == INVALID, n
        assert ggrad(g, **{n: at(5) + 8}) == MISALIGNED, n
    assert ggrad(g, gu=mat(None)) == INVALID and ggrad(g, d=mat(None)) == INVALID
    assert ggrad(g, d=mat(4, 120)) == INVALID and ggrad(g, d=mat(4, 132)) == MISALIGNED
    assert ggrad(g, d=mat(3)) == INVALID and ggrad(g, d=mat(0)) == INVALID and ggrad(g, h=at(3)) == INVALID
    assert ggrad(g, h=at(4)) == INVALID


def ffn(rows=100, x_rows=50, ldx=64, ld_dy=96, E=4, I=128, K=64, H=96, top_k=2, offsets=at(10), perm=at(11)):
    return ops.MoeFeedForward(rows, x_rows, ldx, ld_dy, E, I, K, H, top_k, offsets, perm)


def fgrad(d, dy=at(0), x=at(1), wg=at(2), wd=at(3), gu=mat(4, 256), dx=mat(5, 64), dg=at(6), dd=at(7), t=0, wk=at(8),
          wkb=1 << 40):
    return ops.lib().moe_feed_forward_grad(None if d is None else ctypes.byref(d), dy, x, wg, wd, gu, dx, dg, dd, t, wk,
                                           wkb, None)


def test_feed_forward_gradient_refuses():
    size = ops.lib().moe_feed_forward_grad_workspace_size
    assert fgrad(None) == INVALID and fgrad(ffn(rows=-1)) == INVALID and fgrad(ffn(x_rows=-1)) == INVALID
    for bad in (dict(rows=1 << 31), dict(I=12), dict(I=0), dict(I=-8), dict(I=16392), dict(I=1 << 30), dict(K=60),
                dict(K=16392, ldx=16392), dict(H=12), dict(H=0), dict(E=0), dict(E=1025), dict(top_k=0),
                dict(ld_dy=(1 << 20) + 8), dict(x_rows=1 << 30)):
        assert fgrad(ffn(**bad)) == SHAPE, bad
        assert size(ctypes.byref(ffn(**bad))) == 0, bad
    assert fgrad(ffn(ldx=56)) == INVALID and fgrad(ffn(ld_dy=88)) == INVALID and fgrad(ffn(offsets=None)) == INVALID
    assert fgrad(ffn(ldx=68)) == MISALIGNED and fgrad(ffn(ld_dy=100)) == MISALIGNED
    assert fgrad(ffn(perm=None, x_rows=99)) == INVALID
    d = ffn()
    need = size(ctypes.byref(d))
    assert need >= 100 * 3 * 128 * 2 and need % 256 == 0
    assert fgrad(d, wkb=need - 1) == WS and fgrad(d, wk=at(8) + 16) == MISALIGNED
    for n in ("dy", "x", "wg", "wd", "dg", "dd", "wk"):
        assert fgrad(d, **{n: None}) == INVALID, n
    for n in ("dy", "x", "wg", "wd", "dg", "dd"):
        assert fgrad(d, **{n: at(9) + 8}) == MISALIGNED, n
    assert fgrad(d, gu=mat(None)) == INVALID and fgrad(d, gu=mat(4, 248)) == INVALID and fgrad(d, gu=mat(4, 260)) == MISALIGNED
    assert fgrad(d, dx=mat(None)) == INVALID and fgrad(d, dx=mat(5, 56)) == INVALID
    assert fgrad(d, dx=mat(5, (1 << 20) + 8)) == SHAPE
    assert fgrad(d, t=2) == INVALID
    for n, i in (("dx", mat(0, 64)), ("dg", at(2)), ("dd", at(7)), ("wk", at(4))):
        assert fgrad(d, **{n: i, **({"dg": at(7)} if n == "dd" else {})}) == INVALID, n
    # few experts, long groups: parts of the weight gradients in the workspace
    one = ffn(rows=4096, x_rows=4096, E=1, offsets=None, perm=None)
    assert size(ctypes.byref(one)) > 4096 * 3 * 128 * 2 + 2 * (256 * 64 + 96 * 128) * 4


def comb(tokens=10, rows=20, H=64, k=2, E=4, t=0, inverse=at(6), perm=at(7), offsets=None):
    return ops.MoeCombine(tokens, rows, H, k, E, t, inverse, perm, offsets)


def combine(d, y=mat(0), w=at(1), add=mat(None), out=mat(2)):
    return ops.lib().moe_combine(None if d is None else ctypes.byref(d), y, w, add, out, None)


def cgrad(d, do=mat(0), y=mat(1), w=at(2), dy=mat(3), dw=at(4)):
    return ops.lib().moe_combine_grad(None if d is None else ctypes.byref(d), do, y, w, dy, dw, None)


@pytest.mark.parametrize("call", [combine, cgrad])
def test_combine_refuses(call):
    assert call(None) == INVALID and call(comb(tokens=-1)) == INVALID and call(comb(rows=-1)) == INVALID
    for bad in (dict(H=60), dict(H=0), dict(H=16392), dict(k=0), dict(k=33), dict(rows=1 << 31), dict(tokens=1 << 30)):
        assert call(comb(**bad)) == SHAPE, bad
    assert call(comb(t=2)) == INVALID and call(comb(inverse=None)) == INVALID
    assert call(comb(inverse=at(6) + 2)) == MISALIGNED
    assert call(comb(), y=mat(0, 56)) == INVALID and call(comb(), y=mat(0, 68)) == MISALIGNED
    assert call(comb(), y=ops.MoeMat(at(0) + 8, 64)) == MISALIGNED


def test_combine_refuses_buffers():
    d = comb()
    assert combine(d, y=mat(None)) == INVALID and combine(d, out=mat(None)) == INVALID
    assert combine(d, w=at(1) + 2) == MISALIGNED
    assert combine(d, out=mat(0)) == INVALID and combine(d, out=mat(6)) == INVALID and combine(d, add=mat(2)) == INVALID
    assert combine(comb(tokens=0), y=mat(None), w=None, out=mat(None)) == OK
    for n in ("do", "y", "dy"):
        assert cgrad(d, **{n: mat(None)}) == INVALID, n
    assert cgrad(d, w=None) == INVALID  # a gradient of weights that are not there
    assert cgrad(comb(perm=None)) == INVALID and cgrad(comb(perm=at(7) + 1)) == MISALIGNED
    assert cgrad(comb(offsets=at(8), E=0)) == SHAPE and cgrad(comb(offsets=at(8), E=1025)) == SHAPE
    assert cgrad(d, dy=mat(0)) == INVALID and cgrad(d, dw=at(3)) == INVALID and cgrad(d, dw=at(7)) == INVALID
    assert cgrad(d, dw=at(4) + 2) == MISALIGNED
    assert cgrad(comb(tokens=0, rows=0), do=mat(None), y=mat(None), w=None, dy=mat(None), dw=None) == OK


def test_invert_refuses():
    f = lambda rows=10, p=at(0), o=None, E=0, n=10, i=at(1): ops.lib().moe_invert_permutation(rows, p, o, E, n, i, None)
    assert f(rows=-1) == INVALID and f(n=-1) == INVALID and f(rows=1 << 31) == SHAPE and f(n=1 << 31) == SHAPE
    assert f(o=at(2), E=0) == SHAPE and f(o=at(2), E=1025) == SHAPE
    assert f(p=None) == INVALID and f(i=None) == INVALID
    assert f(p=at(0) + 1) == MISALIGNED and f(i=at(1) + 2) == MISALIGNED and f(o=at(2) + 2, E=4) == MISALIGNED
    assert f(i=at(0)) == INVALID and f(i=at(2), o=at(2), E=4) == INVALID
    assert f(n=0, p=None, i=None) == OK


def tensors(*t):
    return (ops.MoeTensor * len(t))(*(ops.MoeTensor(*x) for x in t))


ONE = (at(0), at(1), 100, 0, 0)


def gnorm(t=(ONE,), count=None, norm=at(20), wk=at(21), wkb=1 << 30):
    return ops.lib().moe_grad_norm(tensors(*t), len(t) if count is None else count, norm, wk, wkb, None)


def clip(t=(ONE,), count=None, m=1.0, eps=1e-6, norm=at(20), given=0, wk=at(21), wkb=1 << 30):
    return ops.lib().moe_clip_grads(tensors(*t), len(t) if count is None else count, m, eps, norm, given, wk, wkb, None)


@pytest.mark.parametrize("call", [gnorm, clip])
def test_clipping_refuses(call):
    assert call(count=-1) == INVALID
    assert ops.lib().moe_grad_norm(None, 1, at(20), at(21), 1 << 30, None) == INVALID
    for t, st in (((at(0), at(1), -1, 0, 0), INVALID), ((at(0), at(1), 1 << 41, 0, 0), SHAPE),
                  ((None, at(1), 5, 0, 0), INVALID), ((at(0), at(1), 5, 2, 0), INVALID),
                  ((at(0) + 1, at(1), 5, 0, 0), MISALIGNED), ((at(0) + 2, at(1), 5, 1, 0), MISALIGNED)):
        assert call(t=(ONE, t)) == st, t
    assert call(norm=None) == INVALID and call(norm=at(20) + 2) == MISALIGNED
    assert call(wk=None) == INVALID and call(wk=at(21) + 16) == MISALIGNED and call(wkb=255) == WS
    assert call(norm=at(0) + 4) == INVALID and call(wk=at(0)) == INVALID and call(wk=at(20)) == INVALID


def test_clipping_refuses_outputs():
    assert clip(t=((at(0), None, 5, 0, 0),)) == INVALID and clip(t=((at(0), at(1) + 2, 5, 0, 1),)) == MISALIGNED
    assert clip(t=((at(0), at(1), 5, 0, 2),)) == INVALID
    for m in (-1.0, math.inf, math.nan):
        assert clip(m=m) == INVALID
    for e in (0.0, -1e-6, math.inf, math.nan):
        assert clip(eps=e) == INVALID
    assert clip(t=((at(0), at(0) + 2, 100, 0, 0),)) == INVALID  # shifted onto itself
    assert clip(t=((at(0), at(0), 100, 0, 1),)) == INVALID  # in place, in another type
    same = (at(0), at(0), 100, 0, 0)
    assert clip(t=(same, same)) == INVALID  # the same tensor twice
    assert clip(t=(ONE, (at(2), at(1) + 100, 100, 0, 0))) == INVALID  # two results on one place
    assert clip(t=((at(0), at(1), 100, 0, 0), (at(1) + 198, at(3), 100, 0, 0))) == INVALID  # a result on another's input
    assert clip(t=tuple((at(2 * i), at(2 * i), 10, 0, 0) for i in range(100)) + ((at(14) + 4, at(300), 1, 0, 0),),
                norm=at(400), wk=at(401)) == INVALID  # many
    assert clip(given=1, norm=None) == INVALID and clip(given=1, norm=at(1)) == INVALID
    none = (None, None, 0, 0, 0)
    assert clip(t=(none, none), given=1, wk=None, wkb=0) == OK  # nothing to scale
    size = ops.lib().moe_grad_norm_workspace_size
    assert size(tensors(ONE), 1) == 256 and size(tensors((None, None, -1, 0, 0)), 1) == 0
    assert size(tensors((at(0), None, 1 << 33, 0, 0)), 1) == 2048 * 8


def loss(rows=10, ldx=64, V=100, H=64, ignore=-100):
    return ops.MoeLoss(rows, ldx, V, H, ignore)


def ce(d, x=at(0), w=at(1), t=at(2), l=at(3), lse=at(4), wk=at(5), wkb=1 << 40):
    return ops.lib().moe_cross_entropy(None if d is None else ctypes.byref(d), x, w, t, l, lse, wk, wkb, None)


def ceg(d, dl=at(6), x=at(0), w=at(1), t=at(2), lse=at(4), dx=mat(7, 64), dxt=0, dw=at(8), dwt=0, wk=at(5), wkb=1 << 40):
    return ops.lib().moe_cross_entropy_grad(None if d is None else ctypes.byref(d), dl, x, w, t, lse, dx, dxt, dw, dwt,
                                            wk, wkb, None)


@pytest.mark.parametrize("call", [ce, ceg])
def test_cross_entropy_refuses(call):
    assert call(None) == INVALID and call(loss(rows=-1)) == INVALID
    for bad in (dict(rows=1 << 31), dict(V=0), dict(V=(1 << 20) + 1), dict(H=60), dict(H=0), dict(H=16392, ldx=16392),
                dict(ldx=(1 << 20) + 8), dict(rows=1 << 22, V=1 << 20)):
        assert call(loss(**bad)) == SHAPE, bad
    assert call(loss(ldx=56)) == INVALID and call(loss(ldx=68)) == MISALIGNED
    d = loss()
    for n in ("x", "w", "t", "wk"):
        assert call(d, **{n: None}) == INVALID, n
    assert call(d, x=at(0) + 8) == MISALIGNED and call(d, w=at(1) + 8) == MISALIGNED
    assert call(d, t=at(2) + 4) == MISALIGNED and call(d, wk=at(5) + 16) == MISALIGNED
    assert call(d, wk=at(0)) == INVALID and call(d, wk=at(1)) == INVALID


def test_cross_entropy_refuses_buffers():
    d = loss()
    L = ops.lib()
    need, gneed = (f(ctypes.byref(d)) for f in (L.moe_cross_entropy_workspace_size, L.moe_cross_entropy_grad_workspace_size))
    assert need > 0 and gneed > 0
    assert L.moe_cross_entropy_workspace_size(ctypes.byref(loss(H=60))) == 0
    assert L.moe_cross_entropy_grad_workspace_size(ctypes.byref(loss(H=60))) == 0
    assert ce(d, wkb=need - 1) == WS and ceg(d, wkb=gneed - 1) == WS
    assert ce(d, l=None) == INVALID and ce(d, l=at(0)) == INVALID and ce(d, lse=at(3)) == INVALID
    assert ce(d, l=at(3) + 2) == MISALIGNED
    assert ce(loss(rows=0), x=None, w=None, t=None, l=None, lse=None, wk=None, wkb=0) == OK
    assert ceg(d, dl=None) == INVALID and ceg(d, lse=None) == INVALID
    assert ceg(d, dx=mat(None), dw=None) == INVALID  # no gradient asked for
    assert ceg(d, dxt=2) == INVALID and ceg(d, dwt=-1) == INVALID
    assert ceg(d, dx=mat(7, 56)) == INVALID and ceg(d, dx=mat(7, 68)) == MISALIGNED and ceg(d, dw=at(8) + 8) == MISALIGNED
    assert ceg(d, dx=mat(0, 64)) == INVALID and ceg(d, dw=at(1)) == INVALID and ceg(d, dw=at(7)) == INVALID
    assert ceg(d, dw=at(6)) == INVALID
    assert ceg(loss(rows=0), dl=None, x=None, w=None, t=None, lse=None, dx=mat(None), dw=None, wk=None, wkb=0) == OK


def test_binding_refuses_cpu_tensors():
    b = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)
    f = lambda *s: torch.zeros(*s)
    for call in (lambda: ops.gated_matmul(b(4, 64), b(2, 64, 64), i(3)),
                 lambda: ops.gated_matmul_grad(b(4, 64), b(2, 64, 32), b(4, 64), i(3)),
                 lambda: ops.feed_forward(b(4, 64), b(2, 64, 64), b(2, 64, 32), i(3)),
                 lambda: ops.feed_forward_grad(b(4, 64), b(4, 64), b(2, 64, 64), b(2, 64, 32), b(4, 64), i(3)),
                 lambda: ops.invert_permutation(i(4)), lambda: ops.combine(b(4, 64), i(4), 2),
                 lambda: ops.combine_grad(b(2, 64), None, i(4), i(4), top_k=2), lambda: ops.grad_norm([f(4)]),
                 lambda: ops.clip_grads([f(4)], 1.0), lambda: ops.cross_entropy(b(4, 64), b(9, 64), torch.zeros(4).long()),
                 lambda: ops.cross_entropy_grad(f(4), b(4, 64), b(9, 64), torch.zeros(4).long(), f(4))):
        with pytest.raises(ValueError, match="GPU"):
            call()
    for bad in ([], ()):
        with pytest.raises(ValueError, match="at least one"):
            ops.grad_norm(bad)
    for bad in (f(4), "ab", None):
        with pytest.raises(TypeError):
            ops.clip_grads(bad, 1.0)
    with pytest.raises(TypeError):
        ops.grad_norm([1.0])
    with pytest.raises(TypeError):
        ops.cross_entropy_grad(f(4), b(4, 64), b(9, 64), torch.zeros(4).long(), f(4), dx_dtype=torch.float16)


def test_clipping_refuses_too_many_elements():
    """2^40 elements in all: none of the sums over the tensors' pieces overflows."""
    half = (at(0), at(0), 1 << 39, 0, 0)
    size = ops.lib().moe_grad_norm_workspace_size
    assert size(tensors(half, half), 2) > 0 and size(tensors(half, half, ONE), 3) == 0
    assert gnorm(t=(half, half, ONE)) == SHAPE and clip(t=(half, half, ONE)) == SHAPE
    assert clip(t=(half, half, ONE), given=1, wk=None, wkb=0) == SHAPE

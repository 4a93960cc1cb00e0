"""The operators' C entry points are exported, refuse bad arguments with the documented status before
launching anything, and the binding refuses tensors the kernels cannot take (CPU only: no call here
reaches a kernel launch)."""
import ctypes
import os
import re

import pytest
import torch

from sparse_moe_router_amd import moe, ops

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, SHAPE, WS, MISALIGNED = 0, 1, 2, 3, 4
FAKE = 0x7F0000000000  # never dereferenced: every call below fails its checks first, or has no rows
GAP = 1 << 32


def at(i):
    return FAKE + i * GAP


def test_exports_every_declared_symbol():
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "moe_ops.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(moe_[a-z0-9_]+)\s*\(", src))
    assert names == set(ops.EXPORTS)
    L = ops.lib()
    for n in names:
        assert hasattr(L, n), n


def test_header_compiles_as_c():
    import shutil
    import subprocess
    import tempfile
    if not shutil.which("gcc"):
        pytest.skip("no host compiler")
    with tempfile.TemporaryDirectory() as d:
        c = os.path.join(d, "use.c")
        with open(c, "w") as f:
            f.write('#include "moe_ops.h"\nint main(void) { moe_groups_t g = {0}; moe_norm_t n = {0};\n'
                    '  return (int)moe_matmul_i8_workspace_size(&g) + (int)moe_norm_grad_workspace_size(&n); }\n')
        subprocess.run(["gcc", "-std=c11", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), "-c", c, "-o",
                        c + ".o"], check=True)


def groups(rows=100, x_rows=50, ldx=64, ldy=128, E=4, N=128, K=64, top_k=2, offsets=at(10), perm=at(11)):
    return ops.MoeGroups(rows, x_rows, ldx, ldy, E, N, K, top_k, offsets, perm)


def fwd(g, x=at(0), w=at(1), y=at(2), t=0):
    return ops.lib().moe_grouped_matmul(None if g is None else ctypes.byref(g), x, w, y, t, None)


def gin(g, dy=at(0), w=at(1), dx=at(2), t=0):
    return ops.lib().moe_grouped_matmul_grad_input(ctypes.byref(g), dy, w, dx, t, None)


def gw(g, x=at(0), dy=at(1), dw=at(2), t=0):
    return ops.lib().moe_grouped_matmul_grad_weight(ctypes.byref(g), x, dy, dw, t, None)


@pytest.mark.parametrize("call", [fwd, gin, gw])
def test_grouped_products_refuse(call):
    assert call(groups(rows=-1)) == INVALID
    assert call(groups(x_rows=-1)) == INVALID
    assert call(groups(rows=1 << 31)) == SHAPE
    for bad in (dict(N=12, ldy=16), dict(N=0), dict(N=(1 << 20) + 8, ldy=(1 << 20) + 8), dict(K=60), dict(K=0),
                dict(K=16392, ldx=16392), dict(E=0), dict(E=1025), dict(top_k=0), dict(top_k=33)):
        assert call(groups(**bad)) == SHAPE, bad
    assert call(groups(ldx=56)) == INVALID and call(groups(ldy=120)) == INVALID
    assert call(groups(ldx=68)) == MISALIGNED and call(groups(ldy=132)) == MISALIGNED
    assert call(groups(offsets=None)) == INVALID  # more than one expert needs offsets
    assert call(groups(offsets=at(10) + 2)) == MISALIGNED and call(groups(perm=at(11) + 1)) == MISALIGNED
    assert call(groups(), t=2) == INVALID
    assert call(groups(rows=(1 << 31) - 1, x_rows=1 << 29, N=1 << 20, ldy=1 << 20, K=16384, ldx=16384, E=1024)) == SHAPE


def test_grouped_products_refuse_pointers():
    g = groups()
    assert fwd(None) == INVALID
    for call, names in ((fwd, ("x", "w", "y")), (gin, ("dy", "w", "dx")), (gw, ("x", "dy", "dw"))):
        for n in names:
            assert call(g, **{n: None}) == INVALID, n
            assert call(g, **{n: at(5) + 8}) == MISALIGNED, n
        out, ins = names[2], names[:2]
        for i in ins:
            assert call(g, **{out: at(5), i: at(5)}) == INVALID
        assert call(g, **{out: at(10)}) == INVALID  # over the offsets
    assert fwd(g, y=at(11) - 64) == INVALID  # over the permutation
    assert fwd(groups(perm=None, top_k=1, x_rows=99)) == INVALID  # fewer rows of x than rows
    assert gw(groups(perm=None, top_k=1, x_rows=99)) == INVALID
    assert fwd(groups(x_rows=1 << 30, top_k=2)) == SHAPE  # assignments past 2^31
    # nothing to do without rows
    assert fwd(groups(rows=0), x=None, w=None, y=None) == OK
    assert gin(groups(rows=0), dy=None, w=None, dx=None) == OK


def i8(g, x=at(0), xs=None, w=at(1), ws=at(3), bias=None, y=at(2), t=0, wk=at(4), wkb=1 << 40):
    return ops.lib().moe_matmul_i8(ctypes.byref(g), x, xs, w, ws, bias, y, t, wk, wkb, None)


def test_matmul_i8_refuses():
    g = groups()
    need = ops.lib().moe_matmul_i8_workspace_size(ctypes.byref(g))
    assert need >= 50 * 64 + 50 * 4 and need % 256 == 0
    assert ops.lib().moe_matmul_i8_workspace_size(ctypes.byref(groups(K=72, ldx=72))) == 0
    assert i8(groups(K=72, ldx=72)) == SHAPE
    assert i8(groups(N=132, ldy=136)) == SHAPE
    assert i8(g, w=None) == INVALID and i8(g, ws=None) == INVALID and i8(g, y=None) == INVALID
    assert i8(g, x=None) == INVALID and i8(g, wk=None) == INVALID
    assert i8(g, wkb=need - 1) == WS
    assert i8(g, wk=at(4) + 16) == MISALIGNED and i8(g, ws=at(3) + 4) == MISALIGNED
    assert i8(g, bias=at(6)) == INVALID  # a bias belongs to one weight matrix
    assert i8(g, wk=at(0)) == INVALID and i8(g, wk=at(2)) == INVALID and i8(g, y=at(3)) == INVALID
    assert i8(groups(ldx=72), xs=at(7)) == MISALIGNED  # rows of codes are 16 bytes apart
    assert i8(g, xs=at(7) + 4) == MISALIGNED
    assert i8(g, t=7) == INVALID
    assert i8(groups(rows=0), x=None, w=None, ws=None, y=None, wk=None, wkb=0) == OK


def test_quantize_refuses():
    q = lambda rows=10, K=64, ldx=64, x=at(0), c=at(1), s=at(2): ops.lib().moe_quantize_i8(rows, K, ldx, x, c, s, None)
    assert q(rows=-1) == INVALID and q(K=24) == SHAPE and q(K=0) == SHAPE and q(K=16400, ldx=16400) == SHAPE
    assert q(ldx=56) == INVALID and q(ldx=68) == MISALIGNED
    assert q(x=None) == INVALID and q(c=None) == INVALID and q(s=None) == INVALID
    assert q(c=at(1) + 8) == MISALIGNED
    assert q(c=at(0)) == INVALID and q(s=at(1)) == INVALID
    assert q(rows=0, x=None, c=None, s=None) == OK


def mat(i, ld=64):
    return ops.MoeMat(None if i is None else at(i), ld)


def desc(rows=10, H=64, st=0, wt=0, gate=0, eps=1e-6, scale=1.0):
    return ops.MoeNorm(rows, H, st, wt, gate, eps, scale)


def norm(d, x=mat(0), w=at(1), h=mat(2)):
    return ops.lib().moe_block_norm(ctypes.byref(d), x, w, h, None)


def merge(d, r=mat(0), y=mat(1), w=at(2), g=mat(None), wn=at(3), out=mat(4), h=mat(5)):
    return ops.lib().moe_block_merge(ctypes.byref(d), r, y, w, g, wn, out, h, None)


def mgrad(d, do=mat(0), dh=mat(1), y=mat(2), w=at(3), g=mat(None), out=mat(4), wn=at(5), dr=mat(6), dy=mat(7),
          dg=mat(None), dw=at(8), dwn=at(9), wk=at(12), wkb=1 << 40):
    return ops.lib().moe_block_merge_grad(ctypes.byref(d), do, dh, y, w, g, out, wn, dr, dy, dg, dw, dwn, wk, wkb, None)


def ngrad(d, dh=mat(0), x=mat(1), w=at(2), da=mat(None), dx=mat(3), dw=at(4), wk=at(12), wkb=1 << 40):
    return ops.lib().moe_block_norm_grad(ctypes.byref(d), dh, x, w, da, dx, dw, wk, wkb, None)


@pytest.mark.parametrize("call", [norm, merge, mgrad, ngrad])
def test_norms_refuse_descriptors(call):
    for bad, st in ((dict(rows=-1), INVALID), (dict(rows=1 << 31), SHAPE), (dict(H=0), SHAPE), (dict(H=60), SHAPE),
                    (dict(H=16392), SHAPE), (dict(st=2), INVALID), (dict(wt=-1), INVALID), (dict(gate=3), INVALID),
                    (dict(eps=0.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID),
                    (dict(scale=float("inf")), INVALID)):
        assert call(desc(**bad)) == st, bad


def test_norms_refuse_buffers():
    d = desc()
    assert norm(d, x=mat(None)) == INVALID and norm(d, w=None) == INVALID and norm(d, h=mat(None)) == INVALID
    assert norm(d, x=mat(0, 56)) == INVALID and norm(d, x=mat(0, 68)) == MISALIGNED
    assert norm(d, h=mat(0)) == INVALID and norm(d, w=at(1) + 4) == MISALIGNED
    assert norm(desc(gate=1)) == INVALID
    assert norm(desc(rows=0), x=mat(None), w=None, h=mat(None)) == OK
    for n in ("r", "y", "out"):
        assert merge(d, **{n: mat(None)}) == INVALID, n
    assert merge(d, w=None) == INVALID
    assert merge(d, h=mat(None)) == INVALID and merge(d, wn=None) == INVALID  # a next norm needs both
    assert merge(d, g=mat(6)) == INVALID and merge(desc(gate=1)) == INVALID  # gate and mode agree
    assert merge(d, out=mat(0)) == INVALID and merge(d, h=mat(1)) == INVALID and merge(d, h=mat(4)) == INVALID
    assert merge(desc(gate=2), g=mat(6, 60)) == INVALID
    need = ops.lib().moe_norm_grad_workspace_size(ctypes.byref(d))
    assert need >= 2 * 64 * 4
    assert ops.lib().moe_norm_grad_workspace_size(ctypes.byref(desc(H=60))) == 0
    assert mgrad(d, wkb=need - 1) == WS and ngrad(d, wkb=need - 1) == WS
    assert mgrad(d, wk=None) == INVALID and mgrad(d, wk=at(12) + 16) == MISALIGNED
    for n in ("y", "dr", "dy", "dh", "out"):
        assert mgrad(d, **{n: mat(None)}) == INVALID, n
    assert mgrad(d, wn=None, dh=mat(None), dwn=None, do=mat(None)) == INVALID  # no gradient at all
    assert mgrad(d, dwn=None) == INVALID and mgrad(d, dw=None) == INVALID
    assert mgrad(desc(gate=2), g=mat(10)) == INVALID and mgrad(d, dg=mat(10)) == INVALID
    assert mgrad(d, dy=mat(2)) == INVALID and mgrad(d, dw=at(9)) == INVALID and mgrad(d, wk=at(6)) == INVALID
    for n in ("dh", "x", "dx"):
        assert ngrad(d, **{n: mat(None)}) == INVALID, n
    assert ngrad(d, dx=mat(1)) == INVALID and ngrad(desc(gate=1)) == INVALID


def test_binding_refuses_cpu_tensors():
    b = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    o = torch.zeros(3, dtype=torch.int32)
    for f in (lambda: ops.grouped_matmul(b(4, 64), b(2, 64, 64), o), lambda: ops.block_norm(b(4, 64), b(64), 1e-6),
              lambda: ops.grouped_matmul_grad_input(b(4, 64), b(2, 64, 64), o),
              lambda: ops.grouped_matmul_grad_weight(b(4, 64), b(4, 64), o), lambda: ops.quantize_i8(b(4, 64)),
              lambda: ops.matmul_i8(b(4, 64), torch.zeros(8, 64, dtype=torch.int8), torch.zeros(8)),
              lambda: ops.block_merge(b(4, 64), b(4, 64), b(64), 1e-6),
              lambda: ops.block_merge_grad(b(4, 64), b(4, 64), b(64), 1e-6),
              lambda: ops.block_norm_grad(b(4, 64), b(4, 64), b(64), 1e-6)):
        with pytest.raises(ValueError, match="GPU"):
            f()
    with pytest.raises(TypeError):
        ops.grouped_matmul([1.0], b(2, 64, 64), o)

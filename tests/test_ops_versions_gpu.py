"""Tensors that the operators write into, as torch's automatic differentiation sees them: each has a new version
afterwards, so that a graph which had saved one before refuses to use the new values as the old ones; those that
are only read keep theirs.  A gradient in a list that requires a gradient itself gives the warning that other
arguments give."""
import warnings

import pytest
import torch

from ops_util import offsets_of, randn
from sparse_moe_router_amd import ops

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def empty(*shape, dtype=BF16):
    return torch.zeros(shape, dtype=dtype, device="cuda")


def calls():
    """name: (call, what it writes, what it reads)"""
    T, K, N, E = 6, 64, 32, 2
    x, w, dy, off = randn(1, T, K).cuda(), randn(2, E, N, K).cuda(), randn(3, T, N).cuda(), offsets_of([4, 2]).cuda()
    perm = torch.tensor([3, 0, 5, 1, 4, 2], dtype=torch.int32, device="cuda")
    inv = torch.argsort(perm).int()
    out = {}

    def add(name, f, written, read=()):
        out[name] = (f, written, read)
    a = empty(T, N)
    add("grouped_matmul", lambda a=a: ops.grouped_matmul(x, w, off, out=a), [a], [x, w, off])
    b = empty(T, K)
    add("grouped_matmul_grad_input", lambda b=b: ops.grouped_matmul_grad_input(dy, w, off, out=b), [b], [dy, w])
    c = empty(E, N, K, dtype=F32)
    add("grouped_matmul_grad_weight", lambda: ops.grouped_matmul_grad_weight(x, dy, off, out=c), [c], [x, dy])
    q, s = empty(T, K, dtype=torch.int8), empty(T, dtype=F32)
    add("quantize_i8", lambda: ops.quantize_i8(x, codes=q, scale=s), [q, s], [x])
    w8, ws = torch.ones(N, K, dtype=torch.int8, device="cuda"), torch.ones(N, device="cuda")
    d = empty(T, N)
    add("matmul_i8", lambda: ops.matmul_i8(x, w8, ws, out=d), [d], [x, w8, ws])
    n, e = torch.ones(K, dtype=BF16, device="cuda"), empty(T, K)
    add("block_norm", lambda: ops.block_norm(x, n, 1e-6, out=e), [e], [x, n])
    m, h = empty(T, K), empty(T, K)
    add("block_merge", lambda: ops.block_merge(x, x, n, 1e-6, next_weight=n, out=m, h=h), [m, h], [x, n])
    g, gu = empty(T, N // 2), empty(T, N)
    add("gated_matmul", lambda: ops.gated_matmul(x, w, off, save=True, out=g, gate_up=gu), [g, gu], [x, w])
    i = empty(T, dtype=torch.int32)
    add("invert_permutation", lambda: ops.invert_permutation(perm, out=i), [i], [perm])
    y, wt, o = randn(4, T, K).cuda(), torch.ones(T // 2, 2, device="cuda"), empty(T // 2, K)
    add("combine", lambda: ops.combine(y, inv, 2, weight=wt, out=o), [o], [y, inv, wt])
    do, gy = randn(5, T // 2, K).cuda(), empty(T, K)
    add("combine_grad", lambda: ops.combine_grad(do, y, perm, inv, wt, dy=gy), [gy], [do, y, perm, inv, wt])
    gr = [randn(6, 9).cuda(), randn(7, 3, 5).cuda().float(), empty(0)]
    add("clip_grads in place", lambda: ops.clip_grads(gr, 0.5), gr)
    gs, go = [randn(8, 9).cuda()], [empty(9, dtype=F32)]
    nm = torch.ones((), device="cuda")
    add("clip_grads", lambda: ops.clip_grads(gs, 0.5, norm=nm, out=go), go, gs + [nm])
    add("grad_norm", lambda: ops.grad_norm(gs), [], gs)
    return out


NAMES = ("grouped_matmul", "grouped_matmul_grad_input", "grouped_matmul_grad_weight", "quantize_i8", "matmul_i8", "block_norm",
         "block_merge", "gated_matmul", "invert_permutation", "combine", "combine_grad", "clip_grads in place", "clip_grads",
         "grad_norm")


@pytest.mark.parametrize("name", NAMES)
def test_what_is_written_has_a_new_version(name):
    f, written, read = calls()[name]
    before = [t._version for t in written], [t._version for t in read]
    f()
    assert all(t._version > v for t, v in zip(written, before[0]))
    assert [t._version for t in read] == before[1]


def test_a_graph_that_saved_a_clipped_tensor_refuses():
    g = randn(1, 100).cuda().float()
    x = torch.ones(100, device="cuda", requires_grad=True)
    y = (x * g).sum()  # saves g
    ops.clip_grads([g], 1e-3)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()


def test_a_view_and_its_base_share_the_version():
    base = empty(10, 128)
    v = base._version
    x, n = randn(1, 10, 64).cuda(), torch.ones(64, dtype=BF16, device="cuda")
    ops.block_norm(x, n, 1e-6, out=base[:, 64:])
    assert base._version > v


def test_inference_tensors_are_written_as_before():
    with torch.inference_mode():
        g, o = randn(1, 100).cuda(), empty(6, 64)
    ops.clip_grads([g], 1e-3)  # outside of the mode: no version to count
    ops.block_norm(randn(2, 6, 64).cuda(), torch.ones(64, dtype=BF16, device="cuda"), 1e-6, out=o)
    assert g.float().norm() < 1.1e-3 and o.any()
    with torch.inference_mode():
        ops.clip_grads([g], 1e-4)
    assert g.float().norm() < 1.1e-4


def test_refused_calls_leave_the_version():
    a = empty(6, 40)
    v = a._version
    with pytest.raises(ValueError):
        ops.grouped_matmul(randn(1, 6, 64).cuda(), randn(2, 1, 32, 64).cuda(), None, out=a)
    g = [randn(1, 100).cuda()]
    with pytest.raises(ops.MoeError):
        ops.clip_grads(g, -1.0)
    assert a._version == v and g[0]._version == 0


def test_lists_warn_where_a_gradient_would_be_recorded():
    p = torch.ones(8, device="cuda", requires_grad=True)
    for call in (lambda: ops.grad_norm([p]), lambda: ops.clip_grads([p], 1.0, out=[torch.empty(8, device="cuda")])):
        with pytest.warns(UserWarning, match="requires a gradient") as w:
            call()
        assert len(w) == 1 and w[0].filename == __file__
        with torch.no_grad(), warnings.catch_warnings():
            warnings.simplefilter("error")
            call()
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        with pytest.raises(UserWarning):
            ops.grad_norm([p])

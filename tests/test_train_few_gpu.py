"""Backward pass of gated feed-forward blocks for few rows, against 64 bits with nothing rounded between, on both
sides of the rule; empty groups, gathered and strided rows, rows behind the last group, entries of the permutation
that are out of range."""
import pytest
import torch

import train_util as U
from ops_util import close, eps_of, offsets_of, randn, source_rows, take
from sparse_moe_router_amd import ops

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def check(g, want, dw, end):
    for name, (v, tol) in want.items():
        t = g[name].dtype
        assert t == (BF16 if name == "x" else dw)
        n = end if name == "x" else len(v)
        close(g[name][:n], v[:n], (tol + eps_of(t) * (v.abs() + tol))[:n], name)


@pytest.mark.parametrize("dw", [BF16, F32])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("counts,I,K,H", [([1], 8, 8, 8), ([1], 136, 520, 72), ([2, 0, 1, 3], 88, 376, 376), ([32], 72, 1032, 136),
                                          ([0, 0, 0, 5], 264, 128, 1048), ([1] * 20 + [0] * 50, 16, 24, 40), ([31, 1], 520, 512, 64),
                                          ([0, 7], 1032, 64, 2056)], ids=lambda v: str(v)[:20])
def test_against_64_bits(counts, I, K, H, gather, dw):
    R, E, k = sum(counts), len(counts), 3 if gather else 1
    T = (R + k - 1) // k
    perm = torch.randperm(T * k, generator=torch.Generator().manual_seed(1))[:R].to(torch.int32) if gather else None
    x, dy, off = randn(2, T, K), randn(3, R, H), offsets_of(counts)
    gu, dn, pre = randn(4, E, 2 * I, K, scale=0.2), randn(5, E, H, I, scale=0.2), randn(6, R, 2 * I)
    want = U.feed_forward_grad_raw(dy, take(x, source_rows(R, perm, k, T)), gu, dn, pre, off)
    c = [v.cuda() for v in (dy, x, gu, dn, pre, off)]
    kw = dict(perm=None if perm is None else perm.cuda(), top_k=k, dw_dtype=dw)
    g = ops.feed_forward_grad(*c, **kw)
    check(g, want, dw, R)
    h = ops.feed_forward_grad(*c, **kw)
    assert all(torch.equal(g[n], h[n]) for n in g), "the same bits again"
    if E == 1:
        h = ops.feed_forward_grad(*c[:5], None, **kw)
        assert all(torch.equal(g[n], h[n]) for n in g), "without offsets"


def test_strided_rows_behind_and_bad_indexes():
    R, E, I, K, H, k = 20, 4, 72, 136, 88, 2
    counts = [6, 0, 3, 2]
    end, off = sum(counts), offsets_of(counts)
    x, dy, pre = randn(1, 12, K + 40)[:, 8:8 + K], randn(2, R, H + 16)[:, 16:], randn(3, R, 2 * I + 24)[:, :2 * I]
    dy[end:], pre[end:] = float("nan"), float("nan")  # of no group: not read
    gu, dn = randn(4, E, 2 * I, K, scale=0.2), randn(5, E, H, I, scale=0.2)
    perm = torch.randint(0, 24, (R,), generator=torch.Generator().manual_seed(6)).to(torch.int32)
    perm[0], perm[3], perm[8] = -1, 24, 1 << 30  # rows of zeros
    want = U.feed_forward_grad_raw(dy, take(x, source_rows(R, perm, k, 12)), gu, dn, pre, off)

    def wide(t, left, right):
        w = torch.full((t.shape[0], t.shape[1] + left + right), 9.0, dtype=BF16, device="cuda")
        w[:, left:left + t.shape[1]] = t.cuda()
        return w[:, left:left + t.shape[1]]
    g = ops.feed_forward_grad(wide(dy, 16, 8), wide(x, 8, 0), gu.cuda(), dn.cuda(), wide(pre, 0, 8), off.cuda(), perm=perm.cuda(),
                              top_k=k)
    check(g, want, F32, end)


@pytest.mark.parametrize("rows", [31, 32, 33])
def test_both_sides_of_the_rule_agree(rows):
    """33 rows go by tiles, whose values between the kernels are bf16: the same gradients of the rows that all have."""
    I, K, H = 72, 136, 88
    x, dy, pre = randn(1, 33, K)[:rows], randn(2, 33, H)[:rows], randn(3, 33, 2 * I)[:rows]
    gu, dn = randn(4, 1, 2 * I, K, scale=0.2), randn(5, 1, H, I, scale=0.2)
    want = U.feed_forward_grad_raw(dy, x.double(), gu, dn, pre, [0, rows])
    g = ops.feed_forward_grad(*(v.cuda() for v in (dy, x, gu, dn, pre)), None)
    if rows <= 32:
        check(g, want, F32, rows)
    for n, (v, _) in want.items():
        # d and h are off by half a unit of bf16, 2^-8 of each; their products add up at worst, and the result rounds
        bound = {"x": None, "w_gate_up": None, "w_down": None}
        (d, td), (h, th) = U.gated_grad_raw(dy, dn, pre, [0, rows])
        bound["x"] = d.abs() @ gu[0].double().abs()
        bound["w_gate_up"] = (d.abs().t() @ x.double().abs())[None]
        bound["w_down"] = (dy.double().abs().t() @ h.abs())[None]
        close(g[n], v, 1.01 * 2.0 ** -8 * (bound[n] + v.abs()), n)


def test_infinities_stay_in_their_rows():
    I, K, H = 40, 72, 24
    x, dy, pre = randn(1, 6, K), randn(2, 6, H), randn(3, 6, 2 * I)
    dy[2, 3] = float("inf")
    dy[4] = float("nan")
    gu, dn = randn(4, 2, 2 * I, K), randn(5, 2, H, I)
    off = torch.tensor([0, 3, 6], dtype=torch.int32)
    g = ops.feed_forward_grad(*(v.cuda() for v in (dy, x, gu, dn, pre)), off.cuda())
    clean = torch.tensor([0, 1, 3, 5])
    assert torch.isfinite(g["x"].cpu()[clean]).all() and torch.isnan(g["x"].cpu()[4]).all()
    assert not torch.isfinite(g["x"].cpu()[2]).any()


def test_captured_and_replayed():
    I, K, H, R = 136, 264, 72, 9
    c = [v.cuda() for v in (randn(1, R, H), randn(2, R, K), randn(3, 3, 2 * I, K), randn(4, 3, H, I), randn(5, R, 2 * I),
                            offsets_of([4, 0, 5]))]
    ops.feed_forward_grad(*c)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g = ops.feed_forward_grad(*c)
    for seed in (10, 20, 30):
        c[0].copy_(randn(seed, R, H))
        c[5].copy_(offsets_of([seed // 10, 2, R - 2 - seed // 10]))
        want = ops.feed_forward_grad(*c)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(g[n], want[n]) for n in g)

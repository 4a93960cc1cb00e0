"""Products grouped by expert and their gradients against plain 64-bit forms."""
import pytest
import torch

from sparse_moe_router_amd import ops
from ops_util import (EPS32, F8, close, eps_of, grad_input_ref, grad_weight_ref, grouped_ref, offsets_of, randn,
                            source_rows, take)

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32

# counts per expert, N, K: one row; empty first, last and inner groups; sizes around the 16, 32, 64 and
# 256 row edges, and past the 8192 rows whose indexes a weight gradient holds at a time; N and K off every tile; more experts than rows; E over the 64 lanes of a wave
CASES = {
    "one": ([1], 8, 8),
    "one_expert": ([70], 136, 264),
    "ragged": ([0, 1, 0, 17, 0, 256, 3, 0], 264, 200),
    "edges": ([15, 16, 17, 31, 32, 33, 63, 64, 65, 255, 257], 72, 136),
    "tall": ([300, 0, 33, 513, 64], 512, 520),
    "wide_k": ([40, 130], 40, 2056),
    "long_groups": ([8300, 0, 100, 16500], 72, 72),
    "long_k": ([3, 0, 20], 24, 16384),
    "decode": ([0] * 100 + [1, 0, 1, 1] + [0] * 120 + [1] * 5 + [0] * 27, 256, 2048),
    "small_batch": ([2, 0, 5, 1, 9, 0, 0, 16, 3, 64, 1, 1], 520, 328),
    "many": ([i % 3 for i in range(1024)], 16, 72),
    "many_tall": ([40 if i % 5 else 0 for i in range(70)], 264, 64),
}


def problem(name, gather, seed=0):
    counts, N, K = CASES[name]
    E, R = len(counts), sum(counts)
    offsets = offsets_of(counts)
    top_k = 2 if gather else 1
    M = (R + 1) // 2 if gather else R
    perm = None
    if gather:
        perm = torch.randperm(M * top_k, generator=torch.Generator().manual_seed(seed + 9))[:R].to(torch.int32)
    return dict(E=E, R=R, N=N, K=K, M=M, offsets=offsets, perm=perm, top_k=top_k, x=randn(seed + 1, M, K),
                w=randn(seed + 2, E, N, K, scale=0.1), dy=randn(seed + 3, R, N))


def dev(t):
    return None if t is None else t.cuda()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("name", list(CASES))
def test_forward(name, gather, dtype):
    p = problem(name, gather)
    y = ops.grouped_matmul(dev(p["x"]), dev(p["w"]), dev(p["offsets"]), perm=dev(p["perm"]), top_k=p["top_k"],
                           out_dtype=dtype)
    want, tol = grouped_ref(take(p["x"], source_rows(p["R"], p["perm"], p["top_k"], p["M"])), p["w"], p["offsets"])
    close(y, want, tol + eps_of(dtype) * want.abs(), name)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("name", list(CASES))
def test_grad_input(name, dtype):
    p = problem(name, False)
    dx = ops.grouped_matmul_grad_input(dev(p["dy"]), dev(p["w"]), dev(p["offsets"]), out_dtype=dtype)
    want, tol = grad_input_ref(p["dy"], p["w"], p["offsets"])
    close(dx, want, tol + eps_of(dtype) * want.abs(), name)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("name", [n for n in CASES if n not in ("long_k", "decode")])
def test_grad_weight(name, gather, dtype):
    p = problem(name, gather)
    dw = ops.grouped_matmul_grad_weight(dev(p["x"]), dev(p["dy"]), dev(p["offsets"]), perm=dev(p["perm"]),
                                        top_k=p["top_k"], out_dtype=dtype)
    rows = take(p["x"], source_rows(p["R"], p["perm"], p["top_k"], p["M"]))
    want, tol = grad_weight_ref(rows, p["dy"], p["offsets"])
    close(dw, want, tol + eps_of(dtype) * want.abs(), name)


@pytest.mark.parametrize("few", [True, False])
def test_rows_behind_the_last_group_stay(few):
    counts = [3, 0, 4] if few else [300, 0, 90]
    R, extra = sum(counts), 37
    off = offsets_of(counts)
    x, w, dy = randn(1, R + extra, 128), randn(2, 3, 72, 128), randn(3, R + extra, 72)
    x[R:], dy[R:] = float("nan"), float("nan")
    y = torch.full((R + extra, 72), 7.0, dtype=BF16, device="cuda")
    dx = torch.full((R + extra, 128), 7.0, dtype=BF16, device="cuda")
    ops.grouped_matmul(dev(x), dev(w), dev(off), out=y)
    ops.grouped_matmul_grad_input(dev(dy), dev(w), dev(off), out=dx)
    dw = ops.grouped_matmul_grad_weight(dev(x), dev(dy), dev(off))
    assert (y[R:] == 7).all() and (dx[R:] == 7).all()
    want, tol = grouped_ref(x[:R].to(F8), w, off)
    close(y[:R], want, tol + eps_of(BF16) * want.abs(), "y")
    want, tol = grad_input_ref(dy[:R], w, off)
    close(dx[:R], want, tol + eps_of(BF16) * want.abs(), "dx")
    want, tol = grad_weight_ref(x[:R].to(F8), dy[:R], off)  # NaN behind the last group reach nothing
    close(dw, want, tol + EPS32 * want.abs(), "dw")


@pytest.mark.parametrize("few", [True, False])
def test_strided_rows_beside_nan(few):
    """Rows that are column slices of wider buffers: nothing beside them is read into a sum or written."""
    counts, N, K = ([2, 0, 7], 88, 200) if few else ([70, 300], 88, 200)
    R, off = sum(counts), offsets_of(counts)
    wide = lambda seed, r, c: torch.full((r, c + 24), float("nan"), dtype=BF16).index_copy_(
        1, torch.arange(8, 8 + c), randn(seed, r, c)).cuda()
    xb, dyb = wide(1, R, K), wide(2, R, N)
    x, dy, w = xb[:, 8:8 + K], dyb[:, 8:8 + N], randn(3, len(counts), N, K).cuda()
    yb = torch.full((R, N + 16), 5.0, dtype=BF16, device="cuda")
    dxb = torch.full((R, K + 16), 5.0, dtype=F32, device="cuda")
    ops.grouped_matmul(x, w, dev(off), out=yb[:, 8:8 + N])
    ops.grouped_matmul_grad_input(dy, w, dev(off), out=dxb[:, 8:8 + K])
    dw = ops.grouped_matmul_grad_weight(x, dy, dev(off))
    for b, n in ((yb, N), (dxb, K)):
        assert (b[:, :8] == 5).all() and (b[:, 8 + n:] == 5).all()
    want, tol = grouped_ref(x.cpu().to(F8), w.cpu(), off)
    close(yb[:, 8:8 + N], want, tol + eps_of(BF16) * want.abs(), "y")
    want, tol = grad_input_ref(dy.cpu(), w.cpu(), off)
    close(dxb[:, 8:8 + K], want, tol + EPS32 * want.abs(), "dx")
    want, tol = grad_weight_ref(x.cpu().to(F8), dy.cpu(), off)
    close(dw, want, tol + EPS32 * want.abs(), "dw")


@pytest.mark.parametrize("few", [True, False])
def test_permutation_entries_out_of_range_are_rows_of_zeros(few):
    counts = [5, 3] if few else [200, 90]
    R, off, M, k = sum(counts), offsets_of(counts), 20, 4
    perm = torch.randint(0, M * k, (R,), generator=torch.Generator().manual_seed(5)).to(torch.int32)
    perm[1], perm[4], perm[R - 1], perm[6] = -1, M * k, 2 ** 31 - 1, -2 ** 31
    x, w, dy = randn(1, M, 72), randn(2, 2, 40, 72), randn(3, R, 40)
    y = ops.grouped_matmul(dev(x), dev(w), dev(off), perm=dev(perm), top_k=k, out_dtype=F32)
    dw = ops.grouped_matmul_grad_weight(dev(x), dev(dy), dev(off), perm=dev(perm), top_k=k)
    rows = take(x, source_rows(R, perm, k, M))
    want, tol = grouped_ref(rows, w, off)
    close(y, want, tol + EPS32 * want.abs(), "y")
    assert (y[1] == 0).all() and (y[R - 1] == 0).all()
    want, tol = grad_weight_ref(rows, dy, off)
    close(dw, want, tol + EPS32 * want.abs(), "dw")


@pytest.mark.parametrize("off", [[-5, 3, 2 ** 30], [4, 2, 8], [0, 100, 3], [2 ** 31 - 1, -1, 0], [0, 0, 0]])
@pytest.mark.parametrize("rows", [8, 400])
def test_offsets_out_of_order_stay_in_bounds(off, rows):
    """Offsets that no routing makes: the calls end, and rows of no group are not written."""
    off = torch.tensor(off, dtype=torch.int32)
    x, w = randn(1, rows, 64).cuda(), randn(2, 2, 32, 64).cuda()
    guard = torch.full((rows + 64, 32), 3.0, dtype=BF16, device="cuda")
    ops.grouped_matmul(x, w, dev(off), out=guard[32:32 + rows])
    dx = ops.grouped_matmul_grad_input(randn(3, rows, 32).cuda(), w, dev(off))
    dw = ops.grouped_matmul_grad_weight(x, randn(3, rows, 32).cuda(), dev(off))
    torch.cuda.synchronize()
    assert (guard[:32] == 3).all() and (guard[32 + rows:] == 3).all()
    assert dx.shape == (rows, 64) and dw.shape == (2, 32, 64)
    if (off == 0).all():
        assert (guard == 3).all() and (dw == 0).all()


@pytest.mark.parametrize("few", [True, False])
def test_nonfinite_values_stay_in_their_rows_and_experts(few):
    counts = [4, 6, 2] if few else [100, 300, 90]
    R, off = sum(counts), offsets_of(counts)
    x, w, dy = randn(1, R, 136), randn(2, 3, 72, 136), randn(3, R, 72)
    x[counts[0]] = float("inf")  # the first row of expert 1
    dy[R - 1, 5] = float("nan")  # the last row of expert 2
    y = ops.grouped_matmul(dev(x), dev(w), dev(off))
    dx = ops.grouped_matmul_grad_input(dev(dy), dev(w), dev(off))
    dw = ops.grouped_matmul_grad_weight(dev(x), dev(dy), dev(off))
    torch.cuda.synchronize()
    bad = ~torch.isfinite(y).all(dim=1).cpu()
    assert bad.nonzero().flatten().tolist() == [counts[0]]
    bad = ~torch.isfinite(dx).all(dim=1).cpu()
    assert bad.nonzero().flatten().tolist() == [R - 1]
    assert torch.isfinite(dw[0]).all() and not torch.isfinite(dw[1]).any()
    assert torch.isnan(dw[2, 5]).all() and torch.isfinite(dw[2, :5]).all() and torch.isfinite(dw[2, 6:]).all()


@pytest.mark.parametrize("rows", [64, 65, 128, 129, 192, 193, 256])
@pytest.mark.parametrize("K", [8, 64, 72, 128, 136, 256, 320])
def test_every_tile_height_and_number_of_steps(rows, K):
    """One group of every height class of tile, reductions of one step up to five, the last one whole or
    not: every pipeline's beginning and end.  (N is large enough for the matrix-matrix kernel.)"""
    N = 16400
    x, w, dy = randn(1, rows, K), randn(2, 1, N, K), randn(3, rows, K)
    y = ops.grouped_matmul(dev(x), dev(w), None, out_dtype=F32)
    off = torch.tensor([0, rows])
    want, tol = grouped_ref(x.to(F8), w, off)
    close(y, want, tol + EPS32 * want.abs(), "y")
    wt = w[0, :600].t().contiguous()[None]  # [1, K, 600]: reduction over K again
    dx = ops.grouped_matmul_grad_input(dev(dy), dev(wt), None, out_dtype=F32)
    want, tol = grad_input_ref(dy, wt, off)
    close(dx, want, tol + EPS32 * want.abs(), "dx")


def test_no_rows():
    off = torch.zeros(5, dtype=torch.int32, device="cuda")
    e = torch.empty(0, 64, dtype=BF16, device="cuda")
    w = randn(1, 4, 32, 64).cuda()
    assert ops.grouped_matmul(e, w, off).shape == (0, 32)
    assert ops.grouped_matmul_grad_input(torch.empty(0, 32, dtype=BF16, device="cuda"), w, off).shape == (0, 64)
    dw = torch.full((4, 32, 64), 9.0, device="cuda")
    ops.grouped_matmul_grad_weight(e, torch.empty(0, 32, dtype=BF16, device="cuda"), off, out=dw)
    assert (dw == 0).all()


def test_gradients_against_differences():
    """The product is linear: <dy, y(x + d) - y(x)> = <dx, d> and the same in w, up to rounding."""
    p = problem("tall", True)
    x, w, dy, off, perm = (dev(p[n]) for n in ("x", "w", "dy", "offsets", "perm"))
    d = torch.randint(-2, 3, x.shape, generator=torch.Generator().manual_seed(3)).to(BF16).cuda()
    x = torch.round(x * 8) / 8  # x + d is exact in bf16
    f = lambda a, b: ops.grouped_matmul(a, b, off, perm=perm, top_k=2, out_dtype=F32).to(F8)
    dx = ops.grouped_matmul_grad_input(dy, w, off, out_dtype=F32).to(F8)
    src = source_rows(p["R"], p["perm"], 2, p["M"]).cuda()
    lhs = (dy.to(F8) * (f(x + d, w) - f(x, w))).sum()
    rhs = (dx * d.to(F8)[src]).sum()
    # both sides sum R * N products of magnitudes up to |dy| |y| with relative errors of K * 2^-23
    mag = (dy.to(F8).abs() * (f((x + d).abs(), w.abs()) + f(x.abs(), w.abs()))).sum()
    assert abs(lhs - rhs) <= 2 * 2 * EPS32 * p["K"] * mag
    dw = ops.grouped_matmul_grad_weight(x, dy, off, perm=perm, top_k=2).to(F8)
    w8 = torch.round(w * 64) / 64
    e = torch.randint(-2, 3, w.shape, generator=torch.Generator().manual_seed(4)).to(BF16).cuda() / 64
    lhs = (dy.to(F8) * (f(x, w8 + e) - f(x, w8))).sum()
    rhs = (dw * e.to(F8)).sum()
    mag = (dy.to(F8).abs() * (f(x.abs(), (w8 + e).abs()) + f(x.abs(), w8.abs()))).sum()
    assert abs(lhs - rhs) <= 2 * 2 * EPS32 * max(p["K"], p["R"]) * mag


@pytest.mark.parametrize("name", ["small_batch", "tall"])
def test_repeated_calls_give_the_same_bits(name):
    p = {k: dev(v) if torch.is_tensor(v) else v for k, v in problem(name, True).items()}
    f = lambda: (ops.grouped_matmul(p["x"], p["w"], p["offsets"], perm=p["perm"], top_k=2, out_dtype=F32),
                 ops.grouped_matmul_grad_input(p["dy"], p["w"], p["offsets"], out_dtype=F32),
                 ops.grouped_matmul_grad_weight(p["x"], p["dy"], p["offsets"], perm=p["perm"], top_k=2))
    a, b = f(), f()
    assert all(torch.equal(i, j) for i, j in zip(a, b))


def test_binding_refusals():
    p = {k: dev(v) if torch.is_tensor(v) else v for k, v in problem("ragged", True).items()}
    ok = dict(perm=p["perm"], top_k=2)
    with pytest.raises(ValueError, match="offsets"):
        ops.grouped_matmul(p["x"], p["w"], p["offsets"][:-1], **ok)
    with pytest.raises(TypeError, match="offsets"):
        ops.grouped_matmul(p["x"], p["w"], p["offsets"].long(), **ok)
    with pytest.raises(ValueError, match="w must be contiguous"):
        ops.grouped_matmul(p["x"], p["w"].transpose(0, 1).contiguous().transpose(0, 1), p["offsets"], **ok)
    with pytest.raises(ValueError, match="contiguous rows"):
        ops.grouped_matmul(p["x"].t().contiguous().t(), p["w"], p["offsets"], **ok)
    with pytest.raises(ValueError, match="overlapping"):
        ops.grouped_matmul(p["x"][:1].expand(p["M"], -1), p["w"], p["offsets"], **ok)
    with pytest.raises(ValueError, match="perm"):
        ops.grouped_matmul(p["x"], p["w"], p["offsets"], perm=p["perm"][:-1], top_k=2,
                           out=torch.empty(p["R"], p["N"], dtype=BF16, device="cuda"))
    with pytest.raises(ValueError, match="offsets"):
        ops.grouped_matmul(p["x"], p["w"], None, **ok)
    with pytest.raises(ops.MoeError, match="INVALID_ARG"):
        ops.grouped_matmul(p["x"], p["w"], p["offsets"], top_k=1, out=torch.empty(p["R"] + 400, p["N"], dtype=BF16,
                                                                                  device="cuda"))
    with pytest.raises(ops.MoeError, match="UNSUPPORTED_SHAPE"):
        ops.grouped_matmul(torch.zeros(4, 12, dtype=BF16, device="cuda"),
                           torch.zeros(1, 8, 12, dtype=BF16, device="cuda"), None)
    with pytest.raises(ops.MoeError, match="MISALIGNED"):
        flat = torch.zeros(4 * 64 + 8, dtype=BF16, device="cuda")
        ops.grouped_matmul(flat[4:4 + 256].view(4, 64), torch.zeros(1, 8, 64, dtype=BF16, device="cuda"), None)

"""The norms around a block and their gradients against plain 64-bit forms."""
import pytest
import torch

from sparse_moe_router_amd import ops
from ops_util import EPS32, F8, close, eps_of, merge_grad_ref, merge_ref, randn, rms, rms_grad, sum_terms

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
EPS = 1e-6

# one row, few and many rows; H of one chunk, at and off the edges of every thread plan
SHAPES = [(1, 8), (1, 2048), (3, 512), (5, 520), (9, 1032), (4, 2056), (6, 4104), (3, 8200), (2, 16384), (1024, 64),
          (1025, 512), (1031, 1000), (1100, 1032), (1026, 2048), (1025, 2056)]


def tensors(M, H, stream, weight, gate, seed=0):
    g = None if gate == "none" else randn(seed + 3, *((M,) if gate == "token" else (M, H)), scale=2.0)
    return dict(x=randn(seed + 1, M, H, dtype=stream), y=randn(seed + 2, M, H, scale=0.5), gate=g,
                w=(randn(seed + 4, H, scale=0.1, dtype=F32) + 1).to(weight),
                wn=(randn(seed + 5, H, scale=0.1, dtype=F32) + 1).to(weight))


def dev(t):
    return None if t is None else t.cuda()


def f8(t):
    return None if t is None else t.cpu().to(F8)


@pytest.mark.parametrize("stream,weight", [(BF16, BF16), (F32, F32), (F32, BF16)])
@pytest.mark.parametrize("M,H", SHAPES)
def test_block_norm(M, H, stream, weight):
    t = tensors(M, H, stream, weight, "none")
    h = ops.block_norm(dev(t["x"]), dev(t["w"]), EPS)
    want = rms(f8(t["x"]), f8(t["w"]), EPS)
    close(h, want, (sum_terms(H) * EPS32 + eps_of(BF16)) * want.abs())


@pytest.mark.parametrize("gate", ["none", "token", "element"])
@pytest.mark.parametrize("stream,weight", [(BF16, BF16), (F32, F32)])
@pytest.mark.parametrize("M,H", SHAPES)
def test_merge(M, H, stream, weight, gate):
    t = tensors(M, H, stream, weight, gate)
    out, h = ops.block_merge(dev(t["x"]), dev(t["y"]), dev(t["w"]), EPS, gate=dev(t["gate"]), scale=0.3,
                             next_weight=dev(t["wn"]))
    only = ops.block_merge(dev(t["x"]), dev(t["y"]), dev(t["w"]), EPS, gate=dev(t["gate"]), scale=0.3)
    assert torch.equal(out, only)
    want = merge_ref(f8(t["x"]), f8(t["y"]), f8(t["w"]), EPS, f8(t["gate"]), 0.3)
    branch = (want - f8(t["x"])).abs()
    close(out, want, sum_terms(H) * EPS32 * branch + (EPS32 + eps_of(stream)) * want.abs(), "out")
    wh = rms(f8(out), f8(t["wn"]), EPS)  # of the stored stream
    close(h, wh, (sum_terms(H) * EPS32 + eps_of(BF16)) * wh.abs(), "h")


@pytest.mark.parametrize("add", [False, True])
@pytest.mark.parametrize("stream,weight", [(BF16, BF16), (F32, F32)])
@pytest.mark.parametrize("M,H", SHAPES)
def test_block_norm_grad(M, H, stream, weight, add):
    t = tensors(M, H, stream, weight, "none")
    d_h, d_add = randn(7, M, H), randn(8, M, H, dtype=stream) if add else None
    g = ops.block_norm_grad(dev(d_h), dev(t["x"]), dev(t["w"]), EPS, d_add=dev(d_add))
    dv, mag, dw = rms_grad(f8(d_h), f8(t["x"]), f8(t["w"]), EPS)
    if add:
        dv, mag = dv + f8(d_add), mag + f8(d_add).abs()
    assert g["x"].dtype == stream and g["weight"].dtype == F32
    close(g["x"], dv, 3 * sum_terms(H) * EPS32 * mag + eps_of(stream) * dv.abs(), "dx")
    close(g["weight"], dw.sum(0), (sum_terms(H) + M) * EPS32 * dw.abs().sum(0), "dw")


@pytest.mark.parametrize("ends", ["both", "out", "h"])
@pytest.mark.parametrize("gate", ["none", "token", "element"])
@pytest.mark.parametrize("stream,weight", [(BF16, BF16), (F32, F32)])
@pytest.mark.parametrize("M,H", SHAPES)
def test_merge_grad(M, H, stream, weight, gate, ends):
    t = tensors(M, H, stream, weight, gate)
    out = randn(6, M, H, dtype=stream)
    d_out = randn(7, M, H, dtype=stream) if ends != "h" else None
    d_h = randn(8, M, H) if ends != "out" else None
    nxt = dict(next_weight=dev(t["wn"]), out=dev(out), d_h=dev(d_h)) if ends != "out" else {}
    g = ops.block_merge_grad(dev(d_out), dev(t["y"]), dev(t["w"]), EPS, gate=dev(t["gate"]), scale=0.3, **nxt)
    want = merge_grad_ref(f8(d_out), f8(d_h), f8(t["y"]), f8(t["w"]), EPS, f8(t["gate"]), 0.3, f8(out), f8(t["wn"]))
    assert set(g) == set(want)
    for n, (v, mag) in want.items():
        # the residual's gradient, the branch's and theirs build on one another: three statistics
        # deep, each within sum_terms; the weights' sums run over the rows as well, a token gate's
        # over the row
        terms = 6 * sum_terms(H) + (M if "weight" in n else 0)
        close(g[n], v, terms * EPS32 * mag + eps_of(g[n].dtype) * v.abs(), n)


def test_reference_gradients_against_differences():
    """The formulas themselves: central differences of the 64-bit forward form."""
    M, H, h = 3, 16, 1e-6
    t = {k: f8(v) for k, v in tensors(M, H, F32, F32, "element").items()}
    d_out, d_h = f8(randn(7, M, H, dtype=F32)), f8(randn(8, M, H, dtype=F32))

    def loss(v):
        out = merge_ref(v["x"], v["y"], v["w"], EPS, v["gate"], 0.3)
        return (out * d_out).sum() + (rms(out, v["wn"], EPS) * d_h).sum()

    out = merge_ref(t["x"], t["y"], t["w"], EPS, t["gate"], 0.3)
    g = merge_grad_ref(d_out, d_h, t["y"], t["w"], EPS, t["gate"], 0.3, out, t["wn"])
    for n, key in (("x", "residual"), ("y", "y"), ("w", "weight"), ("gate", "gate"), ("wn", "next_weight")):
        d = f8(randn(9, *t[n].shape, dtype=F32))
        up, dn = dict(t), dict(t)
        up[n], dn[n] = t[n] + h * d, t[n] - h * d
        diff = (loss(up) - loss(dn)) / (2 * h)
        # truncation h^2 and cancellation 2^-53 / h, times values of order 100
        assert abs(diff - (g[key][0] * d).sum()) < 1e-6, n


def test_gradients_against_differences_of_the_kernels():
    """Directional differences of the forward kernels with an fp32 stream."""
    M, H, s = 64, 256, 2.0 ** -6
    t = {k: dev(v) for k, v in tensors(M, H, F32, F32, "none").items()}
    d_out = randn(7, M, H, dtype=F32).cuda()
    f = lambda y, w: (ops.block_merge(t["x"], y, w, EPS, scale=0.3).to(F8) * d_out.to(F8)).sum()
    g = ops.block_merge_grad(d_out, t["y"], t["w"], EPS, scale=0.3)
    d = randn(9, H, dtype=F32).cuda()
    # linear in the weight: no truncation; 2 M H results with errors of 2^-24 of values below 8
    diff = (f(t["y"], t["w"] + s * d) - f(t["y"], t["w"] - s * d)) / (2 * s)
    want = (g["weight"].to(F8) * d.to(F8)).sum()
    assert abs(diff - want) <= 8 * EPS32 * sum_terms(H) * d_out.to(F8).abs().sum() / s


@pytest.mark.parametrize("M", [3, 1100])
def test_strided_rows(M):
    H = 264
    wide = lambda seed, dt: torch.full((M, H + 24), float("nan"), dtype=dt).index_copy_(
        1, torch.arange(8, 8 + H), randn(seed, M, H, dtype=dt)).cuda()
    cut = lambda b: b[:, 8:8 + H]
    x, y, gate, d_out, d_h, out = (wide(i, dt) for i, dt in enumerate((F32, BF16, BF16, F32, BF16, F32)))
    w, wn = randn(7, H, dtype=F32).cuda(), randn(8, H, dtype=F32).cuda()
    ob, hb = torch.full((M, H + 16), 5.0, device="cuda"), torch.full((M, H + 32), 5.0, dtype=BF16, device="cuda")
    a = ops.block_merge(cut(x), cut(y), w, EPS, gate=cut(gate), scale=0.3, next_weight=wn, out=ob[:, 8:8 + H],
                        h=hb[:, 16:16 + H])
    c = lambda b: cut(b).contiguous()
    b = ops.block_merge(c(x), c(y), w, EPS, gate=c(gate), scale=0.3, next_weight=wn)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert (ob[:, :8] == 5).all() and (ob[:, 8 + H:] == 5).all() and (hb[:, :16] == 5).all()
    kw = dict(scale=0.3, next_weight=wn)
    a = ops.block_merge_grad(cut(d_out), cut(y), w, EPS, gate=cut(gate), out=cut(out), d_h=cut(d_h), **kw)
    b = ops.block_merge_grad(c(d_out), c(y), w, EPS, gate=c(gate), out=c(out), d_h=c(d_h), **kw)
    assert all(torch.equal(a[n], b[n]) for n in b)


def test_extreme_gates_and_zero_rows():
    M, H = 4, 64
    x, y, w = randn(1, M, H, dtype=F32).cuda(), randn(2, M, H).cuda(), torch.ones(H, device="cuda")
    y[1] = 0
    gate = torch.tensor([200.0, 0.0, -200.0, 20.0], dtype=BF16).cuda()
    out = ops.block_merge(x, y, w, EPS, gate=gate)
    assert torch.equal(out[1], x[1]) and torch.equal(out[2], x[2]) and torch.isfinite(out).all()
    g = ops.block_merge_grad(torch.ones_like(x), y, w, EPS, gate=gate)
    assert all(torch.isfinite(v).all() for v in g.values())
    # the slope of a wide open gate keeps its relative accuracy: sigmoid(-20)
    want = merge_grad_ref(torch.ones(M, H, dtype=F8), None, f8(y), f8(w), EPS, f8(gate), 1.0, None, None)["gate"]
    close(g["gate"][3:], want[0][3:], 6 * sum_terms(H) * EPS32 * want[1][3:] + eps_of(BF16) * want[0][3:].abs(), "gate")


def test_nonfinite_rows_stay_alone():
    M, H = 6, 128
    x, y, w = randn(1, M, H), randn(2, M, H), torch.ones(H, dtype=BF16)
    x[2, 5], y[4, 7] = float("nan"), float("inf")
    out, h = ops.block_merge(x.cuda(), y.cuda(), w.cuda(), EPS, next_weight=w.cuda())
    fin = torch.isfinite(h).all(dim=1).cpu()
    assert fin.tolist() == [True, True, False, True, False, True]
    assert torch.isfinite(out[[0, 1, 3, 5]]).all()


def test_no_rows():
    e = lambda dt=BF16: torch.empty(0, 64, dtype=dt, device="cuda")
    w = torch.ones(64, dtype=BF16, device="cuda")
    assert ops.block_norm(e(), w, EPS).shape == (0, 64)
    out, h = ops.block_merge(e(), e(), w, EPS, next_weight=w)
    assert out.shape == h.shape == (0, 64)
    g = ops.block_merge_grad(e(), e(), w, EPS, next_weight=w, out=e(), d_h=e())
    assert (g["weight"] == 0).all() and (g["next_weight"] == 0).all()
    assert (ops.block_norm_grad(e(), e(), w, EPS)["weight"] == 0).all()


def test_binding_refusals():
    x, w = randn(1, 4, 64).cuda(), torch.ones(64, dtype=BF16, device="cuda")
    with pytest.raises(ValueError, match="given together"):
        ops.block_merge_grad(x, x, w, EPS, d_h=x)
    with pytest.raises(ValueError, match="d_out or d_h"):
        ops.block_merge_grad(None, x, w, EPS)
    with pytest.raises(ValueError, match="h needs"):
        ops.block_merge(x, x.clone(), w, EPS, h=torch.empty_like(x))
    with pytest.raises(TypeError, match="next_weight"):
        ops.block_merge(x, x.clone(), w, EPS, next_weight=w.float())
    with pytest.raises(TypeError, match="gate"):
        ops.block_merge(x, x.clone(), w, EPS, gate=torch.zeros(4, device="cuda"))
    with pytest.raises(ValueError, match="gate"):
        ops.block_merge(x, x.clone(), w, EPS, gate=torch.zeros(5, dtype=BF16, device="cuda"))
    with pytest.raises(ops.MoeError, match="INVALID_ARG"):
        ops.block_merge(x, x.clone(), w, EPS, out=x)
    with pytest.raises(ops.MoeError, match="INVALID_ARG"):
        ops.block_norm(x, w, 0.0)

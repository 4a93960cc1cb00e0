"""The norms over the range of eps and of the rows' magnitudes, and streams and weights of different types,
against 64 bits."""
import pytest
import torch

from ops_util import EPS32, F8, close, eps_of, merge_grad_ref, merge_ref, randn, rms, rms_grad, sum_terms
from sparse_moe_router_amd import ops

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
EPS = 1e-28  # rows of 1e-13 have factors of 1e13, whose cube is past fp32


def rows(seed, M, H, dtype, first):
    """Rows of zeros, of sizes about 1e-13, 1 and 1e15, in turn."""
    s = torch.tensor([0.0, 1e-13, 1.0, 1e15])[(torch.arange(M) + first) % 4]
    return (randn(seed, M, H, dtype=F32) * s[:, None]).to(dtype)


def dev(t):
    return None if t is None else t.cuda()


def f8(t):
    return None if t is None else t.to(F8)


@pytest.mark.parametrize("stream,weight", [(BF16, BF16), (F32, F32)])
@pytest.mark.parametrize("M,H", [(5, 264), (6, 2056), (7, 8200), (1100, 264)])
def test_block_norm_grad(M, H, stream, weight):
    x, d_h, w = rows(1, M, H, stream, 0), randn(2, M, H), (randn(3, H, scale=0.1, dtype=F32) + 1).to(weight)
    g = ops.block_norm_grad(dev(d_h), dev(x), dev(w), EPS)
    dv, mag, dw = rms_grad(f8(d_h), f8(x), f8(w), EPS)
    close(g["x"], dv, 3 * sum_terms(H) * EPS32 * mag + eps_of(stream) * dv.abs(), "dx")
    close(g["weight"], dw.sum(0), (sum_terms(H) + M) * EPS32 * dw.abs().sum(0), "dw")


@pytest.mark.parametrize("ends", ["both", "h"])
@pytest.mark.parametrize("gate", ["none", "token", "element"])
@pytest.mark.parametrize("stream,weight", [(BF16, BF16), (F32, F32)])
@pytest.mark.parametrize("M,H", [(5, 264), (6, 2056), (7, 8200), (1100, 264)])
def test_block_merge_grad(M, H, stream, weight, gate, ends):
    y, out = rows(1, M, H, BF16, 0), rows(2, M, H, stream, 1)  # a block's rows and the stream's differ in size
    gt = None if gate == "none" else randn(3, *((M,) if gate == "token" else (M, H)), scale=2.0)
    w, wn = ((randn(s, H, scale=0.1, dtype=F32) + 1).to(weight) for s in (4, 5))
    d_out, d_h = randn(6, M, H, dtype=stream) if ends == "both" else None, randn(7, M, H)
    g = ops.block_merge_grad(dev(d_out), dev(y), dev(w), EPS, gate=dev(gt), scale=0.3, next_weight=dev(wn),
                             out=dev(out), d_h=dev(d_h))
    want = merge_grad_ref(f8(d_out), f8(d_h), f8(y), f8(w), EPS, f8(gt), 0.3, f8(out), f8(wn))
    for n, (v, mag) in want.items():
        terms = 6 * sum_terms(H) + (M if "weight" in n else 0)  # as at ordinary sizes
        close(g[n], v, terms * EPS32 * mag + eps_of(g[n].dtype) * v.abs(), n)


@pytest.mark.parametrize("gate", ["none", "token", "element"])
@pytest.mark.parametrize("stream,weight", [(BF16, F32), (F32, BF16)])
@pytest.mark.parametrize("M,H", [(1, 2048), (5, 264), (6, 4104), (7, 16384), (1027, 520), (1026, 2056)])
def test_stream_and_weights_of_different_types(M, H, stream, weight, gate):
    """Every operator with a bf16 stream and fp32 weights and the other way round, at ordinary sizes."""
    eps = 1e-6
    x, y, out, d_out = (randn(s, M, H, dtype=dt) for s, dt in ((1, stream), (2, BF16), (3, stream), (4, stream)))
    d_h = randn(5, M, H)
    gt = None if gate == "none" else randn(6, *((M,) if gate == "token" else (M, H)), scale=2.0)
    w, wn = ((randn(s, H, scale=0.1, dtype=F32) + 1).to(weight) for s in (7, 8))
    n = sum_terms(H)
    if gate == "none":
        want = rms(f8(x), f8(w), eps)
        close(ops.block_norm(dev(x), dev(w), eps), want, (n * EPS32 + eps_of(BF16)) * want.abs(), "norm")
        g = ops.block_norm_grad(dev(d_h), dev(x), dev(w), eps, d_add=dev(d_out))
        dv, mag, dw = rms_grad(f8(d_h), f8(x), f8(w), eps)
        dv, mag = dv + f8(d_out), mag + f8(d_out).abs()
        assert g["x"].dtype == stream and g["weight"].dtype == F32
        close(g["x"], dv, 3 * n * EPS32 * mag + eps_of(stream) * dv.abs(), "dx")
        close(g["weight"], dw.sum(0), (n + M) * EPS32 * dw.abs().sum(0), "dw")
    got, h = ops.block_merge(dev(x), dev(y), dev(w), eps, gate=dev(gt), scale=0.3, next_weight=dev(wn))
    want = merge_ref(f8(x), f8(y), f8(w), eps, f8(gt), 0.3)
    close(got, want, n * EPS32 * (want - f8(x)).abs() + (EPS32 + eps_of(stream)) * want.abs(), "out")
    wh = rms(f8(got.cpu()), f8(wn), eps)
    close(h, wh, (n * EPS32 + eps_of(BF16)) * wh.abs(), "h")
    g = ops.block_merge_grad(dev(d_out), dev(y), dev(w), eps, gate=dev(gt), scale=0.3, next_weight=dev(wn), out=dev(out),
                             d_h=dev(d_h))
    for name, (v, mag) in merge_grad_ref(f8(d_out), f8(d_h), f8(y), f8(w), eps, f8(gt), 0.3, f8(out), f8(wn)).items():
        terms = 6 * n + (M if "weight" in name else 0)
        close(g[name], v, terms * EPS32 * mag + eps_of(g[name].dtype) * v.abs(), name)

"""The 8-bit products and the token quantiser against plain 64-bit forms."""
import pytest
import torch

from sparse_moe_router_amd import ops
from ops_util import EPS32, F8, close, eps_of, offsets_of, quantize_ref, randn, source_rows

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def codes(seed, *shape):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(-127, 128, shape, generator=g, dtype=torch.int8)


def scales(seed, *shape):
    g = torch.Generator().manual_seed(seed)
    return torch.rand(shape, generator=g) * 0.01 + 1e-3


def i8_ref(q, s, w, ws, bias=None):
    """(y, tolerance without the rounding to the output's type).  The integer sum is exact; its
    conversion, the two scales' product, the product with them and the token's scale itself round once
    each, and so does the sum with a bias."""
    y = (q @ w.to(F8).t()) * (s[:, None] * ws.to(F8))
    tol = 5 * EPS32 * y.abs()
    if bias is not None:
        y = y + bias.to(F8)
        tol = tol + EPS32 * y.abs()
    return y, tol


QUANT = [(1, 16), (1, 2048), (3, 48), (5, 528), (7, 2064), (2, 4112), (3, 8208), (2, 16384), (1025, 64), (1300, 1040),
         (1027, 2048), (1024, 2064)]


@pytest.mark.parametrize("M,K", QUANT)
def test_quantize(M, K):
    x = randn(1, M, K, scale=3.0)
    if M > 2:
        x[1] = 0
        x[2, :7] = torch.tensor([1.0, -1.0, 0.5, 0.25, 3.0, -127.0, 127.0])
        x[2, 7:] = 0
    q, s = ops.quantize_i8(x.cuda())
    want_q, want_s = quantize_ref(x)
    assert q.dtype == torch.int8 and torch.equal(q.cpu().to(F8), want_q)
    close(s, want_s, EPS32 * want_s, "scale")


def test_quantize_borders_and_extremes():
    """Every bf16 magnitude against several row maxima: codes equal the exact ones, borders included."""
    bits = torch.arange(0, 0x7F80, dtype=torch.int32).to(torch.int16)
    vals = bits.view(BF16)
    rows = []
    for m in (1.0, 1.0078125, 1.5, 1.9921875, 127.0, 127.5, 254.0, 3e-39, 1e-40, 2.0 ** 120, 3.3e38):
        mx = torch.tensor(m, dtype=BF16)
        v = vals[vals.float() <= mx.float()]
        v = v[-16384 + 16:]  # the magnitudes next to the maximum
        row = torch.zeros(16384, dtype=BF16)
        row[:len(v)] = v * torch.where(torch.arange(len(v)) % 2 == 0, 1, -1).to(BF16)
        row[16383] = mx
        rows.append(row)
    x = torch.stack(rows)
    q, s = ops.quantize_i8(x.cuda())
    want_q, want_s = quantize_ref(x)
    assert torch.equal(q.cpu().to(F8), want_q)
    # scales below the normal range keep their absolute accuracy: half of 2^-149
    close(s, want_s, EPS32 * want_s + 2.0 ** -150, "scale")


def test_quantize_nonfinite_rows():
    x = randn(1, 6, 64)
    x[1, 3], x[2, 5], x[3, 0], x[3, 1] = float("inf"), float("nan"), float("-inf"), float("nan")
    q, s = ops.quantize_i8(x.cuda())
    want_q, want_s = quantize_ref(x)
    assert torch.equal(q.cpu().to(F8), want_q)
    assert torch.isinf(s[1]) and torch.isnan(s[2]) and torch.isnan(s[3])
    y = ops.matmul_i8(x.cuda(), codes(2, 32, 64).cuda(), scales(3, 32).cuda())
    bad = torch.isnan(y).all(dim=1).cpu()
    assert bad.tolist() == [False, True, True, True, False, False]
    assert torch.isfinite(y[~bad.cuda()]).all()


DENSE = [(3, 24, 4112), (4, 72, 2064), (2, 40, 8192), (1, 16, 16384), (1, 8, 16), (1, 4096, 2048), (2, 136, 528), (16, 264, 272), (17, 72, 64), (33, 1000, 144), (64, 40, 16384),
         (65, 520, 1040), (257, 264, 2064), (600, 328, 4112)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("given", ["bf16", "codes"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("M,N,K", DENSE)
def test_matmul(M, N, K, bias, given, dtype):
    x, w, ws = randn(1, M, K), codes(2, N, K), scales(3, N)
    b = randn(4, N, dtype=F32) if bias else None
    q, s = quantize_ref(x)
    kw = dict(bias=None if b is None else b.cuda(), out_dtype=dtype)
    if given == "codes":
        xs = s.float()
        y = ops.matmul_i8(q.to(torch.int8).cuda(), w.cuda(), ws.cuda(), x_scale=xs.cuda(), **kw)
        s = xs.to(F8)
    else:
        y = ops.matmul_i8(x.cuda(), w.cuda(), ws.cuda(), **kw)
    want, tol = i8_ref(q, s, w, ws, b)
    close(y, want, tol + eps_of(dtype) * want.abs(), f"{M} {N} {K}")


@pytest.mark.parametrize("rows", [64, 65, 128, 129, 192, 193, 256])
@pytest.mark.parametrize("K", [16, 128, 144, 256, 272, 512, 640])
def test_every_tile_height_and_number_of_steps(rows, K):
    N = 16400
    q, w, ws, xs = codes(1, rows, K), codes(2, N, K), scales(3, N), scales(4, rows)
    y = ops.matmul_i8(q.cuda(), w.cuda(), ws.cuda(), x_scale=xs.cuda(), out_dtype=F32)
    want, tol = i8_ref(q.to(F8), xs.to(F8), w, ws)
    close(y, want, tol + EPS32 * want.abs())


def test_extreme_codes_do_not_overflow():
    """The largest sum: K = 16384 products of -128 with -128, 2^28."""
    for M in (1, 300):
        q = torch.full((M, 16384), -128, dtype=torch.int8)
        w = torch.full((24, 16384), -128, dtype=torch.int8)
        y = ops.matmul_i8(q.cuda(), w.cuda(), torch.ones(24, device="cuda"), x_scale=torch.ones(M, device="cuda"),
                          out_dtype=F32)
        assert (y == 2.0 ** 28).all()


GROUPED = {
    "ragged": ([0, 1, 0, 17, 0, 256, 3, 0], 264, 208),
    "edges": ([15, 16, 17, 31, 32, 33, 63, 64, 65, 255, 257], 72, 144),
    "decode": ([0] * 100 + [1, 0, 1, 1] + [0] * 120 + [1] * 5 + [0] * 27, 256, 2048),
    "tall": ([300, 0, 33, 513], 520, 528),
    "many": ([i % 3 for i in range(1024)], 16, 80),
}


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("given", ["bf16", "codes"])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("name", list(GROUPED))
def test_grouped(name, gather, given, dtype):
    counts, N, K = GROUPED[name]
    E, R, off = len(counts), sum(counts), offsets_of(counts)
    k = 2 if gather else 1
    M = (R + 1) // 2 if gather else R
    perm = torch.randperm(M * k, generator=torch.Generator().manual_seed(7))[:R].to(torch.int32) if gather else None
    if gather:
        perm[0] = -1  # a row of zeros
    x, w, ws = randn(1, M, K), codes(2, E, N, K), scales(3, E, N)
    q, s = quantize_ref(x)
    kw = dict(perm=None if perm is None else perm.cuda(), top_k=k, out_dtype=dtype)
    if given == "codes":
        xs = s.float()
        y = ops.grouped_matmul_i8(q.to(torch.int8).cuda(), w.cuda(), ws.cuda(), off.cuda(), x_scale=xs.cuda(), **kw)
        s = xs.to(F8)
    else:
        y = ops.grouped_matmul_i8(x.cuda(), w.cuda(), ws.cuda(), off.cuda(), **kw)
    src = source_rows(R, perm, k, M)
    qr = torch.where((src >= 0)[:, None], q[src.clamp(min=0)], torch.zeros((), dtype=F8))
    sr = torch.where(src >= 0, s[src.clamp(min=0)], torch.zeros((), dtype=F8))
    want, tol = torch.zeros(R, N, dtype=F8), torch.zeros(R, N, dtype=F8)
    for e in range(E):
        a, b = int(off[e]), int(off[e + 1])
        want[a:b], tol[a:b] = i8_ref(qr[a:b], sr[a:b], w[e], ws[e])
    close(y, want, tol + eps_of(dtype) * want.abs(), name)


@pytest.mark.parametrize("M", [5, 300])
def test_strided_codes_and_output(M):
    N, K = 40, 208
    qb = codes(1, M, K + 48)
    q, w, ws, xs = qb[:, 16:16 + K], codes(2, N, K), scales(3, N), scales(4, M)
    yb = torch.full((M, N + 16), 5.0, device="cuda")
    ops.matmul_i8(qb.cuda()[:, 16:16 + K], w.cuda(), ws.cuda(), x_scale=xs.cuda(), out=yb[:, 8:8 + N])
    want, tol = i8_ref(q.to(F8), xs.to(F8), w, ws)
    close(yb[:, 8:8 + N], want, tol + EPS32 * want.abs())
    assert (yb[:, :8] == 5).all() and (yb[:, 8 + N:] == 5).all()
    xb = torch.full((M, K + 24), float("nan"), dtype=BF16)
    xb[:, 8:8 + K] = randn(5, M, K)
    y = ops.matmul_i8(xb.cuda()[:, 8:8 + K], w.cuda(), ws.cuda(), out_dtype=F32)
    qr, sr = quantize_ref(xb[:, 8:8 + K])
    want, tol = i8_ref(qr, sr, w, ws)
    close(y, want, tol + EPS32 * want.abs())


def test_rows_without_tokens():
    """A permutation of rows that no token backs: rows of zeros, for bf16 tokens and for codes."""
    w, ws = codes(1, 2, 32, 64).cuda(), scales(2, 2, 32).cuda()
    off, perm = offsets_of([3, 40]).cuda(), torch.arange(43, dtype=torch.int32, device="cuda")
    for x, xs in ((torch.empty(0, 64, dtype=BF16, device="cuda"), None),
                  (torch.empty(0, 64, dtype=torch.int8, device="cuda"), torch.empty(0, device="cuda"))):
        y = ops.grouped_matmul_i8(x, w, ws, off, perm=perm, top_k=2, x_scale=xs)
        assert y.shape == (43, 32) and (y == 0).all()


def test_no_rows_and_refusals():
    w, ws = codes(1, 32, 64).cuda(), scales(2, 32).cuda()
    assert ops.matmul_i8(torch.empty(0, 64, dtype=BF16, device="cuda"), w, ws).shape == (0, 32)
    x = randn(1, 4, 64).cuda()
    with pytest.raises(ValueError, match="x_scale"):
        ops.matmul_i8(codes(1, 4, 64).cuda(), w, ws)
    with pytest.raises(ValueError, match="x_scale"):
        ops.matmul_i8(x, w, ws, x_scale=torch.ones(4, device="cuda"))
    with pytest.raises(ValueError, match="bias"):
        ops.matmul_i8(x, w, ws, bias=torch.zeros(31, device="cuda"))
    with pytest.raises(ValueError, match="w_scale"):
        ops.matmul_i8(x, w, ws[:-1])
    with pytest.raises(ValueError, match="out"):
        ops.matmul_i8(x, w, ws, out=torch.empty(5, 32, dtype=BF16, device="cuda"))
    with pytest.raises(ops.MoeError, match="WORKSPACE_TOO_SMALL"):
        ops.matmul_i8(randn(1, 40, 64).cuda(), w, ws, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))

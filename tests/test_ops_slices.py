"""Activations that are column slices of one buffer: the overlap check against every byte (on the CPU),
and the operators on slices side by side."""
import ctypes
import os
import random
import shutil
import subprocess

import pytest
import torch

from ops_util import offsets_of, randn
from sparse_moe_router_amd import ops

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF16, F32 = torch.bfloat16, torch.float32
EPS = 1e-6


@pytest.fixture(scope="module")
def overlap(tmp_path_factory):
    """overlap() of two [rows][cols] matrices given as (address, rows, ld, cols, bytes an element)."""
    if not shutil.which("g++"):
        pytest.skip("no host compiler")
    d = tmp_path_factory.mktemp("regions")
    (d / "r.cpp").write_text(
        '#include "regions.h"\nusing namespace moe;\nextern "C" int f(uint64_t p, int64_t r, int64_t l, int64_t c, int e,'
        ' uint64_t q, int64_t s, int64_t m, int64_t k, int g) {\n'
        "  return overlap(matrix_at((void*)p, r, l, c, e), matrix_at((void*)q, s, m, k, g)); }\n")
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-shared", "-fPIC", "-I",
                    os.path.join(ROOT, "sparse_moe_router_amd", "csrc"), str(d / "r.cpp"), "-o", str(d / "r.so")], check=True)
    f = ctypes.CDLL(str(d / "r.so")).f
    i, u, n = ctypes.c_int64, ctypes.c_uint64, ctypes.c_int
    f.argtypes = [u, i, i, i, n, u, i, i, i, n]
    return lambda a, b: bool(f(*a, *b))


def taken(m):
    p, rows, ld, cols, es = m
    return {p + r * ld * es + c for r in range(rows) for c in range(cols * es)}


def test_overlap_of_matrices(overlap):
    """Matrices that share a byte always overlap; column slices that lie side by side do not."""
    rng = random.Random(1)
    interleaved = 0
    for _ in range(20000):
        pitch = rng.choice([8, 12, 16])
        m = []
        for _ in range(2):
            es = rng.choice([1, 2, 4])
            ld = (pitch if rng.random() < 0.8 else rng.choice([8, 12, 16])) // es
            m.append((100 + rng.randrange(0, 40), rng.randrange(0, 4), ld, rng.randrange(1, ld + 1), es))
        a, b = m
        got = overlap(a, b)
        assert got == overlap(b, a)
        assert got or not taken(a) & taken(b), m
        (wa, pa), (wb, pb) = ((x[3] * x[4], x[2] * x[4]) for x in m)
        d = (b[0] - a[0]) % pa
        if a[1] > 1 and b[1] > 1 and pa == pb and d >= wa and d + wb <= pa:
            assert not got, m
            interleaved += max(a[0], b[0]) < min(max(taken(a)), max(taken(b)))
    assert interleaved > 100


@pytest.mark.parametrize("cols,ld", [((0, 64), 128), ((56, 120), 128), ((64, 136), 136)])
def test_overlapping_slices_are_refused(cols, ld):
    """(No address here is ever read: the calls fail their checks.)  x has columns 0 .. 64."""
    base = 0x7F0000000000
    a, b = cols
    if a >= 64:  # other strides: whole extents count
        ld_out = ld + 8
    else:
        ld_out = ld
    d = ops.MoeNorm(10, 64, 0, 0, 0, 1e-6, 1.0)
    st = ops.lib().moe_block_norm(ctypes.byref(d), ops.MoeMat(base, ld), base + (1 << 32), ops.MoeMat(base + 2 * a, ld_out),
                                  None)
    assert st == 1
    g = ops.MoeGroups(10, 10, ld, ld_out, 1, 64, 64, 1, None, None)
    assert ops.lib().moe_grouped_matmul(ctypes.byref(g), base, base + (1 << 32), base + 2 * a, 0, None) == 1


@pytest.mark.gpu
@pytest.mark.parametrize("M", [3, 700])
def test_products_between_slices_of_one_buffer(M):
    """x | y | dy | dx side by side: each call reads one slice and writes its neighbour."""
    K, N = 520, 1048
    counts = [M // 3, M - M // 3]
    off, w = offsets_of(counts).cuda(), randn(1, 2, N, K, scale=0.1).cuda()
    x, dy = randn(2, M, K).cuda(), randn(3, M, N).cuda()
    buf = torch.full((M, 2 * K + 2 * N + 16), 5.0, dtype=BF16, device="cuda")
    cut = [buf[:, a:b] for a, b in ((0, K), (K, K + N), (K + N, K + 2 * N), (K + 2 * N, 2 * K + 2 * N))]
    cut[0].copy_(x)
    cut[2].copy_(dy)
    ops.grouped_matmul(cut[0], w, off, out=cut[1])
    ops.grouped_matmul_grad_input(cut[2], w, off, out=cut[3])
    dw = ops.grouped_matmul_grad_weight(cut[0], cut[2], off)
    assert torch.equal(cut[1], ops.grouped_matmul(x, w, off))
    assert torch.equal(cut[3], ops.grouped_matmul_grad_input(dy, w, off))
    assert torch.equal(dw, ops.grouped_matmul_grad_weight(x, dy, off))
    assert torch.equal(cut[0], x) and torch.equal(cut[2], dy) and (buf[:, -16:] == 5).all()
    wq = torch.randint(-127, 128, (N, 512), generator=torch.Generator().manual_seed(4), dtype=torch.int8).cuda()
    ws = torch.rand(N, generator=torch.Generator().manual_seed(5)).cuda()
    ops.matmul_i8(cut[0][:, :512], wq, ws, out=cut[1])
    assert torch.equal(cut[1], ops.matmul_i8(x[:, :512].contiguous(), wq, ws)) and torch.equal(cut[2], dy)


@pytest.mark.gpu
@pytest.mark.parametrize("M", [3, 1100])
def test_norms_between_slices_of_one_buffer(M):
    H = 264
    x, y, w = randn(1, M, H).cuda(), randn(2, M, H).cuda(), randn(3, H).cuda()
    buf = torch.full((M, 5 * H + 8), 5.0, dtype=BF16, device="cuda")
    cut = [buf[:, i * H:(i + 1) * H] for i in range(5)]
    cut[0].copy_(x)
    cut[1].copy_(y)
    ops.block_merge(cut[0], cut[1], w, EPS, scale=0.5, next_weight=w, out=cut[2], h=cut[3])
    ops.block_norm(cut[0], w, EPS, out=cut[4])
    out, h = ops.block_merge(x, y, w, EPS, scale=0.5, next_weight=w)
    assert torch.equal(cut[2], out) and torch.equal(cut[3], h) and torch.equal(cut[4], ops.block_norm(x, w, EPS))
    assert torch.equal(cut[0], x) and torch.equal(cut[1], y) and (buf[:, -8:] == 5).all()

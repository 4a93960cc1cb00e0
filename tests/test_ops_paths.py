"""The rules that give a forward product to the matrix-vector or the matrix-matrix kernel."""
import ctypes
import os
import random
import shutil
import subprocess

import pytest
import torch

from ops_paths import quantizes_inside, takes_matrix_vector
from ops_util import offsets_of, randn
from sparse_moe_router_amd import ops

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def library_rules(tmp_path_factory):
    if not shutil.which("g++"):
        pytest.skip("no host compiler")
    d = tmp_path_factory.mktemp("paths")
    (d / "r.cpp").write_text(
        '#include "ops_paths.h"\nextern "C" int mv(int64_t r, int e, int n) { return moe::takes_matrix_vector(r, e, n); }\n'
        'extern "C" int qi(int64_t r, int64_t x, int e, int n, int k) { return moe::quantizes_inside(r, x, e, n, k); }\n')
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-shared", "-fPIC", "-I",
                    os.path.join(ROOT, "sparse_moe_router_amd", "csrc"), str(d / "r.cpp"), "-o", str(d / "r.so")], check=True)
    lib = ctypes.CDLL(str(d / "r.so"))
    lib.mv.argtypes = [ctypes.c_int64, ctypes.c_int, ctypes.c_int]
    lib.qi.argtypes = [ctypes.c_int64, ctypes.c_int64, ctypes.c_int, ctypes.c_int, ctypes.c_int]
    return lib


def test_the_tests_rules_are_the_librarys(library_rules):
    rng = random.Random(1)
    log = lambda hi: int(2 ** rng.uniform(0, hi))
    seen = set()
    for _ in range(20000):
        r, x, e, n, k = log(20) if rng.random() < 0.5 else log(9), log(4), log(10), 8 * log(17), 16 * log(10)
        mv, qi = bool(library_rules.mv(r, e, n)), bool(library_rules.qi(r, x, e, n, k))
        assert mv == takes_matrix_vector(r, e, n) and qi == quantizes_inside(r, x, e, n, k)
        seen.add((mv, qi))
    assert seen == {(False, False), (True, False), (True, True)}


def test_no_workgroup_walks_a_long_group(library_rules):
    """The matrix-vector kernel takes a group's rows 64 at a time, one after the other (4 when it quantises
    them): whatever the width of the output and however the rows are shared out, at most four times, and
    twice for a single group."""
    for n in (8, 64, 192, 392, 1024):
        for e in (1, 2, 4, 16, 64, 256):
            for rows in (1, 64, 128, 129, 256, 257, 512, 1024, 5566, 8192):
                if library_rules.mv(rows, e, n):
                    assert rows <= (128 if e == 1 else 256), (rows, e, n)
    # the rows of one group, for all that is known: those of four tokens that each chose it 32 times
    assert not library_rules.qi(128, 4, 1, 64, 512) and library_rules.qi(4, 4, 1, 64, 512)
    assert library_rules.qi(32, 4, 256, 40, 2048)


def kernels(f):
    """The products' kernels that f starts, without their template arguments."""
    with torch.profiler.profile(activities=[torch.profiler.ProfilerActivity.CUDA]) as p:
        for _ in range(3):
            f()
        torch.cuda.synchronize()
    return {n for e in p.events() for n in ("k_op_skinny", "k_op_rows", "k_quantize") if n in e.name}


@pytest.mark.gpu
@pytest.mark.parametrize("rows,E,N", [(128, 1, 64), (129, 1, 64), (256, 4, 64), (257, 4, 64), (5566, 1, 64), (8, 256, 1024),
                                      (32, 256, 1024)])
def test_the_kernel_that_runs(rows, E, N):
    K = 512
    counts = [rows // E + (i < rows % E) for i in range(E)]
    off = None if E == 1 else offsets_of(counts).cuda()
    x, w = randn(1, rows, K).cuda(), randn(2, E, N, K).cuda()
    wq = torch.randint(-127, 128, (E, N, K), generator=torch.Generator().manual_seed(3), dtype=torch.int8).cuda()
    ws = torch.ones(E, N, device="cuda")
    ops.grouped_matmul(x, w, off)
    product = "k_op_skinny" if takes_matrix_vector(rows, E, N) else "k_op_rows"
    assert kernels(lambda: ops.grouped_matmul(x, w, off)) == {product}
    want = {product} if quantizes_inside(rows, rows, E, N, K) else {product, "k_quantize"}
    ops.grouped_matmul_i8(x, wq, ws, off)
    assert kernels(lambda: ops.grouped_matmul_i8(x, wq, ws, off)) == want


@pytest.mark.gpu
def test_rows_without_tokens_quantised_inside():
    """Rows that no token backs, on the path whose workgroups quantise their rows themselves."""
    N, K, R, E = 48, 528, 7, 2
    assert quantizes_inside(R, 0, E, N, K)
    w = torch.randint(-127, 128, (E, N, K), generator=torch.Generator().manual_seed(3), dtype=torch.int8).cuda()
    y = ops.grouped_matmul_i8(torch.empty(0, K, dtype=BF16, device="cuda"), w, torch.ones(E, N, device="cuda"),
                              offsets_of([3, 4]).cuda(), perm=torch.arange(R, dtype=torch.int32, device="cuda"), top_k=2)
    assert y.shape == (R, N) and (y == 0).all()

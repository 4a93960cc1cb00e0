"""The rules of the training operators that the host decides by, compiled by the host's compiler."""
import ctypes
import heapq
import os
import random
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def rules(tmp_path_factory):
    if not shutil.which("g++"):
        pytest.skip("no host compiler")
    d = tmp_path_factory.mktemp("rules")
    (d / "r.cpp").write_text(
        '#include "ops_paths.h"\n'
        'extern "C" int64_t steps(int64_t a, int64_t b, int64_t c, int64_t d) { return moe::launch_steps(a, b, c, d); }\n'
        'extern "C" int next(int n) { return moe::next_parts(n); }\n'
        'extern "C" int few(int64_t r, int64_t e, int64_t h, int64_t i, int64_t k) { return moe::takes_few_rows(r, e, h, i, k); }\n'
        'extern "C" int logits(int64_t r, int64_t c) { return moe::takes_matrix_vector_logits(r, c); }\n')
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-shared", "-fPIC", "-I",
                    os.path.join(ROOT, "sparse_moe_router_amd", "csrc"), str(d / "r.cpp"), "-o", str(d / "r.so")], check=True)
    lib = ctypes.CDLL(str(d / "r.so"))
    lib.steps.restype, lib.steps.argtypes = ctypes.c_int64, [ctypes.c_int64] * 4
    lib.few.argtypes = [ctypes.c_int64] * 5
    lib.logits.argtypes = [ctypes.c_int64] * 2
    return lib


def schedule(*kinds):
    """The time of tiles, (number, steps) of each kind, of which each starts on the first free of 256 workgroups."""
    free = [0] * 256
    for n, steps in kinds:
        for _ in range(n):
            heapq.heapreplace(free, free[0] + steps)
    return max(free)


def test_the_time_of_a_launch(rules):
    rng = random.Random(3)
    edges = [0, 1, 255, 256, 257, 511, 512, 513, 768]
    for _ in range(1500):
        n0, n1 = (rng.choice(edges) if rng.random() < 0.4 else rng.randint(0, 900) for _ in range(2))
        s0, s1 = rng.randint(7, 200), rng.randint(7, 200)
        assert rules.steps(n0, s0, n1, s1) == schedule((n0, s0), (n1, s1)), (n0, s0, n1, s1)


def test_the_counts_of_parts_grow(rules):
    seen, n = [], 1
    while n < 200:
        seen.append(n)
        n = rules.next(n)
    assert seen[:10] == [1, 2, 3, 4, 5, 6, 7, 8, 10, 12] and all(b > a for a, b in zip(seen, seen[1:])) and len(seen) < 30


def test_logits_of_few_tokens_run_at_a_time(rules):
    """64 tokens and 16 columns a workgroup, at most 256 of them."""
    for rows, columns, few in ((1, 16, 1), (64, 4096, 1), (64, 4097, 0), (65, 2048, 1), (65, 2049, 0), (16384, 16, 1),
                               (16385, 16, 0), (1 << 30, 1, 0), (1, 1 << 20, 0)):
        assert bool(rules.logits(rows, columns)) == bool(few), (rows, columns)


def test_few_rows_of_small_blocks(rules):
    """At most 32 rows, 2^28 weights read for them and as many gradients written."""
    for rows, e, h, i, k, few in ((0, 1, 8, 8, 8, 0), (1, 1, 8, 8, 8, 1), (32, 1024, 8, 8, 8, 1), (33, 1, 8, 8, 8, 0),
                                  (32, 1, 2048, 1344, 2048, 1), (32, 1, 2048, 1408, 2048, 0), (1, 42, 2048, 1024, 2048, 1),
                                  (1, 43, 2048, 1024, 2048, 0), (1, 1, 1 << 20, 16384, 16384, 0)):
        assert bool(rules.few(rows, e, h, i, k)) == bool(few), (rows, e, h, i, k)

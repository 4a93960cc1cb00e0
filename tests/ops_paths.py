"""Which kernel a forward product takes: the library's rules once more, for tests that want one side of
them (test_ops_paths.py compares the two)."""


def takes_matrix_vector(rows, E, N):
    groups = min(rows, E)
    return N * (43 * groups + rows) < 43 * 12000 and rows <= (256 if groups > 1 else 128)


def quantizes_inside(rows, x_rows, E, N, K):
    return takes_matrix_vector(rows, E, N) and x_rows <= 4 and x_rows * K <= 16384 and rows <= 4 * E

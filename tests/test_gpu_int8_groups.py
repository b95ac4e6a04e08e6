"""GPU: the grouped integer GEMM over 128 to 1024 groups, every kernel by shapes
that choose it: exact sums rounded once, for rows spread at random, for the
division with the most row tiles there can be, for one group that owns every
row, and for sizes that are negative or pass the rows' end."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
STREAM64, TILED, STREAM128, ROWS = 0, 1, 2, 3

CASES = [  # kernel, G, M, N, K
    (ROWS, 130, 162, 64, 272), (ROWS, 200, 333, 100, 144), (ROWS, 256, 300, 131, 272), (ROWS, 256, 90, 96, 1040),
    (STREAM64, 1024, 1024, 40, 64), (STREAM64, 128, 129, 257, 512), (STREAM64, 256, 257, 520, 1040),
    (STREAM128, 256, 16384, 1024, 512), (STREAM128, 150, 9001, 261, 272), (TILED, 130, 130000, 520, 1040),
]


def _sizes(kind, G, M, g):
    if kind == "random":
        return torch.bincount(torch.randint(0, G, (M,), device=DEV, generator=g), minlength=G)
    if kind == "most":                   # one row in every group but one, which has the rest
        s = torch.zeros(G, dtype=torch.int64, device=DEV)
        s[:min(G, M)] = 1
        s[G // 2] += M - int(s.sum())
        return s
    if kind == "one":
        s = torch.zeros(G, dtype=torch.int64, device=DEV)
        s[G - 2] = M
        return s
    s = torch.randint(-3, 4, (G,), device=DEV, generator=g)       # "wild"
    s[G // 2] = 1 << 40
    s[G // 2 + 1:] = 5
    return s


@pytest.mark.parametrize("kernel,G,M,N,K", CASES)
@pytest.mark.parametrize("kind", ["random", "most", "one", "wild"])
def test_many_groups_are_exact(kernel, G, M, N, K, kind):
    from block_scaled_precision_03_amd import mxgemm as m
    m.init()
    assert m.grouped_int8_variant(G, M, N, K) == kernel
    g = torch.Generator(device=DEV)
    g.manual_seed(G + M + N + K)
    lim = 64                             # sums below 2^24
    A = torch.randint(-lim, lim, (M, K), dtype=torch.int8, device=DEV, generator=g)
    W = torch.randint(-lim, lim, (G, N, K), dtype=torch.int8, device=DEV, generator=g)
    sA = 2.0 ** torch.randint(-3, 4, (M,), device=DEV, generator=g).float()      # powers of two: exact products
    sW = 2.0 ** torch.randint(-3, 4, (G, N), device=DEV, generator=g).float()
    sizes = _sizes(kind, G, M, g)
    full = torch.full((M * N + 4096,), float("nan"), dtype=torch.bfloat16, device=DEV)
    D = full[:M * N].view(M, N)
    m.grouped_int8_run(G, sizes, A, sA, W, sW, D, M, N, K)
    r = 0
    for e, n in enumerate(sizes.tolist()):
        n = max(0, min(n, M - r))
        if n:
            ref = torch.mm(A[r:r + n].double(), W[e].double().t()) * sA[r:r + n].double()[:, None] * sW[e].double()[None, :]
            assert torch.equal(D[r:r + n], ref.float().bfloat16()), e
        r += n
    assert r == M
    assert bool(torch.isnan(full[M * N:]).all())

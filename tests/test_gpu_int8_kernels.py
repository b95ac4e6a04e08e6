"""GPU: every kernel of the 8-bit integer GEMM, by shapes that choose it, with
odd and ragged sizes at its tile edges, one K step per tile, partial last
stages and more tiles than workgroups: exact sums rounded once."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
INT8, NT = 32, 0
ROWS, TILE64, TILE128, TILE256 = 3, 1, 2, 0

CASES = [  # kernel, M, N, K
    (ROWS, 1, 1, 16), (ROWS, 3, 601, 1776), (ROWS, 16, 1024, 528), (ROWS, 17, 333, 144), (ROWS, 40, 250, 2000),
    (ROWS, 33, 1139, 400), (ROWS, 130, 517, 496), (ROWS, 1, 14336, 4096), (ROWS, 5, 131, 9600),
    (TILE64, 257, 4097, 400), (TILE64, 65, 12001, 272), (TILE64, 269, 3715, 1552), (TILE64, 703, 1127, 112),
    (TILE64, 200, 6000, 16),
    (TILE128, 6449, 1003, 1040), (TILE128, 777, 5001, 1040), (TILE128, 717, 9555, 144), (TILE128, 1500, 2501, 400),
    (TILE256, 5000, 3001, 1040), (TILE128, 4097, 4102, 1040), (TILE256, 4097, 8002, 1040), (TILE256, 6831, 6723, 272),
]


@pytest.mark.parametrize("kernel,M,N,K", CASES)
def test_each_kernel_is_exact(kernel, M, N, K):
    from block_scaled_precision_03_amd import mxgemm as m
    m.init()
    assert m.dense_variant(INT8, INT8, NT, M, N, K) == kernel
    g = torch.Generator(device=DEV)
    g.manual_seed(M + N + K)
    lim = 128 if K <= 1000 else 32          # sums below 2^24
    A = torch.randint(-lim, lim, (M, K), dtype=torch.int8, device=DEV, generator=g)
    B = torch.randint(-lim, lim, (N, K), dtype=torch.int8, device=DEV, generator=g)
    sA = 2.0 ** torch.randint(-3, 4, (M,), device=DEV, generator=g).float()   # powers of two: exact products
    sB = 2.0 ** torch.randint(-3, 4, (N,), device=DEV, generator=g).float()
    full = torch.full((M * N + 4096,), float("nan"), dtype=torch.bfloat16, device=DEV)
    D = full[:M * N].view(M, N)
    m.run(INT8, INT8, NT, A, sA, B, sB, D, M, N, K)
    ref = torch.mm(A.double(), B.double().t()) * sA.double()[:, None] * sB.double()[None, :]
    assert torch.equal(D, ref.float().bfloat16())
    assert bool(torch.isnan(full[M * N:]).all())


@pytest.mark.parametrize("sizes,N,K", [([5, 0, 1, 16, 17], 700, 1040), ([64] * 9, 4104, 272), ([300, 0, 129, 400, 3], 2051, 400),
                                       ([2000, 1, 900, 1200], 2050, 144), ([1] * 40, 129, 48)])
def test_grouped_is_exact(sizes, N, K):
    from block_scaled_precision_03_amd import mxgemm as m
    m.init()
    G, M = len(sizes), sum(sizes)
    g = torch.Generator(device=DEV)
    g.manual_seed(N + K)
    lim = 128 if K <= 1000 else 32
    A = torch.randint(-lim, lim, (M, K), dtype=torch.int8, device=DEV, generator=g)
    W = torch.randint(-lim, lim, (G, N, K), dtype=torch.int8, device=DEV, generator=g)
    sA = 2.0 ** torch.randint(-3, 4, (M,), device=DEV, generator=g).float()
    sW = 2.0 ** torch.randint(-3, 4, (G, N), device=DEV, generator=g).float()
    D = torch.empty(M, N, dtype=torch.bfloat16, device=DEV)
    m.grouped_int8_run(G, torch.tensor(sizes, device=DEV), A, sA, W, sW, D, M, N, K)
    r = 0
    for e, n in enumerate(sizes):
        ref = torch.mm(A[r:r + n].double(), W[e].double().t()) * sA[r:r + n].double()[:, None] * sW[e].double()[None, :]
        assert torch.equal(D[r:r + n], ref.float().bfloat16()), e
        r += n

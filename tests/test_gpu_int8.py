"""GPU: the 8-bit integer GEMM, dense and grouped, against 64-bit sums: every
kernel, odd and ragged sizes, all activations, the codes' extremes, K tails
whose neighbours must not leak in, empty groups, K = 0.  With scales of one
and sums below 2^24 the output must be the exact sum rounded once."""
import numpy as np
import pytest
import torch

from tests import moe_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
INT8, NT = 32, 0
PAD = 4096


def _mx():
    from block_scaled_precision_03_amd import mxgemm
    mxgemm.init()
    return mxgemm


def _out(rows, cols):
    """BF16 output inside a NaN-filled buffer, with its guard."""
    full = torch.full((rows * cols + PAD,), float("nan"), dtype=torch.bfloat16, device=DEV)
    return full, full[:rows * cols].view(rows, cols)


def _codes(rng, *shape):
    c = rng.integers(-128, 128, shape).astype(np.int8)
    c.reshape(-1)[:2] = -128
    return c


def _t(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


SHAPES = [  # M, N, K
    (1, 1, 16), (1, 3, 48), (2, 17, 128), (15, 64, 144), (16, 130, 256), (17, 257, 112), (33, 515, 400), (5, 4096, 2064),
    (64, 300, 1040), (65, 129, 4112), (130, 258, 528), (300, 200, 3056), (777, 1002, 1040), (300, 2000, 16),
    (2100, 2056, 144), (1030, 4104, 384), (2049, 2051, 400), (4100, 2060, 128),
]


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_int8_exact_sums(M, N, K):
    m = _mx()
    rng = np.random.default_rng(M + N + K)
    A, B = _codes(rng, M, K), _codes(rng, N, K)
    if K > 1000:                                  # keep the sums below 2^24
        A, B = (A // 4).astype(np.int8), (B // 4).astype(np.int8)
    S = A.astype(np.float64) @ B.astype(np.float64).T
    assert np.abs(S).max() < 2 ** 24
    full, D = _out(M, N)
    # operands inside larger buffers of other codes: a K tail or an edge row
    # that reads past its operand would change the sums
    wide = lambda c: torch.cat([_t(c).reshape(-1), torch.full((65536,), 77, dtype=torch.int8, device=DEV)])
    one = lambda n: torch.ones(n + 512, device=DEV)
    m.run(INT8, INT8, NT, wide(A), one(M), wide(B), one(N), D, M, N, K)
    torch.cuda.synchronize()
    ref = torch.from_numpy(S).float().bfloat16()
    assert torch.equal(D.cpu(), ref)
    assert bool(torch.isnan(full[M * N:]).all())


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("act", [R.ACT_NONE, R.ACT_RELU, R.ACT_GELU, R.ACT_SILU, R.ACT_SWIGLU])
def test_int8_scales_bias_activation(M, N, K, act):
    m = _mx()
    rng = np.random.default_rng(M * N + K + act)
    if act == R.ACT_SWIGLU:
        N += N & 1
    A, B = _codes(rng, M, K), _codes(rng, N, K)
    sA = (rng.uniform(0.5, 1.5, M) * 0.03).astype(np.float32)
    sB = (rng.uniform(0.5, 1.5, N) * 0.5 / (75 * np.sqrt(K))).astype(np.float32)
    bias = torch.from_numpy(rng.normal(size=N).astype(np.float32)).bfloat16() if N % 2 == 0 else None
    No = N // 2 if act == R.ACT_SWIGLU else N
    full, D = _out(M, No)
    m.run_fused(INT8, INT8, NT, _t(A), _t(sA), _t(B), _t(sB), D, M, N, K,
                bias=None if bias is None else bias.to(DEV), activation=act)
    torch.cuda.synchronize()
    ref, tol = R.int8_gemm(A, sA, B, sB, None if bias is None else bias.double().numpy(), act)
    assert np.all(np.abs(D.double().cpu().numpy() - ref) <= tol)
    assert bool(torch.isnan(full[M * No:]).all())


def test_int8_largest_sums():
    """All codes at -128: the sum of the longest K is 2^31 - 2^18."""
    m = _mx()
    K = 131056
    A = torch.full((3, K), -128, dtype=torch.int8, device=DEV)
    D = torch.empty(3, 5, dtype=torch.bfloat16, device=DEV)
    m.run(INT8, INT8, NT, A, torch.ones(3, device=DEV), torch.full((5, K), -128, dtype=torch.int8, device=DEV),
          torch.ones(5, device=DEV), D, 3, 5, K)
    assert (D.float() == torch.tensor(float(128 * 128 * K)).bfloat16().float().to(DEV)).all()


@pytest.mark.parametrize("act", [R.ACT_NONE, R.ACT_GELU, R.ACT_SWIGLU])
@pytest.mark.parametrize("bias", [False, True])
def test_int8_no_k(act, bias):
    m = _mx()
    b = torch.randn(34, device=DEV).bfloat16() if bias else None
    No = 17 if act == R.ACT_SWIGLU else 34
    full, D = _out(9, No)
    m.run_fused(INT8, INT8, NT, None, None, None, None, D, 9, 34, 0, bias=b, activation=act)
    z = (b.double().cpu().numpy() if bias else np.zeros(34))[None].repeat(9, 0)
    ref = R.act(z, act)
    assert np.all(np.abs(D.double().cpu().numpy() - ref) <= np.abs(ref) * (R.HALF_BF16 + 64 * R.HALF_F32) + 2.0 ** -126)
    assert bool(torch.isnan(full[9 * No:]).all())


GROUPS = [  # sizes, N, K
    ([1], 6, 16), ([0, 3, 0, 1], 64, 48), ([5, 0, 17, 2, 40, 0], 130, 400), ([16, 16, 15, 17], 512, 1024),
    ([33, 0, 70, 1, 129, 64], 257 * 2, 272), ([300, 0, 1, 511, 255], 1024, 144), ([2000, 40, 0, 900], 2056, 384),
    ([7] * 33, 320, 528), ([0, 0, 0], 64, 64), ([1500, 700, 3, 2000], 2048, 256),
]


@pytest.mark.parametrize("sizes,N,K", GROUPS)
@pytest.mark.parametrize("act", [R.ACT_NONE, R.ACT_SWIGLU])
@pytest.mark.parametrize("spare", [0, 9])
def test_grouped_int8(sizes, N, K, act, spare):
    m = _mx()
    G, used = len(sizes), sum(sizes)
    M = used + spare                     # trailing rows of no group stay untouched
    if M == 0:
        return
    rng = np.random.default_rng(M + N + K + act)
    A, W = _codes(rng, M, K), _codes(rng, G, N, K)
    sA = (rng.uniform(0.5, 1.5, M) * 0.03).astype(np.float32)
    sW = (rng.uniform(0.5, 1.5, (G, N)) * 0.5 / (75 * np.sqrt(K))).astype(np.float32)
    No = N // 2 if act == R.ACT_SWIGLU else N
    full, D = _out(M, No)
    m.grouped_int8_run(G, _t(np.array(sizes, np.int64)), _t(A), _t(sA), _t(W), _t(sW), D, M, N, K, activation=act)
    torch.cuda.synchronize()
    got, r = D.double().cpu().numpy(), 0
    for g, n in enumerate(sizes):
        if n:
            ref, tol = R.int8_gemm(A[r:r + n], sA[r:r + n], W[g], sW[g], None, act)
            assert np.all(np.abs(got[r:r + n] - ref) <= tol), g
        r += n
    assert np.isnan(got[used:]).all()
    assert bool(torch.isnan(full[M * No:]).all())


def test_grouped_sizes_beyond_the_rows_are_cut():
    m = _mx()
    A = torch.ones(10, 32, dtype=torch.int8, device=DEV)
    W = torch.ones(3, 8, 32, dtype=torch.int8, device=DEV)
    full, D = _out(10, 8)
    m.grouped_int8_run(3, torch.tensor([4, -5, 1 << 40], device=DEV), A, torch.ones(10, device=DEV), W,
                       torch.ones(3, 8, device=DEV), D, 10, 8, 32)
    torch.cuda.synchronize()
    assert (D == 32).all() and bool(torch.isnan(full[80:]).all())


def test_grouped_no_k():
    m = _mx()
    full, D = _out(10, 8)
    m.grouped_int8_run(2, torch.tensor([3, 4], device=DEV), None, None, None, None, D, 10, 8, 0)
    torch.cuda.synchronize()
    assert (D[:7] == 0).all() and bool(torch.isnan(D[7:]).all())


def test_int8_in_a_graph():
    m = _mx()
    rng = np.random.default_rng(1)
    for M, N, K in ((1, 512, 1040), (200, 300, 528), (2100, 2056, 144)):
        A, B, s = _t(_codes(rng, M, K)), _t(_codes(rng, N, K)), torch.rand(4096, device=DEV) * 0.01
        D = torch.empty(M, N, dtype=torch.bfloat16, device=DEV)
        call = lambda: m.run_fused(INT8, INT8, NT, A, s, B, s, D, M, N, K, activation=R.ACT_GELU)
        call()
        ref = D.clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        for _ in range(3):
            D.fill_(float("nan"))
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(D.view(torch.int16), ref.view(torch.int16))

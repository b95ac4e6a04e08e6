"""GPU: operands and outputs past 4 GiB (and 2^31 elements), checked at their
far ends: exact integer sums, codes and combined rows."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _mx():
    from block_scaled_precision_03_amd import mxgemm
    mxgemm.init()
    return mxgemm


def _codes(g, *shape):
    return torch.randint(-8, 9, shape, dtype=torch.int8, device=DEV, generator=g)


@pytest.mark.parametrize("M,N,K", [
    (5, 140032, 32768),       # B past 4 GiB, few rows
    (140001, 130, 32768),     # A past 4 GiB
    (50001, 50003, 64),       # D past 4 GiB
])
def test_int8_far_ends(M, N, K):
    m = _mx()
    g = torch.Generator(device=DEV)
    g.manual_seed(M)
    A, B = _codes(g, M, K), _codes(g, N, K)
    D = torch.zeros(M, N, dtype=torch.bfloat16, device=DEV)
    one = torch.ones(max(M, N), device=DEV)
    m.run(m.INT8, m.INT8, m.NT, A, one, B, one, D, M, N, K)
    for rows in (slice(0, 40), slice(max(0, M - 40), M)):
        for cols in (slice(0, 100), slice(max(0, N - 100), N)):
            ref = torch.mm(A[rows].double(), B[cols].double().t())     # below 2^24: 64 K
            assert torch.equal(D[rows, cols], ref.float().bfloat16())


def test_grouped_far_group():
    m = _mx()
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    G, N, K, sizes = 3, 65540, 32768, [3, 0, 40]
    M = sum(sizes)
    A, W = _codes(g, M, K), _codes(g, G, N, K)
    D = torch.zeros(M, N, dtype=torch.bfloat16, device=DEV)
    m.grouped_int8_run(G, torch.tensor(sizes, device=DEV), A, torch.ones(M, device=DEV), W, torch.ones(G, N, device=DEV),
                       D, M, N, K)
    for rows, e in ((slice(0, 3), 0), (slice(3, 43), 2)):
        for cols in (slice(0, 100), slice(N - 100, N)):
            assert torch.equal(D[rows, cols], torch.mm(A[rows].double(), W[e, cols].double().t()).float().bfloat16())


def test_quantize_and_combine_far_rows():
    m = _mx()
    T, K = 70001, 32768
    x = torch.zeros(T, K, dtype=torch.bfloat16, device=DEV)
    g = torch.Generator(device=DEV)
    g.manual_seed(2)
    for r in (0, 65535, T - 1):
        x[r] = torch.randint(-127, 128, (K,), device=DEV, generator=g).bfloat16()
        x[r, 7] = 127
    q, s = torch.empty(T, K, dtype=torch.int8, device=DEV), torch.empty(T, device=DEV)
    m.quantize_int8(m.BF16, x, q, s, T, K)
    assert bool((s == 1).all())                    # 127 / 127, and zero rows
    for r in (0, 65535, T - 1):
        assert torch.equal(q[r].float(), x[r].float())
    assert not bool(q[1:65535].any())
    # the rows back in reverse order, one slot each, weight 2
    row_of = torch.arange(T - 1, -1, -1, dtype=torch.int32, device=DEV).view(T, 1)
    w, out = torch.full((T, 1), 2.0, device=DEV), torch.empty_like(x)
    m.moe_combine(x, w, row_of, out, T, 1, K, T)
    for r in (0, 65535, T - 1):
        assert torch.equal(out[T - 1 - r], 2 * x[r])
    dy, dw = torch.zeros_like(x), torch.empty(T, 1, device=DEV)
    m.moe_combine_backward(out, x, w, row_of, dy, dw, T, 1, K, T)
    for r in (0, 65535, T - 1):
        assert torch.equal(dy[r], 4 * x[r])
        ref = float(2 * (x[r].double() ** 2).sum())
        # FP32 sums of K products, each partial sum rounded once
        assert abs(float(dw[T - 1 - r]) - ref) <= ref * K * 2.0 ** -24


def test_more_workgroups_than_one_dimension_holds():
    """Grids of 2^32 work-items and more."""
    m = _mx()
    T = (1 << 26) + 5                              # a wave per row
    x = torch.zeros(T, 16, dtype=torch.bfloat16, device=DEV)
    x[-1] = torch.arange(112, 128, device=DEV).bfloat16()
    q, s = torch.empty(T, 16, dtype=torch.int8, device=DEV), torch.zeros(T, device=DEV)
    m.quantize_int8(m.BF16, x, q, s, T, 16)
    assert bool((s == 1).all()) and torch.equal(q[-1].float(), x[-1].float()) and not bool(q[:-1].any())
    T = (1 << 24) + 5                              # a workgroup per token
    d = torch.zeros(T, 2048, dtype=torch.bfloat16, device=DEV)
    d[-1] = 3
    row_of = torch.arange(T, dtype=torch.int32, device=DEV).view(T, 1)
    w, dw, dy = torch.full((T, 1), 2.0, device=DEV), torch.full((T, 1), 9.0, device=DEV), torch.empty_like(d)
    m.moe_combine_backward(d, d, w, row_of, dy, dw, T, 1, 2048, T)
    assert bool((dy[-1] == 6).all()) and float(dw[-1]) == 9.0 * 2048 and not bool(dw[:-1].any())
    D = torch.full((70000, 65536), 7, dtype=torch.bfloat16, device=DEV)   # a value each
    m.run(m.INT8, m.INT8, m.NT, None, None, None, None, D, 70000, 65536, 0)
    assert not bool(D[0].any()) and not bool(D[-1].any()) and not bool(D[65536:65540].any())

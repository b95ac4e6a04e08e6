"""CPU checks of the residual epilogue's entry points (host checks only,
nothing reaches a device), and of the 64-bit gradient against differences."""
import pytest
import torch

from tests import residual_ref as R

P = 1 << 20       # fake, aligned addresses (never dereferenced)
Q, S = 2 << 20, 3 << 20


def _mx():
    from block_scaled_precision_03_amd import mxgemm
    return mxgemm


A = (0, 0, 0, P, P, P, P, P, 64, 66, 256)
I8 = (32, 32, 0, P, P, P, P, P, 64, 66, 256)
FORWARD = [(A, dict(), 0), (A, dict(residual=Q), 0), (A, dict(residual=P), 0), (A, dict(z=Q), 0), (A, dict(residual=Q, z=S, bias=P, activation=2), 0),
           (I8, dict(residual=Q, z=S, activation=8), 0), ((4, 4 | 0x100) + A[2:], dict(residual=Q), 0), ((16, 17) + A[2:], dict(residual=Q), 0),
           (A, dict(residual=Q, activation=8), -1), (A, dict(residual=Q, activation=4), -1), (A, dict(z=P), -1), (A, dict(residual=Q, z=Q), -1),
           (A, dict(residual=Q + 8), -3), (A, dict(z=Q + 2), -3), (A, dict(residual=Q, bias=P + 2), -3),
           ((0, 0, 1) + A[3:9] + (64, 256), dict(residual=Q), -2), ((0, 0, 2) + A[3:9] + (64, 256), dict(z=Q), -2),
           (A[:10] + (200,), dict(residual=Q), -2), (A[:3] + (0,) + A[4:], dict(residual=Q), -1), ((0, 16) + A[2:], dict(residual=Q), -2),
           (A[:9] + (65, 256), dict(residual=Q, bias=P), -2), (A[:9] + (65, 256), dict(residual=Q), 0),
           (A[:8] + (-1, 66, 256), dict(residual=Q), -1), (A[:8] + (0, 66, 256), dict(residual=Q + 8), 0),
           (A[:3] + (0, 0, 0, 0, P, 64, 66, 0), dict(residual=Q, z=S), 0), (I8[:9] + (65, 256), dict(residual=Q, activation=8), -2)]


@pytest.mark.parametrize("args,kw,status", FORWARD)
def test_forward_validate(args, kw, status):
    m = _mx()
    assert m.validate_residual(*args, **kw) == status
    if status != 0:
        with pytest.raises(m.MxgemmError) as err:
            m.run_residual(*args, stream=0, **kw)
        assert err.value.status == status


BACKWARD = [((0, P, 0, 0, Q, 64, 66, P), 0), ((0, P, 0, Q, 0, 64, 66, None), 0), ((2, P, Q, S, P, 64, 66, P), 0), ((2, P, Q, Q, 0, 64, 66, None), 0),
            ((2, P, Q, P, 0, 64, 66, None), 0), ((8, P, Q, Q, P, 64, 66, P), 0), ((1, P, Q, S, P, 8, 65, None), 0),
            ((1, 0, 0, 0, P, 0, 65, None), 0), ((1, 0, 0, 0, P, 64, 0, None), 0),
            ((4, P, Q, S, 0, 64, 66, None), -1), ((-1, P, Q, S, 0, 64, 66, None), -1), ((1, P, Q, 0, 0, 64, 66, None), -1),
            ((1, 0, Q, S, 0, 64, 66, None), -1), ((1, P, 0, S, 0, 64, 66, None), -1), ((1, P, Q, S, P, 300, 66, None), -1),
            ((8, P, Q, P, 0, 64, 66, None), -1), ((1, P, Q, S, 0, -1, 66, None), -1), ((1, P, Q, S, 0, 64, -2, None), -1),
            ((8, P, Q, S, 0, 64, 65, None), -2), ((1, P, Q, S, 0, 1 << 31, 2, None), -2), ((1, P, Q, S, 0, 2, 1 << 31, None), -2),
            ((1, P + 2, Q, S, 0, 64, 66, None), -3), ((1, P, Q + 8, S, 0, 64, 66, None), -3), ((1, P, Q, S + 4, 0, 64, 66, None), -3),
            ((1, P, Q, S, P + 2, 64, 66, P), -3), ((1, P, Q, S, P, 300, 66, P + 8), -3), ((1, P, Q, S, P, 64, 66, None), 0)]


@pytest.mark.parametrize("args,status", BACKWARD)
def test_backward_validate(args, status):
    m = _mx()
    assert m.residual_backward_validate(*args[:7], workspace=args[7]) == status
    if status != 0:
        with pytest.raises(m.MxgemmError) as err:
            m.residual_backward(*args[:7], workspace=args[7], stream=0)
        assert err.value.status == status


def test_backward_workspace():
    m = _mx()
    assert m.residual_backward_workspace_bytes(0, 5) == 0 and m.residual_backward_workspace_bytes(1, 5) == 0
    assert m.residual_backward_workspace_bytes(-1, 5) == -1 and m.residual_backward_workspace_bytes(5, 1 << 31) == -1
    assert m.residual_backward_workspace_bytes(256, 66) == 0           # one part
    need = m.residual_backward_workspace_bytes(300, 66)
    assert need > 0 and need % (4 * 66) == 0
    room = torch.empty(need + 32, dtype=torch.uint8)
    start = -room.data_ptr() % 16
    assert m.residual_backward_validate(1, P, Q, S, P, 300, 66, workspace=room[start:start + need]) == 0
    assert m.residual_backward_validate(1, P, Q, S, P, 300, 66, workspace=room[start:start + need - 1]) == -1


@pytest.mark.parametrize("a", [R.ACT_NONE, R.ACT_RELU, R.ACT_GELU, R.ACT_SILU, R.ACT_SWIGLU])
def test_gradient_against_differences(a):
    g = torch.Generator().manual_seed(a)
    z = torch.randn(4, 6, dtype=torch.float64, generator=g) * 2
    d = torch.randn(4, 3 if a == R.ACT_SWIGLU else 6, dtype=torch.float64, generator=g)
    dz, _, dbias, _ = R.gradient(d, z, a)
    h = 1e-5
    for i in range(4):
        for j in range(6):
            up, down = z.clone(), z.clone()
            up[i, j] += h
            down[i, j] -= h
            diff = ((R.act(up, a) - R.act(down, a)) * d).sum() / (2 * h)
            # a central difference is off by h^2 / 6 times a third derivative
            # (below 10 |d u|), and by the sums' rounding over h
            assert abs(float(diff - dz[i, j])) <= 10 * h * h * 20 + 1e-9
    assert torch.equal(dbias, dz.sum(0))


@pytest.mark.parametrize("fmt", [0, 4, 16, 32])
def test_forward_most_columns(fmt):
    m = _mx()
    most = lambda N, **kw: m.validate_residual(fmt, fmt, 0, P, P, P, P, P, 64, N, 256, **kw)
    for kw in (dict(residual=Q), dict(z=Q)):
        assert most(4194304, **kw) == 0 and most(4194305, **kw) == -2
    assert most(4194305) == 0                  # neither: as run_fused


# (format, preshuffled B, M, N, K, the kernel that was fastest, its us, the others' least us); the measured
# times of the kernel families on 256 compute units, differences of 15 % and more
FASTEST = [(0, False, 1857, 688, 7936, "ROWS", 50, 119), (4, True, 787, 1443, 12544, "ROWS", 40, 83), (0, False, 794, 2496, 7680, "ROWS", 54, 109),
           (0, True, 2243, 872, 12800, "ROWS", 60, 136), (4, False, 824, 1984, 2048, "ROWS", 16, 27), (0, False, 233, 5186, 2432, "ROWS", 23, 41),
           (4, True, 632, 3520, 512, "TILE64", 11, 20), (4, True, 295, 7104, 1024, "TILE64", 18, 21), (4, True, 1991, 1408, 768, "TILE64", 12, 18),
           (0, False, 724, 5499, 256, "TILE64", 21, 34), (0, True, 1690, 6848, 1536, "TILE256", 35, 97), (4, False, 2579, 2752, 512, "TILE256", 19, 28)]


@pytest.mark.parametrize("fmt,psb,M,N,K,kernel,us,others", FASTEST)
def test_forward_kernel_choice(fmt, psb, M, N, K, kernel, us, others):
    """One estimate for all kernels: the choice is the kernel that runs."""
    m = _mx()
    assert 1.15 * us < others
    assert m.residual_variant(fmt, fmt | (m.PRESHUFFLED if psb else 0), m.NT, M, N, K) == getattr(m, "DENSE_" + kernel)

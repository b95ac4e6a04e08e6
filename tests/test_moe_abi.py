"""CPU checks of the 8-bit integer GEMM's and the mixture-of-experts
operators' entry points (host checks only, nothing reaches a device), and of
their 64-bit reference forms: gradients against differences."""
import numpy as np
import pytest

from tests import moe_ref as R

P = 1 << 20       # a fake, aligned address (never dereferenced)


def _mx():
    from block_scaled_precision_03_amd import mxgemm
    return mxgemm


INT8 = 32
DENSE = [
    ((INT8, INT8, 0, P, P, P, P, P, 7, 5, 48), 0),
    ((INT8, INT8, 0, P, P + 4, P, P + 4, P, 7, 5, 48), 0),      # scales 4-byte aligned
    ((INT8, INT8, 0, P, P, P, P, P, 7, 5, 40), -2),             # K % 16
    ((INT8, INT8, 0, P, P, P, P, P, 7, 5, 131056), 0),
    ((INT8, INT8, 0, P, P, P, P, P, 7, 5, 131072), -2),         # sums past 31 bits
    ((INT8, INT8, 1, P, P, P, P, P, 16, 16, 128), -2),          # NT only
    ((INT8, INT8, 2, P, P, P, P, P, 16, 16, 128), -2),
    ((INT8, INT8, 3, P, P, P, P, P, 16, 16, 128), -1),
    ((INT8, INT8 | 0x100, 0, P, P, P, P, P, 16, 16, 128), -2),  # not preshuffled
    ((INT8, 0, 0, P, P, P, P, P, 16, 16, 128), -2),             # with another format
    ((16, INT8, 0, P, P, P, P, P, 16, 16, 128), -2),
    ((INT8, 7, 0, P, P, P, P, P, 16, 16, 128), -1),             # unknown format
    ((INT8, INT8, 0, P, P, P, P, P, -1, 16, 128), -1),
    ((INT8, INT8, 0, 0, P, P, P, P, 16, 16, 128), -1),
    ((INT8, INT8, 0, P, 0, P, P, P, 16, 16, 128), -1),
    ((INT8, INT8, 0, P, P, P, P, 0, 16, 16, 128), -1),
    ((INT8, INT8, 0, P + 8, P, P, P, P, 16, 16, 128), -3),
    ((INT8, INT8, 0, P, P + 2, P, P, P, 16, 16, 128), -3),
    ((INT8, INT8, 0, P, P, P, P, P + 2, 16, 16, 128), -3),
    ((INT8, INT8, 0, 0, 0, 0, 0, 0, 0, 16, 128), 0),            # M = 0
    ((INT8, INT8, 0, 0, 0, 0, 0, P, 16, 16, 0), 0),             # K = 0 reads no operand
]


@pytest.mark.parametrize("args,expect", DENSE)
def test_int8_validate(args, expect):
    assert _mx().validate(*args) == expect


def test_int8_fused_validate():
    m = _mx()
    a = (INT8, INT8, 0, P, P, P, P, P, 16)
    assert m.validate_fused(*a, 16, 128, bias=P, activation=m.ACT_SWIGLU) == 0
    assert m.validate_fused(*a, 17, 128, activation=m.ACT_SWIGLU) == -2       # N even
    assert m.validate_fused(*a, 17, 128, activation=m.ACT_SILU) == 0
    assert m.validate_fused(*a, 17, 128, bias=P) == -2                        # bias: N even
    assert m.validate_fused(*a, 16, 128, bias=P + 2) == -3
    assert m.validate_fused(*a, 16, 128, activation=4) == -1
    # SwiGLU is not built for the block-scaled formats
    assert m.validate_fused(0, 0, 0, P, P, P, P, P, 256, 256, 256, activation=m.ACT_SWIGLU) == -1


GROUPED = [
    ((8, P, P, P, P, P, P, 100, 5, 48, 0), 0),
    ((8, P, P, P, P, P, P, 100, 6, 48, 8), 0),
    ((8, P, P, P, P, P, P, 100, 5, 48, 8), -2),        # SwiGLU: N even
    ((8, P, P, P, P, P, P, 100, 5, 40, 0), -2),
    ((8, P, P, P, P, P, P, 100, 5, 48, 5), -1),        # unknown activation
    ((0, P, P, P, P, P, P, 100, 5, 48, 0), -2),
    ((1025, P, P, P, P, P, P, 100, 5, 48, 0), -2),
    ((8, 0, P, P, P, P, P, 100, 5, 48, 0), -1),
    ((8, P, 0, P, P, P, P, 100, 5, 48, 0), -1),
    ((8, P, P, P, P, P, P + 4, 100, 5, 48, 0), -3),
    ((8, P + 4, P, P, P, P, P, 100, 5, 48, 0), -3),
    ((8, P, P, P, P, P, P, -1, 5, 48, 0), -1),
    ((8, P, 0, 0, 0, 0, 0, 0, 5, 48, 0), 0),
]


@pytest.mark.parametrize("args,expect", GROUPED)
def test_grouped_int8_validate(args, expect):
    assert _mx().lib().grouped_int8_gemm_validate(*args) == expect


B, F = 64, 65
ROUTE = (F, P, P, P, P, 100, 64, 6, 0, 1, 1, 0, 1, 1.0, P, P, P, P, 1 << 20)
CALLS = [
    ("moe_route", dict([(0, 3)]), -1), ("moe_route", {8: 2}, -1), ("moe_route", {11: 5}, -1),
    ("moe_route", {5: -1}, -1), ("moe_route", {6: 0}, -2), ("moe_route", {6: 1025}, -2),
    ("moe_route", {7: 0}, -2), ("moe_route", {7: 65}, -2), ("moe_route", {6: 4, 7: 5}, -2),
    ("moe_route", {9: 3}, -2), ("moe_route", {9: 0}, -2), ("moe_route", {9: 8, 10: 9}, -2),
    ("moe_route", {9: 8, 10: 0}, -2), ("moe_route", {1: 0}, -1), ("moe_route", {3: 0}, -1),
    ("moe_route", {14: 0}, -1), ("moe_route", {15: 0}, -1), ("moe_route", {16: 0}, -1),
    ("moe_route", {17: 0}, -1), ("moe_route", {18: 10}, -1), ("moe_route", {17: P + 8}, -3),
    ("moe_route", {14: P + 4}, -3), ("moe_route", {1: P + 4}, -3), ("moe_route", {5: (1 << 24) + 1}, -2),
    ("moe_route", {5: 0, 14: 0, 15: 0, 16: 0}, 0),
]


@pytest.mark.parametrize("name,change,expect", CALLS)
def test_route_refusals(name, change, expect):
    args = list(ROUTE)
    for k, v in change.items():
        args[k] = v
    assert getattr(_mx().lib(), name)(*args, None) == expect


REJECT = [
    ("moe_route_backward", (F, P, P, P, P, 10, 64, 6, 0, 1, 1.0), {0: 1}, -1),
    ("moe_route_backward", (F, P, P, P, P, 10, 64, 6, 0, 1, 1.0), {1: 0}, -1),
    ("moe_route_backward", (F, P, P, P, P, 10, 64, 6, 0, 1, 1.0), {4: P + 2}, -3),
    ("moe_route_backward", (F, P, P, P, P, 10, 64, 6, 0, 1, 1.0), {7: 33}, -2),
    ("moe_route_backward", (F, P, P, P, P, 10, 64, 6, 0, 1, 1.0), {8: -1}, -1),
    ("moe_route_backward", (F, P, P, P, P, 10, 64, 6, 0, 1, 1.0), {5: 0}, 0),
    ("mxgemm_quantize_int8", (B, P, P, P, 10, 64, P, 2), {0: 0}, -1),
    ("mxgemm_quantize_int8", (B, P, P, P, 10, 64, P, 2), {5: 72}, -2),
    ("mxgemm_quantize_int8", (B, P, P, P, 10, 64, P, 2), {5: 131072}, -2),
    ("mxgemm_quantize_int8", (B, P, P, P, 10, 64, P, 2), {6: 0}, -1),          # topk without rows
    ("mxgemm_quantize_int8", (B, P, P, P, 10, 64, P, 2), {7: 65}, -2),
    ("mxgemm_quantize_int8", (B, P, P, P, 10, 64, P, 2), {2: P + 8}, -3),
    ("mxgemm_quantize_int8", (B, P, P, P, 10, 64, P, 2), {3: 0}, -1),
    ("mxgemm_quantize_int8", (B, P, P, P, 10, 64, P, 2), {4: 0}, 0),
    ("moe_combine", (P, P, P, P, 10, 2, 64, 20), {4: -1}, -1),
    ("moe_combine", (P, P, P, P, 10, 2, 64, 20), {5: 0}, -2),
    ("moe_combine", (P, P, P, P, 10, 2, 64, 20), {0: 0}, -1),
    ("moe_combine", (P, P, P, P, 10, 2, 64, 20), {3: P + 2}, -3),
    ("moe_combine", (P, P, P, P, 10, 2, 64, 20), {6: 0}, 0),
    ("moe_combine_backward", (P, P, P, P, P, P, 10, 2, 64, 20), {4: 0}, -1),
    ("moe_combine_backward", (P, P, P, P, P, P, 10, 2, 64, 20), {5: 0}, -1),
    ("moe_combine_backward", (P, P, P, P, P, P, 10, 2, 64, 20), {0: P + 8}, -3),
    ("moe_combine_backward", (P, P, P, P, P, P, 10, 2, 64, 20), {6: 0}, 0),
]


@pytest.mark.parametrize("name,args,change,expect", REJECT)
def test_operator_refusals(name, args, change, expect):
    args = list(args)
    for k, v in change.items():
        args[k] = v
    assert getattr(_mx().lib(), name)(*args, None) == expect


def test_route_workspace_bytes():
    m = _mx()
    assert m.moe_route_workspace_bytes(64, 256) == 0                  # one block places its own rows
    assert m.moe_route_workspace_bytes(65, 256) == 2 * 256 * 2
    assert m.moe_route_workspace_bytes(65, 250) == 2 * 256 * 2
    assert m.moe_route_workspace_bytes(16384, 256) == 256 * 256 * 2
    assert m.moe_route_workspace_bytes(1 << 20, 256) <= 512 * 256 * 2   # at most 512 blocks
    assert m.moe_route_workspace_bytes(-1, 256) == -1
    assert m.moe_route_workspace_bytes(1, 2000) == -1


def test_int8_variants_cover_every_kernel():
    m = _mx()
    seen = {m.dense_variant(INT8, INT8, 0, M, N, K)
            for M, N, K in ((1, 14336, 4096), (64, 64, 4096), (777, 5002, 4112), (16384, 14336, 4096))}
    assert seen <= {0, 1, 2, 3} and 0 in seen
    assert m.grouped_int8_variant(8, 16384, 4608, 7168) == m.GROUPED_TILED


@pytest.mark.parametrize("score", [R.SOFTMAX, R.SIGMOID])
@pytest.mark.parametrize("renorm", [False, True])
def test_reference_gradient_against_differences(score, renorm):
    """Central differences (step 1e-5, error of order 1e-10) of the weights."""
    rng = np.random.default_rng(5)
    l = rng.normal(size=(3, 11)) * 2
    ids, _ = R.route(l, None, 4, score, renorm=renorm)
    g = rng.normal(size=(3, 4))
    got = R.route_grad(l, ids, g, score, renorm, 1.7)
    for t in range(3):
        for e in range(11):
            d = []
            for h in (1e-5, -1e-5):
                x = l[t].copy()
                x[e] += h
                d.append((1.7 * g[t] * R.chosen_weights(x, ids[t], score, renorm)).sum())
            assert abs((d[0] - d[1]) / 2e-5 - got[t, e]) < 1e-8


def test_quantizer_residual_steps_give_the_correctly_rounded_quotient():
    """The kernel's quotient: q0 = x inv, then twice q + (x - q s) inv, each
    operation one FP32 rounding (the residual's product exact, as in a fused
    multiply-add), against the FP32 division."""
    rng = np.random.default_rng(7)
    f = np.float32

    def fma(a, b, c):
        # a * b is exact in 64 bits; the sum with c is rounded twice, which
        # shows here only if the first rounding lands on an FP32 midpoint
        return (a.astype(np.float64) * b.astype(np.float64) + c.astype(np.float64)).astype(f)

    amax = (rng.uniform(1, 2, 4000) * 2.0 ** rng.integers(-80, 80, 4000)).astype(f)
    s = (amax / f(127)).astype(f)
    inv = (f(1) / s).astype(f)
    for _ in range(40):
        x = (rng.uniform(-1, 1, 4000).astype(f) * amax).astype(f)
        k = rng.integers(0, 127, 4000) + 0.5             # quotients next to the codes' borders
        x = np.where(rng.random(4000) < 0.5, (k * s.astype(np.float64)).astype(f), x)
        x = np.where(rng.random(4000) < 0.3, np.nextafter(x, f(0)), x)
        q = (x * inv).astype(f)
        for _ in range(2):
            q = fma(fma(-q, s, x), inv, q)
        assert np.array_equal(np.rint(q), np.rint((x / s).astype(f)))

"""Plain 64-bit form of the experts of a mixture-of-experts layer and of its
weight formats, in numpy, straight from their definitions, with the error that
the library's arithmetic may have."""
import numpy as np

from tests.moe_ref import ACT_GELU, ACT_NONE, ACT_RELU, ACT_SILU, ACT_SWIGLU, act, logistic  # noqa: F401

INT8, BF16, E4M3, E5M2, E2M1, BLOCK = 32, 64, 0, 1, 4, 18
FORMATS = {"int8": INT8, "bf16": BF16, "e4m3": E4M3, "e5m2": E5M2, "e2m1": E2M1, "block": BLOCK}
UNIT = {INT8: 16, BF16: 8, E4M3: 32, E5M2: 32, E2M1: 32, BLOCK: 128}
HALF_BF16 = 2.0 ** -8
SUM = 2.0 ** -23        # a term's error in an FP32 sum whose order and rounding are the hardware's


def bf16(x):
    """The nearest BF16 of finite FP32 values, ties to even."""
    b = np.ascontiguousarray(x, np.float32).view(np.uint32)
    return ((b + 0x7FFF + ((b >> 16) & 1)) & 0xFFFF0000).astype(np.uint32).view(np.float32)


def _small_float(code, ebits, mbits, bias):
    e, m = (code >> mbits) & ((1 << ebits) - 1), code & ((1 << mbits) - 1)
    v = np.where(e > 0, (1 + m / 2.0 ** mbits) * 2.0 ** (e.astype(np.float64) - bias), m * 2.0 ** (1 - bias - mbits))
    return np.where((code >> (ebits + mbits)) & 1, -v, v)


def encode(rng, fmt, E, N, K, size):
    """Random weights [E, N, K] of the given size in a format: (codes, scales, values)."""
    if fmt == BF16:
        w = bf16(rng.standard_normal((E, N, K)) * size)
        return (w.view(np.uint32) >> 16).astype(np.uint16), None, w.astype(np.float64)
    if fmt == INT8:
        q = rng.integers(-128, 128, (E, N, K)).astype(np.int8)
        s = (rng.random((E, N)) + 0.5).astype(np.float32) * np.float32(size / 74)
        return q, s, q.astype(np.float64) * s.astype(np.float64)[..., None]
    if fmt == BLOCK:
        q = rng.integers(0, 256, (E, N, K)).astype(np.uint8)
        q[(q & 127) == 127] = 0                        # E4M3's NaN
        s = (rng.random((E, N // 128, K // 128)) + 0.5).astype(np.float32) * np.float32(size / 160)
        v = _small_float(q.astype(np.int64), 4, 3, 7)
        return q, s, v * s.astype(np.float64).repeat(128, 1).repeat(128, 2)
    s = (127 + rng.integers(-3, 4, (E, N, K // 32))).astype(np.uint8)
    if fmt == E2M1:
        c = rng.integers(0, 16, (E, N, K)).astype(np.int64)
        v, unit = _small_float(c, 2, 1, 1), size / 3
        q = (c[..., 0::2] | c[..., 1::2] << 4).astype(np.uint8)
    else:
        q = rng.integers(0, 256, (E, N, K)).astype(np.uint8)
        if fmt == E4M3:
            q[(q & 127) == 127] = 0
            v, unit = _small_float(q.astype(np.int64), 4, 3, 7), size / 160
        else:
            q[(q & 124) == 124] = 0                    # infinities and NaN
            v, unit = _small_float(q.astype(np.int64), 5, 2, 15), size / 16000
    s = (s.astype(np.int64) + int(np.floor(np.log2(unit)))).astype(np.uint8)
    return q, s, v * 2.0 ** (s.astype(np.float64) - 127).repeat(32, 2)


def experts(x, ids, w, v1, v2, a, residual=None):
    """(out, tolerance): x [T, D], ids and w [T, topk], v1 [E, N1, D] and
    v2 [E, D, F] as 64-bit values.

    Weights are exact in BF16.  z is an FP32 sum of D products and at most
    four more roundings (channel or block scale); no activation has a slope
    above 1.13, and the logistic form is off by a few units of FP32's last
    place and by its argument's rounding (64 units, as tests/moe_ref.py).  h is
    held as two BF16: off by half a step of the half step that the first
    leaves.  y is an FP32 sum of 2 F products, then scale, share, the sum over the
    token's experts and the residual.  Results below FP32's normal range may
    be flushed."""
    x, w = x.astype(np.float64), w.astype(np.float64)
    T, E = x.shape[0], v1.shape[0]
    out = np.zeros((T, v2.shape[1])) if residual is None else residual.astype(np.float64).copy()
    slip, size = np.zeros_like(out), np.abs(out)
    for t in range(T):
        for e in sorted({int(e) for e in ids[t] if 0 <= e < E}):
            share = sum(float(w[t, j]) for j in range(ids.shape[1]) if ids[t, j] == e)
            bulk = sum(abs(float(w[t, j])) for j in range(ids.shape[1]) if ids[t, j] == e)
            z = (v1[e] @ x[t])[None]
            dz = ((x.shape[1] + 4) * SUM * (np.abs(v1[e]) @ np.abs(x[t])))[None]
            h = act(z, a)
            if a == ACT_SWIGLU:
                g, u = z[:, 0::2], z[:, 1::2]
                dh = 1.13 * dz[:, 0::2] * np.abs(u) + np.abs(g * logistic(g)) * dz[:, 1::2] + dz[:, 0::2] * dz[:, 1::2]
            else:
                dh = 1.13 * dz
            if a not in (ACT_NONE, ACT_RELU):
                dh = dh + 64 * SUM * np.abs(h)
            dh = dh + HALF_BF16 * HALF_BF16 * np.abs(h) + 2.0 ** -126
            y, hull = v2[e] @ h[0], np.abs(v2[e]) @ (np.abs(h) + dh)[0]
            out[t] += share * y
            slip[t] += abs(share) * (np.abs(v2[e]) @ dh[0]) + bulk * (2 * v2.shape[2] + 8 + ids.shape[1]) * SUM * hull
            size[t] += bulk * hull
    slip += (ids.shape[1] + 1) * SUM * size
    return out, (np.abs(out) + slip) * HALF_BF16 + slip + 2.0 ** -126

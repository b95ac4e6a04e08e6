"""Plain 64-bit forms of the 8-bit integer GEMM and of the
mixture-of-experts operators, in numpy, straight from their definitions."""
import numpy as np

ACT_NONE, ACT_RELU, ACT_GELU, ACT_SILU, ACT_SWIGLU = 0, 1, 2, 3, 8
SOFTMAX, SIGMOID = 0, 1
GROUP_MAX, GROUP_TOP2 = 0, 1
HALF_BF16, HALF_F32 = 2.0 ** -8, 2.0 ** -24


def logistic(x):
    x = np.asarray(x, np.float64)
    e = np.exp(-np.abs(x))
    return np.where(x >= 0, 1.0 / (1.0 + e), e / (1.0 + e))


def act(z, a):
    if a == ACT_RELU:
        return np.maximum(z, 0.0)
    if a == ACT_GELU:
        return z * logistic(2 * np.sqrt(2 / np.pi) * (z + 0.044715 * z ** 3))
    if a == ACT_SILU:
        return z * logistic(z)
    if a == ACT_SWIGLU:
        return z[:, 0::2] * logistic(z[:, 0::2]) * z[:, 1::2]
    return z


def int8_gemm(A, sA, B, sB, bias=None, a=ACT_NONE):
    """(result, tolerance) of act(sA sB sum A B + bias) rounded to BF16.

    The kernel rounds the integer sum to FP32, multiplies twice and adds the
    bias with one more rounding: z is off by 3 half steps of the product and
    one of the sum with the bias.  No activation has a slope above 1.13; the
    logistic form is itself off by a few FP32 units of its last place, and by
    the rounding of its argument (at most |z| times a slope of 4 in u, at |z|
    where the result is not yet zero: below 64 units).  Then one rounding to
    BF16; results below FP32's normal range may be flushed."""
    S = A.astype(np.float64) @ B.astype(np.float64).T
    prod = S * sA.astype(np.float64)[:, None] * sB.astype(np.float64)[None, :]
    z = prod if bias is None else prod + bias.astype(np.float64)[None, :]
    dz = HALF_F32 * (3 * np.abs(prod) + np.abs(z)) * 1.01
    r = act(z, a)
    if a == ACT_SWIGLU:
        g, u = z[:, 0::2], z[:, 1::2]
        slip = 1.13 * dz[:, 0::2] * np.abs(u) + np.abs(g * logistic(g)) * dz[:, 1::2]
    else:
        slip = 1.13 * dz
    if a not in (ACT_NONE, ACT_RELU):
        slip = slip + 64 * 2 * HALF_F32 * np.abs(r)
    return r, (np.abs(r) + slip) * HALF_BF16 + slip + 2.0 ** -126


def quantize(x):
    """codes and scales of FP32 rows: s = max|x| / 127, rint(x / s), both as
    FP32 quotients."""
    x = np.asarray(x, np.float32)
    s = (np.abs(x).max(axis=1).astype(np.float32) / np.float32(127)).astype(np.float32)
    s[~(s > 0)] = 1.0
    q = (x / s[:, None]).astype(np.float32)
    return np.clip(np.rint(q), -127, 127).astype(np.int8), s


def scores(l, score):
    """64-bit scores of one token, 0 where an expert is not available."""
    ok = l > -np.inf
    l = np.where(ok, np.minimum(l, np.finfo(np.float32).max), 0.0)
    if score == SIGMOID:
        return np.where(ok, logistic(l), 0.0), ok
    if not ok.any():
        return np.zeros_like(l), ok
    e = np.where(ok, np.exp(l - l[ok].max()), 0.0)
    return e / e.sum(), ok


def chosen_weights(l, ids, score, renorm):
    """64-bit weights (before the scale) of chosen experts ids of one token."""
    s, _ = scores(l, score)
    if not renorm:
        return s[ids]
    x = np.minimum(l[ids], np.finfo(np.float32).max)
    # log of the scores up to a common constant
    lg = x if score == SOFTMAX else np.minimum(x, 0.0) - np.log1p(np.exp(-np.abs(x)))
    w = np.exp(lg - lg.max())
    return w / w.sum()


def route(logits, bias, topk, score, n_group=1, topk_group=1, group_score=GROUP_MAX, renorm=True, scale=1.0):
    logits = np.asarray(logits, np.float64)
    T, E = logits.shape
    n = E // n_group
    ids = np.full((T, topk), -1, np.int32)
    w = np.zeros((T, topk))
    for t in range(T):
        l = logits[t]
        s, ok = scores(l, score)
        sb = s if bias is None else s + bias.astype(np.float64)
        v = np.where(ok, l if bias is None else sb, -np.inf)
        sb = np.where(ok, sb, -np.inf)
        allowed = np.ones(E, bool)
        if n_group > 1:
            gs = []
            for g in range(n_group):
                part = np.sort((sb if group_score == GROUP_TOP2 else v)[g * n:(g + 1) * n])[::-1]
                part = part[part > -np.inf][:2 if group_score == GROUP_TOP2 else 1]
                gs.append(part.sum() if part.size else -np.inf)
            best = sorted(range(n_group), key=lambda g: (-gs[g], g))[:topk_group]
            allowed = np.isin(np.arange(E) // n, best)
        order = [e for e in sorted(range(E), key=lambda e: (-v[e], e)) if allowed[e] and v[e] > -np.inf][:topk]
        if order:
            ids[t, :len(order)] = order
            w[t, :len(order)] = chosen_weights(l, np.array(order), score, renorm) * scale
    return ids, w


def maps(ids, E):
    T, k = ids.shape
    flat = ids.reshape(-1)
    row_of = np.full(T * k, -1, np.int32)
    slot_of = np.full(T * k, -1, np.int32)
    r = 0
    sizes = np.zeros(E, np.int64)
    for e in range(E):
        for s in np.nonzero(flat == e)[0]:
            row_of[s] = r
            slot_of[r] = s
            r += 1
            sizes[e] += 1
    return sizes, row_of.reshape(T, k), slot_of


def route_grad(logits, ids, grad, score, renorm, scale):
    logits = np.asarray(logits, np.float64)
    out = np.zeros_like(logits)
    for t in range(len(logits)):
        l = logits[t]
        s, ok = scores(l, score)
        sel = [(e, j) for j, e in enumerate(ids[t]) if 0 <= e < len(l) and ok[e]]
        e = np.array([x[0] for x in sel], np.int64)
        c = scale * grad[t, [x[1] for x in sel]].astype(np.float64)
        if renorm:
            if len(e):
                w = chosen_weights(l, e, score, True)
                out[t, e] = w * (c - (c * w).sum()) * (logistic(-l[e]) if score == SIGMOID else 1.0)
        elif score == SIGMOID:
            out[t, e] = c * logistic(l[e]) * logistic(-l[e])
        else:
            ds = np.zeros_like(l)
            ds[e] = c
            out[t] = s * (ds - (ds * s).sum())
    return out


def combine(y, w, row_of, N):
    """(result, tolerance): an FP32 sum of topk products, each step one
    rounding, then one to BF16."""
    T, k = row_of.shape
    out, mag = np.zeros((T, N)), np.zeros((T, N))
    for t in range(T):
        for j in range(k):
            r = row_of[t, j]
            if 0 <= r < len(y):
                out[t] += float(w[t, j]) * y[r]
                mag[t] += np.abs(float(w[t, j]) * y[r])
    slip = k * HALF_F32 * mag * 1.01
    return out, np.abs(out) * HALF_BF16 + slip * (1 + HALF_BF16) + 2.0 ** -126

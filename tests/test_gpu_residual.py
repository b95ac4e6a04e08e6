"""GPU: the product with bias, activation and residual in its epilogue, on
every kernel and format, and the epilogue's gradient, against 64-bit forms."""
import numpy as np
import pytest
import torch

import oracle
from block_scaled_precision_03_amd import synth
from tests import residual_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
b16, f32 = torch.bfloat16, torch.float32
ACTS = [R.ACT_NONE, R.ACT_RELU, R.ACT_GELU, R.ACT_SILU]
FORMATS = {"mx44": (0, 0), "mx45": (0, 1), "mx54": (1, 0), "fp4": (4, 4), "tw44": (16, 16), "tw54": (17, 16), "int8": (32, 32)}
ELEM = {0: "e4m3", 1: "e5m2", 4: "e2m1", 16: "e4m3", 17: "e5m2"}
CODE = {"e4m3": oracle.E4M3, "e5m2": oracle.E5M2, "e2m1": oracle.E2M1}


def _mx():
    from block_scaled_precision_03_amd import mxgemm
    return mxgemm


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def operand(fmt, rows, K, seed, size=1.0):
    """(codes, scales, 64-bit values) on the device."""
    rng = np.random.default_rng(seed)
    if fmt == 32:
        q = rng.integers(-128, 128, (rows, K)).astype(np.int8)
        s = ((rng.random(rows) + 0.5) * size / 74).astype(np.float32)
        return dev(q), dev(s), dev(q).double() * dev(s).double()[:, None]
    x = (rng.standard_normal((rows, K)) * size).astype(np.float32)
    e = ELEM[fmt]
    if fmt >= 16:
        q, s = synth.quant_tensor(x, e)
        v = oracle.dequant(CODE[e], oracle.SCALE_TENSOR, 0, q, s, rows, K)
        return dev(q), dev(np.array([s], np.float32)), dev(np.asarray(v, np.float64).reshape(rows, K))
    q, s = synth.quant_mx(x, e)
    v = oracle.dequant(CODE[e], oracle.SCALE_MX, 0, q, s, rows, K)
    return dev(q), dev(s), dev(np.asarray(v, np.float64).reshape(rows, K))


class Case:
    def __init__(self, name, M, N, K, a=R.ACT_NONE, bias=True, residual=True, z=True, psb=False, seed=0):
        m = _mx()
        self.fa, self.fb = FORMATS[name]
        self.M, self.N, self.K, self.a, self.psb = M, N, K, a, psb
        self.No = N // 2 if a == R.ACT_SWIGLU else N
        self.A, self.sA, va = operand(self.fa, M, K, seed + 1)
        self.B, self.sB, vb = operand(self.fb, N, K, seed + 2, K ** -0.5)
        g = torch.Generator(device=DEV)
        g.manual_seed(seed)
        randn = lambda *s: torch.randn(*s, device=DEV, generator=g).to(b16)
        self.bias = randn(N) if bias else None
        self.r = randn(M, self.No) if residual else None
        self.D = torch.full((M + 2, self.No), 7.0, dtype=b16, device=DEV)
        self.Z = torch.full((M + 2, N), 7.0, dtype=b16, device=DEV) if z else None
        bulk = va.abs() @ vb.abs().t()
        # integer codes before their scales: their 64-bit sum is exact, that of
        # scaled ones is off by 2^-53 of the terms where they cancel to zero
        prod = va @ vb.t() if self.fa != 32 else (self.A.double() @ self.B.double().t()) * self.sA.double()[:, None] * self.sB.double()
        self.z = prod if not bias else prod + self.bias.double()
        # integer sums are exact; each product of FP8 and FP4 codes is, and K
        # of them are summed in FP32; scales and the bias: four roundings more
        terms = 4 * prod.abs() if self.fa == 32 else (K + 4) * bulk
        self.dz = R.SUM * (terms + self.z.abs())
        if psb:
            b = torch.empty(m.preshuffle_b_bytes(self.fb, N, K), dtype=torch.uint8, device=DEV)
            m.preshuffle_b(self.fb, m.NT, self.B, b, N, K)
            self.B = b
            if self.fb < 16:
                s = torch.empty(m.preshuffle_scales_bytes(N, K), dtype=torch.uint8, device=DEV)
                m.preshuffle_scales(self.sB, s, N, K)
                self.sB = s

    def rows(self, t):
        """M rows of a guarded buffer, at 16 bytes."""
        flat = t.view(-1)
        start = 8 * -(-t.shape[1] // 8)
        return flat[start:start + self.M * t.shape[1]].view(self.M, t.shape[1])

    def run(self, D=None, residual="own"):
        m = _mx()
        D = self.rows(self.D) if D is None else D
        m.run_residual(self.fa, self.fb | (m.PRESHUFFLED if self.psb else 0), m.NT, self.A, self.sA, self.B, self.sB, D,
                       self.M, self.N, self.K, bias=self.bias, activation=self.a, residual=self.r if residual == "own" else residual,
                       z=None if self.Z is None else self.rows(self.Z))
        return D

    def check(self):
        D = self.run()
        want, tol, ztol = R.epilogue(self.z, self.dz, self.a, self.r)
        bad = (D.double() - want).abs() > tol
        assert not bad.any(), "%d of %d off, first at %s" % (int(bad.sum()), bad.numel(), bad.nonzero()[0].tolist())
        if self.Z is not None:
            bad = (self.rows(self.Z).double() - self.z).abs() > ztol
            assert not bad.any(), "z: %d of %d off, first at %s" % (int(bad.sum()), bad.numel(), bad.nonzero()[0].tolist())
        for t in (self.D, self.Z):
            if t is not None:
                flat, start = t.view(-1), 8 * -(-t.shape[1] // 8)
                end = start + self.M * t.shape[1]
                assert (flat[:start] == 7).all() and (flat[end:] == 7).all()


def k_of(name, K):
    return K if name != "fp4" else -(-K // 256) * 256


@pytest.mark.parametrize("name", sorted(FORMATS))
@pytest.mark.parametrize("M,N,K", [(1, 64, 256), (1, 1026, 2048), (3, 130, 128), (16, 258, 384), (17, 66, 640), (40, 514, 1280),
                                   (70, 130, 256), (333, 1002, 384)])
def test_small_outputs(name, M, N, K):
    Case(name, M, N, k_of(name, K), a=ACTS[M % 4], seed=M).check()


@pytest.mark.parametrize("name", ["mx44", "fp4", "tw54", "mx45"])
@pytest.mark.parametrize("psb", [False, True])
@pytest.mark.parametrize("M,N,K,few", [(3, 70, 1024, True), (25, 1026, 2048, True),        # 8 x 16 tiles, one and several
                                       (37, 1026, 2048, True), (13, 4098, 2048, None),       # 16 x 16
                                       (16, 4098, 4096, True), (40, 2050, 2048, True),       # 32 x 32
                                       (100, 3000, 2048, True), (60, 8194, 2048, True),      # 64 x 32, 64 x 64
                                       (700, 770, 512, None), (4, 40000, 256, False), (300, 6000, 256, False)])
def test_every_kernel(name, psb, M, N, K, few):
    m = _mx()
    fa, fb = FORMATS[name]
    if few is not None:
        got = m.residual_variant(fa, fb | (m.PRESHUFFLED if psb else 0), m.NT, M, N, K)
        assert got == (m.DENSE_ROWS if few else m.DENSE_TILE64)
    Case(name, M, N, K, a=R.ACT_SILU, psb=psb, seed=M).check()


def test_every_kernel_is_chosen_somewhere():
    m = _mx()
    sizes = [(3, 70, 1024), (100, 3000, 2048), (4, 40000, 256), (300, 6000, 256), (2148, 2304, 512)]
    got = {m.residual_variant(f, f, m.NT, *s) for f in (0, 4, 16) for s in sizes}
    assert got == {m.DENSE_ROWS, m.DENSE_TILE64, m.DENSE_TILE256}


@pytest.mark.parametrize("name", ["mx44", "fp4", "tw54", "mx54"])
@pytest.mark.parametrize("M,N", [(1, 130), (9, 4098), (65, 200)])
def test_preshuffled(name, M, N):
    for a in ACTS:
        Case(name, M, N, 1024, a=a, psb=True, seed=a).check()


@pytest.mark.parametrize("name", sorted(FORMATS))
@pytest.mark.parametrize("bias,residual,z", [(False, True, False), (False, False, True), (True, True, False), (False, True, True)])
def test_every_part_alone(name, bias, residual, z):
    """Odd N too, where nothing takes columns in pairs."""
    N = 258 if bias else 259
    Case(name, 37, N, 512, a=R.ACT_SILU, bias=bias, residual=residual, z=z).check()
    Case(name, 2, N, 512, a=R.ACT_NONE, bias=bias, residual=residual, z=z).check()


@pytest.mark.parametrize("name", sorted(FORMATS))
@pytest.mark.parametrize("K", [512, 768])
@pytest.mark.parametrize("a", ACTS)
def test_large_tiles(name, K, a):
    """256 x 256 tiles: whole ones and both ragged edges."""
    m = _mx()
    M, N = 2048 + 100, 2304 + (58 if a else 0)
    fa, fb = FORMATS[name]
    if name != "int8":
        assert m.dense_variant(fa, fb, m.NT, M, N, K) == m.DENSE_TILE256
    Case(name, M, N, K, a=a, psb=name in ("mx44", "fp4") and a == R.ACT_GELU, seed=a).check()


@pytest.mark.parametrize("name,psb", [("mx44", False), ("mx44", True), ("fp4", True), ("tw44", False), ("int8", False)])
@pytest.mark.parametrize("K", [256, 1280, 1536])
def test_several_tiles_per_workgroup(name, psb, K):
    """More tiles than compute units: a tile's epilogue in the next one's first step."""
    K = k_of(name, K)
    M, N = 4352 + 30, 4608
    Case(name, M, N, K, a=R.ACT_GELU if K == 1280 else R.ACT_NONE, z=K != 1536, psb=psb, seed=K).check()


@pytest.mark.parametrize("M,N,K", [(1, 10, 48), (5, 1030, 4096), (33, 514, 512), (300, 642, 1040), (1100, 2562, 272),
                                   (2500, 2560, 1040), (4400, 5122, 272)])
def test_int8_swiglu(M, N, K):
    Case("int8", M, N, K, a=R.ACT_SWIGLU, seed=M).check()
    Case("int8", M, N, K, a=R.ACT_SWIGLU, bias=False, z=False, seed=M).check()


@pytest.mark.parametrize("M,N,K", [(6831, 6723, 48), (777, 5002, 4112), (4400, 5123, 272)])
def test_int8_odd_pitches(M, N, K):
    Case("int8", M, N, K, a=R.ACT_SILU, bias=N % 2 == 0).check()


@pytest.mark.parametrize("name,M,N,K", [("mx44", 4608, 4352, 1280), ("int8", 4608, 4352, 1280), ("mx44", 5, 512, 1024),
                                        ("int8", 5, 512, 1024), ("tw44", 300, 515, 256), ("int8", 300, 515, 272)])
def test_in_place(name, M, N, K):
    """The residual's buffer as the result's."""
    c = Case(name, M, N, K, a=R.ACT_NONE, bias=False, z=False)
    want = c.run().clone()
    r = c.r.clone()
    c.run(D=r, residual=r)
    assert torch.equal(r, want)


@pytest.mark.parametrize("name", sorted(FORMATS))
@pytest.mark.parametrize("M,N,K", [(1, 514, 2048), (130, 258, 512), (2148, 2306, 512)])
def test_without_residual_and_z(name, M, N, K):
    """Bias and activation alone, and nothing: integer sums as run_fused, bit for bit."""
    m = _mx()
    for bias, a in ((True, R.ACT_GELU), (False, R.ACT_NONE)):
        c = Case(name, M, N, K, a=a, bias=bias, residual=False, z=False)
        c.check()
        if name == "int8":
            D = torch.empty(M, N, dtype=b16, device=DEV)
            m.run_fused(c.fa, c.fb, m.NT, c.A, c.sA, c.B, c.sB, D, M, N, K, bias=c.bias, activation=a)
            assert torch.equal(c.run(), D)


@pytest.mark.parametrize("name", ["mx44", "mx54", "fp4", "tw54"])
@pytest.mark.parametrize("N", [2305, 2306, 2308, 2310])
def test_large_tiles_at_any_pitch(name, N):
    Case(name, 2148, N, 512, a=R.ACT_RELU if N == 2306 else R.ACT_NONE, bias=N % 2 == 0, seed=N).check()


@pytest.mark.parametrize("name", ["mx44", "fp4", "tw54"])
@pytest.mark.parametrize("M,N,K", [(635, 194, 2304), (2049, 62, 768), (5000, 130, 512), (777, 770, 1280)])
def test_few_tiles_of_many_rows(name, M, N, K):
    m = _mx()
    for psb in (False, True):
        c = Case(name, M, N, K, a=R.ACT_GELU if psb else R.ACT_NONE, psb=psb, seed=M)
        assert m.residual_variant(c.fa, c.fb, m.NT, M, N, K) == m.DENSE_ROWS
        c.check()


@pytest.mark.parametrize("name", ["mx45", "fp4", "tw44"])
@pytest.mark.parametrize("past", [3, 5, 7, 8, 29, 61, 129, 255])
def test_last_columns_of_large_tiles(name, past):
    """Last column tiles of any width, the last row tile one row high, the
    residual replaced in place, z beside it."""
    m = _mx()
    M, N = 2305, 2048 + past
    c = Case(name, M, N, 512, a=R.ACT_SILU if past & 8 else R.ACT_NONE, bias=False, seed=past)
    assert m.residual_variant(c.fa, c.fb, m.NT, M, N, 512) == m.DENSE_TILE256
    c.check()
    want = c.rows(c.D).clone()
    c.rows(c.D).copy_(c.r)
    c.run(residual=c.rows(c.D))
    assert torch.equal(c.rows(c.D), want)


@pytest.mark.parametrize("name", ["mx44", "int8"])
def test_no_k_and_no_rows(name):
    m = _mx()
    fa, fb = FORMATS[name]
    bias, r = torch.randn(10, device=DEV).to(b16), torch.randn(7, 10, device=DEV).to(b16)
    D, z = torch.zeros(7, 10, dtype=b16, device=DEV), torch.zeros(7, 10, dtype=b16, device=DEV)
    m.run_residual(fa, fb, m.NT, None, None, None, None, D, 7, 10, 0, bias=bias, activation=R.ACT_RELU, residual=r, z=z)
    assert torch.equal(z, bias.expand(7, 10)) and torch.equal(D, (bias.float().clamp(min=0) + r.float()).to(b16))
    m.run_residual(fa, fb, m.NT, None, None, None, None, None, 0, 10, 128, residual=None, z=None)
    if name == "int8":
        r2 = r[:, :5].contiguous()
        D2 = torch.zeros(7, 5, dtype=b16, device=DEV)
        m.run_residual(fa, fb, m.NT, None, None, None, None, D2, 7, 10, 0, bias=bias, activation=R.ACT_SWIGLU, residual=r2, z=z)
        want, tol, _ = R.epilogue(bias.double().expand(7, 10), torch.zeros(7, 10, device=DEV).double(), R.ACT_SWIGLU, r2)
        assert ((D2.double() - want).abs() <= tol).all() and torch.equal(z, bias.expand(7, 10))


@pytest.mark.parametrize("name,M,N,K", [("mx44", 3, 258, 1024), ("mx44", 4608, 4352, 512), ("int8", 300, 642, 1040)])
def test_graph_and_stream(name, M, N, K):
    c = Case(name, M, N, K, a=R.ACT_SILU)
    want, z = c.run().clone(), c.rows(c.Z).clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run()
    s = torch.cuda.Stream()
    for _ in range(3):
        c.D.fill_(3)
        c.Z.fill_(3)
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            g.replay()
        torch.cuda.synchronize()
        assert torch.equal(c.rows(c.D), want) and torch.equal(c.rows(c.Z), z)


# ---- gradient ---------------------------------------------------------------

def backward(a, M, N, dz=True, dbias=True, in_place=None, seed=0, special=False):
    m = _mx()
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    No = N // 2 if a == R.ACT_SWIGLU else N
    d = torch.randn(M, No, device=DEV, generator=g).to(b16)
    z = (torch.randn(M, N, device=DEV, generator=g) * 3).to(b16)
    if special:
        # where the slopes end: far out, and around their zeros
        v = torch.tensor([0.0, -0.0, 1e-3, -1.28, -0.75, 7.9, -8.1, 15.9, -16.2, 40.0, -60.0, 88.0, -90.0, 126.0, -130.0, 3e38, -3e38], device=DEV)
        z.view(-1)[:v.numel()] = v.to(b16)
    want, slip, bias, btol = R.gradient(d, z, a)
    guard = torch.full((M * N + 64,), 7.0, dtype=b16, device=DEV)
    out = guard[:M * N].view(M, N)
    if in_place == "z":
        out = z
    elif in_place == "dD":
        out = d
    db = torch.full((N + 1,), 7.0, dtype=f32, device=DEV)
    need = m.residual_backward_workspace_bytes(M, N)
    ws = torch.full((need + 64,), 0xA5, dtype=torch.uint8, device=DEV)
    m.residual_backward(a, d, None if a == R.ACT_NONE else z, out if dz else None, db[:N] if dbias else None, M, N,
                        workspace=ws[:need] if need else None)
    if dz:
        tol = (want.abs() + slip) * R.HALF_BF16 + slip
        bad = (out.double() - want).abs() > tol
        assert not bad.any(), "%d off, first at %s" % (int(bad.sum()), bad.nonzero()[0].tolist())
    if dbias:
        assert ((db[:N].double() - bias).abs() <= btol).all()
    assert db[N] == 7 and (ws[need:] == 0xA5).all() and (guard[M * N:] == 7).all()
    return out, db


ALL = ACTS + [R.ACT_SWIGLU]


@pytest.mark.parametrize("a", ALL)
@pytest.mark.parametrize("M,N", [(1, 2), (1, 1000), (2, 8), (15, 514), (16, 512), (17, 510), (129, 5002), (256, 258), (257, 260), (300, 4608), (2000, 66), (9327, 146)])
def test_gradient(a, M, N):
    backward(a, M, N, seed=M, special=M * N > 100)


@pytest.mark.parametrize("a", ACTS)
@pytest.mark.parametrize("M,N", [(1, 1), (5, 3), (130, 513), (33, 1023)])
def test_gradient_odd_columns(a, M, N):
    backward(a, M, N)


@pytest.mark.parametrize("a", ALL)
def test_gradient_parts_and_in_place(a):
    backward(a, 70, 1030, dbias=False)
    backward(a, 70, 1030, dz=False)
    backward(a, 70, 1030, in_place="z")
    if a != R.ACT_SWIGLU:
        backward(a, 70, 1030, in_place="dD")


def test_gradient_of_no_rows():
    m = _mx()
    db = torch.full((5,), 7.0, device=DEV)
    m.residual_backward(R.ACT_SILU, None, None, None, db, 0, 5)
    assert (db == 0).all()
    m.residual_backward(R.ACT_SILU, None, None, None, db, 3, 0)


def test_gradient_not_finite():
    m = _mx()
    for a in (R.ACT_GELU, R.ACT_SILU):
        z = torch.tensor([[float("inf"), float("-inf"), float("nan"), 1.0]], dtype=b16, device=DEV)
        d, dz = torch.ones(1, 4, dtype=b16, device=DEV), torch.zeros(1, 4, dtype=b16, device=DEV)
        m.residual_backward(a, d, z, dz, None, 1, 4)
        assert dz[0, 0] == 1 and dz[0, 1] == 0 and torch.isnan(dz[0, 2]) and torch.isfinite(dz[0, 3])


def test_gradient_same_bits_and_graph():
    m = _mx()
    M, N = 1000, 1536
    d, z = torch.randn(M, N, device=DEV).to(b16), torch.randn(M, N, device=DEV).to(b16)
    dz, db = torch.empty_like(z), torch.empty(N, device=DEV)
    ws = torch.empty(m.residual_backward_workspace_bytes(M, N), dtype=torch.uint8, device=DEV)
    run = lambda: m.residual_backward(R.ACT_GELU, d, z, dz, db, M, N, workspace=ws)
    run()
    want = dz.clone(), db.clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    for k in range(4):
        dz.fill_(k), db.fill_(k), ws.fill_(0xFF)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(dz, want[0]) and torch.equal(db, want[1])


def test_gradient_past_4_gib():
    """2^31 elements and more: the last rows and columns."""
    m = _mx()
    M, N = 70000, 32768
    d = torch.zeros(M, N, dtype=b16, device=DEV)
    d[-3:] = torch.randn(3, N, device=DEV).to(b16)
    z = torch.zeros(M, N, dtype=b16, device=DEV)
    z[-3:] = torch.randn(3, N, device=DEV).to(b16)
    want, slip, bias, btol = R.gradient(d[-3:], z[-3:], R.ACT_SILU)
    db = torch.empty(N, device=DEV)
    ws = torch.empty(m.residual_backward_workspace_bytes(M, N), dtype=torch.uint8, device=DEV)
    m.residual_backward(R.ACT_SILU, d, z, z, db, M, N, workspace=ws)
    assert ((z[-3:].double() - want).abs() <= (want.abs() + slip) * R.HALF_BF16 + slip).all()
    assert ((db.double() - bias).abs() <= btol).all() and (z[:-3] == 0).all()


def test_block_forward_and_gradient():
    """A training step's two calls together: y = x + act(x W^T + b), and the
    gradients of z, b and x's residual from y's."""
    c = Case("mx44", 200, 514, 512, a=R.ACT_GELU)
    c.check()
    m = _mx()
    d = torch.randn(200, 514, device=DEV).to(b16)
    z = c.rows(c.Z)
    dz, db = torch.empty(200, 514, dtype=b16, device=DEV), torch.empty(514, device=DEV)
    ws = torch.empty(m.residual_backward_workspace_bytes(200, 514), dtype=torch.uint8, device=DEV)
    m.residual_backward(R.ACT_GELU, d, z, dz, db, 200, 514, workspace=ws)
    leaf, b = z.double().requires_grad_(), torch.zeros(514, dtype=torch.float64, device=DEV, requires_grad=True)
    (R.act(leaf + b, R.ACT_GELU) * d.double()).sum().backward()
    _, slip, _, btol = R.gradient(d, z, R.ACT_GELU)
    assert ((dz.double() - leaf.grad).abs() <= (leaf.grad.abs() + slip) * R.HALF_BF16 + slip).all()
    assert ((db.double() - b.grad).abs() <= btol).all()


@pytest.mark.parametrize("M,N", [(4, 8), (3, 1030), (300, 520)])
def test_gradient_of_dead_units(M, N):
    """ReLU: no gradient where z is not positive, whatever arrives there."""
    m = _mx()
    inf, nan = float("inf"), float("nan")
    d = torch.tensor([inf, -inf, nan, 2.0], device=DEV).repeat(M, N // 4 + 1)[:, :N].to(b16).contiguous()
    z = torch.tensor([-1.0, 0.0, -3.0, -4.0, 5.0, 6.0, 7.0, 8.0], device=DEV).repeat(M, N // 8 + 1)[:, :N].to(b16).contiguous()
    want = torch.where(z > 0, d, torch.zeros_like(d))
    dz, db = torch.empty(M, N, dtype=b16, device=DEV), torch.empty(N, device=DEV)
    ws = torch.empty(m.residual_backward_workspace_bytes(M, N) + 16, dtype=torch.uint8, device=DEV)
    m.residual_backward(R.ACT_RELU, d, z, dz, db, M, N, workspace=ws)
    assert torch.equal(dz.nan_to_num(-9), want.nan_to_num(-9)) and torch.equal(dz.isnan(), want.isnan())
    # sums of equal values, multiples of 2 below 2^24: exact
    sums = M * want[0].float()
    assert torch.equal(db.nan_to_num(-9), sums.nan_to_num(-9)) and torch.equal(db.isnan(), sums.isnan())


def test_gradient_of_very_long_rows():
    """More workgroups than one dimension of a grid holds: 2^29 columns and
    some, and the zeros of no rows."""
    m = _mx()
    N = (1 << 29) + 130
    d = torch.ones(1, N, dtype=b16, device=DEV)
    z = torch.full((1, N), -1.0, dtype=b16, device=DEV)
    at = torch.tensor([0, 1, 127, 128, (1 << 27) - 1, 1 << 27, 1 << 28, (1 << 29) - 1, 1 << 29, N - 3, N - 1], device=DEV)
    z[0, at] = 1.0
    dz, db = torch.full((1, N), 7.0, dtype=b16, device=DEV), torch.full((N,), 7.0, device=DEV)
    assert m.residual_backward_workspace_bytes(1, N) == 0
    m.residual_backward(R.ACT_RELU, d, z, dz, db, 1, N)
    assert (dz[0, at] == 1).all() and (db[at] == 1).all()
    assert int((dz != 0).sum()) == at.numel() and int((db != 0).sum()) == at.numel()
    m.residual_backward(R.ACT_RELU, None, None, None, db, 0, N)
    assert int((db != 0).sum()) == 0

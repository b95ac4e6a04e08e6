"""GPU: the fused ends of a feed-forward block as they are used together: a
shared expert's products with the residual, the router and the chosen experts
on top of it, eager, captured, replayed with other inputs, and first calls of
a new process inside a capture."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from tests import experts_ref as X
from tests import moe_ref as M
from tests import residual_ref as R

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
DEV = "cuda:0"
b16, f32 = torch.bfloat16, torch.float32


def _mx():
    from block_scaled_precision_03_amd import mxgemm
    return mxgemm


class Block:
    """x + shared(x) + experts(x) in 8-bit integers and MXFP4; buffers kept."""

    def __init__(self, T, D, F, E, k, seed=0):
        m = _mx()
        rng = np.random.default_rng(seed)
        self.T, self.D, self.F, self.E, self.k = T, D, F, E, k
        dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(DEV)
        # shared expert: INT8 up with SwiGLU, INT8 down
        self.u, self.su, self.vu = X.encode(rng, X.INT8, 1, 2 * F, D, D ** -0.5)
        self.d, self.sd, self.vd = X.encode(rng, X.INT8, 1, D, F, F ** -0.5)
        self.w1, self.s1, self.v1 = X.encode(rng, X.E2M1, E, 2 * F, D, D ** -0.5)
        self.w2, self.s2, self.v2 = X.encode(rng, X.E2M1, E, D, F, F ** -0.5)
        self.dev = {n: dev(getattr(self, n)) for n in ("u", "su", "d", "sd", "w1", "s1", "w2", "s2")}
        z = lambda dt, *s: torch.zeros(*s, dtype=dt, device=DEV)
        self.x, self.logits = z(b16, T, D), z(f32, T, E)
        self.xq, self.xs, self.h = z(torch.int8, T, D), z(f32, T), z(b16, T, F)
        self.hq, self.hs, self.y, self.out = z(torch.int8, T, F), z(f32, T), z(b16, T, D), z(b16, T, D)
        self.ids, self.w = z(torch.int32, T, k), z(f32, T, k)
        self.ws = z(torch.uint8, m.moe_experts_workspace_bytes(T, k, F))

    def fill(self, seed):
        g = torch.Generator(device=DEV)
        g.manual_seed(seed)
        self.x.copy_(torch.randn(self.T, self.D, device=DEV, generator=g).to(b16))
        self.logits.copy_(torch.randn(self.T, self.E, device=DEV, generator=g))

    def step(self):
        m, v = _mx(), self.dev
        T, D, F = self.T, self.D, self.F
        m.quantize_int8(m.BF16, self.x, self.xq, self.xs, T, D)
        m.run_fused(m.INT8, m.INT8, m.NT, self.xq, self.xs, v["u"], v["su"], self.h, T, 2 * F, D, activation=m.ACT_SWIGLU)
        m.quantize_int8(m.BF16, self.h, self.hq, self.hs, T, F)
        m.run_residual(m.INT8, m.INT8, m.NT, self.hq, self.hs, v["d"], v["sd"], self.y, T, D, F, residual=self.x)
        m.moe_route(m.F32, self.logits, None, self.ids, self.w, T, self.E, self.k)
        m.moe_experts(m.MXFP4_E2M1, self.x, self.ids, self.w, v["w1"], v["s1"], v["w2"], v["s2"], self.out, T, self.E, self.k,
                      D, F, residual=self.y, workspace=self.ws)

    def check(self):
        """The experts' share on top of what the shared expert left, and that
        against its own 64-bit form."""
        n = lambda t: t.float().cpu().numpy().astype(np.float64)
        hq, hs = self.hq.cpu().numpy().astype(np.float64), self.hs.cpu().numpy().astype(np.float64)
        prod = torch.from_numpy((hq @ self.d[0].astype(np.float64).T) * hs[:, None] * self.sd[0].astype(np.float64))
        want, tol, _ = R.epilogue(prod, 4 * R.SUM * prod.abs(), R.ACT_NONE, self.x.cpu())
        assert ((self.y.cpu().double() - want).abs() <= tol).all()
        out, tol = X.experts(n(self.x), self.ids.cpu().numpy(), self.w.cpu().numpy(), self.v1, self.v2, M.ACT_SWIGLU, n(self.y))
        assert (np.abs(n(self.out) - out) <= tol).all()


@pytest.mark.parametrize("T", [1, 2, 9, 50])
def test_block(T):
    b = Block(T, 192, 96, 7, 3)
    b.fill(1)
    b.step()
    b.check()


def test_block_replayed():
    b = Block(6, 256, 160, 5, 2)
    b.fill(1)
    b.step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b.step()
    for seed in range(4):
        b.fill(seed)
        g.replay()
        torch.cuda.synchronize()
        b.check()
        got = b.out.clone()
        b.step()
        assert torch.equal(b.out, got)


def test_two_threads_and_two_streams():
    import threading
    blocks = [Block(4, 192, 96, 7, 3, seed=s) for s in (1, 2)]
    streams = [torch.cuda.Stream() for _ in blocks]
    for b in blocks:
        b.fill(3)
    torch.cuda.synchronize()

    def work(b, s):
        with torch.cuda.stream(s):
            for _ in range(20):
                b.step()

    threads = [threading.Thread(target=work, args=a) for a in zip(blocks, streams)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for b in blocks:
        b.check()


FIRST = """
import torch
from block_scaled_precision_03_amd import mxgemm as m
dev = "cuda:0"
z = lambda dt, *s: torch.zeros(*s, dtype=dt, device=dev)
b16, u8 = torch.bfloat16, torch.uint8
M, N, K = {sizes}
codes = lambda r, c: torch.randint(0, 100, (r, c), dtype=u8, device=dev)
A, B, R = codes(M, K), codes(N, K), torch.randn(M, N, device=dev).to(b16)
s8 = [torch.full((r, K // 32), 120, dtype=u8, device=dev) for r in (M, N)]
sf = [torch.full((r,), 0.01, device=dev) for r in (M, N)]
out = []
fmts = [(0, 0), (1, 0), (16, 16), (17, 16), (4, 4), (32, 32)]
D = [z(b16, M, N) for _ in fmts]
Z = [z(b16, M, N) for _ in fmts]
dz, db = z(b16, M, N), z(torch.float32, N)
ws = z(u8, max(1, m.residual_backward_workspace_bytes(M, N)))
T, E, k, F = 3, 4, 2, 64
x, ids = torch.randn(T, 128, device=dev).to(b16), torch.randint(0, E, (T, k), dtype=torch.int32, device=dev)
w, w1, w2 = torch.rand(T, k, device=dev), codes(E * 2 * F, 128), codes(E * 128, F)
s1, s2 = torch.full((E * 2 * F, 4), 118, dtype=u8, device=dev), torch.full((E * 128, 2), 118, dtype=u8, device=dev)
eo, ews = z(b16, T, 128), z(u8, m.moe_experts_workspace_bytes(T, k, F))
def run():
    for (fa, fb), d, y in zip(fmts, D, Z):
        s = sf if fa >= 16 else s8
        m.run_residual(fa, fb, m.NT, A, s[0], B, s[1], d, M, N, K, activation=m.ACT_SILU, residual=R, z=y)
    m.residual_backward(m.ACT_SILU, D[0], Z[0], dz, db, M, N, workspace=ws)
    m.moe_experts(m.MXFP8_E4M3, x, ids, w, w1, s1, w2, s2, eo, T, E, k, 128, F, workspace=ews)
torch.cuda.synchronize()
m.init()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    run()
got = []
outs = D + Z + [dz, db, eo]
for _ in range(3):
    for t in outs:
        t.fill_(5)
    torch.cuda.synchronize()
    g.replay()
    torch.cuda.synchronize()
    got.append([t.clone() for t in outs])
for t in outs:
    t.fill_(5)
run()
torch.cuda.synchronize()
for r in got:
    for a, b in zip(r, outs):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
print("same")
"""


@pytest.mark.parametrize("sizes", ["5, 70, 512", "300, 6000, 256", "2148, 2304, 512"])
def test_first_calls_in_a_graph(sizes):
    r = subprocess.run([sys.executable, "-c", FIRST.replace("{sizes}", sizes)], cwd=ROOT, capture_output=True, text=True, timeout=100)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]

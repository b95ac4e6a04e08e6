"""GPU: in a new process, the first call after mxgemm_init of the gradients of
router and combine, of the grouped integer GEMM (each of its kernels, SwiGLU
and plain) and of the quantizer into the experts' rows is captured into a graph
(mxgemm_init has loaded their code); replays give the eager results."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

FIRST = """
import torch
from block_scaled_precision_03_amd import mxgemm as m
dev = "cuda:0"
T, E, k, N = 200, 16, 3, 256
n = T * k
z = lambda dt, *s: torch.zeros(*s, dtype=dt, device=dev)
i8, i32, f32, b16 = torch.int8, torch.int32, torch.float32, torch.bfloat16
x, logits, dout, dw = torch.randn(T, N).bfloat16().to(dev), torch.randn(T, E).to(dev), torch.randn(T, N).bfloat16().to(dev), torch.randn(T, k).to(dev)
ids = torch.stack([torch.randperm(E)[:k] for _ in range(T)]).int().to(dev)
rows = torch.randperm(n).int().view(T, k).to(dev)
y, w = torch.randn(n, N).bfloat16().to(dev), torch.rand(T, k).to(dev)
code = lambda *s: torch.randint(-9, 9, s, dtype=i8).to(dev)
# rows, groups, columns, K of a product for each kernel
cases = [(5, 4, 64, 256), (500, 4, 512, 256), (8000, 4, 520, 256), (20000, 3, 2050, 400)]
assert [m.grouped_int8_variant(g, r, c, kk) for r, g, c, kk in cases] == [m.GROUPED_ROWS, m.GROUPED_STREAM64, m.GROUPED_STREAM128, m.GROUPED_TILED]
prods = []
for r, g, c, kk in cases:
    sizes = torch.tensor([r // g] * (g - 1) + [r - r // g * (g - 1)])
    prods.append((g, sizes.to(dev), code(r, kk), torch.rand(r).to(dev), code(g, c, kk), torch.rand(g, c).to(dev), r, c, kk))
o = dict(dl=z(f32, T, E), dy=z(b16, n, N), dw=z(f32, T, k), q=z(i8, n, N), s=z(f32, n))
for i, (r, g, c, kk) in enumerate(cases):
    o["p%d" % i], o["g%d" % i] = z(b16, r, c), z(b16, r, c // 2)
def run():
    m.moe_route_backward(m.F32, logits, ids, dw, o["dl"], T, E, k)
    m.moe_combine_backward(dout, y, w, rows, o["dy"], o["dw"], T, k, N, n)
    m.quantize_int8(m.BF16, x, o["q"], o["s"], T, N, row_of=rows, topk=k)
    for i, (g, sizes, a, sa, b, sb, r, c, kk) in enumerate(prods):
        m.grouped_int8_run(g, sizes, a, sa, b, sb, o["p%d" % i], r, c, kk)
        m.grouped_int8_run(g, sizes, a, sa, b, sb, o["g%d" % i], r, c, kk, activation=m.ACT_SWIGLU)
torch.cuda.synchronize()
m.init()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    run()
got = []
for _ in range(3):
    for v in o.values():
        v.fill_(5)
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    got.append({name: v.clone() for name, v in o.items()})
for v in o.values():
    v.fill_(5)
run()
torch.cuda.synchronize()
for r in got:
    for name, v in o.items():
        assert torch.equal(r[name].view(torch.uint8), v.view(torch.uint8)), name
print("same")
"""


def test_first_calls_in_a_graph():
    r = subprocess.run([sys.executable, "-c", FIRST], cwd=ROOT, capture_output=True, text=True, timeout=100)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]

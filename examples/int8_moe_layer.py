"""A mixture-of-experts feed-forward layer in 8-bit integers, forward and the
gradients of its router and combine, on this library's entry points:

    route -> quantize into the experts' rows -> gate and up product with
    SwiGLU -> quantize -> down product -> combine

and, for a few tokens (a decode step), in three launches from the same weights:

    route -> the chosen experts on unquantized activations, with the residual

Everything but the weights' layout runs on the device from buffers that the
layer keeps, without a host read, so a step can be captured into a graph.

    python examples/int8_moe_layer.py [tokens] [experts] [topk] [dim] [hidden]

prints the time of a step, eager and from a graph, and how far the output is
from the same layer in FP32 with the weights as they were before rounding to
8 bits.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from block_scaled_precision_03_amd import mxgemm as mx  # noqa: E402


class Int8MoE:
    """gate, up: [experts, hidden, dim]; down: [experts, dim, hidden]; FP32 or
    BF16 weights, rounded to 8 bits per output channel once.  dim and hidden
    multiples of 16."""

    def __init__(self, gate, up, down, topk, max_tokens):
        E, F, D = gate.shape
        self.E, self.F, self.D, self.k = E, F, D, topk
        dev = gate.device
        # SwiGLU pairs: row 2j the gate's channel j, row 2j + 1 the up's
        self.w1, self.s1 = self._quantize(torch.stack([gate, up], 2).reshape(E, 2 * F, D).contiguous())
        self.w2, self.s2 = self._quantize(down.contiguous())
        T, n = max_tokens, max_tokens * topk
        new = lambda dt, *s: torch.zeros(*s, dtype=dt, device=dev)
        i8, i32, f32, b16 = torch.int8, torch.int32, torch.float32, torch.bfloat16
        self.ids, self.weights, self.row_of, self.slot_of = new(i32, T, topk), new(f32, T, topk), new(i32, T, topk), new(i32, n)
        self.sizes = new(torch.int64, E)
        self.xq, self.xs, self.h, self.hq, self.hs = new(i8, n, D), new(f32, n), new(b16, n, F), new(i8, n, F), new(f32, n)
        self.y, self.out = new(b16, n, D), new(b16, T, D)
        self.dy, self.dweights, self.dlogits = new(b16, n, D), new(f32, T, topk), new(f32, T, E)
        self.workspace = new(torch.uint8, max(1, mx.moe_route_workspace_bytes(T, E)))
        # a decode step's own choice: forward's waits for its backward
        self.max_few = min(T, 64)
        self.few_ids, self.few_weights = new(i32, self.max_few, topk), new(f32, self.max_few, topk)
        self.few_workspace = new(torch.uint8, mx.moe_experts_workspace_bytes(self.max_few, topk, F))
        self.max_tokens = T

    @staticmethod
    def _quantize(w):
        E, N, K = w.shape
        q = torch.empty(E, N, K, dtype=torch.int8, device=w.device)
        s = torch.empty(E, N, dtype=torch.float32, device=w.device)
        mx.quantize_int8(mx.F32 if w.dtype == torch.float32 else mx.BF16, w, q, s, E * N, K)
        return q, s

    def _check(self, x, logits):
        """The library takes addresses and sizes alone: what does not fit the
        layer's buffers is refused here."""
        T = x.shape[0]
        if T > self.max_tokens:
            raise ValueError("%d tokens, the layer has room for %d" % (T, self.max_tokens))
        for t, shape, dtype in ((x, (T, self.D), torch.bfloat16), (logits, (T, self.E), torch.float32)):
            if tuple(t.shape) != shape or t.dtype != dtype or not t.is_contiguous():
                raise ValueError("expected a contiguous %s of %s, got %s of %s" % (dtype, shape, t.dtype, tuple(t.shape)))

    def forward(self, x, logits):
        """x: BF16 [T, dim], logits: FP32 [T, experts], T <= max_tokens;
        returns BF16 [T, dim] (a view of the layer's buffer)."""
        self._check(x, logits)
        T, E, k, D, F = x.shape[0], self.E, self.k, self.D, self.F
        n = T * k
        mx.moe_route(mx.F32, logits, None, self.ids, self.weights, T, E, k, m_sizes=self.sizes, row_of=self.row_of,
                     slot_of=self.slot_of, workspace=self.workspace)
        mx.quantize_int8(mx.BF16, x, self.xq, self.xs, T, D, row_of=self.row_of, topk=k)
        mx.grouped_int8_run(E, self.sizes, self.xq, self.xs, self.w1, self.s1, self.h, n, 2 * F, D,
                            activation=mx.ACT_SWIGLU)
        mx.quantize_int8(mx.BF16, self.h, self.hq, self.hs, n, F)
        mx.grouped_int8_run(E, self.sizes, self.hq, self.hs, self.w2, self.s2, self.y, n, D, F)
        mx.moe_combine(self.y, self.weights, self.row_of, self.out, T, k, D, n)
        return self.out[:T]

    def decode(self, x, logits, residual=None):
        """forward for at most 64 tokens, plus `residual` (BF16, x's shape).
        The activations stay in BF16 and FP32, so its result is closer to the
        FP32 layer's than forward's.  It returns a view of the buffer that
        forward's result is in, and leaves what backward needs as it is."""
        self._check(x, logits)
        T, k = x.shape[0], self.k
        if T > self.max_few:
            raise ValueError("%d tokens, decode takes %d" % (T, self.max_few))
        if residual is not None and (residual.shape != x.shape or residual.dtype != x.dtype or not residual.is_contiguous()):
            raise ValueError("expected a residual like x")
        mx.moe_route(mx.F32, logits, None, self.few_ids, self.few_weights, T, self.E, k)
        mx.moe_experts(mx.INT8, x, self.few_ids, self.few_weights, self.w1, self.s1, self.w2, self.s2, self.out, T, self.E, k,
                       self.D, self.F, residual=residual, workspace=self.few_workspace)
        return self.out[:T]

    def backward(self, dout, logits):
        """Gradients after forward(x, logits): of the experts' outputs (BF16,
        in their rows' order) and of the logits."""
        self._check(dout, logits)
        T, k, n = dout.shape[0], self.k, dout.shape[0] * self.k
        mx.moe_combine_backward(dout, self.y, self.weights, self.row_of, self.dy, self.dweights, T, k, self.D, n)
        mx.moe_route_backward(mx.F32, logits, self.ids, self.dweights, self.dlogits, T, self.E, k)
        return self.dy[:n], self.dlogits[:T]


def plain(x, logits, gate, up, down, topk):
    """The layer in FP32, weights as given."""
    x = x.float()
    top = torch.topk(logits, topk, dim=1)
    w = torch.softmax(top.values, dim=1)
    out = torch.zeros_like(x)
    for e in range(gate.shape[0]):
        t, slot = (top.indices == e).nonzero(as_tuple=True)
        if t.numel():
            g, u = x[t] @ gate[e].float().t(), x[t] @ up[e].float().t()
            out.index_add_(0, t, w[t, slot, None] * ((torch.nn.functional.silu(g) * u) @ down[e].float().t()))
    return out


def main(argv):
    T, E, k, D, F = [int(a) for a in argv] + [2048, 32, 4, 1024, 512][len(argv):]
    mx.init()
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    rand = lambda *s: torch.randn(*s, device="cuda", generator=gen)
    gate, up, down = rand(E, F, D) * D ** -0.5, rand(E, F, D) * D ** -0.5, rand(E, D, F) * F ** -0.5
    x, logits, dout = rand(T, D).bfloat16(), rand(T, E), rand(T, D).bfloat16()
    layer = Int8MoE(gate, up, down, k, T)
    step = lambda: (layer.forward(x, logits), layer.backward(dout, logits))
    out = step()[0].float().clone()
    ref = plain(x, logits, gate, up, down, k)
    error = float((out - ref).norm() / ref.norm())

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()

    def timed(f, n=20):
        f()
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        for _ in range(n):
            f()
        b.record()
        b.synchronize()
        return a.elapsed_time(b) * 1e3 / n

    print("tokens %d, %d experts, topk %d, dim %d, hidden %d: %.1f us a step, %.1f us from a graph; "
          "relative error against FP32 %.4f" % (T, E, k, D, F, timed(step), timed(graph.replay), error))
    return error


if __name__ == "__main__":
    main(sys.argv[1:])

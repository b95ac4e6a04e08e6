"""GPU: the example layer's decode step runs, eager and from a graph, on the
weights of its forward, and refuses what does not fit."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def test_decode():
    from examples import int8_moe_layer as ex
    from block_scaled_precision_03_amd import mxgemm as m
    m.init()
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    rand = lambda *s: torch.randn(*s, device=DEV, generator=g)
    E, F, D, k = 8, 96, 160, 2
    gate, up, down = rand(E, F, D) * D ** -0.5, rand(E, F, D) * D ** -0.5, rand(E, D, F) * F ** -0.5
    layer = ex.Int8MoE(gate, up, down, k, 70)
    x, logits = rand(70, D).bfloat16(), rand(70, E)
    for T in (1, 5, 64):
        ref = ex.plain(x[:T], logits[:T], gate, up, down, k)
        full = layer.forward(x[:T], logits[:T]).float().clone()
        few = layer.decode(x[:T], logits[:T]).float().clone()
        both = layer.decode(x[:T], logits[:T], residual=x[:T]).float().clone()
        # rounding to 8 bits leaves r / (127 sqrt 12) of an operand, r its rows'
        # largest value over their root mean square (about 4): 0.9 % each for gate, up
        # and down, 1.6 % together in squares; twice that.  forward rounds the
        # activations too (tests/test_gpu_int8_example.py)
        error = lambda a: float((a - ref).norm() / ref.norm())
        assert error(few) < 0.033 and error(full) < 0.066
        # each of the two results is rounded once
        assert float((both - few - x[:T].float()).abs().max()) <= 1.01 * 2 ** -8 * float(both.abs().max() + few.abs().max())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            layer.decode(x[:T], logits[:T])
        layer.out.fill_(9)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(layer.out[:T].float(), few) and (layer.out[T:] == 9).all()
    with pytest.raises(ValueError):
        layer.decode(x, logits)
    with pytest.raises(ValueError):
        layer.decode(x[:3], logits[:3], residual=x[:2])


def test_decode_between_forward_and_backward():
    """Gradients of a step with a decode of other tokens inside are the step's own."""
    from examples import int8_moe_layer as ex
    from block_scaled_precision_03_amd import mxgemm as m
    m.init()
    g = torch.Generator(device=DEV)
    g.manual_seed(4)
    rand = lambda *s: torch.randn(*s, device=DEV, generator=g)
    E, F, D, k, T = 8, 96, 160, 2, 40
    layer = ex.Int8MoE(rand(E, F, D) * D ** -0.5, rand(E, F, D) * D ** -0.5, rand(E, D, F) * F ** -0.5, k, T)
    x, logits, dout = rand(T, D).bfloat16(), rand(T, E), rand(T, D).bfloat16()
    layer.forward(x, logits)
    want = [t.clone() for t in layer.backward(dout, logits)]
    layer.forward(x, logits)
    for n in (1, 40):
        layer.decode(rand(n, D).bfloat16(), rand(n, E))
    for t in (layer.dy, layer.dlogits):
        t.fill_(5)
    assert all(torch.equal(a, b) for a, b in zip(layer.backward(dout, logits), want))

"""GPU: the example layer against the same layer in FP32.  Rounding to 8 bits
with a scale from the row's largest value leaves each operand a relative error
of r / (127 sqrt 12), r the row's largest value over its root mean square: 0.9 %
for the activations and 0.8 % for the weights (r about 4), 2 % for the products
after SwiGLU (r about 9).  The gate's and the up's errors (1.2 % each) and
those of the down product add up in squares to about 3.3 %; twice that is the
bound."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("size", [(), (1, 8, 2, 256, 128), (130, 16, 3, 528, 272), (700, 40, 8, 256, 384)])
def test_example_layer(size):
    from examples import int8_moe_layer
    assert int8_moe_layer.main([str(s) for s in size]) < 0.066

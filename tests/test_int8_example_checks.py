"""CPU: the example layer refuses what does not fit its buffers before any
library call."""
import pytest
import torch

E, D, MAX = 8, 32, 16


@pytest.fixture
def layer(monkeypatch):
    from examples import int8_moe_layer as ex

    def called(*args, **kw):
        raise AssertionError("a library call was made")
    for name in ("moe_route", "quantize_int8", "grouped_int8_run", "moe_combine", "moe_combine_backward", "moe_route_backward"):
        monkeypatch.setattr(ex.mx, name, called)
    z = lambda dt, *s: torch.zeros(*s, dtype=dt)
    monkeypatch.setattr(ex.Int8MoE, "_quantize", staticmethod(lambda w: (z(torch.int8, *w.shape), z(torch.float32, *w.shape[:2]))))
    w = torch.zeros(E, 48, D)
    return ex.Int8MoE(w, w, torch.zeros(E, D, 48), 2, MAX)


x, l = torch.zeros(4, D, dtype=torch.bfloat16), torch.zeros(4, E)
BAD = [
    (torch.zeros(MAX + 1, D, dtype=torch.bfloat16), torch.zeros(MAX + 1, E)),     # more tokens than the buffers hold
    (torch.zeros(4, D + 16, dtype=torch.bfloat16), l), (x.float(), l), (torch.zeros(D, 4, dtype=torch.bfloat16).t(), l),
    (x, torch.zeros(3, E)), (x, torch.zeros(4, E - 1)), (x, l.bfloat16()), (x, torch.zeros(E, 4).t()),
]


@pytest.mark.parametrize("which", range(len(BAD)))
def test_refused(layer, which):
    a, b = BAD[which]
    with pytest.raises(ValueError):
        layer.forward(a, b)
    with pytest.raises(ValueError):
        layer.backward(a, b)


def test_what_fits_reaches_the_library(layer):
    for T in (0, 4, MAX):
        with pytest.raises(AssertionError, match="library call"):
            layer.forward(torch.zeros(T, D, dtype=torch.bfloat16), torch.zeros(T, E))

"""GPU: groups chosen by the sum of their two best values where the balance
biases are large: two values of opposite sign cancel, so that the sum says
nothing of how far rounding has moved it, and sums pass the 32-bit range.  The
choice is that of 64-bit values."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _choose(x, bias, topk, score, n_group, topk_group, top2=True):
    from block_scaled_precision_03_amd import mxgemm as m
    m.init()
    T, E = x.shape
    ids = torch.full((T, topk), 7, dtype=torch.int32, device=DEV)
    w = torch.empty(T, topk, device=DEV)
    m.moe_route(m.BF16 if x.dtype == torch.bfloat16 else m.F32, x, bias, ids, w, T, E, topk, score=score,
                n_group=n_group, topk_group=topk_group, group_score=m.MOE_GROUP_TOP2 if top2 else m.MOE_GROUP_MAX)
    return ids.long().cpu()


def _definition(x, bias, topk, score, n_group, topk_group, top2=True):
    """In 64 bits on the host; every expert is available."""
    return _decided(x, bias, topk, score, n_group, topk_group, top2)[0]


def _decided(x, bias, topk, score, n_group, topk_group, top2=True):
    """The choice, and how far it is from another one: the least gap between
    neighbours of the order, of groups at the border and of chosen experts."""
    l = x.double().cpu()
    s = torch.softmax(l, dim=1) if score == 0 else torch.special.expit(l)
    v = s + bias.double().cpu()
    T, E = v.shape
    best = torch.sort(v.view(T, n_group, E // n_group), dim=2, descending=True).values[:, :, :2 if top2 else 1].sum(2)
    order = torch.sort(best, dim=1, descending=True, stable=True)
    keep, gap = order.indices[:, :topk_group], order.values[:, topk_group - 1] - order.values[:, topk_group]
    on = torch.zeros(T, n_group, dtype=torch.bool).scatter_(1, keep, True).repeat_interleave(E // n_group, dim=1)
    top = torch.sort(torch.where(on, v, -float("inf")), dim=1, descending=True, stable=True)
    near = (top.values[:, :topk] - top.values[:, 1:topk + 1]).amin(1)
    return top.indices[:, :topk], torch.minimum(gap, near)


@pytest.mark.parametrize("T", [1, 17, 300])
def test_sums_that_cancel(T):
    """Group 0's exact sum is 1.3819155, group 1's 1.3819124; with s + bias
    rounded to 32 bits they come out as 1.3818970 and 1.3819580."""
    x = torch.tensor([[1.9814709, 0.0123108, 0.1749193, 1.6455866]], device=DEV).repeat(T, 1)
    bias = torch.tensor([1000.0, -1000.0, 1000.0, -1000.0], device=DEV)
    ref = _definition(x, bias, 2, 1, 2, 1)
    assert ref.tolist() == [[0, 1]] * T
    assert torch.equal(_choose(x, bias, 2, 1, 2, 1), ref)


@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("size", [64.0, 1024.0, 4096.0, 1e5])
@pytest.mark.parametrize("E,n_group", [(16, 8), (256, 8), (40, 20), (1020, 60)])
def test_large_biases_of_either_sign(score, size, E, n_group):
    T, n = (4000 if E > 64 else 40000), E // n_group
    g = torch.Generator(device=DEV)
    g.manual_seed(E + int(size))
    x = torch.randn(T, E, device=DEV, generator=g)
    # one expert of each group far up, the others far down: the two best cancel
    bias = torch.full((n_group, n), -size, device=DEV)
    bias[:, 0] = size
    bias = bias.reshape(-1)
    for l in (x, x.bfloat16()):
        ref, gap = _decided(l, bias, 6, score, n_group, 4)
        # a 64-bit score is off by a few units of its last place and its sum
        # with the bias by half a unit of the bias's: what is closer than that
        # (BF16 logits repeat) may come out either way
        sure = gap > 8 * 2.0 ** -52 * size
        assert float(sure.double().mean()) > 0.5
        assert torch.equal(_choose(l, bias, 6, score, n_group, 4)[sure], ref[sure])


@pytest.mark.parametrize("top2", [False, True])
@pytest.mark.parametrize("T", [9, 200])
def test_sums_past_the_32_bit_range(top2, T):
    g = torch.Generator(device=DEV)
    g.manual_seed(T)
    x = torch.randn(T, 32, device=DEV, generator=g)
    big = torch.tensor([3.0e38, 3.2e38, -3.0e38, -3.2e38, 3.4e38, -3.4e38, 0.0, 1.0], device=DEV)
    for _ in range(8):
        bias = big[torch.randint(0, 8, (32,), device=DEV, generator=g)]
        for n_group, kept in ((4, 2), (16, 5)):
            args = (x, bias, 5, 1, n_group, kept, top2)
            assert torch.equal(_choose(*args), _definition(*args))
    # every group's sum past the range, upwards or downwards: the larger one wins
    for lo, hi in ((3.0e38, 3.2e38), (-3.2e38, -3.0e38)):
        bias = torch.tensor([lo] * 16 + [hi] * 16, device=DEV)
        assert torch.equal(_choose(x, bias, 5, 1, 2, 1, top2), _definition(x, bias, 5, 1, 2, 1, top2))

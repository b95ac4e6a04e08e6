"""GPU: the experts of a mixture-of-experts layer for a few tokens against
their 64-bit form: every weight format, odd sizes, tokens without an expert,
experts named twice, buffers that are shared, graphs, streams, large offsets."""
import numpy as np
import pytest
import torch

from tests import experts_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
b16 = torch.bfloat16


def _mx():
    from block_scaled_precision_03_amd import mxgemm
    return mxgemm


def dev(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


class Case:
    """Inputs on the host and the device; `guard` rows and bytes around what
    the call may write."""

    def __init__(self, fmt, T, E, k, D, F, a=R.ACT_SWIGLU, residual=True, seed=0, ids=None):
        rng = np.random.default_rng(seed)
        self.fmt, self.T, self.E, self.k, self.D, self.F, self.a = fmt, T, E, k, D, F, a
        N1 = 2 * F if a == R.ACT_SWIGLU else F
        self.x = R.bf16(rng.standard_normal((T, D)))
        if ids is None:
            ids = np.argsort(rng.random((T, max(E, k))), axis=1)[:, :k]
            ids = np.where(ids < E, ids, -1)
        self.ids = np.asarray(ids, np.int32).reshape(T, k)
        self.w = (rng.random((T, k)) + 0.1).astype(np.float32)
        self.c1, self.s1, self.v1 = R.encode(rng, fmt, E, N1, D, D ** -0.5)
        self.c2, self.s2, self.v2 = R.encode(rng, fmt, E, D, F, F ** -0.5)
        self.r = R.bf16(rng.standard_normal((T, D))) if residual else None
        m = _mx()
        self.d = dict(x=dev(self.x).to(b16), ids=dev(self.ids), w=dev(self.w), s1=dev(self.s1), s2=dev(self.s2),
                      r=None if self.r is None else dev(self.r).to(b16))
        for n, c in (("w1", self.c1), ("w2", self.c2)):
            self.d[n] = dev(c.view(np.int16)) if fmt == R.BF16 else dev(c)
        self.nbytes = m.moe_experts_workspace_bytes(T, k, F)
        self.ws = torch.full((self.nbytes + 64,), 0xA5, dtype=torch.uint8, device=DEV)
        self.out = torch.full((T + 2, D), 7.0, dtype=b16, device=DEV)

    def run(self, out=None, ws=None, **kw):
        d, m = self.d, _mx()
        out = self.out[1:self.T + 1] if out is None else out
        m.moe_experts(self.fmt, d["x"], d["ids"], d["w"], d["w1"], d["s1"], d["w2"], d["s2"], out, self.T, self.E, self.k,
                      self.D, self.F, activation=self.a, residual=kw.get("residual", d["r"]),
                      workspace=self.ws[:self.nbytes] if ws is None else ws, stream=kw.get("stream"))
        return out

    def check(self):
        got = self.run().float().cpu().numpy().astype(np.float64)
        ref, tol = R.experts(self.x, self.ids, self.w, self.v1, self.v2, self.a, self.r)
        bad = np.abs(got - ref) > tol
        assert not bad.any(), "%d of %d off, worst %.3g of the tolerance" % (bad.sum(), bad.size, (np.abs(got - ref) / tol).max())
        assert (self.out[0] == 7).all() and (self.out[-1] == 7).all()
        assert (self.ws[self.nbytes:] == 0xA5).all()


SIZES = {"int8": (80, 48), "bf16": (88, 24), "e4m3": (96, 160), "e5m2": (32, 96), "e2m1": (288, 96), "block": (128, 384)}


@pytest.mark.parametrize("name", sorted(R.FORMATS))
@pytest.mark.parametrize("T,E,k", [(1, 5, 2), (3, 1, 1), (16, 7, 3), (17, 4, 2), (33, 3, 2), (64, 2, 1), (64, 33, 5)])
def test_formats_and_tokens(name, T, E, k):
    D, F = SIZES[name]
    Case(R.FORMATS[name], T, E, k, D, F, residual=T % 2 == 1, seed=T).check()


@pytest.mark.parametrize("name", sorted(R.FORMATS))
@pytest.mark.parametrize("a", [R.ACT_NONE, R.ACT_RELU, R.ACT_GELU, R.ACT_SILU])
def test_activations(name, a):
    D, F = SIZES[name]
    Case(R.FORMATS[name], 5, 6, 2, D, F, a=a, seed=a).check()


@pytest.mark.parametrize("name", sorted(R.FORMATS))
def test_several_units_of_k(name):
    u = R.UNIT[R.FORMATS[name]]
    Case(R.FORMATS[name], 2, 3, 2, u * (1100 // u), u * (1300 // u), seed=3).check()


@pytest.mark.parametrize("name", sorted(R.FORMATS))
def test_smallest(name):
    u = R.UNIT[R.FORMATS[name]]
    Case(R.FORMATS[name], 1, 1, 1, u, u, seed=4).check()


def test_tokens_without_an_expert():
    ids = np.array([[0, 2], [-1, -1], [1, -1], [5, 4], [-7, 3], [2, 1 << 30]], np.int32)
    c = Case(R.INT8, 6, 4, 2, 64, 32, ids=ids)
    c.check()
    assert torch.equal(c.out[2], c.d["r"][1]) and torch.equal(c.out[4], c.d["r"][3])
    c = Case(R.INT8, 3, 4, 2, 64, 32, ids=-np.ones((3, 2)), residual=False)
    c.check()
    assert (c.out[1:4] == 0).all()


def test_an_expert_named_twice_counts_with_both_weights():
    Case(R.E4M3, 4, 3, 4, 64, 64, ids=[[1, 1, 1, 1], [0, 2, 0, 2], [2, -1, 2, 1], [0, 1, 2, 0]]).check()
    Case(R.INT8, 40, 2, 32, 64, 64, ids=np.random.default_rng(1).integers(-1, 3, (40, 32))).check()


@pytest.mark.parametrize("T", [1, 2])
def test_most_slots_of_one_and_two_tokens(T):
    """The choice of one or two tokens is read in registers: up to 64 slots,
    named in any order, twice, by both tokens, or not at all."""
    rng = np.random.default_rng(T)
    for ids in (rng.integers(-1, 4, (T, 32)), rng.permutation(200)[:32 * T].reshape(T, 32), np.full((T, 32), -1),
                np.concatenate([np.full((T, 31), 1 << 20), np.full((T, 1), 3)], 1), np.full((T, 32), 199)):
        Case(R.INT8, T, 200, 32, 48, 32, ids=ids, seed=T).check()
    if T == 2:
        # the second token alone, and the first alone, name an expert
        Case(R.E4M3, 2, 5, 2, 64, 64, ids=[[3, -1], [4, 3]]).check()
        Case(R.E4M3, 2, 5, 2, 64, 64, ids=[[-1, -1], [4, 0]]).check()


@pytest.mark.parametrize("T", [1, 5])
@pytest.mark.parametrize("D,F", [(131072, 16), (16, 131072)])
def test_longest_rows(T, D, F):
    c = Case(R.INT8, T, 2, 1, D, F, ids=np.arange(T)[:, None] % 2, a=R.ACT_NONE)
    c.check()


@pytest.mark.parametrize("name", sorted(R.FORMATS))
@pytest.mark.parametrize("T", [1, 2])
def test_many_rows_of_the_first_weight(name, T):
    """One or two tokens, enough short rows for 64 of them per workgroup (the
    last of them not full), and so many that K is long as well."""
    u = R.UNIT[R.FORMATS[name]]
    F = u * (3300 // u) + (u if u < 64 else 0)
    Case(R.FORMATS[name], T, 4, 4, u * (280 // u), F, seed=T).check()
    Case(R.FORMATS[name], T, 4, 1, u * (6200 // u), u * max(300 // u, 1), a=R.ACT_NONE, seed=T).check()


def test_most_experts():
    Case(R.INT8, 64, 1024, 32, 16, 16, seed=2).check()
    Case(R.INT8, 1, 1024, 32, 16, 16, seed=3).check()


def test_every_token_to_one_expert():
    for n in (15, 16, 31, 32, 48, 49, 64):
        Case(R.E2M1, n, 3, 1, 64, 96, ids=np.full((n, 1), 2)).check()


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_not_finite_stays_where_it_is(value):
    c = Case(R.E4M3, 20, 4, 2, 64, 64, ids=np.array([[t % 3, (t + 1) % 3] for t in range(20)]))
    clean = c.run().clone()
    c.d["x"][7, 5] = value
    c.d["s1"][3].fill_(255)                    # an expert that no token chose
    c.d["w2"][3].fill_(127)
    got = c.run()
    keep = torch.arange(20, device=DEV) != 7
    assert torch.equal(got[keep], clean[keep]) and not torch.isfinite(got[7].float()).any()


def test_infinite_activation():
    """A sum past FP32's range makes h infinite, and the result infinite or NaN."""
    c = Case(R.BF16, 2, 1, 1, 16, 8, a=R.ACT_RELU, residual=False)
    c.d["x"][0].fill_(3e38)
    c.d["w1"].copy_(torch.full((1, 8, 16), 2.0, dtype=b16, device=DEV).view(torch.int16))
    c.d["w2"].copy_(torch.full((1, 16, 8), 1.0, dtype=b16, device=DEV).view(torch.int16))
    got = c.run().float()
    assert torch.isinf(got[0]).all() and torch.isfinite(got[1]).all()


@pytest.mark.parametrize("code", [0, 1, 100, 254])
def test_extreme_scales(code):
    """E8M0 codes over the whole range: 2^(code - 127), exactly."""
    c = Case(R.E4M3, 1, 1, 1, 32, 32, a=R.ACT_NONE, residual=False)
    c.d["w1"].fill_(0x38)                      # 1.0
    c.d["w2"].fill_(0x38)
    c.d["s1"].fill_(code)
    c.d["s2"].fill_(254 - code)
    c.d["x"].fill_(0)
    c.d["x"][0, 3] = 1.0
    c.d["w"].fill_(0.5)
    # h = 2^(code - 127), y = 32 h 2^(127 - code)
    assert (c.run() == 16.0).all()


def test_nan_scale():
    c = Case(R.E2M1, 1, 1, 1, 32, 64, residual=False)
    c.d["s2"][0, 5, 1] = 255
    got = c.run()[0].float()
    assert torch.isnan(got[5]) and torch.isfinite(torch.cat([got[:5], got[6:]])).all()


def test_shared_buffers():
    c = Case(R.INT8, 9, 5, 2, 160, 64)
    want = c.run().clone()
    r = c.d["r"].clone()
    assert torch.equal(c.run(out=r, residual=r), want)
    c.d["x"] = c.d["x"].clone()
    assert torch.equal(c.run(out=c.d["x"]), want)


def test_same_bits_every_time():
    c = Case(R.E4M3, 64, 9, 4, 256, 512)
    want = c.run().clone()
    for _ in range(10):
        c.ws.fill_(0xFF)
        assert torch.equal(c.run(), want)


@pytest.mark.parametrize("name", sorted(R.FORMATS))
@pytest.mark.parametrize("T", [1, 2, 5, 40])
def test_few_columns_many_units(name, T):
    """Lists split over workgroups, whose sums meet."""
    u = R.UNIT[R.FORMATS[name]]
    c = Case(R.FORMATS[name], T, 6, 4, max(u, 128), u * (2600 // u), seed=T)
    c.check()
    want = c.out.clone()
    for _ in range(5):
        c.ws.fill_(0xEE)
        c.run()
        assert torch.equal(c.out, want)


def test_empty_sizes():
    c = Case(R.INT8, 3, 2, 1, 32, 16)
    m, d = _mx(), c.d
    m.moe_experts(R.INT8, None, None, None, None, None, None, None, None, 0, 2, 1, 32, 16, workspace=c.ws)
    m.moe_experts(R.INT8, None, d["ids"], d["w"], None, None, None, None, c.out[1:4], 3, 2, 1, 32, 0, residual=d["r"], workspace=c.ws)
    assert torch.equal(c.out[1:4], d["r"])


def test_graph_stream_and_two_workspaces():
    a, b = Case(R.E2M1, 5, 6, 3, 96, 160, seed=1), Case(R.INT8, 31, 6, 3, 96, 160, seed=2)
    want = [c.run().clone() for c in (a, b)]
    torch.cuda.synchronize()
    graphs = []
    for c in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.run()
        graphs.append(g)
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    for rep in range(4):
        for c in (a, b):
            c.out.fill_(3)
            c.ws.fill_(rep)
        torch.cuda.synchronize()
        for g, st in zip(graphs, s):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for c, w in zip((a, b), want):
            assert torch.equal(c.out[1:c.T + 1], w)
    # new choices in the captured buffers
    a.d["ids"].copy_(torch.flip(a.d["ids"], [0]))
    graphs[0].replay()
    torch.cuda.synchronize()
    got = a.out[1:6].clone()
    assert torch.equal(a.run(), got)
    torch.cuda.synchronize()
    with torch.cuda.stream(s[0]):
        a.run()
    torch.cuda.synchronize()
    assert torch.equal(a.out[1:6], got)
    a.run(stream=s[1])
    torch.cuda.synchronize()
    assert torch.equal(a.out[1:6], got)


def test_choice_from_the_router():
    m = _mx()
    c = Case(R.INT8, 12, 16, 4, 64, 96)
    logits = torch.randn(12, 16, device=DEV)
    logits[3] = float("-inf")
    m.moe_route(m.F32, logits, None, c.d["ids"], c.d["w"], 12, 16, 4)
    c.ids, c.w = c.d["ids"].cpu().numpy(), c.d["w"].cpu().numpy()
    assert (c.ids[3] == -1).all()
    c.check()


@pytest.mark.parametrize("fmt", [R.INT8, R.E2M1])
def test_weights_past_4_gib(fmt):
    """The last of the experts whose weights lie past 2^32 bytes."""
    m = _mx()
    D, F, T, k = 16384, 4096, 2, 1
    E = 40 if fmt == R.INT8 else 80            # w1 5.4 GB in either format
    g = torch.Generator(device=DEV)
    g.manual_seed(5)
    one = Case(fmt, T, 1, k, D, F, ids=np.zeros((T, k)))
    kb = {R.INT8: 1, R.E2M1: 2}[fmt]
    w1 = torch.zeros(E, 2 * F, D // kb, dtype=one.d["w1"].dtype, device=DEV)
    w2 = torch.zeros(E, D, F // kb, dtype=one.d["w2"].dtype, device=DEV)
    s1 = torch.zeros(E, *one.d["s1"].shape[1:], dtype=one.d["s1"].dtype, device=DEV)
    s2 = torch.zeros(E, *one.d["s2"].shape[1:], dtype=one.d["s2"].dtype, device=DEV)
    assert w1.numel() > 1 << 32
    for big, small in ((w1, "w1"), (w2, "w2"), (s1, "s1"), (s2, "s2")):
        big[-1] = one.d[small][0]
    want = one.run().clone()
    one.d.update(w1=w1, w2=w2, s1=s1, s2=s2, ids=torch.full((T, k), E - 1, dtype=torch.int32, device=DEV))
    one.E = E
    assert torch.equal(one.run(), want)


INFINITE = {"bf16": (0x7F80, 0xFF80), "e5m2": (0x7C, 0xFC)}        # codes of plus and minus infinity


@pytest.mark.parametrize("name", sorted(INFINITE))
@pytest.mark.parametrize("T,E,k,F", [(1, 5, 2, 96), (2, 4, 3, 2592), (6, 3, 2, 96), (40, 6, 4, 2592)])
@pytest.mark.parametrize("a", [R.ACT_NONE, R.ACT_RELU, R.ACT_SWIGLU])
def test_infinite_weights_of_the_second_product(name, T, E, k, F, a):
    """Columns with one infinity, with two (of both signs or not), and without:
    infinite with the argument's sign, NaN where infinities of both signs meet or one
    meets a zero, and the others as they were."""
    fmt = R.FORMATS[name]
    c = Case(fmt, T, E, k, 96, F, a=a, seed=T)
    plus, minus = (dev(np.array([v]).astype(c.c2.dtype)).view(c.d["w2"].dtype) for v in INFINITE[name])
    v2 = c.v2.copy()
    for d, marks in ((3, ((5, 1),)), (17, ((F - 1, -1),)), (40, ((7, 1), (60, 1))), (41, ((0, 1), (33, -1))), (95, ((64, -1), (65, -1)))):
        for f, sign in marks:
            c.d["w2"][:, d, f] = plus if sign > 0 else minus
            v2[:, d, f] = sign * np.inf
    got = c.run().float().cpu().numpy().astype(np.float64)
    with np.errstate(invalid="ignore"):
        want, _ = R.experts(c.x, c.ids, c.w, c.v1, v2, a, c.r)
        clean, tol = R.experts(c.x, c.ids, c.w, c.v1, c.v2, a, c.r)
    hot = ~np.isfinite(want)
    assert hot.any() and np.array_equal(got[hot], want[hot], equal_nan=True)
    assert (np.abs(got - clean) <= tol)[~hot].all()


@pytest.mark.parametrize("name", sorted(INFINITE))
@pytest.mark.parametrize("T", [1, 5])
def test_infinite_weights_and_arguments_without_a_low_part(name, T):
    """Arguments that one BF16 holds exactly."""
    fmt = R.FORMATS[name]
    c = Case(fmt, T, 1, 1, 96, 96, ids=np.zeros((T, 1)), a=R.ACT_NONE, residual=False)
    one = 0x3F80 if fmt == R.BF16 else 0x3C
    minus = INFINITE[name][1] - (1 << 16 if fmt == R.BF16 else 0)
    for n in ("w1", "w2"):
        c.d[n].zero_()
    if fmt != R.BF16:
        c.d["s1"].fill_(127)
        c.d["s2"].fill_(127)
    c.d["x"].zero_()
    c.d["w"].fill_(1.0)
    i = torch.arange(96, device=DEV)
    c.d["w1"][0, i, i] = one                   # h = x
    for d, f, code in ((10, 0, INFINITE[name][0]), (11, 1, minus), (12, 2, minus), (13, 3, one)):
        c.d["w2"][0, d, f] = code
    c.d["x"][0, 0], c.d["x"][0, 1], c.d["x"][0, 2], c.d["x"][0, 3] = 1.0, -2.0, 3e38, -2.0
    got = c.run().float()
    inf = float("inf")
    assert got[0, 10] == inf and got[0, 11] == inf and got[0, 12] == -inf and got[0, 13] == -2.0
    # zeros beside infinite weights are NaN, whoever's token they are
    assert torch.isnan(got[1:, 10:13]).all() and (got[:, :10] == 0).all() and (got[:, 14:] == 0).all()


@pytest.mark.parametrize("T,D,F", [(1, 160, 64), (9, 160, 64), (40, 128, 2592)])
def test_stream_updated_in_place(T, D, F):
    """x, the residual and out one buffer: a residual stream in place."""
    c = Case(R.INT8, T, 5, 2, D, F, a=R.ACT_SILU)
    c.d["r"] = c.d["x"].clone()
    want = c.run().clone()
    x = c.d["x"]
    assert torch.equal(c.run(out=x, residual=x), want)

"""The operators of a mixture-of-experts layer in 8-bit integers, as measured
cases: routing and its gradient, per-token quantization, the integer matrix
product (dense and grouped by expert), and the weighted combine of the
experts' rows with its gradient.

`own` chooses what `run` computes with: elementary torch operations (False)
or this library's entry points (True).  `exact` is the definition in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
FLT_MAX = torch.finfo(torch.float32).max


# ---- cases ------------------------------------------------------------------

def listed():
    return [
        # one token of a chat reply: latency alone
        dict(name="route_token", op="route", dtype="bf16", T=1, E=64, topk=6, score="softmax", bias=False,
             n_group=1, topk_group=1, group_score="max", renorm=True, scale=1.0, masked=0.0),
        # a prompt batch: sigmoid scores, balance bias, group-limited choice, some padding tokens
        dict(name="route_prompt", op="route", dtype="f32", T=16384, E=256, topk=8, score="sigmoid", bias=True,
             n_group=8, topk_group=4, group_score="top2", renorm=True, scale=2.5, masked=0.03),
        # a training step's router gradient
        dict(name="route_grad", op="route_grad", dtype="f32", T=16384, E=128, topk=8, score="softmax",
             renorm=False, scale=1.0),
        # the activations of a dense layer before an integer product
        dict(name="quant_rows", op="quant", dtype="bf16", T=4096, K=14336, topk=0, experts=0),
        # the tokens of a prompt batch, each to its experts' rows
        dict(name="quant_permute", op="quant", dtype="bf16", T=2049, K=7168, topk=8, experts=64),
        # one token through a dense layer: weight streaming
        dict(name="int8_token", op="int8", M=1, N=14336, K=4096, bias=False, act="none"),
        # a short prompt with ragged sizes, fused bias and activation
        dict(name="int8_ragged", op="int8", M=777, N=5002, K=4112, bias=True, act="gelu"),
        # a long prompt through a dense layer: matrix-core bound
        dict(name="int8_large", op="int8", M=16384, N=14336, K=4096, bias=False, act="none"),
        # a few tokens per expert, gate and up projection with SwiGLU
        dict(name="grouped_decode", op="grouped", G=8, totM=128, N=4608, K=7168, act="swiglu"),
        # a prompt batch's gate and up projection, uneven groups
        dict(name="grouped_prompt", op="grouped", G=8, totM=16384, N=4608, K=7168, act="swiglu"),
        # the experts' rows back to their tokens
        dict(name="combine", op="combine", T=4096, topk=8, N=7168),
        # the same in a training step, backwards
        dict(name="combine_grad", op="combine_grad", T=2049, topk=8, N=4096),
    ]


def _log(rng, lo, hi):
    return math.exp(rng.uniform(math.log(lo), math.log(hi)))


def _odd(rng, lo, hi):
    """An odd number spread over [lo, hi] on a logarithmic scale."""
    return max(1, int(_log(rng, lo, hi))) | 1


def draw(rng):
    op = rng.choice(["route", "route", "route_grad", "quant", "quant", "int8", "int8", "grouped", "grouped",
                     "combine", "combine_grad"])
    if op == "route":
        n_group = rng.choice([1, 1, 4, 5, 8])
        E = n_group * rng.randint(8, 250 // n_group)
        topk_group = max(1, n_group // 2)
        topk = rng.randint(1, min(12, topk_group * (E // n_group)))
        bias = rng.random() < 0.5
        return dict(op=op, dtype=rng.choice(["bf16", "f32"]), T=_odd(rng, 1, 20000), E=E, topk=topk,
                    score=rng.choice(["softmax", "sigmoid"]), bias=bias, n_group=n_group, topk_group=topk_group,
                    group_score="top2" if bias else "max", renorm=rng.random() < 0.7,
                    scale=rng.choice([1.0, 2.5]), masked=rng.choice([0.0, 0.05]))
    if op == "route_grad":
        E = rng.randint(8, 250)
        return dict(op=op, dtype=rng.choice(["bf16", "f32"]), T=_odd(rng, 16, 20000), E=E,
                    topk=rng.randint(1, min(12, E)), score=rng.choice(["softmax", "sigmoid"]),
                    renorm=rng.random() < 0.5, scale=rng.choice([1.0, 2.5]))
    if op == "quant":
        permute = rng.random() < 0.5
        return dict(op=op, dtype=rng.choice(["bf16", "f32"]), T=_odd(rng, 1, 4000), K=16 * _odd(rng, 16, 800),
                    topk=rng.randint(1, 8) if permute else 0, experts=rng.randint(8, 96) if permute else 0)
    if op == "int8":
        act = rng.choice(["none", "none", "gelu", "silu", "relu", "swiglu"])
        bias = rng.random() < 0.4
        N = _odd(rng, 128, 12000)
        if bias or act == "swiglu":
            N = 2 * (N // 2 | 1)
        return dict(op=op, M=_odd(rng, 1, 8000), N=N, K=16 * _odd(rng, 8, 600), bias=bias, act=act)
    if op == "grouped":
        G = rng.randint(2, 33)
        return dict(op=op, G=G, totM=_odd(rng, 8, 8000), N=64 * _odd(rng, 4, 64), K=16 * _odd(rng, 16, 400),
                    act=rng.choice(["none", "swiglu"]))
    if op == "combine":
        return dict(op=op, T=_odd(rng, 1, 4000), topk=rng.randint(1, 8), N=8 * _odd(rng, 32, 800))
    return dict(op=op, T=_odd(rng, 1, 2000), topk=rng.randint(1, 8), N=8 * _odd(rng, 32, 800))


def _out_cols(c):
    return c["N"] // 2 if c["act"] == "swiglu" else c["N"]


def work(c):
    op = c["op"]
    if op in ("route", "route_grad"):
        T, E, k, b = c["T"], c["E"], c["topk"], (2 if c["dtype"] == "bf16" else 4)
        if op == "route":
            # logits in; ids, weights, the two row maps and the counts out; a score per expert
            return {"bytes": T * E * b + 16 * T * k + 8 * E + (4 * E if c["bias"] else 0), "flops": 10 * T * E}
        return {"bytes": 2 * T * E * b + 8 * T * k, "flops": 10 * T * E}
    if op == "quant":
        T, K, b = c["T"], c["K"], (2 if c["dtype"] == "bf16" else 4)
        rows = T * max(1, c["topk"])
        return {"bytes": T * K * b + rows * (K + 4) + (4 * rows if c["topk"] else 0), "flops": 3 * T * K}
    if op == "int8":
        M, N, K = c["M"], c["N"], c["K"]
        return {"bytes": M * K + N * K + 4 * (M + N) + 2 * M * _out_cols(c) + (2 * N if c["bias"] else 0),
                "flops": 2 * M * N * K}
    if op == "grouped":
        M, N, K, G = c["totM"], c["N"], c["K"], c["G"]
        live = min(G, M)
        return {"bytes": M * K + live * N * K + 4 * (M + live * N) + 2 * M * _out_cols(c) + 8 * G,
                "flops": 2 * M * N * K}
    T, k, N = c["T"], c["topk"], c["N"]
    if op == "combine":
        return {"bytes": 2 * T * k * N + 2 * T * N + 8 * T * k, "flops": 2 * T * k * N}
    return {"bytes": 4 * T * k * N + 2 * T * N + 12 * T * k, "flops": 3 * T * k * N}


# ---- inputs -----------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _dtype(c):
    return torch.bfloat16 if c["dtype"] == "bf16" else torch.float32


def _codes(g, *shape):
    """int8 codes as per-row quantization of roughly normal data leaves them."""
    return (torch.randn(*shape, device=DEV, generator=g) * 34.0).round_().clamp_(-127, 127).to(torch.int8)


def _routes(g, T, topk, experts):
    """topk different experts for every token, and the rows of each slot in
    expert order (by token within an expert)."""
    ids = torch.rand(T, experts, device=DEV, generator=g).argsort(dim=1)[:, :topk].reshape(-1)
    order = torch.sort(ids, stable=True).indices
    row_of = torch.empty(T * topk, dtype=torch.int32, device=DEV)
    row_of[order] = torch.arange(T * topk, dtype=torch.int32, device=DEV)
    return row_of.view(T, topk)


def _inputs(c, seed):
    g = _gen(seed)
    op = c["op"]
    st = {"case": c}
    if op in ("route", "route_grad"):
        T, E, k = c["T"], c["E"], c["topk"]
        st["logits"] = (torch.randn(T, E, device=DEV, generator=g) * 1.5).to(_dtype(c))
        if op == "route":
            if c["masked"] > 0:
                # padding tokens: no expert is available to them
                st["logits"][torch.rand(T, device=DEV, generator=g) < c["masked"]] = -math.inf
            st["bias"] = torch.randn(E, device=DEV, generator=g) * 0.05 if c["bias"] else None
        else:
            st["ids"] = torch.topk(st["logits"].float(), k, dim=1).indices.to(torch.int32)
            st["grad"] = torch.randn(T, k, device=DEV, generator=g)
    elif op == "quant":
        st["x"] = torch.randn(c["T"], c["K"], device=DEV, generator=g).to(_dtype(c))
        st["row_of"] = _routes(g, c["T"], c["topk"], c["experts"]) if c["topk"] else None
    elif op == "int8":
        M, N, K = c["M"], c["N"], c["K"]
        st["a"], st["b"] = _codes(g, M, K), _codes(g, N, K)
        st["sa"] = torch.rand(M, device=DEV, generator=g) * 0.02 + 0.02
        st["sb"] = (torch.rand(N, device=DEV, generator=g) + 0.5) * (0.5 / (34.0 * math.sqrt(K)))
        st["bias"] = torch.randn(N, device=DEV, generator=g).to(torch.bfloat16) if c["bias"] else None
    elif op == "grouped":
        G, M, N, K = c["G"], c["totM"], c["N"], c["K"]
        st["a"], st["w"] = _codes(g, M, K), _codes(g, G, N, K)
        st["sa"] = torch.rand(M, device=DEV, generator=g) * 0.02 + 0.02
        st["sw"] = (torch.rand(G, N, device=DEV, generator=g) + 0.5) * (0.5 / (34.0 * math.sqrt(K)))
        # uneven popularity of the experts, the last of them often without a row
        share = torch.rand(G, device=DEV, generator=g) + 0.1
        share[-1] = 0.0
        cuts = (torch.cumsum(share, 0) / share.sum() * M).round().long()
        sizes = torch.diff(cuts, prepend=cuts.new_zeros(1))
        st["m_sizes"] = sizes
        st["m_host"] = sizes.tolist()
    else:
        T, k, N = c["T"], c["topk"], c["N"]
        st["row_of"] = _routes(g, T, k, max(k, 16))
        st["y"] = torch.randn(T * k, N, device=DEV, generator=g).to(torch.bfloat16)
        w = torch.rand(T, k, device=DEV, generator=g) + 0.05
        st["w"] = w / w.sum(1, keepdim=True)
        if op == "combine_grad":
            st["dout"] = torch.randn(T, N, device=DEV, generator=g).to(torch.bfloat16)
    return st


def prepare(case, seed):
    c = dict(case)
    st = _inputs(c, seed)
    if not own:
        return st
    from block_scaled_precision_03_amd import mxgemm as mx
    op = c["op"]
    e32, ei = dict(dtype=torch.float32, device=DEV), dict(dtype=torch.int32, device=DEV)
    eb = dict(dtype=torch.bfloat16, device=DEV)
    mx.init()
    if op == "route":
        T, E, k = c["T"], c["E"], c["topk"]
        st["out"] = (torch.empty(T, k, **ei), torch.empty(T, k, **e32),
                     torch.empty(E, dtype=torch.int64, device=DEV), torch.empty(T, k, **ei),
                     torch.empty(T * k, **ei))
        st["ws"] = torch.empty(mx.moe_route_workspace_bytes(T, E), dtype=torch.uint8, device=DEV)
    elif op == "route_grad":
        st["out"] = torch.empty_like(st["logits"])
    elif op == "quant":
        rows = c["T"] * max(1, c["topk"])
        st["out"] = (torch.empty(rows, c["K"], dtype=torch.int8, device=DEV), torch.empty(rows, **e32))
    elif op == "int8":
        st["out"] = torch.empty(c["M"], _out_cols(c), **eb)
    elif op == "grouped":
        st["out"] = torch.empty(c["totM"], _out_cols(c), **eb)
    elif op == "combine":
        st["out"] = torch.empty(c["T"], c["N"], **eb)
    else:
        st["out"] = (torch.empty_like(st["y"]), torch.empty_like(st["w"]))
    return st


# ---- this library -----------------------------------------------------------

def _run_own(st):
    from block_scaled_precision_03_amd import mxgemm as mx
    c, out = st["case"], st["out"]
    op = c["op"]
    if op in ("route", "route_grad"):
        dt = mx.BF16 if c["dtype"] == "bf16" else mx.F32
        score = mx.MOE_SOFTMAX if c["score"] == "softmax" else mx.MOE_SIGMOID
    if op == "route":
        ids, weights, m_sizes, row_of, slot_of = out
        mx.moe_route(dt, st["logits"], st["bias"], ids, weights, c["T"], c["E"], c["topk"], score=score,
                     n_group=c["n_group"], topk_group=c["topk_group"],
                     group_score=mx.MOE_GROUP_TOP2 if c["group_score"] == "top2" else mx.MOE_GROUP_MAX,
                     renormalize=c["renorm"], scale=c["scale"], m_sizes=m_sizes, row_of=row_of, slot_of=slot_of,
                     workspace=st["ws"])
    elif op == "route_grad":
        mx.moe_route_backward(dt, st["logits"], st["ids"], st["grad"], out, c["T"], c["E"], c["topk"],
                              score=score, renormalize=c["renorm"], scale=c["scale"])
    elif op == "quant":
        mx.quantize_int8(mx.BF16 if c["dtype"] == "bf16" else mx.F32, st["x"], out[0], out[1], c["T"], c["K"],
                         row_of=st["row_of"], topk=max(1, c["topk"]))
    elif op in ("int8", "grouped"):
        act = {"none": mx.ACT_NONE, "relu": mx.ACT_RELU, "gelu": mx.ACT_GELU_TANH, "silu": mx.ACT_SILU,
               "swiglu": mx.ACT_SWIGLU}[c["act"]]
        if op == "int8":
            mx.run_fused(mx.INT8, mx.INT8, mx.NT, st["a"], st["sa"], st["b"], st["sb"], out, c["M"], c["N"],
                         c["K"], bias=st["bias"], activation=act)
        else:
            mx.grouped_int8_run(c["G"], st["m_sizes"], st["a"], st["sa"], st["w"], st["sw"], out, c["totM"],
                                c["N"], c["K"], activation=act)
    elif op == "combine":
        mx.moe_combine(st["y"], st["w"], st["row_of"], out, c["T"], c["topk"], c["N"], c["T"] * c["topk"])
    else:
        mx.moe_combine_backward(st["dout"], st["y"], st["w"], st["row_of"], out[0], out[1], c["T"], c["topk"],
                                c["N"], c["T"] * c["topk"])
    return out


# ---- plain form -------------------------------------------------------------

def _act(z, act):
    if act == "relu":
        return torch.clamp_min(z, 0)
    if act == "gelu":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "swiglu":
        g, u = z[:, 0::2], z[:, 1::2]
        return g / (1 + torch.exp(-g)) * u
    return z


def _plain_scores(l, score):
    """Scores of 64-bit logits, 0 where an expert is not available."""
    ok = l > -math.inf
    l = torch.where(ok, l.clamp(max=FLT_MAX), torch.zeros_like(l))
    if score == "sigmoid":
        return torch.where(ok, 1 / (1 + torch.exp(-l)), 0), ok
    m = torch.where(ok, l, -math.inf).amax(1, keepdim=True)
    e = torch.where(ok, torch.exp(l - m), 0)
    return e / e.sum(1, keepdim=True).clamp(min=1), ok


def _plain_route(st):
    c = st["case"]
    T, E, k, ng = c["T"], c["E"], c["topk"], c["n_group"]
    # values next to a border decide between experts: scores in 64 bits
    l = st["logits"].double()
    s, ok = _plain_scores(l, c["score"])
    b = st["bias"].double() if st["bias"] is not None else None
    choice = torch.where(ok, l if b is None else s + b, -math.inf)
    if ng > 1:
        per = choice.view(T, ng, E // ng)
        if c["group_score"] == "top2":
            sb = torch.where(ok, s if b is None else s + b, -math.inf).view(T, ng, E // ng)
            top = torch.sort(sb, dim=2, descending=True).values[:, :, :2]
            gs = torch.where(top[:, :, 0] > -math.inf, torch.where(top > -math.inf, top, 0).sum(2), -math.inf)
        else:
            gs = per.amax(2)
        order = torch.sort(gs, dim=1, descending=True, stable=True).indices[:, :c["topk_group"]]
        keep = torch.zeros_like(gs, dtype=torch.bool).scatter_(1, order, True)
        choice = torch.where(keep.unsqueeze(2), per, -math.inf).view(T, E)
    top = torch.sort(choice, dim=1, descending=True, stable=True)
    ids, live = top.indices[:, :k], top.values[:, :k] > -math.inf
    w = torch.where(live, s.gather(1, ids), 0)
    if c["renorm"]:
        w = torch.where(live, w / w.sum(1, keepdim=True), 0)
    ids = torch.where(live, ids, -1)
    flat = ids.reshape(-1)
    key = torch.where(flat < 0, E, flat)
    srt = torch.sort(key, stable=True)
    rows = torch.arange(T * k, dtype=torch.int32, device=DEV)
    used = srt.values < E
    slot_of = torch.where(used, srt.indices, -1).to(torch.int32)
    row_of = torch.empty(T * k, dtype=torch.int32, device=DEV)
    row_of[srt.indices] = torch.where(used, rows, -1)
    m_sizes = torch.bincount(key, minlength=E + 1)[:E]
    return ids.to(torch.int32), (w * c["scale"]).float(), m_sizes, row_of.view(T, k), slot_of


def _plain_route_grad(st):
    c = st["case"]
    l, ids, g = st["logits"].float(), st["ids"].long(), st["grad"]
    if c["score"] == "sigmoid":
        s = 1 / (1 + torch.exp(-l))
    else:
        e = torch.exp(l - l.amax(1, keepdim=True))
        s = e / e.sum(1, keepdim=True)
    sk = s.gather(1, ids)
    if c["renorm"]:
        tot = sk.sum(1, keepdim=True)
        ds = c["scale"] * (g - (g * sk).sum(1, keepdim=True) / tot) / tot
    else:
        ds = c["scale"] * g
    ds = torch.zeros_like(s).scatter_(1, ids, ds)
    if c["score"] == "sigmoid":
        dl = ds * s * (1 - s)
    else:
        dl = s * (ds - (ds * s).sum(1, keepdim=True))
    return dl.to(st["logits"].dtype)


def _run_plain(st):
    c = st["case"]
    op = c["op"]
    if op == "route":
        return _plain_route(st)
    if op == "route_grad":
        return _plain_route_grad(st)
    if op == "quant":
        x = st["x"].float()
        top = x.abs().amax(1)
        # a tensor of 127: torch multiplies by a rounded 1/127 for a number
        s = top / torch.full_like(top, 127.0)
        s = torch.where(s > 0, s, 1.0)
        q = torch.round(x / s[:, None]).clamp_(-127, 127).to(torch.int8)
        if st["row_of"] is None:
            return q, s
        rows, k = st["row_of"].reshape(-1).long(), c["topk"]
        codes = torch.empty(c["T"] * k, c["K"], dtype=torch.int8, device=DEV)
        scales = torch.empty(c["T"] * k, dtype=torch.float32, device=DEV)
        codes[rows] = q.repeat_interleave(k, dim=0)
        scales[rows] = s.repeat_interleave(k)
        return codes, scales
    if op == "int8":
        z = st["a"].float() @ st["b"].float().t() * st["sa"][:, None] * st["sb"]
        if st["bias"] is not None:
            z = z + st["bias"].float()
        return _act(z, c["act"]).to(torch.bfloat16)
    if op == "grouped":
        parts, r = [], 0
        for g, m in enumerate(st["m_host"]):
            if m:
                z = st["a"][r:r + m].float() @ st["w"][g].float().t() * st["sa"][r:r + m, None] * st["sw"][g]
                parts.append(_act(z, c["act"]).to(torch.bfloat16))
            r += m
        return torch.cat(parts)
    T, k, N = c["T"], c["topk"], c["N"]
    rows = st["row_of"].reshape(-1).long()
    y = st["y"][rows].float().view(T, k, N)
    if op == "combine":
        return (y * st["w"][:, :, None]).sum(1).to(torch.bfloat16)
    d = st["dout"].float()[:, None, :]
    dy = torch.empty_like(st["y"])
    dy[rows] = (d * st["w"][:, :, None]).to(torch.bfloat16).view(T * k, N)
    return dy, (y * d).sum(2)


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---- 64-bit definition ------------------------------------------------------

def _exact_select(c, l, b):
    """ids and weights from ranks: an expert's rank is the number of experts
    that come before it (larger choice, or equal and of lower index)."""
    T, E, k, ng = l.shape[0], c["E"], c["topk"], c["n_group"]
    idx = torch.arange(E, device=DEV)
    avail = torch.isfinite(l) | (l == math.inf)
    if c["score"] == "sigmoid":
        s = torch.special.expit(l)
    else:
        s = torch.softmax(torch.where(avail, l, -math.inf), dim=1)
    s = torch.where(avail, s, 0.0)
    v = l if b is None else s + b
    v = torch.where(avail, v, -math.inf)
    if ng > 1:
        n = E // ng
        score = v if c["group_score"] == "max" else torch.where(avail, s if b is None else s + b, -math.inf)
        score = score.reshape(T, ng, n)
        best = score.max(2)
        gs = best.values
        if c["group_score"] == "top2":
            second = score.scatter(2, best.indices[:, :, None], -math.inf).max(2).values
            gs = gs + torch.where(second > -math.inf, second, 0.0)
        gi = torch.arange(ng, device=DEV)
        before = (gs[:, None, :] > gs[:, :, None]) | ((gs[:, None, :] == gs[:, :, None]) & (gi[None, :] < gi[:, None]))
        chosen = (before.sum(2) < c["topk_group"]).repeat_interleave(n, dim=1)
        v = torch.where(chosen, v, -math.inf)
    before = (v[:, None, :] > v[:, :, None]) | ((v[:, None, :] == v[:, :, None]) & (idx[None, :] < idx[:, None]))
    rank = before.sum(2)
    ids = torch.full((T, k), -1, dtype=torch.int64, device=DEV)
    w = torch.zeros(T, k, dtype=torch.float64, device=DEV)
    t, e = torch.nonzero((rank < k) & (v > -math.inf), as_tuple=True)
    ids[t, rank[t, e]] = e
    w[t, rank[t, e]] = s[t, e]
    if c["renorm"]:
        w = w / torch.where(ids[:, :1] >= 0, w.sum(1, keepdim=True), 1.0)
    return ids, w * c["scale"]


def _exact_route(c, st):
    T, E, k = c["T"], c["E"], c["topk"]
    b = st["bias"].double() if st["bias"] is not None else None
    part = [_exact_select(c, x.double(), b) for x in torch.split(st["logits"], max(1, (1 << 26) // (E * E)))]
    ids, w = torch.cat([p[0] for p in part]), torch.cat([p[1] for p in part])
    # every expert's rows follow those of the experts before it, in token order
    used = torch.zeros(T, E + 1, dtype=torch.int64, device=DEV).scatter_(1, torch.where(ids < 0, E, ids), 1)[:, :E]
    m_sizes = used.sum(0)
    first = torch.cumsum(m_sizes, 0) - m_sizes
    place = torch.cumsum(used, 0) - used + first
    row_of = torch.where(ids < 0, -1, place.gather(1, ids.clamp(min=0)))
    slot_of = torch.full((T * k,), -1, dtype=torch.int64, device=DEV)
    flat = row_of.reshape(-1)
    slots = torch.arange(T * k, device=DEV)
    slot_of[flat[flat >= 0]] = slots[flat >= 0]
    i32 = torch.int32
    return ids.to(i32), w, m_sizes, row_of.to(i32), slot_of.to(i32)


def _exact_route_grad(c, st):
    l, ids, g = st["logits"].double(), st["ids"].long(), st["grad"].double()
    lk = l.gather(1, ids)
    dl = torch.zeros_like(l)
    if c["score"] == "sigmoid":
        p = torch.special.expit(lk)
        slope = p * torch.special.expit(-lk)
        w = p / p.sum(1, keepdim=True)
        up = (g - (g * w).sum(1, keepdim=True)) / p.sum(1, keepdim=True) if c["renorm"] else g
        return dl.scatter_(1, ids, c["scale"] * up * slope)
    if c["renorm"]:
        w = torch.softmax(lk, dim=1)
        return dl.scatter_(1, ids, c["scale"] * w * (g - (g * w).sum(1, keepdim=True)))
    s = torch.softmax(l, dim=1)
    sk = s.gather(1, ids)
    return c["scale"] * (dl.scatter_(1, ids, sk * g) - s * (sk * g).sum(1, keepdim=True))


def _exact_act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, 0.0)
    if act == "gelu":
        u = math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
        return z * torch.special.expit(2 * u)
    if act == "silu":
        return z * torch.special.expit(z)
    if act == "swiglu":
        m, n = z.shape
        pair = z.reshape(m, n // 2, 2)
        return pair[:, :, 0] * torch.special.expit(pair[:, :, 0]) * pair[:, :, 1]
    return z


def exact(case, seed):
    c = dict(case)
    st = _inputs(c, seed)
    op = c["op"]
    if op == "route":
        return _exact_route(c, st)
    if op == "route_grad":
        return _exact_route_grad(c, st)
    if op == "quant":
        # the scale and the quotients are defined as 32-bit numbers; a 64-bit
        # quotient rounded to 32 bits is the correctly rounded one
        x = st["x"].double()
        top = torch.maximum(x.max(1).values, -x.min(1).values)
        s = (top / 127).float().double()
        s[s == 0] = 1
        q = (x / s[:, None]).float().round().clamp(-127, 127).to(torch.int8)
        if not c["topk"]:
            return q, s
        row_of = st["row_of"].long()
        token = torch.empty(row_of.numel(), dtype=torch.int64, device=DEV)
        for j in range(c["topk"]):
            token[row_of[:, j]] = torch.arange(c["T"], device=DEV)
        return q[token], s[token]
    if op == "int8":
        z = torch.mm(st["a"].double(), st["b"].double().t())
        z.mul_(st["sa"].double()[:, None]).mul_(st["sb"].double()[None, :])
        if st["bias"] is not None:
            z += st["bias"].double()[None, :]
        return _exact_act(z, c["act"])
    if op == "grouped":
        z = torch.empty(c["totM"], c["N"], dtype=torch.float64, device=DEV)
        ends = torch.cumsum(st["m_sizes"], 0).tolist()
        for g, hi in enumerate(ends):
            lo = ends[g - 1] if g else 0
            if hi > lo:
                torch.mm(st["a"][lo:hi].double(), st["w"][g].double().t(), out=z[lo:hi])
                z[lo:hi] *= st["sa"][lo:hi].double()[:, None] * st["sw"][g].double()[None, :]
        return _exact_act(z, c["act"])
    T, k, N = c["T"], c["topk"], c["N"]
    row_of, w, y = st["row_of"].long(), st["w"].double(), st["y"]
    if op == "combine":
        out = torch.zeros(T, N, dtype=torch.float64, device=DEV)
        for j in range(k):
            out += w[:, j, None] * y[row_of[:, j]].double()
        return out
    dy = torch.empty(T * k, N, dtype=torch.float64, device=DEV)
    dw = torch.empty(T, k, dtype=torch.float64, device=DEV)
    for j in range(k):
        dy[row_of[:, j]] = w[:, j, None] * st["dout"].double()
        dw[:, j] = (st["dout"].double() * y[row_of[:, j]].double()).sum(1)
    return dy, dw

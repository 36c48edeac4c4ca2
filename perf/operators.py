"""Measured cases of the few-token operators: products with 4-bit weights and whole MoE layers.

Four operators, each called with 1 to 16 tokens as a decode or a speculative-verification step does:

* ``linear``    y = x W^T, W in 4-bit codes with a BF16 scale per row and group of 32, 64 or 128
* ``dense``     the dense SwiGLU MLP with such weights
* ``few``       the whole sparse-MoE layer (router to combine), BF16 expert weights
* ``few_int4``  the same layer with 4-bit expert weights

Definitions (sums over the whole row; the layer's routing is that of ``beam_moe_route``):

    s[n, g] = bf16(max_{k in g} |W[n, k]| / 7),   q[n, k] = clamp(rne(W[n, k] / s[n, g(k)]), -8, 7)
    y[t, n] = sum_k x[t, k] s[n, g(k)] q[n, k]
    mlp(x)  = W_down ( silu(W_gate x) * (W_up x) )
    layer   = sum_j w_j mlp_{e_j}(x),  e = group-limited top-k of sigmoid(x W_r^T) + bias

``own`` false computes them with elementary torch operations in FP32 (the router's logits in FP64,
rounded to FP32: a choice of experts hangs on their last bits); ``own`` true calls the library.
"""
import math

import torch

own = False

MAX_TOKENS = 16


# ------------------------------------------------------------------ cases

def _linear(T, N, K, group, out):
    return dict(op="linear", T=T, N=N, K=K, group=group, out=out)


def _dense(T, d, I, group):
    return dict(op="dense", T=T, d=d, I=I, group=group)


def _few(T, d, E, n_group, topk_group, k, I, skew=False):
    return dict(op="few", T=T, d=d, E=E, n_group=n_group, topk_group=topk_group, k=k, I=I, skew=skew)


def _few_int4(T, d, E, n_group, topk_group, k, I, group, skew=False):
    return dict(_few(T, d, E, n_group, topk_group, k, I, skew), op="few_int4", group=group)


def listed():
    beam = dict(d=5120, E=256, n_group=8, topk_group=4, k=8, I=2560)
    tiny = dict(d=256, E=16, n_group=4, topk_group=2, k=4, I=128)
    return [
        # a small projection with an odd number of rows, three drafted tokens: latency counts
        dict(_linear(3, 1283, 2560, 32, "bf16"), name="linear T3 1283x2560 g32"),
        # one decode token through the gate and up halves of a dense layer
        dict(_linear(1, 40960, 5120, 64, "bf16"), name="linear T1 40960x5120 g64"),
        # the logits of 16 verified tokens over the whole vocabulary, FP32
        dict(_linear(16, 151936, 5120, 128, "fp32"), name="linear T16 vocab g128"),
        # a small dense MLP, five tokens
        dict(_dense(5, 1024, 2816, 32), name="dense T5 1024x2816 g32"),
        # Beam's dense layers at decode: one stream, then eight
        dict(_dense(1, 5120, 20480, 128), name="dense T1 beam g128"),
        dict(_dense(8, 5120, 20480, 128), name="dense T8 beam g128"),
        # the smallest layer: launches and latency
        dict(_few(1, **tiny), name="few T1 tiny"),
        # Beam's layer for one decode stream, and for the 16 tokens of one verification step
        dict(_few(1, **beam), name="few T1 beam"),
        dict(_few(16, **beam), name="few T16 beam"),
        # the 4-bit layer: small and ragged, one decode stream, eight streams on hot experts
        dict(_few_int4(7, **tiny, group=32), name="few_int4 T7 tiny g32"),
        dict(_few_int4(1, **beam, group=128), name="few_int4 T1 beam g128"),
        dict(_few_int4(8, **beam, group=64, skew=True), name="few_int4 T8 skewed g64"),
    ]


def _log(rng, lo, hi):
    return math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))


def draw(rng):
    op = rng.choice(["linear", "dense", "few", "few_int4"])
    T, group = rng.randint(1, MAX_TOKENS), rng.choice([32, 64, 128])
    if op == "linear":
        K = 128 * min(160, int(_log(rng, 2, 160)))
        N = int(_log(rng, 64, min(151936, 151936 * 5120 // K)))
        return _linear(T, N, K, group, rng.choice(["bf16", "fp32"]))
    if op == "dense":
        return _dense(T, 256 * min(20, int(_log(rng, 1, 20))), 128 * min(160, int(_log(rng, 1, 160))), group)
    n_group = rng.choice([1, 2, 4, 8])
    per = rng.choice([4, 8, 16, 32])
    topk_group = rng.randint(1, n_group)
    k = rng.randint(1, min(8, topk_group * per))
    d, I = 256 * min(20, int(_log(rng, 1, 20))), 128 * min(20, int(_log(rng, 1, 20)))
    skew = rng.random() < 0.5
    if op == "few":
        return _few(T, d, n_group * per, n_group, topk_group, k, I, skew)
    return _few_int4(T, d, n_group * per, n_group, topk_group, k, I, group, skew)


# ------------------------------------------------------------------ inputs

def _normal(gen, std, *shape, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, std, generator=gen)


def _bias(case, gen):
    """Near-uniform loads, or 0.5 / rank over a permutation: a few experts take most tokens."""
    E = case["E"]
    if case["skew"]:
        rank = torch.randperm(E, generator=gen, device=gen.device).float() + 1.0
        return 0.5 / rank
    return (torch.rand(E, generator=gen, device=gen.device) - 0.5) * 0.1


def _inputs(case, seed):
    """Every input of a case, weights in BF16, on the GPU: a function of the case and the seed."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    op, T = case["op"], case["T"]
    if op == "linear":
        N, K = case["N"], case["K"]
        return dict(x=_normal(gen, 1.0, T, K), w=_normal(gen, K ** -0.5, 1, N, K))
    d, I = case["d"], case["I"]
    E = 1 if op == "dense" else case["E"]
    s = dict(x=_normal(gen, 1.0, T, d), w_gate=_normal(gen, d ** -0.5, E, I, d),
             w_up=_normal(gen, d ** -0.5, E, I, d), w_down=_normal(gen, I ** -0.5, E, d, I))
    if op != "dense":
        # logits of standard deviation 0.7, as the repository's Beam workloads have
        s["router_w"] = _normal(gen, 0.7 * d ** -0.5, E, d, dtype=torch.float32)
        s["bias"] = _bias(case, gen)
    return s


def _codes(w, group):
    """(q int8 [E, R, K], s BF16 [E, R, K / group]) of BF16 weights w [E, R, K]."""
    E, R, K = w.shape
    q = torch.empty((E, R, K), dtype=torch.int8, device=w.device)
    s = torch.empty((E, R, K // group), dtype=torch.bfloat16, device=w.device)
    step = max(1, (1 << 28) // (R * K))
    for e in range(0, E, step):
        x = w[e:e + step].float().view(-1, R, K // group, group)
        sc = (x.abs().amax(-1) / 7.0).bfloat16()
        s[e:e + step] = sc
        sc = sc.float()[..., None]
        x = torch.where(sc > 0, x / sc, torch.zeros((), device=x.device))
        q[e:e + step] = x.round_().clamp_(-8, 7).view(-1, R, K)
    return q, s


def prepare(case, seed):
    """Inputs, and the weights in the form that the program keeps them in: as the library lays them
    out where ``own`` is true, plain codes and scales (or the BF16 weights) otherwise."""
    s = _inputs(case, seed)
    op, T = case["op"], case["T"]
    if op == "linear":
        s["out"] = torch.empty(T, case["N"], device="cuda", dtype=torch.float32 if case["out"] == "fp32" else torch.bfloat16)
    else:
        s["out"] = torch.empty(T, case["d"], dtype=torch.bfloat16, device="cuda")
        if op != "dense":
            s["idx"] = torch.empty(T, case["k"], dtype=torch.int32, device="cuda")
            s["w"] = torch.empty(T, case["k"], dtype=torch.float32, device="cuda")
    s["case"] = case
    if own:
        from sparse_moe_transformer_fp32_b200 import beam_moe as bm
        s["bm"] = bm
        if op == "linear":
            s["packed"] = bm.beam_int4_quantize(s.pop("w"), group_size=case["group"])
            s["shape"] = bm.int4_shape(T, case["N"], case["K"], case["group"])
        elif op == "dense":
            s["gate_up"] = bm.beam_int4_quantize(s.pop("w_gate"), s.pop("w_up"), group_size=case["group"])
            s["down"] = bm.beam_int4_quantize(s.pop("w_down"), group_size=case["group"])
            s["shape"] = bm.dense_shape(T, case["d"], case["I"])
            s["ws"] = bm.dense_int4_workspace(s["shape"])
        else:
            s["shape"] = bm.make_shape(T, case["d"], case["E"], case["n_group"], case["topk_group"], case["k"], case["I"])
            s["ws"] = bm.few_workspace(s["shape"])
            if op == "few_int4":
                s["gate_up"] = bm.beam_int4_quantize(s.pop("w_gate"), s.pop("w_up"), group_size=case["group"])
                s["down"] = bm.beam_int4_quantize(s.pop("w_down"), group_size=case["group"])
    elif op != "few":
        for name in [n for n in ("w_gate", "w_up", "w_down") if n in s] or ["w"]:
            s[name] = _codes(s[name], case["group"]) if op != "linear" else tuple(t[0] for t in _codes(s[name], case["group"]))
    return s


# ------------------------------------------------------------------ one pass

def _value(w, at=None):
    """FP32 weights: BF16 ones widened, codes times their scales; of the rows ``at`` of the first axis."""
    if isinstance(w, tuple):
        q, sc = w if at is None else (w[0][at], w[1][at])
        return (q.float().unflatten(-1, (sc.shape[-1], -1)) * sc.float()[..., None]).flatten(-2)
    return (w if at is None else w[at]).float()


def _choose(sb, case):
    """The chosen experts [T, k] of biased scores sb [T, E], ascending; ties to the lower index."""
    T, E = sb.shape
    per = E // case["n_group"]
    grouped = sb.view(T, case["n_group"], per)
    top = grouped.sort(dim=-1, descending=True).values
    gs = top[..., 0] + top[..., 1] if per > 1 else top[..., 0]
    kept = gs.sort(dim=-1, descending=True, stable=True).indices[:, :case["topk_group"]]
    open_ = torch.zeros_like(gs, dtype=torch.bool).scatter_(1, kept, True)
    cand = grouped.masked_fill(~open_[..., None], -math.inf).view(T, E)
    return cand.sort(dim=-1, descending=True, stable=True).indices[:, :case["k"]].sort(dim=-1).values


def _route(x, router_w, bias, case):
    logits = (x.double() @ router_w.double().T).float()
    score = torch.sigmoid(logits.double()).float()
    idx = _choose(score + bias, case)
    chosen = score.gather(1, idx)
    return idx, 2.5 * chosen / chosen.sum(dim=1, keepdim=True)


def _silu(v):
    return v / (1.0 + torch.exp(-v))


def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        bm = s["bm"]
        if op == "linear":
            bm.beam_int4_linear(s["shape"], s["x"], s["packed"], s["out"])
            return {"out": s["out"]}
        if op == "dense":
            bm.beam_dense_forward_int4(s["shape"], case["group"], s["x"], s["gate_up"], s["down"], s["out"], ws=s["ws"])
            return {"out": s["out"]}
        if op == "few":
            bm.beam_moe_forward_few(s["shape"], s["x"], s["router_w"], s["bias"], s["w_gate"], s["w_up"], s["w_down"],
                                    s["out"], s["idx"], s["w"], ws=s["ws"])
        else:
            bm.beam_moe_forward_few_int4(s["shape"], case["group"], s["x"], s["router_w"], s["bias"], s["gate_up"], s["down"],
                                         s["out"], s["idx"], s["w"], ws=s["ws"])
        return {"out": s["out"], "topk_idx": s["idx"], "topk_w": s["w"]}
    x = s["x"].float()
    if op == "linear":
        return {"out": (x @ _value(s["w"]).T).to(s["out"].dtype)}
    if op == "dense":
        a = _silu(x @ _value(s["w_gate"])[0].T) * (x @ _value(s["w_up"])[0].T)
        return {"out": (a @ _value(s["w_down"])[0].T).bfloat16()}
    idx, w = _route(s["x"], s["router_w"], s["bias"], case)
    col = x[:, None, :, None]
    a = _silu(_value(s["w_gate"], idx) @ col) * (_value(s["w_up"], idx) @ col)
    y = (_value(s["w_down"], idx) @ a).squeeze(-1)
    out = (w[..., None] * y).sum(dim=1)
    return {"out": out.bfloat16(), "topk_idx": idx.int(), "topk_w": w}


# ------------------------------------------------------------------ definition in 64 bits

def exact(case, seed):
    """The definitions above in FP64, expert by expert; written apart from ``run``."""
    s = _inputs(case, seed)
    x = s["x"].to(torch.float64)

    def weight(w):  # [R, K] BF16 -> the FP64 values that the operator multiplies with
        w = w.to(torch.float64)
        if case["op"] == "few":
            return w
        parts = w.split(case["group"], dim=1)
        vals = []
        for p in parts:
            sc = (p.abs().max(dim=1, keepdim=True).values.float() / 7.0).to(torch.bfloat16).to(torch.float64)
            q = torch.round(p / torch.where(sc == 0, torch.ones_like(sc), sc))
            vals.append(sc * torch.minimum(torch.maximum(q, torch.full_like(q, -8)), torch.full_like(q, 7)))
        return torch.cat(vals, dim=1)

    def product(v, w):  # v [n, K] FP64, w [R, K] BF16; a few thousand rows at a time
        return torch.cat([torch.mm(v, weight(c).t()) for c in w.split(16384)], dim=1)

    if case["op"] == "linear":
        return {"out": product(x, s["w"][0])}

    def mlp(v, e):
        g, u = product(v, s["w_gate"][e]), product(v, s["w_up"][e])
        return product(g / (torch.exp(-g) + 1) * u, s["w_down"][e])

    if case["op"] == "dense":
        return {"out": mlp(x, 0)}

    # the routing's decisions are taken on FP32 scores by definition; the weights are not rounded
    score = 1.0 / (1.0 + torch.exp(-torch.mm(x, s["router_w"].to(torch.float64).t())))
    logit32 = torch.mm(x, s["router_w"].to(torch.float64).t()).float()
    sb = ((1.0 / (1.0 + torch.exp(-logit32.double()))).float() + s["bias"]).cpu().tolist()
    per, T, k = case["E"] // case["n_group"], case["T"], case["k"]
    idx = []
    for t in range(T):
        total = []
        for g in range(case["n_group"]):
            two = sorted(sb[t][g * per:(g + 1) * per], reverse=True)[:2]
            total.append(float(torch.tensor(two, dtype=torch.float32).sum()))
        groups = sorted(range(case["n_group"]), key=lambda g: (-total[g], g))[:case["topk_group"]]
        cand = [e for g in groups for e in range(g * per, (g + 1) * per)]
        idx.append(sorted(sorted(cand, key=lambda e: (-sb[t][e], e))[:k]))
    idx = torch.tensor(idx, device=x.device)
    w = torch.gather(score, 1, idx)
    w = w / w.sum(dim=1, keepdim=True) * 2.5
    out = torch.zeros_like(x)
    for e in sorted(set(idx.flatten().tolist())):
        t, j = (idx == e).nonzero(as_tuple=True)
        out.index_add_(0, t, mlp(x[t], e) * w[t, j][:, None])
    return {"out": out, "topk_idx": idx.int(), "topk_w": w}


# ------------------------------------------------------------------ work of one pass

def _touched(case):
    """Experts that hold a token, as a mean over routings drawn with the cases' distributions."""
    gen = torch.Generator()
    gen.manual_seed(1)
    n = 0
    for _ in range(8):
        sb = torch.sigmoid(torch.randn(case["T"], case["E"], generator=gen) * 0.7) + _bias(case, gen)
        n += len(set(_choose(sb, case).flatten().tolist()))
    return n / 8


def work(case):
    """Weights of the experts touched, inputs and outputs, each once; two operations a product."""
    T, op = case["T"], case["op"]
    per = 2.0 if op == "few" else 0.5 + 2.0 / case["group"]  # bytes of a weight
    if op == "linear":
        N, K = case["N"], case["K"]
        return {"bytes": N * K * per + 2 * T * K + T * N * (4 if case["out"] == "fp32" else 2), "flops": 2.0 * T * N * K}
    d, I = case["d"], case["I"]
    if op == "dense":
        return {"bytes": 3 * d * I * per + 4 * T * d, "flops": 6.0 * T * d * I}
    E, k = case["E"], case["k"]
    return {"bytes": _touched(case) * 3 * d * I * per + 4 * E * (d + 1) + T * (4 * d + 8 * k),
            "flops": 6.0 * T * k * d * I + 2.0 * T * d * E}

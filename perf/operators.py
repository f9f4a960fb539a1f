"""Cases of the operators around dispatch and combine: the gate that makes the routing (forward and gradient),
microscaled quantisation, and the experts' grouped product on microscaled rows and 4-bit weights.

`run` computes each operator from elementary torch operations where `own` is false, and through the package where it
is true, on what `prepare` made. `exact` is the definition in binary64.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
BLOCK = 32                                    # elements that share one scale byte
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # one token from each of 8 ranks: the decode step's routing, where latency is all
        {"name": "gate 8 of 64", "op": "gate", "tokens": 8, "experts": 64, "topk": 8, "dtype": "bf16",
         "score": "softmax", "bias": False, "groups": 1, "topk_groups": 1, "renorm": True, "scale": 1.0,
         "masked": False},
        # 16 ranks x 256 tokens: sigmoid scores, balance bias, 4 of 8 groups by their two best experts
        {"name": "gate 4096 of 256 grouped", "op": "gate", "tokens": 4096, "experts": 256, "topk": 8, "dtype": "fp32",
         "score": "sigmoid", "bias": True, "groups": 8, "topk_groups": 4, "renorm": True, "scale": 2.5,
         "masked": False},
        # a long prefill with an odd token count, 48 special experts beside 256, and padded tokens
        {"name": "gate 65521 of 304 masked", "op": "gate", "tokens": 65521, "experts": 304, "topk": 8, "dtype": "bf16",
         "score": "softmax", "bias": True, "groups": 1, "topk_groups": 1, "renorm": False, "scale": 1.0,
         "masked": True},
        # the training step's gradient at 16 ranks x 256 tokens
        {"name": "gate gradient 4096 of 256", "op": "gate_backward", "tokens": 4096, "experts": 256, "topk": 8,
         "dtype": "fp32", "score": "sigmoid", "renorm": True, "scale": 2.5, "masked": False},
        # a long batch whose weights are the plain softmax scores: every expert's logit gets a gradient
        {"name": "gate gradient 65521 of 304", "op": "gate_backward", "tokens": 65521, "experts": 304, "topk": 8,
         "dtype": "bf16", "score": "softmax", "renorm": False, "scale": 1.0, "masked": True},
        # the rows of 8 ranks x 4 tokens, top-8: activations between two products at small batch
        {"name": "quantize 256 x 7168 e2m1", "op": "quantize", "rows": 256, "cols": 7168, "dtype": "bf16",
         "element": "e2m1"},
        # every row of 16 ranks x 256 tokens, top-8
        {"name": "quantize 32768 x 7168 e2m1", "op": "quantize", "rows": 32768, "cols": 7168, "dtype": "bf16",
         "element": "e2m1"},
        # odd row count, a last block of 16, 8-bit elements from half precision
        {"name": "quantize 4099 x 2064 e4m3", "op": "quantize", "rows": 4099, "cols": 2064, "dtype": "fp16",
         "element": "e4m3"},
        # one token on each of 2 ranks: single-token decode, bound by the weights of the experts hit
        {"name": "product 2 tokens", "op": "product", "ranks": 2, "tokens": 1, "experts_per_rank": 4, "topk": 4,
         "k": 7168, "n": 4096, "element": "e4m3", "activation": True, "dtype": "bf16", "routing": "uniform",
         "masked": False},
        # 8 ranks x 32 tokens: the first product on the MXFP8 rows that dispatch writes
        {"name": "product 8x32 up", "op": "product", "ranks": 8, "tokens": 32, "experts_per_rank": 8, "topk": 8,
         "k": 7168, "n": 4096, "element": "e4m3", "activation": True, "dtype": "bf16", "routing": "uniform",
         "masked": False},
        # 16 ranks x 256 tokens with a quarter of the pairs masked: the second product, rows left behind the last
        {"name": "product 16x256 down", "op": "product", "ranks": 16, "tokens": 256, "experts_per_rank": 16,
         "topk": 8, "k": 2048, "n": 7168, "element": "e2m1", "activation": False, "dtype": "bf16",
         "routing": "uniform", "masked": True},
        # 8 ranks x 1024 tokens, Zipf routing: long prefill with one very popular expert, both sides 4-bit
        {"name": "product 8x1024 up zipf", "op": "product", "ranks": 8, "tokens": 1024, "experts_per_rank": 8,
         "topk": 8, "k": 7168, "n": 4096, "element": "e2m1", "activation": True, "dtype": "bf16", "routing": "zipf",
         "masked": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gate", "gate", "gate_backward", "quantize", "product", "product"])
    if op == "gate":
        groups = rng.choice([1, 1, 2, 4, 8])
        experts = groups * rng.randint(max(2, 64 // groups), 304 // groups)
        return {"op": op, "tokens": _log(rng, 1, 65521), "experts": experts, "topk": rng.randint(1, 16),
                "dtype": rng.choice(sorted(DTYPES)), "score": rng.choice(["softmax", "sigmoid"]),
                "bias": rng.random() < 0.6, "groups": groups, "topk_groups": max(1, groups // 2),
                "renorm": rng.random() < 0.6, "scale": rng.choice([1.0, 2.5]), "masked": rng.random() < 0.3}
    if op == "gate_backward":
        return {"op": op, "tokens": _log(rng, 1, 65521), "experts": rng.randint(64, 304), "topk": rng.randint(1, 16),
                "dtype": rng.choice(sorted(DTYPES)), "score": rng.choice(["softmax", "sigmoid"]),
                "renorm": rng.random() < 0.5, "scale": rng.choice([1.0, 2.5]), "masked": rng.random() < 0.3}
    if op == "quantize":
        return {"op": op, "rows": _log(rng, 1, 32768), "cols": 16 * _log(rng, 1, 448),
                "dtype": rng.choice(sorted(DTYPES)), "element": rng.choice(["e2m1", "e4m3"])}
    ranks = rng.choice([2, 4, 8, 16])
    epr = rng.choice([1, 2, 4, 8][:3 if ranks == 16 else 4])
    topk = rng.randint(1, min(8, ranks * epr))
    k, n = 16 * _log(rng, 8, 448), 2 * _log(rng, 64, 2048)
    most = 8192 // ranks
    return {"op": op, "ranks": ranks, "tokens": _log(rng, 1, most), "experts_per_rank": epr, "topk": topk,
            "k": k, "n": n, "element": rng.choice(["e2m1", "e4m3"]), "activation": rng.random() < 0.5,
            "dtype": rng.choice(["bf16", "fp16"]), "routing": rng.choice(["uniform", "zipf"]),
            "masked": rng.random() < 0.3}


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(0x5EED + 7919 * int(seed))


def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(shape, generator=g, device=DEV, dtype=dtype)


def _rand(g, *shape):
    return torch.rand(shape, generator=g, device=DEV)


# ---- inputs ----

def _gate_inputs(case, g):
    N, E = case["tokens"], case["experts"]
    # a router's logits: a token's own spread around an expert's popularity
    logits = (_randn(g, N, E) * 1.5 + _randn(g, 1, E) * 0.5).to(DTYPES[case["dtype"]])
    bias = _randn(g, E) * (0.05 if case["score"] == "sigmoid" else 0.01) if case.get("bias") else None
    mask = _rand(g, N) < 0.75 if case["masked"] else None
    return logits, bias, mask


def _routing(case, g):
    """Row counts as dispatch forms them: ep_recv_count and the most rows that an expert has."""
    W, bs, epr, K = case["ranks"], case["tokens"], case["experts_per_rank"], case["topk"]
    E, N = W * epr, W * bs
    pop = torch.arange(1, E + 1, device=DEV, dtype=torch.float32).log() * -1.2
    z = _randn(g, N, E) + (pop if case["routing"] == "zipf" else 0.0)
    ids = z.argsort(dim=1, descending=True, stable=True)[:, :K]
    src = (torch.arange(N, device=DEV) // bs)[:, None]
    keep = _rand(g, N, K) < 0.75 if case["masked"] else torch.ones((N, K), device=DEV, dtype=torch.bool)
    seg = torch.bincount((ids * W + src)[keep], minlength=E * W)         # (expert, source rank), experts rank-major
    counts = seg.view(W, epr * W).cumsum(1).to(torch.int32).contiguous()
    return counts, int(seg.view(E, W).sum(1).max())


def _quantise(x, element):
    """(codes as values times no scale, shared exponents) of rows whose length is a multiple of 16, in binary32."""
    rows, cols = x.shape
    pad = -cols % BLOCK
    b = torch.nn.functional.pad(x.float(), (0, pad)).view(rows, -1, BLOCK)
    top = torch.frexp(b.abs().amax(2))[1] - 1                     # floor(log2 max|x|)
    zero = b.abs().amax(2) == 0
    shared = (top - (2 if element == "e2m1" else 8)).clamp(-127, 127).masked_fill(zero, -127).to(torch.int32)
    y = b * ((127 - shared) << 23).view(torch.float32)[:, :, None]       # an exact power of two
    a = y.abs()
    if element == "e2m1":
        step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
        q = (torch.round(a / step) * step).clamp(max=6.0)
    else:
        e = (torch.frexp(a)[1] - 1).clamp(min=-6)                 # eight steps a binade, 2^-9 the smallest
        step = ((e - 3 + 127) << 23).view(torch.float32)
        q = (torch.round(a / step) * step).clamp(max=448.0)
    return torch.copysign(q, b), shared


def _power(byte):
    """2^(byte - 127) of scale bytes, as binary32."""
    b = byte.to(torch.int32)
    return torch.where(b > 0, b << 23, torch.full_like(b, 1 << 22)).view(torch.float32)


def _pack(q, shared, element, cols):
    """Codes and scale bytes as the operators take them."""
    q = q.flatten(1)[:, :cols]
    if element == "e4m3":
        codes = q.to(torch.float8_e4m3fn)
    else:
        a = q.abs() * 2                                           # 0 1 2 3 4 6 8 12 are the codes 0 to 7
        code = torch.where(a < 4, a, torch.where(a < 8, a / 2 + 2, a / 4 + 4)).to(torch.uint8)
        code = code | (torch.signbit(q).to(torch.uint8) << 3)
        codes = (code[:, 0::2] | (code[:, 1::2] << 4)).contiguous()
    return codes, (shared + 127).to(torch.uint8)


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op == "gate":
        logits, bias, mask = _gate_inputs(case, g)
        return {"case": case, "logits": logits, "bias": bias, "mask": mask}
    if op == "gate_backward":
        logits, _, mask = _gate_inputs(case, g)
        full = dict(case, bias=False, groups=1, topk_groups=1)
        ids, w, _ = _gate_plain(full, logits, None, mask)
        return {"case": case, "logits": logits, "ids": ids, "weights": w, "grad": _randn(g, *w.shape)}
    if op == "quantize":
        # activations: a normal, rows of different size, a few columns that stand out
        x = _randn(g, case["rows"], case["cols"]) * torch.exp(_randn(g, case["rows"], 1))
        x = x * torch.where(_rand(g, 1, case["cols"]) < 0.01, 20.0, 1.0)
        return {"case": case, "x": x.to(DTYPES[case["dtype"]])}
    E, k, n = case["ranks"] * case["experts_per_rank"], case["k"], case["n"]
    rows = case["ranks"] * case["tokens"] * case["topk"]
    counts, most = _routing(case, g)
    x, xs = [], []
    for at in range(0, rows, 8192):
        part = _randn(g, min(8192, rows - at), k) * torch.where(_rand(g, 1, k) < 0.01, 8.0, 1.0)
        c, s = _pack(*_quantise(part.bfloat16(), case["element"]), case["element"], k)
        x.append(c.view(torch.uint8))
        xs.append(s)
    x = torch.cat(x)
    w = torch.empty((E, n, k // 2), dtype=torch.uint8, device=DEV)
    ws = torch.empty((E, n, -(-k // BLOCK)), dtype=torch.uint8, device=DEV)
    for e in range(E):
        w[e], ws[e] = _pack(*_quantise(_randn(g, n, k) * k ** -0.5, "e2m1"), "e2m1", k)
    out = torch.zeros((rows, n // 2 if case["activation"] else n), dtype=DTYPES[case["dtype"]], device=DEV)
    return {"case": case, "x": x.view(torch.float8_e4m3fn) if case["element"] == "e4m3" else x, "xs": torch.cat(xs),
            "w": w, "ws": ws, "counts": counts, "most": most, "out": out}


# ---- the plain forms ----

def _gate_plain(case, logits, bias, mask):
    """(ids, weights, pair mask): scores and choices in binary64, where two experts' order may hang on the last bits."""
    N, E = logits.shape
    K, G = case["topk"], case["groups"]
    low = float("-inf")
    l = logits.double()
    ok = l > low
    if bias is not None:
        ok = ok & (bias > low)
    if mask is not None:
        ok = ok & mask[:, None]
    l = torch.where(ok, l, low)
    if case["score"] == "softmax":
        top = l.amax(1, keepdim=True).clamp(min=-1e300)
        e = torch.exp(l - top)
        s = e / e.sum(1, keepdim=True).clamp(min=1e-300)
    else:
        s = 1.0 / (1.0 + torch.exp(-l))
    c = torch.where(ok, s + bias.double() if bias is not None else l, low)
    if G > 1:
        v = torch.where(ok, s + bias.double() if bias is not None else s, low)
        two = v.view(N, G, E // G).sort(dim=2, descending=True).values[:, :, :2]
        of = two[:, :, 0] + (two[:, :, 1].clamp(min=-1e300) * (two[:, :, 1] > low) if two.shape[2] > 1 else 0.0)
        best = of.sort(dim=1, descending=True, stable=True).indices[:, :case["topk_groups"]]
        kept = torch.zeros((N, G), dtype=torch.bool, device=DEV).scatter_(1, best, True)
        c = torch.where(kept.repeat_interleave(E // G, dim=1), c, low)
    c, at = c.sort(dim=1, descending=True, stable=True)
    c, at = c[:, :K], at[:, :K]
    on = c > low
    w = torch.where(on, s.gather(1, at), 0.0)
    if case["renorm"]:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, 0.0)
    w = w * case["scale"]
    return torch.where(on, at, -1).to(torch.int32), w.float(), on


def _gate_backward_plain(case, logits, ids, w, grad):
    l, w, g = logits.float(), w, grad
    on = ids >= 0
    at = ids.clamp(min=0).long()
    g = torch.where(on, g, 0.0)
    dot = (g.double() * w.double()).sum(1, keepdim=True).float()
    if case["renorm"]:
        d = w * (g - dot / case["scale"])
        if case["score"] == "sigmoid":
            d = d / (1.0 + torch.exp(l.gather(1, at)))            # 1 - sigmoid
    elif case["score"] == "sigmoid":
        s = 1.0 / (1.0 + torch.exp(-l.gather(1, at)))
        d = case["scale"] * g * s / (1.0 + torch.exp(l.gather(1, at)))
    else:
        d = case["scale"] * g
    d = torch.where(on, d, 0.0)
    full = torch.zeros_like(l).scatter_add_(1, at, d)
    if case["score"] == "softmax" and not case["renorm"]:
        e = torch.exp(l - l.amax(1, keepdim=True))
        full = e / e.sum(1, keepdim=True) * (full - dot)
        full = torch.where(on.any(1, keepdim=True), full, 0.0)
    return full.to(logits.dtype)


def _nibbles(codes):
    """What packed 4-bit codes stand for, [..., 2 per byte], in binary32."""
    v = torch.stack((codes & 15, codes >> 4), dim=-1).flatten(-2)
    m = (v & 7).float()
    a = torch.where(m < 4, m * 0.5, torch.where(m < 6, m - 2, m * 2 - 8))
    return torch.where(v > 7, -a, a)


def _scaled(values, bytes_):
    """values [..., k] times each block's power of two."""
    return values * _power(bytes_).repeat_interleave(BLOCK, dim=-1)[..., :values.shape[-1]]


def _product_plain(case, s):
    counts, out = s["counts"], torch.zeros_like(s["out"])
    W, E = counts.shape[0], s["w"].shape[0]
    base = (counts[:, -1].cumsum(0) - counts[:, -1])[:, None]
    ends = (counts[:, W - 1::W] + base).reshape(E).contiguous()   # one past each expert's last row
    row = torch.arange(out.shape[0], device=DEV, dtype=torch.int32)
    expert = torch.searchsorted(ends, row, right=True)
    start = torch.cat((ends.new_zeros(1), ends))
    x = _nibbles(s["x"]) if case["element"] == "e2m1" else s["x"].float()
    x = _scaled(x, s["xs"])
    m = s["most"]
    # every expert's rows, padded to the longest: row p of expert e is input row start[e] + p
    index = start[:E, None] + torch.arange(m, device=DEV)
    padded = x[index.clamp(max=out.shape[0] - 1)].transpose(1, 2).contiguous()
    y = torch.bmm(_scaled(_nibbles(s["w"]), s["ws"]), padded)     # [expert, n, row]
    if case["activation"]:
        gate, up = y.chunk(2, dim=1)
        y = gate / (1.0 + torch.exp(-gate)) * up
    live = expert < E
    expert = expert.clamp(max=E - 1)
    rows = y.transpose(1, 2)[expert, (row - start[expert]).clamp(0, m - 1)]
    return torch.where(live[:, None], rows.to(out.dtype), out)


def run(state):
    case = state["case"]
    if own:
        return _own(case, state)
    if case["op"] == "gate":
        return _gate_plain(case, state["logits"], state["bias"], state["mask"])
    if case["op"] == "gate_backward":
        return _gate_backward_plain(case, state["logits"], state["ids"], state["weights"], state["grad"])
    if case["op"] == "quantize":
        q, shared = _quantise(state["x"], case["element"])
        v = q * _power(shared + 127)[:, :, None]
        return v.flatten(1)[:, :case["cols"]].bfloat16()
    return _product_plain(case, state)


def _own(case, s):
    import combine_ep_recv_amd as moe

    score = {"softmax": moe.MOE_SCORE_SOFTMAX, "sigmoid": moe.MOE_SCORE_SIGMOID}.get(case.get("score"))
    if case["op"] == "gate":
        ids, w, on = moe.gate(s["logits"], case["topk"], score, bias=s["bias"], groups=case["groups"],
                              topk_groups=case["topk_groups"], group_score=moe.MOE_GROUP_TOP2,
                              renormalize=case["renorm"], scale=case["scale"], token_mask=s["mask"],
                              with_pair_mask=True)
        return ids, w, on
    if case["op"] == "gate_backward":
        return moe.gate_backward(s["logits"], s["ids"], s["weights"], s["grad"], score,
                                 renormalize=case["renorm"], scale=case["scale"])
    if case["op"] == "quantize":
        element = {"e2m1": moe.MOE_MX_E2M1, "e4m3": moe.MOE_MX_E4M3}[case["element"]]
        codes, scales = moe.quantize_mx(s["x"], element)
        return moe.dequantize_mx(codes, scales, torch.bfloat16)   # the values that the codes stand for
    act = moe.MOE_ACT_SWIGLU if case["activation"] else moe.MOE_ACT_NONE
    return moe.expert_product_into(s["out"], s["x"], s["xs"], s["w"], s["ws"], s["counts"], activation=act)


# ---- what a pass cannot do without ----

def _hit(case):
    """Experts that get a row, as expected from the routing: (experts, rows)."""
    E, N, K = case["ranks"] * case["experts_per_rank"], case["ranks"] * case["tokens"], case["topk"]
    p = np.arange(1, E + 1) ** (-1.2 if case["routing"] == "zipf" else 0.0)
    keep = 0.75 if case["masked"] else 1.0
    p = np.minimum(1.0, keep * K * p / p.sum())
    return float((1.0 - (1.0 - p) ** N).sum()), N * K * keep


def work(case):
    if case["op"] in ("gate", "gate_backward"):
        N, E, K = case["tokens"], case["experts"], case["topk"]
        on = 0.75 if case["masked"] else 1.0
        table = N * E * DTYPES[case["dtype"]].itemsize
        if case["op"] == "gate":
            return {"bytes": table * on + N * K * 9 + (N if case["masked"] else 0) + (4 * E if case["bias"] else 0),
                    "flops": 10.0 * N * E * on}
        dense = case["score"] == "softmax" and not case["renorm"]
        picked = 0 if case["renorm"] and case["score"] == "softmax" else N * K * on * DTYPES[case["dtype"]].itemsize
        return {"bytes": table + (table * on if dense else picked) + 12 * N * K, "flops": (6.0 if dense else 1.0) * N * E}
    if case["op"] == "quantize":
        n = case["rows"] * case["cols"]
        packed = n * (0.5 if case["element"] == "e2m1" else 1.0) + case["rows"] * -(-case["cols"] // BLOCK)
        return {"bytes": n * DTYPES[case["dtype"]].itemsize + 2 * packed + 2 * n, "flops": 4.0 * n}
    hit, rows = _hit(case)
    k, n = case["k"], case["n"]
    scale = -(-k // BLOCK)
    made = n // 2 if case["activation"] else n
    return {"bytes": hit * n * (k / 2 + scale) + rows * (k * (0.5 if case["element"] == "e2m1" else 1.0) + scale)
            + rows * made * 2, "flops": 2.0 * rows * n * k}


# ---- the definitions, in binary64 ----

def _exact_scores(l, ok, score):
    if score == "sigmoid":
        return torch.where(ok, torch.sigmoid(l), 0.0)
    l = torch.where(ok, l, -1e300)
    return torch.where(ok, torch.softmax(l, dim=1), 0.0)


def _exact_gate(case, s):
    l = s["logits"].double().cpu()
    N, E = l.shape
    K, G = case["topk"], case["groups"]
    ok = torch.ones((N, E), dtype=torch.bool) if s["mask"] is None else s["mask"].cpu()[:, None].expand(N, E)
    sc = _exact_scores(l, ok, case["score"])
    b = torch.zeros(E, dtype=torch.float64) if s["bias"] is None else s["bias"].double().cpu()
    value = (sc + b).numpy()
    key = l.numpy() if s["bias"] is None else value
    live = np.repeat(ok.numpy().any(1)[:, None], K, 1)
    usable = np.ones((N, E), dtype=bool)
    if G > 1:
        of = np.sort(value.reshape(N, G, E // G), axis=2)[:, :, -2:].sum(2)
        order = np.argsort(-of, axis=1, kind="stable")[:, :case["topk_groups"]]
        usable = (order[:, :, None] == (np.arange(E) // (E // G))[None, None, :]).any(1)
    ids = np.argsort(np.where(usable, -key, np.inf), axis=1, kind="stable")[:, :K]
    live = live & np.take_along_axis(usable, ids, 1)
    w = np.where(live, np.take_along_axis(sc.numpy(), ids, 1), 0.0)
    if case["renorm"]:
        w = w / np.maximum(w.sum(1, keepdims=True), 1e-300)
    return np.where(live, ids, -1).astype(np.int32), w * case["scale"], live


def _exact_gate_backward(case, s):
    l, w, g = s["logits"].double(), s["weights"].double(), s["grad"].double()
    ids = s["ids"].long()
    on = (ids >= 0).double()
    E, c = l.shape[1], case["scale"]
    pick = torch.nn.functional.one_hot(ids.clamp(min=0), E).double() * on[:, :, None]    # [N, K, E]
    dot = (on * g * w).sum(1, keepdim=True)
    if case["renorm"]:
        dw = w * (g - dot / c)
    else:
        dw = c * g
    full = torch.matmul(dw[:, None, :], pick)[:, 0]
    sig = torch.sigmoid(l)
    if case["score"] == "sigmoid":
        return full * torch.sigmoid(-l) * (1.0 if case["renorm"] else sig)
    if case["renorm"]:
        return full
    return torch.softmax(l, dim=1) * (full - dot) * on.amax(1, keepdim=True)


def _exact_table(element):
    if element == "e2m1":
        return torch.tensor([v for v in E2M1] + [-v for v in E2M1], dtype=torch.float64, device=DEV)
    return torch.arange(256, device=DEV).to(torch.uint8).view(torch.float8_e4m3fn).double()


def _exact_quantize(case, s):
    x = s["x"].double()
    rows, cols = x.shape
    b = torch.zeros((rows, -(-cols // BLOCK) * BLOCK), dtype=torch.float64, device=DEV)
    b[:, :cols] = x
    b = b.view(rows, -1, BLOCK)
    top = b.abs().amax(2)
    emax = 2 if case["element"] == "e2m1" else 8
    # floor(log2): the exponent field of the binary64 (every input is normal there)
    shared = ((top.view(torch.int64) >> 52) - 1023 - emax).clamp(-127, 127)
    scale = ((shared + 1023) << 52).view(torch.float64)[:, :, None]
    table = _exact_table(case["element"])[:8 if emax == 2 else 127]          # the finite values from 0 up
    a = (b.abs() / scale).clamp(max=float(table[-1]))
    low = (torch.searchsorted(table, a.contiguous(), right=True) - 1).clamp(max=len(table) - 2)
    below, above = a - table[low], table[low + 1] - a
    up = (above < below) | ((above == below) & (low % 2 == 1))               # a tie goes to the even code
    v = table[low + up.long()] * scale
    return torch.copysign(v, b).reshape(rows, -1)[:, :cols]


def _exact_product(case, s):
    W = case["ranks"]
    counts = s["counts"].cpu().numpy().astype(np.int64)
    nib, table = _exact_table("e2m1"), _exact_table(case["element"])
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)

    def values(codes, scales, t, packed):
        c = codes.view(torch.uint8)
        v = torch.stack((t[(c & 15).int()], t[(c >> 4).int()]), -1).flatten(-2) if packed else t[c.int()]
        two = ((scales.long() - 127 + 1023) << 52).view(torch.float64)
        return v * two.repeat_interleave(BLOCK, -1)[..., :v.shape[-1]]

    row = 0
    for r in range(W):
        first = row
        for el in range(case["experts_per_rank"]):
            end = first + int(counts[r, (el + 1) * W - 1])
            if end > row:
                e = r * case["experts_per_rank"] + el
                a = values(s["x"][row:end], s["xs"][row:end], table, case["element"] == "e2m1")
                y = a @ values(s["w"][e], s["ws"][e], nib, True).t()
                if case["activation"]:
                    half = y.shape[1] // 2
                    y = y[:, :half] * torch.sigmoid(y[:, :half]) * y[:, half:]
                out[row:end] = y
            row = end
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "gate":
        return _exact_gate(case, s)
    if case["op"] == "gate_backward":
        return _exact_gate_backward(case, s)
    if case["op"] == "quantize":
        return _exact_quantize(case, s)
    return _exact_product(case, s)

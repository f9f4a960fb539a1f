"""Cases of the operators that close a training step and an int8 layer around dispatch and combine: the gradients of
both calls, rows of 8-bit integers with a scale each, and the experts' grouped product on such rows and weights.

`run` computes each operator from elementary torch operations where `own` is false, and through the package where it
is true, on what `prepare` made. `exact` is the definition in binary64.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # one token from each of 8 ranks: the shortest step, where latency is all
        {"name": "combine gradient 8x1", "op": "combine_backward", "ranks": 8, "tokens": 1, "experts_per_rank": 8,
         "topk": 8, "h": 7168, "dtype": "bf16", "masked": False, "zero": 0, "copy": 0, "const": 0},
        # 16 ranks x 256 tokens: the training step of the layer that the benchmark runs
        {"name": "combine gradient 16x256", "op": "combine_backward", "ranks": 16, "tokens": 256,
         "experts_per_rank": 16, "topk": 8, "h": 7168, "dtype": "bf16", "masked": False, "zero": 0, "copy": 0,
         "const": 0},
        # a padded batch of odd size with zero, copy and const experts, rows that are no multiple of 16 bytes
        {"name": "combine gradient 4x515 special", "op": "combine_backward", "ranks": 4, "tokens": 515,
         "experts_per_rank": 5, "topk": 6, "h": 1037, "dtype": "fp16", "masked": True, "zero": 1, "copy": 2,
         "const": 3},
        # the same three steps one call further back: the gradient of the tokens
        {"name": "dispatch gradient 8x1", "op": "dispatch_backward", "ranks": 8, "tokens": 1, "experts_per_rank": 8,
         "topk": 8, "h": 7168, "dtype": "bf16", "masked": False, "special": 0, "add": False, "scales": False},
        {"name": "dispatch gradient 16x256", "op": "dispatch_backward", "ranks": 16, "tokens": 256,
         "experts_per_rank": 16, "topk": 8, "h": 7168, "dtype": "bf16", "masked": False, "special": 0, "add": False,
         "scales": False},
        # with what else flows back to the tokens (a residual, copy experts), and the moved weights' gradient
        {"name": "dispatch gradient 4x515 add", "op": "dispatch_backward", "ranks": 4, "tokens": 515,
         "experts_per_rank": 5, "topk": 6, "h": 1037, "dtype": "fp16", "masked": True, "special": 6, "add": True,
         "scales": True},
        # one token on each of 2 ranks: single-token decode, bound by the weights of the experts hit
        {"name": "int8 product 2 tokens", "op": "product", "ranks": 2, "tokens": 1, "experts_per_rank": 4, "topk": 4,
         "k": 7168, "n": 4096, "activation": True, "dtype": "bf16", "routing": "uniform", "masked": False,
         "row_scales": True},
        # 8 ranks x 32 tokens: the first product on the int8 rows that dispatch writes
        {"name": "int8 product 8x32 up", "op": "product", "ranks": 8, "tokens": 32, "experts_per_rank": 8, "topk": 8,
         "k": 7168, "n": 4096, "activation": True, "dtype": "bf16", "routing": "uniform", "masked": False,
         "row_scales": True},
        # 16 ranks x 256 tokens with a quarter of the pairs masked: the second product, rows left behind the last
        {"name": "int8 product 16x256 down", "op": "product", "ranks": 16, "tokens": 256, "experts_per_rank": 16,
         "topk": 8, "k": 2048, "n": 7168, "activation": False, "dtype": "bf16", "routing": "uniform", "masked": True,
         "row_scales": True},
        # 8 ranks x 1024 tokens, Zipf routing: long prefill with one very popular expert
        {"name": "int8 product 8x1024 up zipf", "op": "product", "ranks": 8, "tokens": 1024, "experts_per_rank": 8,
         "topk": 8, "k": 7168, "n": 4096, "activation": True, "dtype": "bf16", "routing": "zipf", "masked": False,
         "row_scales": True},
        # the rows between two products of 8 ranks x 4 tokens, top-8
        {"name": "int8 rows 256 x 2048", "op": "quantize", "rows": 256, "cols": 2048, "dtype": "bf16"},
        # every row of 16 ranks x 256 tokens, top-8
        {"name": "int8 rows 32768 x 7168", "op": "quantize", "rows": 32768, "cols": 7168, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["combine_backward", "dispatch_backward", "product", "product", "quantize"])
    ranks = rng.choice([2, 4, 8, 16])
    if op in ("combine_backward", "dispatch_backward"):
        h = rng.choice([8 * _log(rng, 2, 896), 8 * _log(rng, 2, 896), _log(rng, 1, 2400)])
        epr = rng.randint(1, 16)
        topk = rng.randint(1, min(8, ranks * epr))
        case = {"op": op, "ranks": ranks, "tokens": _log(rng, 1, 4096 // ranks), "experts_per_rank": epr, "topk": topk,
                "h": h, "dtype": rng.choice(["bf16", "fp16"]), "masked": rng.random() < 0.4}
        special = rng.random() < 0.4
        if op == "combine_backward":
            return dict(case, zero=rng.randint(0, 2) if special else 0, copy=rng.randint(0, 2) if special else 0,
                        const=rng.randint(0, 16) if special else 0)
        return dict(case, special=rng.randint(1, 6) if special else 0, add=rng.random() < 0.5,
                    scales=rng.random() < 0.3)
    if op == "quantize":
        return {"op": op, "rows": _log(rng, 1, 32768), "cols": 16 * _log(rng, 1, 448),
                "dtype": rng.choice(["bf16", "bf16", "fp16", "fp32"])}
    epr = rng.choice([1, 2, 4, 8][:3 if ranks == 16 else 4])
    topk = rng.randint(1, min(8, ranks * epr))
    return {"op": op, "ranks": ranks, "tokens": _log(rng, 1, 8192 // ranks), "experts_per_rank": epr, "topk": topk,
            "k": 16 * _log(rng, 8, 448), "n": 2 * _log(rng, 64, 2048), "activation": rng.random() < 0.5,
            "dtype": rng.choice(["bf16", "fp16"]), "routing": rng.choice(["uniform", "zipf"]),
            "masked": rng.random() < 0.3, "row_scales": rng.random() < 0.8}


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(0xACE5 + 7919 * int(seed))


def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(shape, generator=g, device=DEV, dtype=dtype)


def _rand(g, *shape):
    return torch.rand(shape, generator=g, device=DEV)


# ---- inputs ----

def _special(case):
    return case["zero"] + case["copy"] + case["const"] if case["op"] == "combine_backward" else case.get("special", 0)


def _routing(case, g):
    """What dispatch leaves behind: ids, weights, mask, assist_info, ep_recv_count, and the most rows of an expert."""
    W, bs, epr, K = case["ranks"], case["tokens"], case["experts_per_rank"], case["topk"]
    E, N = W * epr, W * bs
    z = _randn(g, N, E + _special(case))
    if case.get("routing") == "zipf":
        z = z - 1.2 * torch.arange(1, E + 1, device=DEV, dtype=torch.float32).log()
    top, ids = z.sort(dim=1, descending=True, stable=True)
    w = torch.softmax(top[:, :K], dim=1)
    ids = ids[:, :K].contiguous()
    mask = _rand(g, N, K) < 0.75 if case["masked"] else None
    on = ids < E if mask is None else mask & (ids < E)
    # rows by rank, local expert, source rank and token: by (expert, token), the missing pairs behind all others
    t = torch.arange(N, device=DEV)[:, None]
    key = torch.where(on, ids * N + t, (E + 1) * N).flatten()
    pair = key.argsort(stable=True)
    live = torch.arange(N * K, device=DEV) < on.sum()
    token = pair // K
    assist = torch.stack((token // bs, token % bs, pair % K), 1)
    assist = torch.where(live[:, None], assist, 0).to(torch.int32).contiguous()
    seg = torch.bincount((ids * W + t // bs)[on], minlength=E * W)          # (expert, source rank), rank-major
    counts = seg.view(W, epr * W).cumsum(1).to(torch.int32).contiguous()
    return ids.to(torch.int32), w.contiguous(), mask, assist, counts, int(seg.view(E, W).sum(1).max())


def prepare(case, seed):
    g = _gen(seed)
    op, dtype = case["op"], DTYPES[case["dtype"]]
    if op == "quantize":
        # activations: a normal, rows of different size, a few columns that stand out, and a row of zeros
        x = _randn(g, case["rows"], case["cols"]) * torch.exp(_randn(g, case["rows"], 1))
        x = x * torch.where(_rand(g, 1, case["cols"]) < 0.01, 20.0, 1.0)
        x[case["rows"] // 2] *= 0.0 if case["rows"] > 1 else 1.0
        return {"case": case, "x": x.to(dtype)}
    ids, w, mask, assist, counts, most = _routing(case, g)
    N, K = ids.shape
    s = {"case": case, "ids": ids, "weights": w, "mask": mask, "assist": assist, "counts": counts, "most": most}
    if op == "combine_backward":
        h = case["h"]
        s["rows"] = _randn(g, N * K, h, dtype=dtype)
        s["grad"] = (_randn(g, N, h) * torch.exp(_randn(g, N, 1))).to(dtype)
        s["x"] = _randn(g, N, h, dtype=dtype) if case["copy"] else None
        s["const_x"] = _randn(g, case["const"], h, dtype=dtype) if case["const"] else None
        s["grad_rows"] = torch.zeros((N * K, h), dtype=dtype, device=DEV)
        return s
    if op == "dispatch_backward":
        h = case["h"]
        s["grad"] = _randn(g, N * K, h, dtype=dtype)
        s["add"] = _randn(g, N, h, dtype=dtype) if case["add"] else None
        s["grad_scales"] = _randn(g, N * K) if case["scales"] else None
        return s
    E, k, n = case["ranks"] * case["experts_per_rank"], case["k"], case["n"]
    # codes as they come out of rows whose largest element is 127
    s["x"] = (_randn(g, N * K, k, dtype=torch.bfloat16) * 32).round().clamp(-127, 127).to(torch.int8)
    s["xs"] = torch.exp(_randn(g, N * K) * 0.5) * (4.0 / 127) if case["row_scales"] else None
    s["w"] = torch.empty((E, n, k), dtype=torch.int8, device=DEV)
    for e in range(E):
        s["w"][e] = (_randn(g, n, k, dtype=torch.bfloat16) * 32).round().clamp(-127, 127).to(torch.int8)
    s["ws"] = torch.exp(_randn(g, E, n) * 0.2) * (k ** -0.5 / (32 if case["row_scales"] else 1024))
    s["out"] = torch.zeros((N * K, n // 2 if case["activation"] else n), dtype=dtype, device=DEV)
    return s


# ---- the plain forms ----

def _live(s):
    """(rows that exist, the pair of each row: one past the last where there is none)."""
    bs, (N, K) = s["case"]["tokens"], s["ids"].shape
    live = torch.arange(N * K, device=DEV) < s["counts"][:, -1].sum()
    a = s["assist"].long()
    return live, torch.where(live, (a[:, 0] * bs + a[:, 1]) * K + a[:, 2], N * K)


def _combine_backward_plain(case, s):
    ids, w, g = s["ids"].long(), s["weights"], s["grad"].float()
    N, K = ids.shape
    live, pair = _live(s)
    p = pair.clamp(max=N * K - 1)
    gt = g[p // K]
    rows = torch.where(live[:, None], (w.flatten()[p][:, None] * gt).to(s["grad"].dtype), s["grad_rows"])
    gw = torch.zeros(N * K + 1, device=DEV).scatter_(0, pair, (s["rows"].float() * gt).sum(1))[:-1].view(N, K)
    on = torch.ones_like(ids, dtype=torch.bool) if s["mask"] is None else s["mask"]
    first = case["ranks"] * case["experts_per_rank"] + case["zero"]
    out = [rows]
    if case["copy"]:
        is_copy = on & (ids >= first) & (ids < first + case["copy"])
        gw = torch.where(is_copy, (s["x"].float() * g).sum(1, keepdim=True), gw)
        out.append((torch.where(is_copy, w, 0.0).sum(1, keepdim=True) * g).to(s["x"].dtype))
    if case["const"]:
        c = ids - first - case["copy"]
        is_const = on & (c >= 0)
        c = c.clamp(min=0)
        gw = torch.where(is_const, (g @ s["const_x"].float().t().contiguous()).gather(1, c), gw)
        share = torch.zeros((N, case["const"]), dtype=torch.float64, device=DEV)
        share.scatter_add_(1, c, torch.where(is_const, w, 0.0).double())
        out.append((share.t().contiguous() @ g.double()).to(s["const_x"].dtype))
    return [gw] + out


def _dispatch_backward_plain(case, s):
    N, K = s["ids"].shape
    _, pair = _live(s)
    # the row of each pair; pairs without one read a row of zeros behind the last
    row = torch.full((N * K + 1,), N * K, device=DEV).scatter_(0, pair, torch.arange(N * K, device=DEV))[:-1].view(N, K)
    row = torch.where(_has_row(case, s), row, N * K)
    g = torch.cat((s["grad"].float(), torch.zeros((1, case["h"]), device=DEV)))
    total = g[row].sum(1)
    if s["add"] is not None:
        total = total + s["add"].float()
    out = [total.to(s["grad"].dtype)]
    if s["grad_scales"] is not None:
        out.append(torch.cat((s["grad_scales"], torch.zeros(1, device=DEV)))[row])
    return out


def _has_row(case, s):
    real = s["ids"] < case["ranks"] * case["experts_per_rank"]
    return real if s["mask"] is None else real & s["mask"]


def _product_plain(case, s):
    counts, out = s["counts"], s["out"]
    W, E = counts.shape[0], s["w"].shape[0]
    base = (counts[:, -1].cumsum(0) - counts[:, -1])[:, None]
    ends = (counts[:, W - 1::W] + base).reshape(E).contiguous()   # one past each expert's last row
    row = torch.arange(out.shape[0], device=DEV, dtype=torch.int32)
    expert = torch.searchsorted(ends, row, right=True)
    start = torch.cat((ends.new_zeros(1), ends))
    m = max(s["most"], 1)
    # every expert's rows, padded to the longest: row p of expert e is input row start[e] + p
    index = (start[:E, None] + torch.arange(m, device=DEV)).clamp(max=out.shape[0] - 1)
    padded = s["x"][index].transpose(1, 2).contiguous().float()
    y = torch.bmm(s["w"].float(), padded) * s["ws"][:, :, None]   # [expert, n, row]
    if s["xs"] is not None:
        y = y * s["xs"][index][:, None, :]
    if case["activation"]:
        gate, up = y.chunk(2, dim=1)
        y = gate / (1.0 + torch.exp(-gate)) * up
    live = expert < E
    expert = expert.clamp(max=E - 1)
    rows = y.transpose(1, 2)[expert, (row - start[expert]).clamp(0, m - 1)]
    return torch.where(live[:, None], rows.to(out.dtype), out)


def _quantize_plain(s):
    x = s["x"].float()
    scale = x.abs().amax(1, keepdim=True) / 127.0
    codes = torch.where(scale > 0, torch.round(x / scale), 0.0).clamp(-127, 127)
    return (codes * scale).bfloat16(), scale[:, 0]


def run(state):
    case = state["case"]
    if own:
        return _own(case, state)
    if case["op"] == "combine_backward":
        return _combine_backward_plain(case, state)
    if case["op"] == "dispatch_backward":
        return _dispatch_backward_plain(case, state)
    if case["op"] == "quantize":
        return _quantize_plain(state)
    return _product_plain(case, state)


def _own(case, s):
    import combine_ep_recv_amd as moe

    if case["op"] == "combine_backward":
        gw = torch.empty_like(s["weights"])
        ori = torch.empty_like(s["x"]) if case["copy"] else None
        const = torch.empty_like(s["const_x"]) if case["const"] else None
        moe.combine_backward_into(s["grad_rows"], gw, s["grad"], s["rows"], s["assist"], s["counts"], s["ids"],
                                  s["weights"], case["ranks"], case["experts_per_rank"], x_active_mask=s["mask"],
                                  zero_experts=case["zero"], copy_experts=case["copy"], ori_x=s["x"], grad_ori_x=ori,
                                  const_experts=case["const"], const_x=s["const_x"], grad_const_x=const)
        return [gw, s["grad_rows"]] + [v for v in (ori, const) if v is not None]
    if case["op"] == "dispatch_backward":
        out = moe.dispatch_backward(s["grad"], s["assist"], s["counts"], s["ids"], case["ranks"],
                                    case["experts_per_rank"], x_active_mask=s["mask"], add=s["add"],
                                    grad_expand_scales=s["grad_scales"])
        return list(out) if isinstance(out, tuple) else [out]
    if case["op"] == "quantize":
        codes, scales = moe.quantize_int8(s["x"])
        return moe.dequantize_int8(codes, scales, torch.bfloat16), scales    # the values that the codes stand for
    act = moe.MOE_ACT_SWIGLU if case["activation"] else moe.MOE_ACT_NONE
    return moe.expert_product_into(s["out"], s["x"], s["xs"], s["w"], s["ws"], s["counts"], activation=act)


# ---- what a pass cannot do without ----

def _share(case):
    """The part of all pairs that has a row, as expected from the routing."""
    E = case["ranks"] * case["experts_per_rank"]
    return (0.75 if case["masked"] else 1.0) * E / (E + _special(case))


def _hit(case):
    """Experts that get a row, as expected from the routing: (experts, rows)."""
    E, N, K = case["ranks"] * case["experts_per_rank"], case["ranks"] * case["tokens"], case["topk"]
    p = np.arange(1, E + 1) ** (-1.2 if case["routing"] == "zipf" else 0.0)
    keep = 0.75 if case["masked"] else 1.0
    p = np.minimum(1.0, keep * K * p / p.sum())
    return float((1.0 - (1.0 - p) ** N).sum()), N * K * keep


def work(case):
    if case["op"] == "quantize":
        n, size = case["rows"] * case["cols"], DTYPES[case["dtype"]].itemsize
        return {"bytes": n * (size + 1) + 4 * case["rows"] + n * (1 + 2) + 4 * case["rows"], "flops": 4.0 * n}
    N, K, E = case["ranks"] * case["tokens"], case["topk"], case["ranks"] * case["experts_per_rank"]
    if case["op"] == "product":
        hit, rows = _hit(case)
        k, n = case["k"], case["n"]
        made = n // 2 if case["activation"] else n
        return {"bytes": hit * n * (k + 4) + rows * (k + (4 if case["row_scales"] else 0) + made * 2)
                + case["ranks"] * E * 4, "flops": 2.0 * rows * n * k}
    h, rows = case["h"], N * K * _share(case)
    routing = rows * 12 + N * K * (5 if case["masked"] else 4) + case["ranks"] * E * 4
    if case["op"] == "dispatch_backward":
        moved = rows * h * 2 + N * h * (4 if case["add"] else 2) + (rows + N * K) * (4 if case["scales"] else 0)
        return {"bytes": moved + routing, "flops": float(rows * h)}
    pairs = N * K * (0.75 if case["masked"] else 1.0) / (E + _special(case))     # pairs of each special expert
    copied = min(N, pairs * case["copy"])
    moved = 2 * rows * h * 2 + N * h * 2 + N * K * 8
    if case["copy"]:
        moved += copied * h * 2 + N * h * 2
    return {"bytes": moved + 4 * case["const"] * h + routing,
            "flops": 3.0 * h * (rows + pairs * (case["copy"] + case["const"]))}


# ---- the definitions, in binary64 ----

def _exact_rows(case, s):
    """The row of each pair from the ids alone, -1 where there is none: rows lie by (expert, token)."""
    N, K = s["ids"].shape
    ids = s["ids"].cpu().numpy().astype(np.int64)
    on = ids < case["ranks"] * case["experts_per_rank"]
    if s["mask"] is not None:
        on &= s["mask"].cpu().numpy()
    t, k = np.nonzero(on)
    order = np.lexsort((t, ids[t, k]))
    row = np.full((N, K), -1, dtype=np.int64)
    row[t[order], k[order]] = np.arange(len(order))
    return torch.from_numpy(row).to(DEV)


def _exact_combine_backward(case, s):
    row, w, g = _exact_rows(case, s), s["weights"].double(), s["grad"].double()
    N, K = row.shape
    ids, on = s["ids"].long(), (torch.ones_like(row) if s["mask"] is None else s["mask"]).bool()
    zero_end = case["ranks"] * case["experts_per_rank"] + case["zero"]
    copy_end = zero_end + case["copy"]
    rows = s["grad_rows"].double()
    gw = torch.zeros((N, K), dtype=torch.float64, device=DEV)
    ori = torch.zeros_like(g)
    const = torch.zeros((case["const"], case["h"]), dtype=torch.float64, device=DEV)
    for k in range(K):
        at = row[:, k]
        t = torch.nonzero(at >= 0)[:, 0]
        rows[at[t]] = w[t, k, None] * g[t]
        gw[t, k] = torch.linalg.vecdot(s["rows"][at[t]].double(), g[t])
        t = torch.nonzero(on[:, k] & (ids[:, k] >= zero_end) & (ids[:, k] < copy_end))[:, 0]
        if len(t):
            gw[t, k] = torch.linalg.vecdot(s["x"][t].double(), g[t])
            ori[t] += w[t, k, None] * g[t]
        for j in range(case["const"]):
            t = torch.nonzero(on[:, k] & (ids[:, k] == copy_end + j))[:, 0]
            gw[t, k] = torch.linalg.vecdot(s["const_x"][j].double().expand(len(t), -1), g[t])
            const[j] += (w[t, k, None] * g[t]).sum(0)
    return [gw, rows] + ([ori] if case["copy"] else []) + ([const] if case["const"] else [])


def _exact_dispatch_backward(case, s):
    row = _exact_rows(case, s)
    total = torch.zeros((row.shape[0], case["h"]), dtype=torch.float64, device=DEV)
    if s["add"] is not None:
        total += s["add"].double()
    scales = torch.zeros(row.shape, dtype=torch.float64, device=DEV)
    for k in range(row.shape[1]):
        t = torch.nonzero(row[:, k] >= 0)[:, 0]
        total[t] += s["grad"][row[t, k]].double()
        if s["grad_scales"] is not None:
            scales[t, k] = s["grad_scales"][row[t, k]].double()
    return [total] + ([scales] if s["grad_scales"] is not None else [])


def _exact_product(case, s):
    W = case["ranks"]
    counts = s["counts"].cpu().numpy().astype(np.int64)
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
    row = 0
    for r in range(W):
        first = row
        for el in range(case["experts_per_rank"]):
            end = first + int(counts[r, (el + 1) * W - 1])
            if end > row:
                e = r * case["experts_per_rank"] + el
                y = s["x"][row:end].double() @ s["w"][e].double().t() * s["ws"][e].double()
                if s["xs"] is not None:
                    y = y * s["xs"][row:end, None].double()
                if case["activation"]:
                    half = y.shape[1] // 2
                    y = y[:, :half] * torch.sigmoid(y[:, :half]) * y[:, half:]
                out[row:end] = y
            row = end
    return out


def _exact_quantize(case, s):
    # the definition divides in binary32 and rounds what that gives: a quotient next to a half goes by it
    x = s["x"].float().cpu().numpy()
    scale = (np.abs(x).max(1, keepdims=True) / np.float32(127)).astype(np.float32)
    with np.errstate(divide="ignore", invalid="ignore"):
        codes = np.where(scale > 0, np.rint(x / scale), 0).clip(-127, 127)
    value = codes.astype(np.float64) * scale.astype(np.float64)
    return torch.from_numpy(value), torch.from_numpy(scale[:, 0].astype(np.float64))


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "combine_backward":
        return _exact_combine_backward(case, s)
    if case["op"] == "dispatch_backward":
        return _exact_dispatch_backward(case, s)
    if case["op"] == "quantize":
        return _exact_quantize(case, s)
    return _exact_product(case, s)

"""The gate: choice of experts and weights from a router's logits, and its gradient.

The plain implementation below works in binary64 on the CPU, one token at a time, from the definition in
include/moe_ep.h. Ids and pair masks must be equal to it.

Tolerances, u = 2^-24 (half a step of fp32). A weight's score is exp(l - m) / Z: the difference carries one rounding,
which exp turns into a relative |l - m| u; exp itself, the products and the division take a few roundings, and the sum
over E experts at most E / 64 + 6 in a row. Weights are allowed (|l - m| + E / 64 + 16) u, twice that where they are
renormalised. A gradient is a product of such a weight and a difference whose terms add up to A = |g| + sum |g w|; it
is allowed the same count of u times the product of the magnitudes, then half a step of the logits' type.
"""
import ctypes
import itertools

import numpy as np
import pytest
import torch

import combine_ep_recv_amd as moe

DEV = "cuda"
U = 2.0 ** -24
SOFTMAX, SIGMOID = moe.MOE_SCORE_SOFTMAX, moe.MOE_SCORE_SIGMOID
MAX, TOP2 = moe.MOE_GROUP_MAX, moe.MOE_GROUP_TOP2
TYPES = [torch.bfloat16, torch.float16, torch.float32]


def scores(l, score):
    """Scores of one token's logits in binary64; logits of -inf and NaN are not there."""
    l = np.asarray(l, np.float64)
    there = l > -np.inf
    s = np.zeros_like(l)
    if not there.any():
        return s, there
    if score == SIGMOID:
        with np.errstate(over="ignore"):
            s[there] = 1.0 / (1.0 + np.exp(-l[there]))
        return s, there
    m = l[there].max()
    with np.errstate(invalid="ignore"):
        e = np.where(l[there] == m, 1.0, np.exp(l[there] - m))
    s[there] = e / e.sum()
    return s, there


def plain_gate(logits, topk, score=SOFTMAX, bias=None, groups=1, topk_groups=1, group_score=MAX, renormalize=True,
               scale=1.0, token_mask=None):
    L = logits.detach().cpu().double().numpy()
    B = None if bias is None else bias.detach().cpu().double().numpy()
    N, E = L.shape
    ids, w = np.full((N, topk), -1, np.int32), np.zeros((N, topk))
    for t in range(N):
        if token_mask is not None and not token_mask[t]:
            continue
        s, there = scores(L[t], score)
        c = s + B if B is not None else np.where(there, L[t], 0.0)
        v = s + B if B is not None else (s if group_score == TOP2 else c)
        ok = there & (np.ones(E, bool) if B is None else B > -np.inf)
        cand = [e for e in range(E) if ok[e]]
        if topk_groups < groups:
            size, worth = E // groups, {}
            for e in cand:
                worth.setdefault(e // size, []).append(v[e])
            value = {g: (sum(sorted(x, reverse=True)[:2]) if group_score == TOP2 else max(x))
                     for g, x in worth.items()}
            best = sorted(value, key=lambda g: (-value[g], g))[:topk_groups]
            cand = [e for e in cand if e // size in best]
        cand = sorted(cand, key=lambda e: (-c[e], e))[:topk]
        total = sum(s[e] for e in cand)
        for k, e in enumerate(cand):
            ids[t, k] = e
            w[t, k] = scale * (s[e] if not renormalize else (s[e] / total if total > 0 else 0.0))
    return ids, w


def plain_backward(logits, ids, w, grad, score, renormalize, scale):
    """(gradient, magnitude that its rounding errors scale with), binary64."""
    L, W, G = (x.detach().cpu().double().numpy() for x in (logits, w, grad))
    I = ids.cpu().numpy()
    out, mag = np.zeros_like(L), np.zeros_like(L)
    for t in range(L.shape[0]):
        on = [k for k in range(I.shape[1]) if 0 <= I[t, k] < L.shape[1]]
        if not on:
            continue
        s, _ = scores(L[t], score)
        D = sum(G[t, k] * W[t, k] for k in on)
        A = sum(abs(G[t, k] * W[t, k]) for k in on)
        if score == SOFTMAX and not renormalize:
            g = np.zeros(L.shape[1])
            for k in on:
                g[I[t, k]] += scale * G[t, k]
            out[t], mag[t] = s * (g - D), s * (np.abs(g) + A)
            continue
        for k in on:
            e = I[t, k]
            if renormalize:
                d, m = W[t, k] * (G[t, k] - D / scale), abs(W[t, k]) * (abs(G[t, k]) + A / abs(scale))
                f = 1.0 - s[e] if score == SIGMOID else 1.0
                if score == SIGMOID:
                    f = 1.0 / (1.0 + np.exp(L[t, e]))          # 1 - s without the cancellation
            else:
                f = s[e] / (1.0 + np.exp(L[t, e]))
                d, m = scale * G[t, k], abs(scale * G[t, k])
            out[t, e] += d * f
            mag[t, e] += m * f
    return out, mag


def draw(N, E, dtype, seed, spread=1.5):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(N, E, generator=g) * spread).to(dtype)


def check(logits, ids, w, pair=None, **kw):
    N, E = logits.shape
    want, ww = plain_gate(logits, ids.shape[1], **kw)
    got = ids.cpu().numpy()
    assert (got == want).all(), (np.argwhere(got != want)[:5], got[(got != want).any(1)][:2], want[(got != want).any(1)][:2])
    L = logits.cpu().double().numpy()
    top = np.max(np.where(L > -np.inf, L, -1e9), axis=1, keepdims=True)
    far = np.abs(np.take_along_axis(L, np.maximum(want, 0), 1) - top)
    far = np.where(np.isfinite(far), far, 0.0)
    room = (far + E / 64 + 16) * U * (2 if kw.get("renormalize", True) else 1)
    if kw.get("renormalize", True):
        room = np.broadcast_to(room.max(1, keepdims=True), want.shape)
    err = np.abs(w.cpu().double().numpy() - ww)
    assert (err <= room * np.abs(ww) + 2.0 ** -149).all(), (err.max(), (err / np.maximum(np.abs(ww), 1e-300)).max())
    if pair is not None:
        assert (pair.cpu().numpy().astype(bool) == (want >= 0)).all()


# ---- host only: refusals ----

A = 1 << 20


def _c_gate(**kw):
    p = dict(logits=A, bias=None, mask=None, N=4, E=16, K=2, dtype=2, score=0, groups=1, tg=1, gs=0, renorm=1, scale=1.0,
             ids=2 * A, w=3 * A, pm=None)
    p.update(kw)
    P = lambda v: None if v is None else ctypes.c_void_p(v)
    return moe.library().moe_gate(P(p["logits"]), P(p["bias"]), P(p["mask"]), p["N"], p["E"], p["K"], p["dtype"],
                                  p["score"], p["groups"], p["tg"], p["gs"], p["renorm"], p["scale"], P(p["ids"]),
                                  P(p["w"]), P(p["pm"]), None)


@pytest.mark.parametrize("kw,want", [
    (dict(N=-1), moe.MOE_ERR_SHAPE), (dict(N=1 << 24), moe.MOE_ERR_SHAPE), (dict(E=0), moe.MOE_ERR_SHAPE),
    (dict(E=2049), moe.MOE_ERR_SHAPE), (dict(K=0), moe.MOE_ERR_SHAPE), (dict(K=17), moe.MOE_ERR_SHAPE),
    (dict(E=128, K=65), moe.MOE_ERR_SHAPE), (dict(groups=3), moe.MOE_ERR_SHAPE), (dict(groups=0), moe.MOE_ERR_SHAPE),
    (dict(E=130, groups=65), moe.MOE_ERR_SHAPE), (dict(groups=4, tg=5), moe.MOE_ERR_SHAPE),
    (dict(groups=4, tg=0), moe.MOE_ERR_SHAPE), (dict(groups=16, tg=1), moe.MOE_ERR_SHAPE),
    (dict(gs=2), moe.MOE_ERR_SHAPE), (dict(score=2), moe.MOE_ERR_SHAPE), (dict(dtype=0), moe.MOE_ERR_DTYPE),
    (dict(dtype=4), moe.MOE_ERR_DTYPE), (dict(scale=0.0), moe.MOE_ERR_SHAPE),
    (dict(scale=float("nan")), moe.MOE_ERR_SHAPE), (dict(scale=float("inf")), moe.MOE_ERR_SHAPE),
    (dict(logits=None), moe.MOE_ERR_NULLPTR), (dict(ids=None), moe.MOE_ERR_NULLPTR),
    (dict(w=None), moe.MOE_ERR_NULLPTR), (dict(logits=A + 1), moe.MOE_ERR_ALIGN),
    (dict(bias=A + 2), moe.MOE_ERR_ALIGN), (dict(dtype=3, logits=A + 2), moe.MOE_ERR_ALIGN),
    (dict(N=0, logits=None, ids=None, w=None), moe.MOE_OK),
])
def test_gate_refuses_before_a_launch(kw, want):
    assert _c_gate(**kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(N=-1), moe.MOE_ERR_SHAPE), (dict(E=2049), moe.MOE_ERR_SHAPE), (dict(K=0), moe.MOE_ERR_SHAPE),
    (dict(dtype=0), moe.MOE_ERR_DTYPE), (dict(score=-1), moe.MOE_ERR_SHAPE), (dict(scale=0.0), moe.MOE_ERR_SHAPE),
    (dict(grad=None), moe.MOE_ERR_NULLPTR), (dict(out=None), moe.MOE_ERR_NULLPTR),
    (dict(out=A + 1), moe.MOE_ERR_ALIGN), (dict(N=0, out=None), moe.MOE_OK),
])
def test_gate_backward_refuses_before_a_launch(kw, want):
    p = dict(logits=A, ids=2 * A, w=3 * A, grad=4 * A, N=4, E=16, K=2, dtype=2, score=0, renorm=1, scale=1.0, out=5 * A)
    p.update(kw)
    P = lambda v: None if v is None else ctypes.c_void_p(v)
    assert moe.library().moe_gate_backward(P(p["logits"]), P(p["ids"]), P(p["w"]), P(p["grad"]), p["N"], p["E"], p["K"],
                                           p["dtype"], p["score"], p["renorm"], p["scale"], P(p["out"]), None) == want


class _Recorder:
    def __init__(self):
        self.calls = []
        self.moe_status_str = moe.library().moe_status_str

    def __getattr__(self, name):
        def call(*args):
            self.calls.append(name)
            return moe.MOE_OK
        return call


@pytest.fixture
def rec(monkeypatch):
    r = _Recorder()
    monkeypatch.setattr(moe, "library", lambda: r)
    monkeypatch.setattr(moe, "_gpu_device", lambda name, t: t.device)
    monkeypatch.setattr(moe, "_stream_ptr", lambda device: 0)
    return r


def _gate_args(N=4, E=16, K=2):
    return dict(expert_ids=torch.zeros((N, K), dtype=torch.int32), expert_scales=torch.zeros((N, K)),
                logits=torch.zeros((N, E), dtype=torch.bfloat16))


def test_well_formed_gate_calls_reach_the_library(rec):
    moe.gate_into(**_gate_args(), bias=torch.zeros(16), token_mask=torch.ones(4, dtype=torch.bool),
                  pair_mask=torch.zeros((4, 2), dtype=torch.uint8))
    ids, w, on = moe.gate(torch.zeros(4, 16), 2, with_pair_mask=True)
    assert ids.shape == w.shape == on.shape == (4, 2) and on.dtype == torch.bool
    g = moe.gate_backward(torch.zeros(4, 16), ids, w, w)
    assert g.shape == (4, 16) and rec.calls == ["moe_gate", "moe_gate", "moe_gate_backward"]


@pytest.mark.parametrize("field,value", [
    ("logits", torch.zeros((4, 16), dtype=torch.float64)), ("logits", torch.zeros((16, 4)).t()),
    ("logits", torch.zeros(16)), ("expert_ids", torch.zeros((4, 2), dtype=torch.int64)),
    ("expert_ids", torch.zeros((3, 2), dtype=torch.int32)), ("expert_scales", torch.zeros((4, 3))),
    ("expert_scales", torch.zeros((4, 2), dtype=torch.float16)), ("bias", torch.zeros(15)),
    ("bias", torch.zeros(16, dtype=torch.bfloat16)), ("token_mask", torch.zeros(5, dtype=torch.bool)),
    ("token_mask", torch.zeros(4)), ("pair_mask", torch.zeros((4, 3), dtype=torch.bool)),
    ("pair_mask", torch.zeros((4, 2), dtype=torch.int32)),
], ids=lambda v: v if isinstance(v, str) else "")
def test_gate_into_rejects_before_the_call(rec, field, value):
    args = _gate_args()
    args[field] = value
    with pytest.raises(moe.MoeError):
        moe.gate_into(**args)
    assert rec.calls == []


def test_gate_rejects_cpu_tensors_and_bad_topk():
    with pytest.raises(moe.MoeError):
        moe.gate(torch.zeros(4, 16), 2)
    with pytest.raises(moe.MoeError):
        moe.gate_backward(torch.zeros(4, 16), torch.zeros((4, 2), dtype=torch.int32), torch.zeros(4, 2), torch.zeros(4, 2))


def test_the_plain_gradient_is_the_gates_derivative():
    """plain_backward against central differences of plain_gate's weights, step 1e-5 in binary64: the quotient is
    off by h^2 / 6 times the third derivative (at most about 10 here), under 1e-8, and by 1e-16 / h = 1e-11."""
    for score, renorm in itertools.product((SOFTMAX, SIGMOID), (True, False)):
        L = draw(3, 12, torch.float64, 5)
        grad = torch.randn(3, 4, generator=torch.Generator().manual_seed(1), dtype=torch.float64)
        kw = dict(score=score, renormalize=renorm, scale=1.7)
        ids, w = plain_gate(L, 4, **kw)
        got, _ = plain_backward(L, torch.from_numpy(ids), torch.from_numpy(w), grad, score, renorm, 1.7)
        for t, e in itertools.product(range(3), range(12)):
            ends = []
            for h in (1e-5, -1e-5):
                M = L.clone()
                M[t, e] += h
                i2, w2 = plain_gate(M, 4, **kw)
                assert (i2 == ids).all()
                ends.append((w2 * grad.numpy()).sum())
            assert abs((ends[0] - ends[1]) / 2e-5 - got[t, e]) < 1e-7


# ---- GPU ----

@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID])
@pytest.mark.parametrize("N,E,K", [(1, 1, 1), (1, 8, 8), (3, 63, 5), (5, 64, 8), (7, 65, 64), (129, 128, 1), (65, 256, 8),
                                   (33, 304, 8), (9, 385, 6), (6, 1000, 16), (2, 1025, 8), (3, 2048, 64)])
def test_gate_matches_the_definition(dtype, score, N, E, K):
    L = draw(N, E, dtype, 100 + N)
    for bias, renorm in ((False, True), (True, False)):
        b = torch.randn(E, generator=torch.Generator().manual_seed(2)) * 0.05 if bias else None
        kw = dict(score=score, renormalize=renorm, scale=2.5 if bias else 1.0)
        ids, w, on = moe.gate(L.to(DEV), K, bias=None if b is None else b.to(DEV), with_pair_mask=True, **kw)
        check(L, ids, w, on, bias=b, **kw)


@pytest.mark.gpu
@pytest.mark.parametrize("E,groups,topk_groups,K", [(64, 8, 3, 8), (256, 8, 4, 8), (256, 32, 2, 3), (60, 6, 2, 7),
                                                    (64, 64, 5, 5), (130, 2, 1, 9), (1024, 16, 4, 8), (63, 7, 7, 4),
                                                    (305, 5, 2, 8), (2048, 64, 8, 16)])
@pytest.mark.parametrize("group_score", [MAX, TOP2])
def test_gate_groups(E, groups, topk_groups, K, group_score):
    for seed, (score, bias, dtype) in enumerate(itertools.product((SOFTMAX, SIGMOID), (False, True),
                                                                  (torch.bfloat16, torch.float32))):
        L = draw(21, E, dtype, seed)
        b = torch.randn(E, generator=torch.Generator().manual_seed(3)) * 0.03 if bias else None
        kw = dict(score=score, groups=groups, topk_groups=topk_groups, group_score=group_score)
        ids, w = moe.gate(L.to(DEV), K, bias=None if b is None else b.to(DEV), **kw)
        check(L, ids, w, bias=b, **kw)


@pytest.mark.gpu
@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID])
@pytest.mark.parametrize("groups", [1, 4])
def test_gate_ties_go_to_the_lower_id(score, groups):
    """Few distinct logits, biases that are equal, zero or on a grid: many exact ties, and ties of sums."""
    g = torch.Generator().manual_seed(9)
    L = torch.randint(-2, 3, (64, 256), generator=g).float()
    for b in (None, torch.zeros(256), torch.full((256,), -0.25), torch.randint(0, 2, (256,), generator=g) * 0.5):
        kw = dict(score=score, groups=groups, topk_groups=1 if groups == 1 else 2, group_score=TOP2)
        ids, w = moe.gate(L.to(DEV), 8, bias=None if b is None else b.to(DEV), **kw)
        check(L, ids, w, bias=b, **kw)
    L = torch.zeros(3, 100)
    ids, w = moe.gate(L.to(DEV), 4)
    assert ids.cpu().tolist() == [[0, 1, 2, 3]] * 3 and (w.cpu() == 0.25).all()


@pytest.mark.gpu
@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID])
def test_gate_choices_that_hang_on_the_last_bits(score):
    """Choices a few 1e-9 apart, closer than fp32 scores can tell: the order is that of binary64."""
    N, E = 32, 64
    L = draw(N, E, torch.float32, 12)
    s = np.stack([scores(L[t].numpy(), score)[0] for t in range(1)])[0]
    # a bias that levels the first token's scores to within fp32's rounding of the bias
    b = torch.from_numpy((0.5 - s).astype(np.float32))
    L = L[:1].expand(N, E).contiguous() + 0.0
    for renorm in (True, False):
        kw = dict(score=score, renormalize=renorm)
        ids, w = moe.gate(L.to(DEV), 8, bias=b.to(DEV), **kw)
        check(L, ids, w, bias=b, **kw)


@pytest.mark.gpu
@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID])
@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_gate_missing_experts_and_extremes(score, dtype):
    inf, nan, low = float("inf"), float("nan"), torch.finfo(dtype).min
    L = draw(12, 70, dtype, 4)
    L[0] = -inf
    L[1] = nan
    L[2] = -inf
    L[2, 69] = 1.0
    L[3] = low                        # the type's lowest value is a logit like any other
    L[4, ::2] = -inf
    L[5, 3:] = nan
    L[6] = low
    L[6, 5] = 0.0
    L[7, 66] = inf
    L[8, 66] = L[8, 2] = inf
    L[9] = torch.finfo(dtype).max
    L[10] = -100.0
    for bias in (None, torch.linspace(-0.1, 0.1, 70)):
        if bias is not None:
            bias[7], bias[9] = -inf, nan
        for groups in (1, 7):
            for renorm in (True, False):
                kw = dict(score=score, groups=groups, topk_groups=1 if groups == 1 else 2, group_score=TOP2,
                          renormalize=renorm)
                ids, w, on = moe.gate(L.to(DEV), 6, bias=None if bias is None else bias.to(DEV), with_pair_mask=True,
                                      **kw)
                assert torch.isfinite(w).all()
                check(L, ids, w, on, bias=bias, **kw)


@pytest.mark.gpu
def test_gate_token_mask_hides_its_rows():
    L = draw(50, 96, torch.bfloat16, 6)
    m = torch.rand(50, generator=torch.Generator().manual_seed(0)) < 0.5
    L[~m] = float("nan")
    for mask in (m, m.to(torch.uint8) * 7):
        ids, w, on = moe.gate(L.to(DEV), 4, token_mask=mask.to(DEV), with_pair_mask=True)
        check(L, ids, w, on, token_mask=m)
    ids, w = moe.gate(L.to(DEV), 4, token_mask=torch.zeros(50, dtype=torch.bool, device=DEV))
    assert (ids.cpu() == -1).all() and (w.cpu() == 0).all()
    ids, w = moe.gate(torch.zeros((0, 96), device=DEV), 4)
    assert ids.shape == (0, 4)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("N,E,K", [(1, 1, 1), (1, 8, 8), (3, 63, 5), (7, 65, 64), (65, 256, 8), (33, 304, 8), (6, 1000, 16),
                                   (3, 2048, 64), (5, 130, 3)])
def test_gate_backward_matches_the_formula(dtype, score, renorm, N, E, K):
    scale = 2.5
    L = draw(N, E, dtype, 40 + N)
    m = torch.ones(N, dtype=torch.bool)
    m[N // 2:N // 2 + 1] = N == 1
    ids, w = moe.gate(L.to(DEV), K, score, renormalize=renorm, scale=scale, token_mask=m.to(DEV))
    g = torch.randn(N, K, generator=torch.Generator().manual_seed(8))
    g[~m] = float("nan")                                  # what belongs to no pair is not used
    LL = L.clone()
    LL[~m] = float("nan")
    got = moe.gate_backward(LL.to(DEV), ids, w, g.to(DEV), score, renormalize=renorm, scale=scale)
    assert got.dtype == dtype
    want, mag = plain_backward(L, ids, w, torch.nan_to_num(g), score, renorm, scale)
    Ld = L.double().numpy()
    far = np.abs(Ld - Ld.max(1, keepdims=True)) if score == SOFTMAX and not renorm else np.abs(Ld)
    f = torch.finfo(dtype)
    room = (far + E / 64 + K + 24) * U * mag + f.eps / 2 * np.abs(want) * 1.01 + f.tiny * f.eps
    err = np.abs(got.cpu().double().numpy() - want)
    assert (err <= room).all(), (err.max(), np.argwhere(err > room)[:4])
    assert (got.cpu()[~m] == 0).all()


@pytest.mark.gpu
def test_gate_backward_of_rows_with_missing_pairs():
    L = draw(6, 40, torch.float32, 3)
    L[1, 3:] = -float("inf")
    L[2] = -float("inf")
    L[3] = float("nan")
    for score, renorm in itertools.product((SOFTMAX, SIGMOID), (True, False)):
        ids, w = moe.gate(L.to(DEV), 5, score, renormalize=renorm)
        g = torch.randn(6, 5, generator=torch.Generator().manual_seed(8))
        got = moe.gate_backward(L.to(DEV), ids, w, g.to(DEV), score, renormalize=renorm).cpu()
        want, mag = plain_backward(L, ids, w, g, score, renorm, 1.0)
        far = np.where(np.isfinite(L.numpy()), np.abs(L.numpy() - 4.0), 0.0)
        assert torch.isfinite(got).all()
        assert (np.abs(got.numpy() - want) <= (far + 40) * U * mag + U * np.abs(want)).all()
        assert (got[2:4] == 0).all() and (got[1, 3:] == 0).all()
        far = moe.gate_backward(L.to(DEV), torch.full_like(ids, 99), w, g.to(DEV), score, renormalize=renorm)
        assert (far.cpu() == 0).all()                     # ids that name no expert count as missing


@pytest.mark.gpu
def test_gate_replays_from_a_graph():
    L = draw(300, 256, torch.bfloat16, 1).to(DEV)
    b = (torch.randn(256, generator=torch.Generator().manual_seed(2)) * 0.05).to(DEV)
    ids = torch.empty((300, 8), dtype=torch.int32, device=DEV)
    w, grad = torch.empty((300, 8), device=DEV), torch.empty_like(L)
    gw = torch.randn(300, 8, device=DEV)
    kw = dict(score=SIGMOID, scale=2.0)

    def step():
        moe.gate_into(ids, w, L, bias=b, groups=8, topk_groups=4, group_score=TOP2, **kw)
        moe.gate_backward_into(grad, L, ids, w, gw, **kw)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        L.copy_(draw(300, 256, torch.bfloat16, 50 + i))
        graph.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in (ids, w, grad)]
        step()
        torch.cuda.synchronize()
        for x, y in zip(got, (ids, w, grad)):
            assert torch.equal(x, y)


@pytest.mark.gpu
def test_gate_feeds_dispatch_and_combine():
    """Identity experts: the combine returns each token times the sum of its weights, over the pairs that exist."""
    W, bs, epr, h, K = 4, 16, 4, 64, 4
    L = draw(W * bs, W * epr, torch.float32, 21)
    L[5, 2:] = -float("inf")                              # two experts only
    m = torch.ones(W * bs, dtype=torch.bool)
    m[7] = False
    x = torch.randn(W * bs, h, generator=torch.Generator().manual_seed(1)).half().to(DEV)
    ids, w, on = moe.gate(L.to(DEV), K, token_mask=m.to(DEV), with_pair_mask=True)
    ex, _, assist, erc = moe.dispatch(x, ids, W, epr, x_active_mask=on)
    out = moe.combine(ex, assist, erc, ids, w, W, epr, x_active_mask=on).float().cpu()
    want = x.float().cpu() * w.sum(1, keepdim=True).cpu()
    # K products of fp16 values summed in fp32 and one rounding to fp16
    assert (out - want).abs().le(want.abs() * (2.0 ** -11 + 2 * K * U) + 2.0 ** -24).all()
    assert (out[7] == 0).all() and int(erc[:, -1].sum()) == int(on.sum())


@pytest.mark.gpu
@pytest.mark.parametrize("N,E,K,groups,topk_groups", [(513, 16, 4, 1, 1), (1061, 33, 8, 1, 1), (2049, 64, 16, 8, 3),
                                                      (4099, 128, 1, 1, 1), (6001, 160, 8, 16, 4), (8197, 256, 8, 8, 4),
                                                      (9731, 304, 8, 1, 1), (10243, 320, 15, 5, 2), (21001, 96, 3, 6, 6)])
@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID])
def test_gate_of_long_batches(N, E, K, groups, topk_groups, score):
    """Batches long enough for several tokens to share a wavefront; a third of the rows hold few distinct logits (ties),
    some have missing experts or infinities, some tokens are masked. 300 rows are looked at, the last ones among them."""
    g = torch.Generator().manual_seed(N)
    for dtype, bias, group_score in ((torch.bfloat16, False, MAX), (torch.float32, True, TOP2), (torch.float16, True, MAX),
                                     (torch.float32, False, TOP2)):
        L = draw(N, E, dtype, N + 1)
        L[::3] = L[::3].round()
        L[7::31, :E // 2] = -float("inf")
        L[11::37] = float("nan")
        L[13::41, E - 1] = float("inf")
        L[17::43] -= 90.0
        m = torch.rand(N, generator=g) < 0.8
        L[~m] = float("nan")
        b = torch.randint(-2, 3, (E,), generator=g) * 0.25 if bias and dtype == torch.float16 else (
            torch.randn(E, generator=g) * 0.05 if bias else None)
        kw = dict(score=score, groups=groups, topk_groups=topk_groups, group_score=group_score, renormalize=bias, scale=1.5)
        ids, w, on = moe.gate(L.to(DEV), K, bias=None if b is None else b.to(DEV), token_mask=m.to(DEV),
                              with_pair_mask=True, **kw)
        rows = torch.cat((torch.randperm(N, generator=g)[:280], torch.arange(N - 20, N)))
        at = rows.to(DEV)
        check(L[rows], ids[at], w[at], on[at], bias=b, token_mask=m[rows], **kw)


@pytest.mark.gpu
@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID])
def test_gate_of_long_batches_on_the_last_bits(score):
    """As test_gate_choices_that_hang_on_the_last_bits, several tokens to a wavefront: every token is decided anew."""
    N, E = 1100, 32
    L = draw(1, E, torch.float32, 12)
    b = torch.from_numpy((0.5 - scores(L[0].numpy(), score)[0]).astype(np.float32))
    L = L.expand(N, E).contiguous()
    L[::2] = draw(N, E, torch.float32, 13)[::2]
    ids, w = moe.gate(L.to(DEV), 8, score, bias=b.to(DEV))
    check(L[:40], ids[:40], w[:40], bias=b, score=score)
    assert (ids[1::2] == ids[1]).all() and (w[1::2] == w[1]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID])
@pytest.mark.parametrize("N,E", [(300, 64), (2100, 64), (300, 300), (9700, 300), (200, 1500)])
@pytest.mark.parametrize("spread", [3e-7, 3e-6, 3e-5])
def test_gate_choices_about_as_far_apart_as_fp32_can_tell(score, N, E, spread):
    """Tokens whose choices lie around the distance below which fp32 scores are not trusted, on either side of it, with
    scores that differ much under biases that level them: the order is that of binary64 for every token."""
    g = torch.Generator().manual_seed(E)
    base = 2 * torch.randn(E, generator=g)
    b = torch.from_numpy((0.5 - scores(base.numpy(), score)[0]).astype(np.float32))
    L = base * (1 + spread * torch.randn((N, E), generator=g))
    at = torch.randperm(N, generator=g)[:200]
    for groups, kind in ((1, moe.MOE_GROUP_MAX), (4, moe.MOE_GROUP_MAX), (4, moe.MOE_GROUP_TOP2)):
        kw = dict(score=score, groups=groups, topk_groups=(groups + 1) // 2, group_score=kind)
        ids, w = moe.gate(L.to(DEV), 8, bias=b.to(DEV), **kw)
        check(L[at], ids[at.to(DEV)], w[at.to(DEV)], bias=b, **kw)

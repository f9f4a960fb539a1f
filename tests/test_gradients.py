"""Gradients of combine and dispatch: refusals on the CPU, and on the GPU the formulas in binary64, differences of the
forward calls, and calls at sizes, masks and alignments where they could go wrong."""
import ctypes

import numpy as np
import pytest
import torch

import combine_ep_recv_amd as moe
from test_gate import rec  # noqa: F401  (the fixture that records the library's calls)

DEV = "cuda"
A = 1 << 20
BIG = 2 ** 32


def P(v):
    return None if v is None else ctypes.c_void_p(v)


# ---- host only ----

def _special(zero=0, copy=0, const=0, ori=None, cx=None):
    return ctypes.byref(moe.MoeSpecialExperts(zero, copy, const, 0, ori, cx))


COMBINE = dict(grad=A, y=2 * A, assist=3 * A, erc=4 * A, ids=5 * A, w=6 * A, mask=None, kind=0, special=None, W=2, bs=4, epr=2,
               h=8, K=2, dtype=2, gy=7 * A, gw=8 * A, gori=None, gconst=None, ws=None, wsn=0)


@pytest.mark.parametrize("kw,want", [
    (dict(W=1), moe.MOE_ERR_SHAPE), (dict(W=769), moe.MOE_ERR_SHAPE), (dict(epr=0), moe.MOE_ERR_SHAPE),
    (dict(epr=513), moe.MOE_ERR_SHAPE), (dict(h=0), moe.MOE_ERR_SHAPE), (dict(K=0), moe.MOE_ERR_SHAPE),
    (dict(K=5), moe.MOE_ERR_SHAPE), (dict(bs=-1), moe.MOE_ERR_SHAPE), (dict(bs=1 << 23), moe.MOE_ERR_SHAPE),
    (dict(h=1 << 31 - 1, bs=1 << 8), moe.MOE_ERR_SHAPE), (dict(dtype=0), moe.MOE_ERR_DTYPE),
    (dict(dtype=3), moe.MOE_ERR_DTYPE), (dict(grad=None), moe.MOE_ERR_NULLPTR), (dict(y=None), moe.MOE_ERR_NULLPTR),
    (dict(assist=None), moe.MOE_ERR_NULLPTR), (dict(erc=None), moe.MOE_ERR_NULLPTR), (dict(ids=None), moe.MOE_ERR_NULLPTR),
    (dict(w=None), moe.MOE_ERR_NULLPTR), (dict(gy=None), moe.MOE_ERR_NULLPTR), (dict(gw=None), moe.MOE_ERR_NULLPTR),
    (dict(grad=A + 1), moe.MOE_ERR_ALIGN), (dict(y=A + 1), moe.MOE_ERR_ALIGN), (dict(w=A + 2), moe.MOE_ERR_ALIGN),
    (dict(gw=A + 2), moe.MOE_ERR_ALIGN), (dict(gy=A + 1), moe.MOE_ERR_ALIGN), (dict(assist=A + 2), moe.MOE_ERR_ALIGN),
    (dict(kind=3), moe.MOE_ERR_MASK), (dict(kind=1), moe.MOE_ERR_MASK), (dict(mask=A), moe.MOE_ERR_MASK),
    (dict(gori=A), moe.MOE_ERR_NULLPTR), (dict(gconst=A), moe.MOE_ERR_NULLPTR),
    (dict(special=(0, 1, 0, None, None)), moe.MOE_ERR_NULLPTR), (dict(special=(0, 0, 1, None, None)), moe.MOE_ERR_NULLPTR),
    (dict(special=(-1, 0, 0, None, None)), moe.MOE_ERR_SHAPE), (dict(special=(0, -1, 0, A, A)), moe.MOE_ERR_SHAPE),
    (dict(special=(1 << 30, 1 << 30, 0, A, A)), moe.MOE_ERR_SHAPE),
    (dict(special=(0, 0, 1 << 24, None, A), gconst=A), moe.MOE_ERR_SHAPE),
    (dict(special=(0, 0, 3, None, A), gconst=A, bs=200), moe.MOE_ERR_NULLPTR),
    (dict(special=(0, 0, 3, None, A), gconst=A, bs=200, ws=A, wsn=-1), moe.MOE_ERR_WORKSPACE),
    (dict(special=(0, 0, 3, None, A), gconst=A, bs=200, ws=A + 8), moe.MOE_ERR_ALIGN),
    (dict(bs=0, grad=None, y=None, assist=None, ids=None, w=None, gy=None, gw=None), moe.MOE_OK),
])
def test_combine_backward_refuses_before_a_launch(kw, want):
    p = dict(COMBINE, **kw)
    sp = None if p["special"] is None else _special(*p["special"])
    if p["gconst"] and p["special"] and want in (moe.MOE_ERR_WORKSPACE, moe.MOE_ERR_ALIGN):      # wsn: beside what it needs
        p["wsn"] += moe.combine_backward_workspace_size(p["W"], p["bs"], p["epr"], p["h"], p["K"], p["dtype"], p["special"][2])
    assert moe.library().moe_combine_backward(
        P(p["grad"]), P(p["y"]), P(p["assist"]), P(p["erc"]), P(p["ids"]), P(p["w"]), P(p["mask"]), p["kind"], sp, p["W"],
        p["bs"], p["epr"], p["h"], p["K"], p["dtype"], P(p["gy"]), P(p["gw"]), P(p["gori"]), P(p["gconst"]), P(p["ws"]),
        p["wsn"], None) == want


@pytest.mark.parametrize("kw,want", [
    (dict(W=1), moe.MOE_ERR_SHAPE), (dict(K=5), moe.MOE_ERR_SHAPE), (dict(h=0), moe.MOE_ERR_SHAPE),
    (dict(dtype=0), moe.MOE_ERR_DTYPE), (dict(dtype=3), moe.MOE_ERR_DTYPE), (dict(grad=None), moe.MOE_ERR_NULLPTR),
    (dict(assist=None), moe.MOE_ERR_NULLPTR), (dict(erc=None), moe.MOE_ERR_NULLPTR), (dict(ids=None), moe.MOE_ERR_NULLPTR),
    (dict(gx=None), moe.MOE_ERR_NULLPTR), (dict(gs=A), moe.MOE_ERR_NULLPTR), (dict(gw=A), moe.MOE_ERR_NULLPTR),
    (dict(kind=2), moe.MOE_ERR_MASK), (dict(kind=-1), moe.MOE_ERR_MASK), (dict(grad=A + 1), moe.MOE_ERR_ALIGN),
    (dict(add=A + 1), moe.MOE_ERR_ALIGN), (dict(gs=A + 2, gw=A), moe.MOE_ERR_ALIGN), (dict(gx=A + 1), moe.MOE_ERR_ALIGN),
    (dict(bs=0, grad=None, assist=None, ids=None, gx=None), moe.MOE_OK),
])
def test_dispatch_backward_refuses_before_a_launch(kw, want):
    p = dict(grad=A, assist=2 * A, erc=3 * A, ids=4 * A, gs=None, add=None, mask=None, kind=0, W=2, bs=4, epr=2, h=8, K=2,
             dtype=2, gx=5 * A, gw=None)
    p.update(kw)
    assert moe.library().moe_dispatch_backward(
        P(p["grad"]), P(p["assist"]), P(p["erc"]), P(p["ids"]), P(p["gs"]), P(p["add"]), P(p["mask"]), p["kind"], p["W"],
        p["bs"], p["epr"], p["h"], p["K"], p["dtype"], P(p["gx"]), P(p["gw"]), None) == want


def test_workspace_is_for_the_const_experts_parts():
    size = moe.combine_backward_workspace_size
    assert size(4, 1, 2, 24, 2, moe.MOE_BF16, 5) == 0                     # one part: no sums to join
    few, many = (size(4, n, 2, 24, 2, moe.MOE_BF16, 5) for n in (100, 1 << 20))
    assert 0 < few < many <= 64 * 5 * 24 * 4 and few % (5 * 24 * 4) == many % (5 * 24 * 4) == 0
    assert size(4, 1 << 20, 2, 24, 2, moe.MOE_BF16) == 0
    for args in ((4, 65, 2, 24, 2, moe.MOE_BF16, BIG), (4, 65, 2, 24, 2, moe.MOE_BF16, 1 << 24),
                 (2, 0, 1, 2 ** 31 - 1, 1, moe.MOE_BF16, 2)):
        with pytest.raises(moe.MoeError) as e:
            size(*args)
        assert e.value.status == moe.MOE_ERR_SHAPE


W_, BS, EPR, H, K_ = 2, 3, 2, 8, 2
N_ = W_ * BS


def _combine_args():
    z = torch.zeros
    return dict(grad_expand_x=z(N_ * K_, H).bfloat16(), grad_scales=z(N_, K_), grad_out=z(N_, H).bfloat16(),
                expand_x=z(N_ * K_, H).bfloat16(), assist_info=z(N_ * K_, 3, dtype=torch.int32),
                ep_recv_count=z(W_, EPR * W_, dtype=torch.int32), expert_ids=z(N_, K_, dtype=torch.int32),
                expert_scales=z(N_, K_), ep_world=W_, experts_per_rank=EPR)


def _dispatch_args():
    a = _combine_args()
    return dict(grad_x=a["grad_out"], grad_expand_x=a["expand_x"], **{k: a[k] for k in (
        "assist_info", "ep_recv_count", "expert_ids", "ep_world", "experts_per_rank")})


def test_well_formed_gradient_calls_reach_the_library(rec):  # noqa: F811
    a = _combine_args()
    moe.combine_backward_into(**a)
    moe.combine_backward_into(**a, x_active_mask=torch.ones(N_, dtype=torch.bool), copy_experts=1, ori_x=a["grad_out"],
                              grad_ori_x=a["grad_out"].clone(), zero_experts=2)
    del a["grad_expand_x"], a["grad_scales"]
    assert [t.shape for t in moe.combine_backward(**a, const_experts=0)] == [(N_ * K_, H), (N_, K_)]
    out = moe.combine_backward(**a, copy_experts=1, ori_x=a["grad_out"])
    assert len(out) == 3 and out[2].shape == (N_, H)
    d = _dispatch_args()
    moe.dispatch_backward_into(**d)
    del d["grad_x"]
    assert moe.dispatch_backward(**d).shape == (N_, H)
    x, w = moe.dispatch_backward(**d, add=torch.zeros(N_, H).bfloat16(), grad_expand_scales=torch.zeros(N_ * K_))
    assert x.shape == (N_, H) and w.shape == (N_, K_)
    assert rec.calls == ["moe_combine_backward"] * 4 + ["moe_dispatch_backward"] * 3


@pytest.mark.parametrize("field,value", [
    ("grad_out", torch.zeros(N_, H)), ("grad_out", torch.zeros(N_, H + 1).bfloat16()),
    ("grad_out", torch.zeros(H, N_).bfloat16().t()), ("grad_out", None), ("expand_x", torch.zeros(N_ * K_, H)),
    ("expand_x", torch.zeros(N_ * K_, H, dtype=torch.int32)), ("expand_x", torch.zeros(N_ * K_ - 1, H).bfloat16()),
    ("assist_info", torch.zeros(N_ * K_, 3, dtype=torch.int64)), ("assist_info", torch.zeros(N_ * K_, 2, dtype=torch.int32)),
    ("ep_recv_count", torch.zeros(W_, EPR * W_ + 1, dtype=torch.int32)), ("expert_ids", torch.zeros(N_, K_)),
    ("expert_ids", torch.zeros(N_ + 1, K_, dtype=torch.int32)), ("expert_ids", torch.zeros(N_, dtype=torch.int32)),
    ("expert_scales", torch.zeros(N_, K_).bfloat16()), ("grad_expand_x", torch.zeros(N_ * K_, H).half()),
    ("grad_scales", torch.zeros(N_ * K_)), ("ep_world", 4), ("ep_world", 0), ("experts_per_rank", 3),
    ("experts_per_rank", BIG + 2), ("ep_world", BIG + 2),
    ("x_active_mask", torch.zeros(N_ + 1, dtype=torch.bool)), ("x_active_mask", torch.zeros(N_, K_)),
    ("copy_experts", 1), ("const_experts", 1), ("zero_experts", BIG), ("zero_experts", -1),
    ("grad_ori_x", torch.zeros(N_, H).bfloat16()), ("grad_const_x", torch.zeros(1, H).bfloat16()),
], ids=lambda v: v if isinstance(v, str) else "")
def test_combine_backward_rejects_before_the_call(rec, field, value):  # noqa: F811
    a = _combine_args()
    a[field] = value
    with pytest.raises(moe.MoeError):
        moe.combine_backward_into(**a)
    assert rec.calls == []


@pytest.mark.parametrize("field,value", [
    ("grad_x", torch.zeros(N_, H)), ("grad_x", torch.zeros(N_, H + 1).bfloat16()),
    ("grad_expand_x", torch.zeros(N_ * K_, H)), ("grad_expand_x", torch.zeros(H, N_ * K_).bfloat16().t()),
    ("add", torch.zeros(N_, H)), ("grad_expand_scales", torch.zeros(N_ * K_)), ("grad_scales", torch.zeros(N_, K_)),
    ("assist_info", torch.zeros(N_, 3, dtype=torch.int32)), ("ep_recv_count", torch.zeros(4, 4, dtype=torch.int32)),
    ("x_active_mask", torch.zeros(K_, N_, dtype=torch.bool).t()), ("expert_ids", torch.zeros(N_, K_, dtype=torch.int64)),
], ids=lambda v: v if isinstance(v, str) else "")
def test_dispatch_backward_rejects_before_the_call(rec, field, value):  # noqa: F811
    d = _dispatch_args()
    d[field] = value
    with pytest.raises(moe.MoeError):
        moe.dispatch_backward_into(**d)
    assert rec.calls == []


@pytest.mark.parametrize("kw", [dict(const_experts=BIG, const_x=torch.zeros(1, H).bfloat16()), dict(const_experts=2),
                                dict(const_experts=2, const_x=torch.zeros(1, H).bfloat16()), dict(copy_experts=1),
                                dict(copy_experts=1, ori_x=torch.zeros(N_, H)), dict(const_experts=1, const_x=3),
                                dict(const_experts=2, const_x=torch.zeros(H, 2).bfloat16().t()), dict(zero_experts=-1),
                                dict(expand_x=torch.zeros(N_ * K_, H, dtype=torch.int32)), dict(ep_world=4)], ids=str)
def test_combine_backward_refuses_before_it_makes_room(rec, kw):  # noqa: F811
    a = _combine_args()
    del a["grad_expand_x"], a["grad_scales"]
    a.update(kw)
    with pytest.raises(moe.MoeError):
        moe.combine_backward(**a)
    assert rec.calls == []


def test_gradients_of_cpu_tensors_are_rejected():
    with pytest.raises(moe.MoeError):
        moe.combine_backward_into(**_combine_args())
    with pytest.raises(moe.MoeError):
        moe.dispatch_backward_into(**_dispatch_args())


# ---- on the GPU ----

def route(W, bs, epr, K, special=0, mask=None, seed=0, skew=0.0):
    """Distinct ids of each token, a mask of the given kind, and the row of each pair (-1: none) by the definition: rows
    lie by expert, then token."""
    rng = np.random.default_rng(seed)
    N, E = W * bs, W * epr
    z = rng.standard_normal((N, E + special)) - skew * np.arange(E + special)
    ids = np.argsort(-z, axis=1, kind="stable")[:, :K].astype(np.int32)
    m = {None: None, "token": rng.random(N) < 0.7, "pair": rng.random((N, K)) < 0.6,
         "none": np.zeros((N, K), bool), "no token": np.zeros(N, bool)}[mask]
    on = np.ones((N, K), bool) if m is None else np.broadcast_to(m if m.ndim == 2 else m[:, None], (N, K))
    t, k = np.nonzero(on & (ids < E))
    order = np.lexsort((t, ids[t, k]))
    row = np.full((N, K), -1)
    row[t[order], k[order]] = np.arange(len(order))
    return torch.from_numpy(ids), None if m is None else torch.from_numpy(m), torch.from_numpy(row), torch.from_numpy(on.copy())


def dispatched(ids, mask, row, W, epr, special):
    """assist_info and ep_recv_count of dispatch itself for this routing."""
    x = torch.zeros((ids.shape[0], 8), dtype=torch.bfloat16, device=DEV)
    m = None if mask is None else mask.to(DEV)
    _, _, assist, counts = moe.dispatch(x, ids.to(DEV), W, epr, x_active_mask=m, zero_experts=special)
    A = int((row >= 0).sum())
    a = assist.cpu()[:A].long()
    bs = ids.shape[0] // W
    assert torch.equal(row[a[:, 0] * bs + a[:, 1], a[:, 2]], torch.arange(A))
    return assist, counts


SHAPES = [
    # W, bs, epr, K, h, special (zero, copy, const), mask, skew
    (2, 1, 1, 1, 1, (0, 0, 0), None, 0.0), (2, 1, 2, 2, 7, (0, 0, 0), None, 0.0), (8, 1, 8, 8, 7168, (0, 0, 0), None, 0.0),
    (4, 9, 3, 5, 8, (0, 0, 0), "pair", 0.0), (2, 20, 4, 8, 2048, (0, 0, 0), "token", 0.0),
    (4, 33, 2, 3, 2057, (1, 2, 3), "pair", 0.0), (3, 50, 5, 9, 300, (2, 1, 4), "token", 0.0),
    (2, 40, 1, 2, 136, (0, 0, 2), None, 0.0), (2, 40, 1, 2, 33, (0, 3, 0), None, 0.0), (2, 7, 2, 3, 64, (2, 0, 0), None, 0.0),
    (2, 600, 2, 4, 40, (0, 0, 0), None, 0.0),            # segments of every token
    (2, 700, 4, 3, 264, (1, 1, 2), "pair", 2.0),         # one expert with nearly every row
    (16, 40, 16, 8, 520, (0, 0, 0), None, 0.0), (4, 300, 16, 7, 2049, (1, 1, 1), "token", 0.0),
    (768, 2, 1, 3, 24, (0, 0, 0), "pair", 0.0), (70, 9, 14, 70, 48, (3, 3, 3), "pair", 0.0),
    (2, 4, 512, 200, 32, (0, 0, 0), "pair", 0.0), (2, 9, 512, 1000, 16, (1, 1, 1), None, 0.0),
    (4, 5, 2, 2, 24, (0, 1, 1), "none", 0.0), (4, 5, 2, 2, 24, (1, 1, 1), "no token", 0.0),
    (4, 9000, 2, 3, 20, (1, 1, 2), "pair", 0.0),         # parts of the tokens that are listed in several pieces
    (2, 40000, 1, 1, 9, (0, 0, 1), None, -9.0),          # a const expert with nearly every pair: full lists
    (4, 2100, 2, 4, 4099, (0, 1, 1), "token", 0.0),      # rows that fill the Infinity Cache, at odd offsets
    (2, 1, 2, 2, 200003, (0, 1, 1), None, 0.0),
]
TYPES = [torch.bfloat16, torch.float16]


def inputs(ids, h, special, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    N, K = ids.shape
    r = lambda *s: torch.randn(s, generator=g)
    return dict(y=r(N * K, h).to(dtype), g=(r(N, h) * torch.exp(r(N, 1))).to(dtype), w=r(N, K), x=r(N, h).to(dtype),
                cx=r(special[2], h).to(dtype))


def sources(ids, row, on, E, special, v):
    """Each pair's row as binary64 [N, K, h] (zeros: none), and which pairs are a copy's and a const's ([N, K, C])."""
    ids = ids.long()
    src = torch.where((row >= 0)[..., None], v["y"].double()[row.clamp(min=0)], 0.0)
    first = E + special[0]
    copy = on & (ids >= first) & (ids < first + special[1])
    src = torch.where(copy[..., None], v["x"].double()[:, None], src)
    j = ids - first - special[1]
    const = (on & (j >= 0))[..., None] & (j[..., None] == torch.arange(special[2]))
    if special[2]:
        src = torch.where(const.any(2)[..., None], v["cx"].double()[j.clamp(min=0)], src)
    return src, copy, const


def chain(h):
    """Additions that a product of rows goes through: 8 for each 512 columns (a wavefront's; 2048 where four take a row of
    more), the tail, 6 in a wavefront and 3 beyond."""
    return 8 * -(-h // (512 if h <= 2048 else 2048)) + 1 + 6 + 3


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_combine_backward(shape, dtype):
    W, bs, epr, K, h, special, mask, skew = shape
    E, N = W * epr, W * bs
    ids, m, row, on = route(W, bs, epr, K, sum(special), mask, 5, skew)
    assist, counts = dispatched(ids, m, row, W, epr, sum(special))
    v = inputs(ids, h, special, dtype, 7)
    d = {k: t.to(DEV) for k, t in v.items()}
    gy = torch.full((N * K, h), 7.0, dtype=dtype, device=DEV)
    gw = torch.full((N, K), 7.0, device=DEV)
    ori = torch.full((N, h), 7.0, dtype=dtype, device=DEV) if special[1] else None
    const = torch.full((special[2], h), 7.0, dtype=dtype, device=DEV) if special[2] else None
    moe.combine_backward_into(gy, gw, d["g"], d["y"], assist, counts, ids.to(DEV), d["w"], W, epr,
                              x_active_mask=None if m is None else m.to(DEV), zero_experts=special[0],
                              copy_experts=special[1], ori_x=d["x"], grad_ori_x=ori, const_experts=special[2],
                              const_x=d["cx"], grad_const_x=const)
    f, u = torch.finfo(dtype), 2.0 ** -24
    # one product in binary32, rounded to the type: the same two roundings
    live = row >= 0
    want = torch.full((N * K, h), 7.0, dtype=dtype)
    pairs = (v["w"][..., None] * v["g"].float()[:, None]).to(dtype)
    want[row[live]] = pairs[live]
    assert torch.equal(gy.cpu(), want)
    src, copy, const_on = sources(ids, row, on, E, special, v)
    g = v["g"].double()
    ref, size = (src * g[:, None]).sum(2), (src * g[:, None]).abs().sum(2)
    assert ((gw.cpu().double() - ref).abs() <= 1.01 * chain(h) * u * size).all()
    assert (gw.cpu()[~(live | copy | const_on.any(2))] == 0).all()

    def close(got, ref, size, terms):
        room = 1.01 * terms * u * size
        limit = room + f.eps / 2 * (ref.abs() + room) + f.tiny * f.eps
        assert ((got.cpu().double() - ref).abs() <= limit).all()

    if special[1]:
        share = torch.where(copy, v["w"].double(), 0.0)
        close(ori, share.sum(1)[:, None] * g, share.abs().sum(1)[:, None] * g.abs(), K + 8)
    if special[2]:
        share = (const_on * v["w"].double()[..., None]).sum(1).t()
        close(const, share @ g, share.abs() @ g.abs(), int(const_on.sum((0, 1)).max()) + 64)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_dispatch_backward(shape, dtype):
    W, bs, epr, K, h, special, mask, skew = shape
    N = W * bs
    ids, m, row, on = route(W, bs, epr, K, sum(special), mask, 11, skew)
    assist, counts = dispatched(ids, m, row, W, epr, sum(special))
    gen = torch.Generator().manual_seed(13)
    rows = torch.randn(N * K, h, generator=gen).to(dtype)
    rows[int((row >= 0).sum()):] = float("nan")                    # rows that no pair has
    add = torch.randn(N, h, generator=gen).to(dtype)
    gs = torch.randn(N * K, generator=gen)
    f, u = torch.finfo(dtype), 2.0 ** -24
    args = (rows.to(DEV), assist, counts, ids.to(DEV), W, epr, None if m is None else m.to(DEV))
    live = row >= 0
    parts = torch.where(live[..., None], rows.double()[row.clamp(min=0)], 0.0)
    for extra in (None, add):
        ref, size = parts.sum(1), parts.abs().sum(1)
        if extra is not None:
            ref, size = ref + extra.double(), size + extra.double().abs()
        got, w = moe.dispatch_backward(*args, None if extra is None else extra.to(DEV), gs.to(DEV))
        room = 1.01 * (K + 1) * u * size
        assert ((got.cpu().double() - ref).abs() <= room + f.eps / 2 * (ref.abs() + room) + f.tiny * f.eps).all()
        assert torch.equal(w.cpu(), torch.where(live, gs[row.clamp(min=0)], 0.0))
    x = add.to(DEV)
    assert torch.equal(moe.dispatch_backward_into(x, *args, x), got)      # into add itself


@pytest.mark.gpu
def test_gradients_against_differences():
    """Small whole numbers in fp16, whose sums all come out exactly: a step d of an input moves the loss <G, output> by
    exactly <gradient, d>, both inputs of combine and the tokens of dispatch."""
    W, bs, epr, K, h = 4, 11, 2, 3, 40
    ids, m, row, on = route(W, bs, epr, K, 4, "pair", 3)
    assist, counts = dispatched(ids, m, row, W, epr, 4)
    gen = torch.Generator().manual_seed(4)
    whole = lambda *s: torch.randint(-2, 3, s, generator=gen).to(DEV)
    N = W * bs
    y, x, G, w, cx = whole(N * K, h).half(), whole(N, h).half(), whole(N, h).half(), whole(N, K).float(), whole(2, h).half()
    idd, md = ids.to(DEV), m.to(DEV)
    kw = dict(x_active_mask=md, zero_experts=1, copy_experts=1, const_experts=2)
    out = lambda y, w, x, cx: moe.combine(y, assist, counts, idd, w, W, epr, ori_x=x, const_x=cx, **kw).double()
    gy, gw, gx, gc = moe.combine_backward(G, y, assist, counts, idd, w, W, epr, ori_x=x, const_x=cx, **kw)
    live = torch.arange(N * K, device=DEV)[:, None] < int((row >= 0).sum())
    base = out(y, w, x, cx)
    for i, (grad, at) in enumerate(((gy, y), (gw, w), (gx, x), (gc, cx))):
        d = whole(*at.shape).to(at.dtype)
        moved = [y, w, x, cx]
        moved[i] = at + d
        step = ((out(*moved) - base) * G.double()).sum()
        move = grad.double() * d.double()
        assert step == (torch.where(live, move, 0.0) if i == 0 else move).sum() and step != 0
    Gr = whole(N * K, h).half()
    send = lambda x: torch.where(live, moe.dispatch(x, idd, W, epr, x_active_mask=md, zero_experts=4)[0].double(), 0.0)
    d = whole(N, h).half()
    step = ((send(x + d) - send(x)) * Gr.double()).sum()
    assert step == (moe.dispatch_backward(Gr, assist, counts, idd, W, epr, md).double() * d.double()).sum() and step != 0


@pytest.mark.gpu
def test_values_in_places_that_do_not_count():
    """NaN and infinity in an inactive pair's weight, in rows behind the last, and in a token that only masked pairs and
    zero experts have."""
    W, bs, epr, K, h = 2, 30, 2, 3, 72
    ids, m, row, on = route(W, bs, epr, K, 2, "pair", 8)
    assist, counts = dispatched(ids, m, row, W, epr, 2)
    v = inputs(ids, h, (2, 0, 0), torch.bfloat16, 9)
    clean = [t.to(DEV) for t in (v["g"], v["y"], v["w"])]
    A, live = int((row >= 0).sum()), row >= 0
    v["w"][~live] = float("nan")
    v["y"][A:] = float("inf")
    alone = ~live.any(1)
    v["g"][alone] = float("nan")
    args = (assist, counts, ids.to(DEV))
    kw = dict(x_active_mask=m.to(DEV), zero_experts=2)
    got = moe.combine_backward(v["g"].to(DEV), v["y"].to(DEV), *args, v["w"].to(DEV), W, epr, **kw)
    want = moe.combine_backward(clean[0], clean[1], *args, clean[2], W, epr, **kw)
    assert alone.any() and torch.equal(got[0][:A], want[0][:A]) and torch.equal(got[1], want[1])
    assert (got[1][~live] == 0).all() and torch.isfinite(got[1]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("bs", [6, 400], ids=["workgroup a pair", "workgroup a token"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")], ids=str)
@pytest.mark.parametrize("mask", ["pair", "token"])
def test_a_padded_tokens_gradient_reaches_no_token_nor_const_expert(bs, bad, mask):
    """What x_out's gradient holds at a token without active pairs (padding) flows back to nothing: neither its own
    grad_ori_x nor the const experts' table, and dispatch's gradient adds 0."""
    W, epr, K, h = 2, 2, 3, 77
    N, E, special = W * bs, W * epr, (1, 1, 2)
    ids, m, row, on = route(W, bs, epr, K, sum(special), mask, 12)
    assist, counts = dispatched(ids, m, row, W, epr, sum(special))
    v = inputs(ids, h, special, torch.bfloat16, 13)
    clean, copy = v["g"].to(DEV), on & (ids == E + 1)
    idle, d = ~on.any(1), {k: t.to(DEV) for k, t in v.items()}
    assert idle.any() and copy.any() and (on.any(1) & ~copy.any(1)).any()
    d["g"][idle.to(DEV)] = bad
    kw = dict(x_active_mask=m.to(DEV), zero_experts=1, copy_experts=1, ori_x=d["x"], const_experts=2, const_x=d["cx"])
    args = (d["y"], assist, counts, ids.to(DEV), d["w"], W, epr)
    got, want = moe.combine_backward(d["g"], *args, **kw), moe.combine_backward(clean, *args, **kw)
    A = int((row >= 0).sum())
    assert torch.equal(got[0][:A], want[0][:A])
    assert all(torch.equal(a, b) for a, b in zip(got[1:], want[1:]))
    assert (got[2][~copy.any(1).to(DEV)] == 0).all() and torch.isfinite(got[2]).all()
    back = [moe.dispatch_backward(r[0], assist, counts, ids.to(DEV), W, epr, m.to(DEV), r[2]) for r in (got, want)]
    assert torch.equal(*back) and (back[0][idle.to(DEV)] == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("h", [8, 61, 2056])
def test_gradients_at_any_alignment_leave_the_neighbours_alone(h):
    W, bs, epr, K = 2, 9, 3, 4
    N = W * bs
    ids, m, row, on = route(W, bs, epr, K, 2, "pair", 21)
    assist, counts = dispatched(ids, m, row, W, epr, 2)
    v = {k: t.to(DEV) for k, t in inputs(ids, h, (0, 1, 1), torch.bfloat16, 22).items()}
    idd, md, A = ids.to(DEV), m.to(DEV), int((row >= 0).sum())
    kw = dict(x_active_mask=md, copy_experts=1, const_experts=1)
    want = moe.combine_backward(v["g"], v["y"], assist, counts, idd, v["w"], W, epr, ori_x=v["x"], const_x=v["cx"], **kw)
    back = moe.dispatch_backward(v["y"], assist, counts, idd, W, epr, md, v["x"])

    def odd(t, fill=None):
        whole = torch.full((t.numel() + 40,), 7.0, dtype=t.dtype, device=DEV)
        part = whole[19:19 + t.numel()].view(t.shape)
        if fill is None:
            part.copy_(t)
        return whole, part

    g, y, x, cx = (odd(v[k])[1] for k in ("g", "y", "x", "cx"))
    outs = [odd(t, 7.0) for t in want]
    moe.combine_backward_into(outs[0][1], outs[1][1], g, y, assist, counts, idd, v["w"], W, epr, ori_x=x,
                              grad_ori_x=outs[2][1], const_x=cx, grad_const_x=outs[3][1], **kw)
    dx = odd(back, 7.0)
    moe.dispatch_backward_into(dx[1], y, assist, counts, idd, W, epr, md, x)
    for (whole, part), t in zip(outs + [dx], [*want, back]):
        n = A * h if part.shape == (N * K, h) else part.numel()
        assert torch.equal(part.flatten()[:n], t.flatten()[:n])
        assert (whole[:19] == 7).all() and (whole[19 + n:] == 7).all()


@pytest.mark.gpu
@pytest.mark.parametrize("h", [520, 2064])
def test_a_tokens_gradients_do_not_depend_on_how_many_there_are(h):
    """A call of few tokens and one of many, each with its own split of the work, add in the same order."""
    W, epr, K, big = 2, 4, 8, 400
    ids, _, row, on = route(W, big, epr, K, 0, None, 31)
    small = 30
    pick = torch.cat([torch.arange(small) + s * big for s in range(W)])
    v = inputs(ids, h, (0, 0, 0), torch.bfloat16, 32)
    full = dispatched(ids, None, row, W, epr, 0)
    few_ids = ids[pick].contiguous()
    N = W * small
    order = np.lexsort((np.repeat(np.arange(N), K), few_ids.numpy().ravel()))
    few_row = torch.empty(N * K, dtype=torch.int64)
    few_row[torch.from_numpy(order)] = torch.arange(N * K)
    few_row = few_row.view(N, K)
    few = dispatched(few_ids, None, few_row, W, epr, 0)
    y = torch.empty(N * K, h, dtype=torch.bfloat16)
    y[few_row.flatten()] = v["y"][row[pick].flatten()]
    a = moe.combine_backward(v["g"].to(DEV), v["y"].to(DEV), *full, ids.to(DEV), v["w"].to(DEV), W, epr)
    b = moe.combine_backward(v["g"][pick].to(DEV), y.to(DEV), *few, few_ids.to(DEV), v["w"][pick].to(DEV), W, epr)
    assert torch.equal(a[1].cpu()[pick], b[1].cpu())
    assert torch.equal(a[0].cpu()[row[pick].flatten()], b[0].cpu()[few_row.flatten()])
    c = moe.dispatch_backward(v["y"].to(DEV), *full, ids.to(DEV), W, epr)
    d = moe.dispatch_backward(y.to(DEV), *few, few_ids.to(DEV), W, epr)
    assert torch.equal(c.cpu()[pick], d.cpu())


@pytest.mark.gpu
def test_gradients_of_nothing():
    W, epr, K, h = 4, 2, 3, 16
    z = lambda *s, dt=torch.bfloat16: torch.zeros(s, dtype=dt, device=DEV)
    assist, counts, ids = z(0, 3, dt=torch.int32), z(W, epr * W, dt=torch.int32), z(0, K, dt=torch.int32)
    gy, gw, gc = moe.combine_backward(z(0, h), z(0, h), assist, counts, ids, z(0, K, dt=torch.float32), W, epr,
                                      const_experts=2, const_x=z(2, h) + 1)
    assert gy.shape == (0, h) and gw.shape == (0, K) and (gc == 0).all()
    assert moe.dispatch_backward(z(0, h), assist, counts, ids, W, epr).shape == (0, h)


@pytest.mark.gpu
@pytest.mark.parametrize("bad", ["negative", "descending", "huge", "tokens", "ids"])
def test_gradients_stay_in_bounds_on_routing_they_should_not_get(bad):
    W, bs, epr, K, h = 4, 50, 2, 4, 72
    N = W * bs
    ids, m, row, on = route(W, bs, epr, K, 0, None, 41)
    assist, counts = dispatched(ids, m, row, W, epr, 0)
    v = {k: t.to(DEV) for k, t in inputs(ids, h, (0, 1, 1), torch.bfloat16, 42).items()}
    ids = ids.to(DEV)
    if bad == "tokens":
        assist = torch.full_like(assist, -2 ** 31)
        assist[::2] = 2 ** 31 - 1
    elif bad == "ids":
        ids = torch.randint(-2 ** 31, 2 ** 31 - 1, (N, K), device=DEV, dtype=torch.int32)
    else:
        counts = {"negative": -counts, "descending": counts.flip(1).contiguous(),
                  "huge": torch.full_like(counts, 2 ** 31 - 1)}[bad]
    whole = [torch.full((n + 64, h), 7.0, dtype=torch.bfloat16, device=DEV) for n in (N * K, N, 1, N)]
    parts = [w[32:-32] for w in whole]
    gw = torch.full((N * K + 64,), 7.0, device=DEV)
    moe.combine_backward_into(parts[0], gw[32:-32].view(N, K), v["g"], v["y"], assist, counts, ids, v["w"], W, epr,
                              copy_experts=1, ori_x=v["x"], grad_ori_x=parts[1], const_experts=1, const_x=v["cx"],
                              grad_const_x=parts[2])
    moe.dispatch_backward_into(parts[3], v["y"], assist, counts, ids, W, epr, None, v["x"])
    for w in whole + [gw]:
        assert (w[:32] == 7).all() and (w[-32:] == 7).all()


@pytest.mark.gpu
def test_gradients_at_once_and_replayed():
    """Two streams at a time, and a captured step (combine's gradient into dispatch's) replayed as its inputs change."""
    W, bs, epr, K, h = 4, 60, 4, 4, 520
    N, zero = W * bs, 1
    sets = []
    for seed in range(4):
        ids, m, row, on = route(W, bs, epr, K, 3, "pair", seed)
        assist, counts = dispatched(ids, m, row, W, epr, 3)
        v = {k: t.to(DEV) for k, t in inputs(ids, h, (1, 1, 1), torch.bfloat16, seed).items()}
        sets.append([v["g"], v["y"], assist, counts, ids.to(DEV), v["w"], m.to(DEV), v["x"], v["cx"]])

    def outputs():
        e = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device=DEV)
        return [e(N * K, h), torch.zeros(N, K, device=DEV), e(N, h), e(1, h), e(N, h),
                moe.combine_backward_workspace(W, bs, epr, h, K, torch.bfloat16, 1, DEV)]

    def step(s, o):
        g, y, assist, counts, ids, w, m, x, cx = s
        moe.combine_backward_into(o[0], o[1], g, y, assist, counts, ids, w, W, epr, o[5], m, zero, 1, x, o[2], 1, cx, o[3])
        moe.dispatch_backward_into(o[4], o[0], assist, counts, ids, W, epr, m, o[2])

    want = []
    for s in sets:
        o = outputs()
        step(s, o)
        want.append([t.clone() for t in o[:5]])
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream(), torch.cuda.Stream()], [outputs(), outputs()]
    torch.cuda.synchronize()
    for _ in range(5):
        for st, s, o in zip(streams, sets, outs):
            with torch.cuda.stream(st):
                step(s, o)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert all(torch.equal(a, b) for a, b in zip(o, w))
    held, o = [t.clone() for t in sets[0]], outputs()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(held, o)
    for i in (1, 2, 0, 3):
        for a, b in zip(held, sets[i]):
            a.copy_(b)
        o[0].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(o, want[i])), i


@pytest.mark.gpu
def test_a_training_step_of_the_layer():
    """gate -> dispatch -> experts -> combine and all the way back, against binary64 autograd of the whole function.

    An expert multiplies by a power of two of its own and a copy expert gives the token itself, so that 16-bit rows hold
    the experts' outputs exactly; what is left are the gate's weights (some 2^-22 of themselves), the sums' roundings in
    fp32, and one rounding to 16 bits of each row's gradient and of the tokens'."""
    W, bs, epr, K, h = 4, 40, 4, 4, 264
    N, E = W * bs, W * epr
    gen = torch.Generator().manual_seed(51)
    x = torch.randn(N, h, generator=gen).bfloat16()
    logits = torch.randn(N, E + 2, generator=gen)                          # two copy experts among them
    G = torch.randn(N, h, generator=gen).bfloat16()
    power = 2.0 ** torch.randint(-1, 2, (E,), generator=gen).double()

    xd, ld, gd = x.to(DEV), logits.to(DEV), G.to(DEV)
    ids, w, on = moe.gate(ld, K, moe.MOE_SCORE_SIGMOID, scale=2.0, with_pair_mask=True)
    rows, _, assist, counts = moe.dispatch(xd, ids, W, epr, x_active_mask=on, copy_experts=2)
    ends = (counts[:, W - 1::W].cpu().long() + torch.cat((torch.zeros(1).long(), counts[:, -1].cpu().long().cumsum(0)[:-1]))[:, None]).flatten()
    A = int(ends[-1])
    expert = torch.searchsorted(ends, torch.arange(N * K), right=True).clamp(max=E - 1)
    p = power[expert].bfloat16().to(DEV)[:, None]
    y = rows * p
    out = moe.combine(y, assist, counts, ids, w, W, epr, x_active_mask=on, copy_experts=2, ori_x=xd)
    gy, gw, gori = moe.combine_backward(gd, y, assist, counts, ids, w, W, epr, x_active_mask=on, copy_experts=2, ori_x=xd)
    gx = moe.dispatch_backward(gy * p, assist, counts, ids, W, epr, on, gori)
    gl = moe.gate_backward(ld, ids, w, gw, moe.MOE_SCORE_SIGMOID, scale=2.0)

    X, L = x.double().requires_grad_(), logits.double().requires_grad_()
    at = ids.cpu().long()
    s = torch.sigmoid(L).gather(1, at)
    wt = 2.0 * s / s.sum(1, keepdim=True)
    f = torch.cat((power, torch.ones(2).double()))[at]
    ref = ((wt * f).sum(1)[:, None] * X)
    (ref * G.double()).sum().backward()
    eps, u, size = 2.0 ** -8, 2.0 ** -24, (wt * f).detach()
    mag = size.sum(1)[:, None] * X.detach().abs()
    assert ((out.cpu().double() - ref).abs() <= eps * ref.abs() + 40 * u * mag).all()
    gmag = size.sum(1)[:, None] * G.double().abs()
    assert ((gx.cpu().double() - X.grad).abs() <= (2 * eps + 80 * u + eps * eps) * gmag).all()
    # the weights' gradients are off by chain(h) u of the sum of sizes; the logits' by that, the weights' own error and a
    # few roundings, each times a weight of at most 2 and summed over K of them
    dot = (f * (X.detach().abs() * G.double().abs()).sum(1)[:, None]).max(1).values[:, None]
    assert ((gl.cpu().double() - L.grad).abs() <= 2 * (1 + K) * (chain(h) + 40) * u * dot).all()
    assert A < N * K and (gl != 0).any()


@pytest.mark.gpu
def test_gradients_of_rows_beyond_4_gib():
    """300000 rows of 14336 bytes: tokens whose rows lie on both sides of the 4 GiB line, the first and the last ones."""
    W, bs, epr, K, h = 2, 18750, 4, 8, 7168
    N = W * bs
    g = torch.Generator(DEV).manual_seed(61)
    ids = torch.rand(N, W * epr, generator=g, device=DEV).argsort(dim=1)[:, :K].int().contiguous()   # every expert
    w = torch.randn(N, K, generator=g, device=DEV)
    x = torch.randn(N, h, generator=g, device=DEV, dtype=torch.bfloat16)
    y, _, assist, counts = moe.dispatch(x, ids, W, epr)
    assert y.numel() * 2 > 1 << 32
    gy, gw = moe.combine_backward(x, y, assist, counts, ids, w, W, epr)
    gx = moe.dispatch_backward(y, assist, counts, ids, W, epr)
    row = torch.empty(N * K, dtype=torch.int64, device=DEV)
    a = assist.long()
    row[(a[:, 0] * bs + a[:, 1]) * K + a[:, 2]] = torch.arange(N * K, device=DEV)
    row = row.view(N, K)
    line = (1 << 32) // (2 * h)
    near = a[line - 20:line + 20, 0] * bs + a[line - 20:line + 20, 1]
    for t in torch.cat((torch.tensor([0, 1, bs - 1, bs, N - 1], device=DEV), near)).tolist():
        assert torch.equal(gy[row[t]], (w[t][:, None] * x[t].float()).bfloat16())
        # dispatch's rows are the token: the weights' gradients are its square, the tokens' eight times itself
        size = x[t].double().square().sum()
        assert ((gw[t].double() - size).abs() <= 1.01 * chain(h) * 2.0 ** -24 * size).all()
        assert torch.equal(gx[t], x[t] * 8)
    torch.cuda.empty_cache()

"""Rows of 8-bit integers and the experts' product on them: refusals on the CPU, and on the GPU the quantiser's definition in
numpy, the product against exact integer sums, and whole layers."""
import ctypes

import numpy as np
import pytest
import torch

import combine_ep_recv_amd as moe
from test_gate import rec  # noqa: F401  (the fixture that records the library's calls)
from test_mx_rows import counts_for

DEV = "cuda"
NONE, SWIGLU = moe.MOE_ACT_NONE, moe.MOE_ACT_SWIGLU
TYPES = [torch.bfloat16, torch.float16, torch.float32]
A = 1 << 20
BIG = 2 ** 32
U = 2.0 ** -24


def P(v):
    return None if v is None else ctypes.c_void_p(v)


# ---- host only ----

@pytest.mark.parametrize("kw,want", [
    (dict(rows=-1), moe.MOE_ERR_SHAPE), (dict(cols=0), moe.MOE_ERR_SHAPE), (dict(cols=(1 << 30) + 1), moe.MOE_ERR_SHAPE),
    (dict(dtype=0), moe.MOE_ERR_DTYPE), (dict(dtype=4), moe.MOE_ERR_DTYPE), (dict(rows=1 << 31, cols=16), moe.MOE_ERR_SHAPE),
    (dict(rows=(1 << 31) - 255, cols=1), moe.MOE_ERR_SHAPE), (dict(rows=1 << 62, cols=1 << 20), moe.MOE_ERR_SHAPE),
    (dict(rows=(1 << 30) - 127, cols=17), moe.MOE_ERR_SHAPE),
    (dict(x=None), moe.MOE_ERR_NULLPTR), (dict(codes=None), moe.MOE_ERR_NULLPTR), (dict(scales=None), moe.MOE_ERR_NULLPTR),
    (dict(x=A + 1), moe.MOE_ERR_ALIGN), (dict(x=A + 2, dtype=3), moe.MOE_ERR_ALIGN), (dict(scales=A + 2), moe.MOE_ERR_ALIGN),
    (dict(rows=0, x=None, codes=None, scales=None), moe.MOE_OK),
])
def test_int8_rows_refuse_before_a_launch(kw, want):
    p = dict(x=A, rows=4, cols=64, dtype=2, codes=2 * A, scales=3 * A)
    p.update(kw)
    lib = moe.library()
    assert lib.moe_int8_quantize(P(p["x"]), p["rows"], p["cols"], p["dtype"], P(p["codes"]), P(p["scales"]), None) == want
    assert lib.moe_int8_dequantize(P(p["codes"]), P(p["scales"]), p["rows"], p["cols"], p["dtype"], P(p["x"]), None) == want


@pytest.mark.parametrize("kw,want", [
    (dict(W=1), moe.MOE_ERR_SHAPE), (dict(W=769), moe.MOE_ERR_SHAPE), (dict(epr=0), moe.MOE_ERR_SHAPE),
    (dict(W=8, epr=129), moe.MOE_ERR_SHAPE), (dict(rows=-1), moe.MOE_ERR_SHAPE), (dict(k=8), moe.MOE_ERR_SHAPE),
    (dict(k=72), moe.MOE_ERR_SHAPE), (dict(k=131072), moe.MOE_ERR_SHAPE), (dict(n=0), moe.MOE_ERR_SHAPE),
    (dict(act=1, n=7), moe.MOE_ERR_SHAPE), (dict(act=2), moe.MOE_ERR_SHAPE), (dict(dtype=0), moe.MOE_ERR_DTYPE),
    (dict(dtype=3), moe.MOE_ERR_DTYPE), (dict(rows=1 << 30, n=1 << 20), moe.MOE_ERR_SHAPE),
    (dict(rows=(1 << 31) - 200, n=2), moe.MOE_ERR_SHAPE), (dict(k=1 << 16, n=(1 << 15) + 1), moe.MOE_ERR_SHAPE),
    (dict(x=None), moe.MOE_ERR_NULLPTR), (dict(w=None), moe.MOE_ERR_NULLPTR), (dict(ws=None), moe.MOE_ERR_NULLPTR),
    (dict(erc=None), moe.MOE_ERR_NULLPTR), (dict(out=None), moe.MOE_ERR_NULLPTR), (dict(x=A + 8), moe.MOE_ERR_ALIGN),
    (dict(w=A + 4), moe.MOE_ERR_ALIGN), (dict(xs=A + 2), moe.MOE_ERR_ALIGN), (dict(ws=A + 1), moe.MOE_ERR_ALIGN),
    (dict(erc=A + 2), moe.MOE_ERR_ALIGN), (dict(out=A + 1), moe.MOE_ERR_ALIGN),
    (dict(rows=0, x=None, xs=None, out=None), moe.MOE_OK),
])
def test_int8_product_refuses_before_a_launch(kw, want):
    p = dict(x=A, xs=2 * A, w=3 * A, ws=4 * A, erc=5 * A, W=2, epr=2, rows=8, k=64, n=32, act=0, dtype=2, out=6 * A)
    p.update(kw)
    assert moe.library().moe_expert_product_int8(P(p["x"]), P(p["xs"]), P(p["w"]), P(p["ws"]), P(p["erc"]), p["W"], p["epr"],
                                                 p["rows"], p["k"], p["n"], p["act"], p["dtype"], P(p["out"]), None) == want


def _args(W=2, epr=3, rows=10, k=48, n=32):
    E, i8 = W * epr, dict(dtype=torch.int8)
    return dict(out=torch.zeros((rows, n), dtype=torch.bfloat16), x=torch.zeros((rows, k), **i8), x_scales=torch.zeros(rows),
                weights=torch.zeros((E, n, k), **i8), weight_scales=torch.zeros((E, n)),
                ep_recv_count=torch.zeros((W, E), dtype=torch.int32))


def test_well_formed_int8_calls_reach_the_library(rec):  # noqa: F811
    moe.expert_product_into(**_args())
    a = _args()
    del a["out"]
    assert moe.expert_product(**dict(a, x_scales=None), activation=SWIGLU, dtype=torch.float16).shape == (10, 16)
    c, s = moe.quantize_int8(torch.zeros(3, 2, 37))
    assert c.shape == (3, 2, 37) and c.dtype == torch.int8 and s.shape == (3, 2)
    assert moe.dequantize_int8(c, s).shape == (3, 2, 37)
    c, s = moe.quantize_int8(torch.zeros(5).half())
    assert c.shape == (5,) and s.shape == () and moe.dequantize_int8(c, s, torch.float32).shape == (5,)
    assert rec.calls == ["moe_expert_product_int8"] * 2 + ["moe_int8_quantize", "moe_int8_dequantize"] * 2


@pytest.mark.parametrize("field,value", [
    ("x", torch.zeros((9, 48), dtype=torch.int8)), ("x", torch.zeros((48, 10), dtype=torch.int8).t()),
    ("x", torch.zeros((10, 47), dtype=torch.int8)), ("x_scales", torch.zeros(9)), ("x_scales", torch.zeros(10, 1)),
    ("x_scales", torch.zeros(10).bfloat16()), ("weights", torch.zeros((6, 32, 48), dtype=torch.uint8)),
    ("weights", torch.zeros((7, 32, 48), dtype=torch.int8)), ("weights", torch.zeros((6, 32, 64), dtype=torch.int8)),
    ("weight_scales", torch.zeros(6, 31)), ("weight_scales", torch.zeros((6, 32), dtype=torch.uint8)), ("weight_scales", None),
    ("ep_recv_count", torch.zeros((2, 5), dtype=torch.int32)), ("ep_recv_count", torch.zeros((4, 6), dtype=torch.int32)),
    ("ep_recv_count", torch.zeros((2, 6), dtype=torch.int64)), ("out", torch.zeros((10, 32))),
    ("out", torch.zeros((10, 16), dtype=torch.bfloat16)), ("out", torch.zeros((9, 32), dtype=torch.bfloat16)),
], ids=lambda v: v if isinstance(v, str) else "")
def test_int8_product_rejects_before_the_call(rec, field, value):  # noqa: F811
    with pytest.raises(moe.MoeError):
        moe.expert_product_into(**dict(_args(), **{field: value}))
    assert rec.calls == []


def test_int8_wrappers_reject_before_the_call(rec):  # noqa: F811
    c, s, x = torch.zeros((4, 24), dtype=torch.int8), torch.zeros(4), torch.zeros(4, 24)
    for call in (lambda: moe.quantize_int8(x.double()), lambda: moe.quantize_int8(x.t()), lambda: moe.quantize_int8(x[:, :0]),
                 lambda: moe.quantize_int8(torch.tensor(1.0)), lambda: moe.quantize_int8_into(c, s[:3], x),
                 lambda: moe.quantize_int8_into(c.view(torch.uint8), s, x), lambda: moe.quantize_int8_into(c[:3], s, x),
                 lambda: moe.quantize_int8_into(c, s.double(), x), lambda: moe.dequantize_int8(c, s, torch.int32),
                 lambda: moe.dequantize_int8(c.view(torch.uint8), s), lambda: moe.dequantize_int8(c, s[:, None]),
                 lambda: moe.dequantize_int8(torch.tensor(1, dtype=torch.int8), s),
                 lambda: moe.dequantize_int8_into(torch.zeros(4, 25), c, s)):
        with pytest.raises(moe.MoeError):
            call()
    assert rec.calls == []


def _meta(*shape, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device="meta")


@pytest.mark.parametrize("kw", [dict(rows=BIG + 4), dict(k=BIG + 64), dict(n=BIG + 32), dict(activation=BIG)])
def test_int8_sizes_beyond_a_c_int_are_refused_not_cut_off(rec, kw):  # noqa: F811
    p = dict(dict(rows=4, k=64, n=32, activation=NONE), **kw)
    with pytest.raises(moe.MoeError) as e:
        moe.expert_product(_meta(p["rows"], p["k"], dtype=torch.int8), None, _meta(4, p["n"], p["k"], dtype=torch.int8),
                           _meta(4, p["n"], dtype=torch.float32), _meta(2, 4, dtype=torch.int32), p["activation"])
    assert e.value.status == moe.MOE_ERR_SHAPE and rec.calls == []
    with pytest.raises(moe.MoeError):
        moe.quantize_int8(_meta(1, BIG + 32))


def test_int8_calls_reject_cpu_tensors():
    with pytest.raises(moe.MoeError):
        moe.quantize_int8(torch.zeros(4, 64))
    with pytest.raises(moe.MoeError):
        moe.expert_product_into(**_args())


# ---- rows, on the GPU ----

def plain_rows(x):
    """Codes and scales by the definition, binary32 divisions in numpy."""
    v = x.float().numpy()
    top = np.abs(v).max(1, keepdims=True)
    fine = np.isfinite(v).all(1, keepdims=True)
    with np.errstate(all="ignore"):
        scale = np.where(fine, top / np.float32(127), np.float32("nan")).astype(np.float32)
        codes = np.where(fine & (scale > 0), np.rint(v / scale), 0).clip(-127, 127)
    return codes.astype(np.int8), scale[:, 0]


def rows_of(n, cols, dtype, seed):
    """Rows of different size with outliers, zeros, negative zeros, subnormals, ties, the largest values, and some that are
    not finite."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, cols, generator=g) * torch.exp(2 * torch.randn(n, 1, generator=g))
    x[:, ::7] *= 20
    x = x.to(dtype)
    f = torch.finfo(dtype)
    if n > 8:
        x[1] = 0
        x[2] = -0.0
        x[3] = f.tiny * torch.randn(cols, generator=g).to(dtype)
        x[4] = f.max
        x[4, ::2] = -f.max
        x[5] = (torch.arange(cols) % 255 - 127).to(dtype) / 2         # quotients of whole and half codes
        x[5, 0] = 127
        x[6] = f.smallest_normal * f.eps                              # the smallest subnormal
        x[7, cols // 2] = float("inf")
        x[8, cols - 1] = float("nan")
    return x


COLS = [1, 15, 16, 17, 48, 255, 256, 257, 1000, 1024, 1025, 2048, 2049, 2064, 4096, 4111, 7168, 8192, 8193, 16384, 16400, 40000]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("cols", COLS)
def test_int8_rows_are_the_definitions(cols, dtype):
    x = rows_of(37, cols, dtype, cols)
    codes, scales = moe.quantize_int8(x.to(DEV))
    c, s = plain_rows(x)
    assert np.array_equal(codes.cpu().numpy(), c) and np.array_equal(scales.cpu().numpy(), s, equal_nan=True)
    for out in TYPES:
        # one product in binary32, rounded to the type
        want = (torch.from_numpy(c).float() * torch.from_numpy(s)[:, None]).to(out)
        got = moe.dequantize_int8(codes, scales, out).cpu()
        bits = torch.int32 if out == torch.float32 else torch.int16
        assert torch.equal(got.isnan(), want.isnan())
        assert torch.equal(got.view(bits)[~want.isnan()], want.view(bits)[~want.isnan()])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=str)
@pytest.mark.parametrize("h", [64, 520, 7168])
def test_int8_rows_are_dispatchs(h, dtype):
    W, bs, epr, K = 4, 30, 2, 3
    g = torch.Generator().manual_seed(h)
    x = rows_of(W * bs, h, dtype, h)
    x[7:9] = 1                                                         # dispatch takes finite tokens
    ids = torch.rand(W * bs, W * epr, generator=g).argsort(dim=1)[:, :K].int().contiguous().to(DEV)
    rows, scales, assist, _ = moe.dispatch(x.to(DEV), ids, W, epr, moe.MOE_QUANT_DYN_TOKEN)
    codes, mine = moe.quantize_int8(x.to(DEV))
    token = (assist[:, 0] * bs + assist[:, 1]).long()
    assert torch.equal(rows, codes[token]) and torch.equal(scales, mine[token])


@pytest.mark.gpu
def test_int8_rows_of_many_and_none():
    """More rows than workgroups, and rows of fewer pieces than lanes; calls without rows."""
    x = torch.randn(300001, 24, generator=torch.Generator().manual_seed(2)).bfloat16()
    codes, scales = moe.quantize_int8(x.to(DEV))
    c, s = plain_rows(x)
    assert np.array_equal(codes.cpu().numpy(), c) and np.array_equal(scales.cpu().numpy(), s)
    codes, scales = moe.quantize_int8(x[:0].to(DEV))
    assert codes.shape == (0, 24) and scales.shape == (0,) and moe.dequantize_int8(codes, scales).shape == (0, 24)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("cols", [5, 48, 1037, 9000])
def test_int8_rows_at_any_alignment_leave_the_neighbours_alone(cols, dtype):
    n = 13
    x = rows_of(n, cols, dtype, 3).to(DEV)
    want = moe.quantize_int8(x)
    back = moe.dequantize_int8(*want, dtype)

    def odd(shape, dt, fill=7, pad=3):
        whole = torch.full((int(np.prod(shape)) + 40,), fill, dtype=dt, device=DEV)
        return whole, whole[pad:pad + int(np.prod(shape))].view(shape)

    _, xo = odd((n, cols), dtype)
    xo.copy_(x)
    cw, co = odd((n, cols), torch.int8)
    sw, so = odd((n,), torch.float32)
    moe.quantize_int8_into(co, so, xo)
    ow, oo = odd((n, cols), dtype)
    moe.dequantize_int8_into(oo, co, so)
    assert torch.equal(co, want[0]) and torch.equal(so.isnan(), want[1].isnan())
    assert torch.equal(so.nan_to_num(), want[1].nan_to_num()) and torch.equal(oo.nan_to_num(), back.nan_to_num())
    for whole, size in ((cw, n * cols), (sw, n), (ow, n * cols)):
        assert (whole[:3] == 7).all() and (whole[3 + size:] == 7).all()


# ---- the product, on the GPU ----

def draw(per_expert, W, k, n, seed, spare=0, scaled=True, full=False):
    """Codes over the whole range of int8 and scales: (x, xs, w, ws, counts)."""
    g = torch.Generator().manual_seed(seed)
    E, rows = len(per_expert), int(sum(per_expert)) + spare
    i8 = lambda *s: torch.randint(-128, 128, s, generator=g, dtype=torch.int8) if not full else torch.full(s, -128, dtype=torch.int8)
    x, w = i8(rows, k), i8(E, n, k)
    xs = torch.exp(torch.randn(rows, generator=g)) / 100 if scaled else None
    ws = torch.exp(torch.randn(E, n, generator=g)) * k ** -0.5 / 100
    return x, xs, w, ws, counts_for(per_expert, W, seed)


def on_gpu(args):
    return [None if t is None else t.to(DEV) for t in args]


def check(per_expert, W, k, n, act=NONE, dtype=torch.bfloat16, seed=0, spare=0, scaled=True, full=False):
    x, xs, w, ws, counts = args = draw(per_expert, W, k, n, seed, spare, scaled, full)
    fo = n // 2 if act == SWIGLU else n
    out = torch.full((x.shape[0], fo), 7.0, dtype=dtype, device=DEV)
    x, xs, w, ws, counts = args = on_gpu(args)
    moe.expert_product_into(out, *args, activation=act)
    got, f, row = out.double(), torch.finfo(dtype), 0
    for e, c in enumerate(per_expert):
        if c == 0:
            continue
        y = x[row:row + c].double() @ w[e].double().t()        # whole numbers below 2^31: exact in binary64
        y = y * ws[e].double()
        if scaled:
            y = y * xs[row:row + c, None].double()
        room = 3.01 * U * y.abs()                              # the sum as binary32, and two products
        if act == SWIGLU:
            g, u, dg, du = y[:, :fo], y[:, fo:], room[:, :fo], room[:, fo:]
            s = g / (1 + torch.exp(-g))
            y = s * u
            # silu of a gate that is off by dg: its slope is at most 1.1 in size; an exponential and a reciprocal off by a few
            # units, the exponent's argument by |g| half steps
            room = 1.1 * dg * (u.abs() + du) + s.abs() * du + (16 + g.abs()) * U * y.abs()
        ref, mine = y, got[row:row + c]
        if dtype == torch.float16:
            ref, mine = ref.clamp(-f.max, f.max), mine.clamp(-f.max, f.max)
        limit = room + f.eps / 2 * (ref.abs() + room) + f.tiny * f.eps
        err = (mine - ref).abs()
        assert (err <= limit).all(), (e, c, float((err / limit).max()), torch.nonzero(err > limit)[:4])
        row += c
    assert (got[row:] == 7.0).all()                            # rows behind the last are left alone
    return got


@pytest.mark.gpu
@pytest.mark.parametrize("act", [NONE, SWIGLU])
@pytest.mark.parametrize("k,n", [(16, 2), (32, 16), (48, 30), (64, 64), (80, 34), (128, 66), (144, 130), (192, 64), (256, 96),
                                 (320, 258), (384, 34), (400, 2), (512, 514), (640, 62), (1040, 96), (2064, 18)])
@pytest.mark.parametrize("per_expert", [[20, 1], [100, 60], [300, 180]], ids=str)
def test_int8_product_shapes(per_expert, act, k, n):
    check(per_expert, 2, k, n, act, seed=k + n)


# Rows and columns by which a call takes each shape of a tile (rows x weight rows), with last tiles of every number of
# fragments, and lengths of no, one, two, ... seven whole stages and a rest.
TILES = {"256x256": ([2078, 2148, 2228, 2000], 4096), "128x256": ([100, 40, 128, 64, 65, 1, 0, 200, 129, 100, 96, 33] + [100] * 4, 7168),
         "128x128": ([1000, 929, 1090, 0], 800), "32x128": ([31, 33, 64, 1], 1000),         # 32x64 from k 512 on
         "32x128 of long rows": ([31, 33, 64, 1], 4600)}


@pytest.mark.gpu
@pytest.mark.parametrize("act", [NONE, SWIGLU])
@pytest.mark.parametrize("k", [48, 128, 272, 384, 640, 768, 1008])
@pytest.mark.parametrize("tile", list(TILES))
def test_int8_product_in_every_shape_of_a_tile(tile, k, act):
    per_expert, n = TILES[tile]
    check(per_expert, 2, k, n, act, seed=k, spare=5)
    if k == 272:
        check(per_expert, 2, k, n - 118, act, torch.float16, seed=1)      # a last tile of few columns


@pytest.mark.gpu
@pytest.mark.parametrize("act", [NONE, SWIGLU])
@pytest.mark.parametrize("k", [512, 528, 656, 896, 1040, 2064, 7168])
@pytest.mark.parametrize("per_expert", [[1, 0], [16, 17], [0, 32, 33, 3], [100, 2], [1] * 16], ids=str)
def test_int8_product_of_few_tiles(per_expert, k, act):
    check(per_expert, 2, k, 134, act, seed=k, spare=3)
    check(per_expert, 2, k, 66, act, torch.float16, seed=k + 1, scaled=False)


@pytest.mark.gpu
@pytest.mark.parametrize("per_expert,W", [([0, 0], 2), ([1, 0], 2), ([0, 17], 2), ([40, 0, 0, 5], 4), ([33] * 8, 8),
                                          ([64, 128, 129, 63], 2), ([256, 257, 0, 255], 4), ([700, 3], 2), ([0, 0, 900], 3)], ids=str)
@pytest.mark.parametrize("spare", [0, 9])
def test_int8_product_rows_per_expert(per_expert, W, spare):
    if sum(per_expert) + spare:
        check(per_expert, W, 208, 70, seed=W, spare=spare)


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1, 3, 33, 127, 129, 255, 257])
def test_int8_product_odd_columns(n):
    check([20, 5], 2, 96, n, seed=n)
    check([200, 90], 2, 96, n, seed=n)
    check([20, 350], 2, 96, 2 * n, SWIGLU, seed=n)


@pytest.mark.gpu
@pytest.mark.parametrize("per_expert,n,act", [([(17 * e) % 90 for e in range(1024)], 34, SWIGLU), ([260, 0] * 120, 514, NONE),
                                              ([100] * 300, 300, SWIGLU)], ids=["1024 experts", "tall", "middle"])
def test_int8_product_of_more_tiles_than_workgroups(per_expert, n, act):
    check(per_expert, 4, 272, n, act, seed=3)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=str)
@pytest.mark.parametrize("act", [NONE, SWIGLU])
@pytest.mark.parametrize("scaled", [True, False])
@pytest.mark.parametrize("per_expert", [[20, 1], [200, 50], [700, 90]], ids=str)
def test_int8_product_types(dtype, act, scaled, per_expert):
    check(per_expert, 2, 528, 96, act, dtype, seed=7, spare=3, scaled=scaled)


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [5, 100, 300])
def test_int8_product_of_the_longest_rows_at_the_largest_sum(rows):
    """131056 products of -128 by -128: 2147221504, the largest sum there is, and random ones of that length."""
    check([rows, 3], 2, 131056, 40, full=True, seed=1)
    check([rows, 3], 2, 131056, 40, SWIGLU, seed=2)


@pytest.mark.gpu
def test_int8_product_rows_do_not_depend_on_each_other():
    """An expert's rows by themselves and among many: all shapes of a tile give the same bits. Scales that are not finite
    stay in their row or column."""
    per, W, k, n = [30, 2500, 5], 3, 656, 4096
    x, xs, w, ws, counts = draw(per, W, k, n, 11)
    bad = xs.clone()
    bad[3], bad[100] = float("nan"), float("inf")
    wbad = ws.clone()
    wbad[1, 7] = float("nan")
    for act in (NONE, SWIGLU):
        whole = moe.expert_product(*on_gpu((x, xs, w, ws, counts)), act)
        for rows in ([30, 0, 0], [0, 40, 0], [0, 300, 0], [0, 1200, 0], [0, 2500, 0], [0, 0, 5]):
            e = int(np.argmax(rows))
            first = sum(per[:e])
            part = slice(first, first + rows[e])
            alone = moe.expert_product(*on_gpu((x[part].contiguous(), xs[part].contiguous(), w, ws, counts_for(rows, W, 1))), act)
            assert torch.equal(alone, whole[part]), (act, rows)
        got = moe.expert_product(*on_gpu((x, bad, w, wbad, counts)), act)
        fine = torch.ones(2535, whole.shape[1], dtype=torch.bool, device=DEV)
        fine[3], fine[100], fine[30:2530, 7] = False, False, False
        assert torch.equal(got[fine], whole[fine]) and got[3].isnan().all() and got[30:2530, 7].isnan().all()
        assert not torch.isfinite(got[100]).any() or act == SWIGLU


@pytest.mark.gpu
@pytest.mark.parametrize("bad", ["negative", "descending", "huge"])
def test_int8_product_stays_in_bounds_on_counts_it_should_not_get(bad):
    for per, n in [([30, 70, 1, 20], 48), *TILES.values()]:
        x, xs, w, ws, counts = draw(per, 2, 160, n, 3)
        counts = {"negative": -counts, "descending": counts.flip(1).contiguous(),
                  "huge": torch.full_like(counts, 2 ** 31 - 1)}[bad]
        rows = x.shape[0]
        whole = torch.full((rows + 64, n), 7.0, dtype=torch.bfloat16, device=DEV)
        moe.expert_product_into(whole[32:32 + rows], *on_gpu((x, xs, w, ws, counts)))
        assert (whole[:32] == 7.0).all() and (whole[32 + rows:] == 7.0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1, 3, 37, 66])
def test_int8_product_into_an_output_of_any_alignment(n):
    args = on_gpu(draw([20, 5], 2, 96, n, n))
    want = moe.expert_product(*args)
    flat = torch.full((25 * n + 9,), 7.0, dtype=torch.bfloat16, device=DEV)
    out = flat[5:5 + 25 * n].view(25, n)
    moe.expert_product_into(out, *args)
    assert torch.equal(out, want) and (flat[:5] == 7.0).all() and (flat[5 + 25 * n:] == 7.0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("act", [NONE, SWIGLU])
def test_int8_product_of_operands_beyond_4_gib(act):
    """2^20 rows and more of 4112 bytes, results of as many columns: rows on both sides of the 4 GiB line and at the end are
    those of a call with these rows alone."""
    k, n = 4112, 4112 * (1 if act == NONE else 2)
    per, W = [5, 1 << 20, 0, 777], 2
    rows = sum(per)
    g = torch.Generator(DEV).manual_seed(5)
    x = torch.randint(-128, 128, (rows, k), generator=g, device=DEV, dtype=torch.int8)
    w = torch.randint(-128, 128, (4, n, k), generator=g, device=DEV, dtype=torch.int8)
    xs = torch.rand(rows, generator=g, device=DEV) / 1000
    ws = torch.rand(4, n, generator=g, device=DEV) / 1000

    def totals(per):
        a, b, c, d = per
        return torch.tensor([[a, a, a + b, a + b], [c, c, c + d, c + d]], dtype=torch.int32, device=DEV)

    out = moe.expert_product(x, xs, w, ws, totals(per), act)
    line = (1 << 32) // 4112
    for at, part in ((slice(0, 5), [5, 0, 0, 0]), (slice(5, 100), [0, 95, 0, 0]),
                     (slice(line - 60, line + 60), [0, 120, 0, 0]), (slice(line // 2 - 60, line // 2 + 60), [0, 120, 0, 0]),
                     (slice(rows - 777, rows), [0, 0, 0, 777])):
        small = moe.expert_product(x[at].contiguous(), xs[at].contiguous(), w, ws, totals(part), act)
        assert torch.equal(small, out[at]), at
    del out
    torch.cuda.empty_cache()
    codes, scales = moe.quantize_int8(x.view(torch.bfloat16)[:, :2048].nan_to_num().contiguous())
    back = moe.dequantize_int8(codes, scales)
    for at in (slice(0, 50), slice((1 << 31) // 2048 - 50, (1 << 31) // 2048 + 50), slice(rows - 50, rows)):
        c, s = moe.quantize_int8(x[at].view(torch.bfloat16)[:, :2048].nan_to_num().contiguous())
        assert torch.equal(c, codes[at]) and torch.equal(s, scales[at]) and torch.equal(moe.dequantize_int8(c, s), back[at])


@pytest.mark.gpu
def test_two_int8_products_at_once_and_replayed():
    sets = [on_gpu(draw(per, 2, 1040, 96, s)) for s, per in ((1, [40, 3, 0, 90]), (2, [10, 400, 300, 0]))]
    want = [moe.expert_product(*d, SWIGLU) for d in sets]
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream(), torch.cuda.Stream()], [torch.empty_like(w) for w in want]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, d, o in zip(streams, sets, outs):
            with torch.cuda.stream(s):
                moe.expert_product_into(o, *d, activation=SWIGLU)
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, want))
    x = torch.randn(133, 1040, device=DEV)
    codes, scales = moe.quantize_int8(x)
    y, d = torch.empty_like(want[0]), sets[0]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.quantize_int8_into(codes, scales, x)
        moe.expert_product_into(y, codes, scales, *d[2:], activation=SWIGLU)
    for i in range(4):
        x.copy_(torch.randn(133, 1040, generator=torch.Generator().manual_seed(i)))
        d[4].copy_(counts_for([40 - i, 3 + i, 0, 90], 2, i))
        graph.replay()
        torch.cuda.synchronize()
        got = y.clone()
        ref = moe.expert_product(*moe.quantize_int8(x), *d[2:], SWIGLU)
        torch.cuda.synchronize()
        assert torch.equal(got, ref)


@pytest.mark.gpu
@pytest.mark.parametrize("mode", [moe.MOE_QUANT_DYN_TOKEN, moe.MOE_QUANT_STATIC])
def test_the_whole_layer_on_int8_rows(mode):
    """gate -> dispatch (int8) -> product with SwiGLU -> quantise -> product -> combine, each product against binary64 from
    its own inputs; the combined tokens against the second product's rows."""
    W, bs, epr, h, f, K = 4, 12, 4, 160, 96, 4
    N, E = W * bs, W * epr
    g = torch.Generator().manual_seed(17)
    x = torch.randn(N, h, generator=g).bfloat16()
    logits = torch.randn(N, E, generator=g)
    logits[3, 2:] = -float("inf")
    w1, w2 = torch.randn(E, 2 * f, h, generator=g) * h ** -0.5, torch.randn(E, h, f, generator=g) * f ** -0.5
    q1, s1 = moe.quantize_int8(w1.to(DEV))
    q2, s2 = moe.quantize_int8(w2.to(DEV))
    ids, wt, on = moe.gate(logits.to(DEV), K, moe.MOE_SCORE_SIGMOID, with_pair_mask=True)
    coefficient = 32.0
    qs = torch.full((1,), coefficient, device=DEV) if mode == moe.MOE_QUANT_STATIC else None
    rows, rs, assist, erc = moe.dispatch(x.to(DEV), ids, W, epr, mode, x_active_mask=on, quant_scales=qs)
    if mode == moe.MOE_QUANT_STATIC:
        assert rs is None
        s1 = s1 / coefficient
    A = int(on.sum())
    y1 = moe.expert_product(rows, rs, q1, s1, erc, SWIGLU)
    y1[A:] = 0
    r2, rs2 = moe.quantize_int8(y1)
    y2 = moe.expert_product(r2, rs2, q2, s2, erc)
    out = moe.combine(y2, assist, erc, ids, wt, W, epr, x_active_mask=on).cpu().double()

    ends = (erc.cpu()[:, W - 1::W].long() + torch.cat((torch.zeros(1).long(), erc.cpu()[:, -1].long().cumsum(0)[:-1]))[:, None]).flatten()
    assert int(ends[-1]) == A < N * K
    expert = torch.searchsorted(ends, torch.arange(A), right=True)
    a = assist.cpu()[:A].long()
    tok = a[:, 0] * bs + a[:, 1]
    assert torch.equal(ids.cpu()[tok, a[:, 2]].long(), expert)
    # whole sums first (exact in binary64), then the scales: a sum of 0 has to come out as 0
    sums = lambda r, rs, q, qs: (torch.linalg.vecdot(r[:A].cpu().double()[:, None], q.cpu().double()[expert])
                                 * qs.cpu().double()[expert] * (1.0 if rs is None else rs[:A].cpu().double()[:, None]))
    z = sums(rows, rs, q1, s1)
    G, Up = z[:, :f], z[:, f:]
    want = G / (1 + torch.exp(-G)) * Up
    room = (1.1 * 3.01 * U * G.abs() + 3.01 * U * G.abs() + (16 + G.abs()) * U * G.abs()) * Up.abs() * 1.01
    assert ((y1[:A].cpu().double() - want).abs() <= room + 2.0 ** -8 * (want.abs() + room) + 1e-38).all()
    z2 = sums(r2, rs2, q2, s2)
    got2 = y2[:A].cpu().double()
    assert ((got2 - z2).abs() <= (2.0 ** -8 + 4 * U) * z2.abs() + 1e-38).all()
    part = got2 * wt.cpu().double()[tok, a[:, 2]][:, None]
    ref, size = torch.zeros(N, h).double().index_add_(0, tok, part), torch.zeros(N, h).double().index_add_(0, tok, part.abs())
    assert ((out - ref).abs() <= 2.0 ** -8 * ref.abs() + (2 * K) * U * 1.01 * size + 1e-38).all()
    assert (out[~on.cpu().any(1)] == 0).all()

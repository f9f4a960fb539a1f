"""The int8 product in every shape of a tile: more tiles than workgroups, rows without scales, odd columns, the longest rows and
the largest sum, and rows that give the same bits whichever shape takes them. Sizes are those by which a call takes the shape
that a case is named after."""
import pytest
import torch

import combine_ep_recv_amd as moe
import test_int8
from test_int8 import NONE, SWIGLU, check, draw, on_gpu
from test_mx_rows import counts_for

DEV = "cuda"


@pytest.mark.gpu
@pytest.mark.parametrize("k", [528, 1040])
@pytest.mark.parametrize("act", [NONE, SWIGLU])
@pytest.mark.parametrize("tile", ["32x128", "32x64"])
def test_int8_product_of_more_small_tiles_than_workgroups(tile, act, k):
    """Eight rounds of 32 x 128, two of 32 x 64: experts without rows, one of two row tiles, a last tile of few columns."""
    if tile == "32x128":
        per_expert, n = [(5 * e) % 11 for e in range(63)] + [40], 4108 if act == SWIGLU else 4102
    else:
        per_expert, n = [e % 6 for e in range(639)] + [40], 58
    check(per_expert, 4, k, n, act, seed=k, spare=3)
    check(per_expert, 4, k, n, act, torch.float16, seed=k + 1, scaled=False)


SHAPES = {"256x256": ([2078, 2148, 2228, 2000], 400, 4091), "128x128": ([1000, 929, 1090, 0], 400, 801),
          "128x256": ([100, 40, 128, 64, 65, 1, 0, 200, 129, 100, 96, 33] + [100] * 4, 400, 7161),
          "32x128": ([31, 33, 64, 1], 400, 997), "32x64": ([31, 33, 64, 1], 528, 133)}


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=str)
@pytest.mark.parametrize("scaled", [True, False])
@pytest.mark.parametrize("tile", list(SHAPES))
def test_int8_product_of_odd_columns_in_every_shape_of_a_tile(tile, scaled, dtype):
    per_expert, k, n = SHAPES[tile]
    check(per_expert, 2, k, n, NONE, dtype, seed=7, spare=3, scaled=scaled)
    check(per_expert, 2, k, n // 4 * 4 + 2, SWIGLU, dtype, seed=8, spare=3, scaled=scaled)


@pytest.fixture
def codes_from_the_gpu(monkeypatch):
    """check's inputs, made on the GPU: gigabytes of them."""
    def draw(per_expert, W, k, n, seed, spare=0, scaled=True, full=False):
        g = torch.Generator(DEV).manual_seed(seed)
        E, rows = len(per_expert), sum(per_expert) + spare
        i8 = lambda *s: (torch.full(s, -128, dtype=torch.int8, device=DEV) if full else
                         torch.randint(-128, 128, s, generator=g, dtype=torch.int8, device=DEV))
        x, w = i8(rows, k), i8(E, n, k)
        xs = torch.exp(torch.randn(rows, generator=g, device=DEV)) / 100 if scaled else None
        ws = torch.exp(torch.randn(E, n, generator=g, device=DEV)) * k ** -0.5 / 100
        return x, xs, w, ws, counts_for(per_expert, W, seed)

    monkeypatch.setattr(test_int8, "draw", draw)
    yield
    torch.cuda.empty_cache()


@pytest.mark.gpu
@pytest.mark.parametrize("per_expert,n", [([1500, 1500], 2815), ([500, 420], 4999), ([300, 270], 2001), ([40, 500], 1001)],
                         ids=["256x256", "128x256", "128x128", "32x128"])
def test_int8_product_of_the_longest_rows_in_the_larger_tiles(codes_from_the_gpu, per_expert, n):
    """131056 products of -128 by -128: 2147221504, the largest sum there is, and random ones of that length."""
    check(per_expert, 2, 131056, n, full=True, seed=1)
    check(per_expert, 2, 131056, n - 1, SWIGLU, seed=2)


@pytest.mark.gpu
def test_int8_product_rows_of_fewer_columns_do_not_depend_on_each_other():
    """Below 512 columns few rows go in tiles of 32 x 128, others of 128 x 128, 128 x 256 and 256 x 256: the same bits."""
    per, W, k, n = [30, 2500, 5], 3, 400, 4096
    x, xs, w, ws, counts = draw(per, W, k, n, 12)
    for act in (NONE, SWIGLU):
        whole = moe.expert_product(*on_gpu((x, xs, w, ws, counts)), act)
        for rows in ([30, 0, 0], [0, 40, 0], [0, 300, 0], [0, 1200, 0], [0, 2500, 0], [0, 0, 5]):
            e = max(range(3), key=rows.__getitem__)
            first = sum(per[:e])
            part = slice(first, first + rows[e])
            alone = moe.expert_product(*on_gpu((x[part].contiguous(), xs[part].contiguous(), w, ws, counts_for(rows, W, 1))), act)
            assert torch.equal(alone, whole[part]), (act, rows)

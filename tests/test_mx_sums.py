"""The sums of the experts' product: every product of an E4M3 row counts, in every tile.

Tolerance of a result. Inside a block of 32 the products of a part (E4M3 rows are multiplied in two, E2M1 rows in one) add
up exactly: they are multiples of one power of two, and 32 of the largest stay below 2^20 of it. A matrix instruction
then adds four such blocks and the accumulator, four additions in fp32 that may cut off as well as round, 2^-23 of the
sum of magnitudes M = sum |x w| each. A row of k elements takes ceil(k / 128) steps of one or two instructions: at most
4 parts ceil(k / 128) 2^-23 M in all. The output is rounded once, half a step. SwiGLU passes an error e of the gate on as at
most 1.1 |up| e and one of the up projection as |silu(gate)| e, and its own exponential, reciprocal and products take
up to (16 + |gate|) 2^-24 of the result.
"""
import numpy as np
import pytest
import torch

import combine_ep_recv_amd as moe
from test_mx_rows import DEV, E2M1, E4M3, NONE, SWIGLU, counts_for, draw_product, on_gpu, values


def check_sums(per_expert, W, k, n, element, act=NONE, dtype=torch.bfloat16, seed=0, spare=0, spread=2):
    x, xs, w, ws, counts = draw_product(per_expert, W, k, n, element, seed, spare, spread)
    fo = n // 2 if act == SWIGLU else n
    out = torch.full((x.shape[0], fo), 7.0, dtype=dtype, device=DEV)
    moe.expert_product_into(out, *on_gpu(x, xs, w, ws, counts, element), activation=act)
    got = out.cpu().double().numpy()
    X, row, f = values(x, xs, element), 0, torch.finfo(dtype)
    part = 4 * (1 if element == E2M1 else 2) * -(-k // 128) * 2.0 ** -23
    for e, c in enumerate(per_expert):
        V = values(w[e], ws[e], E2M1)
        y, room = X[row:row + c] @ V.T, part * (np.abs(X[row:row + c]) @ np.abs(V).T)
        if act == SWIGLU:
            g, u, dg, du = y[:, :fo], y[:, fo:], room[:, :fo], room[:, fo:]
            with np.errstate(over="ignore"):
                s = g / (1 + np.exp(-g))
            y = s * u
            room = 1.1 * dg * (np.abs(u) + du) + np.abs(s) * du + (16 + np.abs(g)) * 2.0 ** -24 * np.abs(y)
        ref = np.clip(y, -f.max, f.max) if dtype == torch.float16 else y
        err = np.abs(np.clip(got[row:row + c], -f.max, f.max) - ref)
        limit = room + f.eps / 2 * (np.abs(ref) + room) + f.tiny * f.eps
        assert (err <= limit).all(), (e, c, err.max(), np.argwhere(err > limit)[:4], (err / limit).max())
        row += c
    assert (got[row:] == 7.0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("k", [128, 528, 1040])
@pytest.mark.parametrize("rows", [5, 60, 300])
def test_product_counts_every_product_of_e4m3_rows(k, rows):
    """Large products that cancel beside ones 2^-21 as large. All are multiples of 2^-10, and their magnitudes add up to
    less than 2^14 (four of 448 * 6 and 1040 of 1/2 * 6), so that fp32 holds every sum of them: the result is the
    exact one, rounded once."""
    rng = np.random.default_rng(k + rows)
    per, W, n = [rows, 0, 3, rows], 2, 48
    total, nb = sum(per), -(-k // 32)
    x = rng.integers(0, 0x31, (total, k)).astype(np.uint8) | (rng.integers(0, 2, (total, k)) << 7).astype(np.uint8)
    w = rng.integers(0, 16, (4, n, k)).astype(np.uint8)
    for at, other in ((3, 9), (40, 100)):             # neighbours, and elements of different blocks
        x[:, at] = x[:, other] = rng.integers(0x78, 0x7f, total)
        w[:, :, at] = 7
        w[:, :, other] = 15
    xs, ws = np.full((total, nb), 127, np.uint8), np.full((4, n, nb), 127, np.uint8)
    counts = counts_for(per, W, 1)
    out = moe.expert_product(*on_gpu(x, xs, w, ws, counts, E4M3)).cpu()
    X, row = values(x, xs, E4M3), 0
    for e, c in enumerate(per):
        V = values(w[e], ws[e], E2M1)
        assert (np.abs(X[row:row + c]) @ np.abs(V).T).max(initial=0) < 2 ** 14
        y = torch.from_numpy(X[row:row + c] @ V.T).to(torch.bfloat16)
        assert torch.equal(out[row:row + c], y), (e, c, (out[row:row + c] != y).sum())
        row += c


@pytest.mark.gpu
@pytest.mark.parametrize("element", [E2M1, E4M3])
@pytest.mark.parametrize("act", [NONE, SWIGLU])
@pytest.mark.parametrize("per_expert", [[30, 1], [120, 90], [500, 300]], ids=str)
@pytest.mark.parametrize("k", [112, 512, 1168])
def test_product_sums_in_fp32(element, act, per_expert, k):
    check_sums(per_expert, 2, k, 150, element, act, seed=k, spare=2)


@pytest.mark.gpu
@pytest.mark.parametrize("element", [E2M1, E4M3])
@pytest.mark.parametrize("per_expert,k", [([100, 90, 130, 70], 528), ([100, 90, 130, 70], 1040), ([300, 250, 17, 400], 528),
                                          ([300, 250, 17, 400], 1040), ([300, 200] * 24, 528)],
                         ids=["128 rows, 528", "128 rows, 1040", "256 rows, 528", "256 rows, 1040", "many tiles"])
def test_swiglu_of_tall_tiles_and_several_columns(element, per_expert, k):
    """SwiGLU where a tile has 128 or 256 rows: three tiles of columns, the last one ragged and of an odd width, and a
    rest of k behind the whole groups; with more tiles than workgroups a workgroup goes from column tile to column tile."""
    check_sums(per_expert, 2, k, 2 * (2 * 128 + 37), element, SWIGLU, seed=k, spare=2)


@pytest.mark.gpu
def test_product_of_e4m3_rows_replayed_with_other_row_counts():
    """One captured call, replayed as the experts' row counts change under it: tiles with one to four fragments of rows,
    whole tiles and none."""
    per, W, k, n = [64, 64, 64, 64], 2, 656, 96
    x, xs, w, ws, counts = draw_product(per, W, k, n, E4M3, 4, spread=2)
    dev = on_gpu(x, xs, w, ws, counts, E4M3)
    out = torch.empty((256, n // 2), dtype=torch.bfloat16, device=DEV)
    moe.expert_product_into(out, *dev, activation=SWIGLU)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.expert_product_into(out, *dev, activation=SWIGLU)
    for i, now in enumerate(([64, 64, 64, 64], [1, 16, 17, 222], [0, 256, 0, 0], [33, 48, 49, 126], [5, 0, 130, 65])):
        dev[4].copy_(counts_for(now, W, i))
        out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        want = torch.full_like(out, 7.0)
        moe.expert_product_into(want, *dev, activation=SWIGLU)
        torch.cuda.synchronize()
        assert torch.equal(got, want)
        if i == 0:
            first = got
    # expert 0's first five rows are the same in every call that gives them to it
    assert torch.equal(got[:5], first[:5])

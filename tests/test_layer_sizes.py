"""The gate, the microscaled rows and the experts' product at the largest sizes they take, and where offsets pass 32 bits.

Rows stand for themselves in all of these operators, so the last rows of a large call must be those of a small one, bit
for bit; the longest rows hold few elements that are not zero, so that their products are whole numbers.
"""
import pytest
import torch

import combine_ep_recv_amd as moe
from test_gate import DEV, SIGMOID, SOFTMAX
from test_mx_rows import E2M1, E4M3, SWIGLU

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def free_memory():
    yield
    torch.cuda.empty_cache()


def _codes(g, shape, element):
    """Random codes of at most 7.5 in size, without NaN, as the bytes that hold them."""
    v = torch.randint(0, 256, shape, generator=g, device=DEV, dtype=torch.uint8)
    return v if element == E2M1 else v & 0xCF


@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID])
def test_gate_of_the_most_tokens(score):
    """2^24 - 1 tokens of 304 experts: 10 GB of logits, and of gradients."""
    N, E = (1 << 24) - 1, 304
    L = torch.randn(N, E, device=DEV, dtype=torch.bfloat16, generator=torch.Generator(DEV).manual_seed(1))
    kw = dict(score=score, renormalize=False, scale=2.0)
    ids, w, on = moe.gate(L, 8, with_pair_mask=True, **kw)
    grad = moe.gate_backward(L, ids, w, w, **kw)
    crossing = (1 << 32) // E
    for rows in (slice(0, 50), slice(crossing - 50, crossing + 50), slice(N - 200, N)):
        part = L[rows].contiguous()
        i, v = moe.gate(part, 8, **kw)
        assert torch.equal(i, ids[rows]) and torch.equal(v, w[rows]) and on[rows].all()
        assert torch.equal(moe.gate_backward(part, i, v, v, **kw), grad[rows])


@pytest.mark.parametrize("element", [E2M1, E4M3])
@pytest.mark.parametrize("cols", [32, 48])
def test_quantize_of_more_than_32_bits_of_elements(element, cols):
    rows = (1 << 27) + 3
    x = torch.randn(rows, cols, device=DEV, dtype=torch.bfloat16, generator=torch.Generator(DEV).manual_seed(2))
    codes, scales = moe.quantize_mx(x, element)
    back = moe.dequantize_mx(codes, scales)
    for at in (slice(0, 100), slice((1 << 32) // cols - 50, (1 << 32) // cols + 50), slice(rows - 100, rows)):
        c, s = moe.quantize_mx(x[at].contiguous(), element)
        assert torch.equal(codes[at].view(torch.uint8), c.view(torch.uint8)) and torch.equal(scales[at], s)
        assert torch.equal(back[at], moe.dequantize_mx(c, s))


@pytest.mark.parametrize("element", [E2M1, E4M3])
@pytest.mark.parametrize("rows", [5, 600])
def test_product_of_the_longest_rows(element, rows):
    """k = 2^24 and n * k = 2^32: codes of whole numbers in 200 columns, the first and last among them. Their products add
    up to at most 200 * 4 * 4 in size, which fp32 holds exactly."""
    k, n, W, g = 1 << 24, 256, 2, torch.Generator(DEV).manual_seed(rows)
    at = torch.cat((torch.tensor([0, 1, (1 << 23) - 1, 1 << 23, k - 2, k - 1], device=DEV),
                    torch.randint(2, k - 2, (194,), generator=g, device=DEV))).unique()
    whole = torch.tensor([0, 2, 4, 6, 10, 12, 14] if element == E2M1 else [0, 56, 64, 72, 184, 192, 200], device=DEV,
                         dtype=torch.uint8)                               # 0, 1, 2, 4, -1, -2, -4
    value = torch.tensor([0, 1, 2, 4, -1, -2, -4], device=DEV, dtype=torch.float64)
    pick = torch.randint(0, 7, (rows, len(at)), generator=g, device=DEV)
    wpick = torch.randint(0, 7, (4, n, len(at)), generator=g, device=DEV)
    w4 = torch.tensor([0, 2, 4, 6, 10, 12, 14], device=DEV, dtype=torch.uint8)

    def place(to, codes, packed):
        for j, c in enumerate(at.tolist()):
            if packed:
                to[..., c // 2] |= codes[..., j] << (4 * (c % 2))
            else:
                to[..., c] = codes[..., j]

    x = torch.zeros((rows, k // 2 if element == E2M1 else k), dtype=torch.uint8, device=DEV)
    w = torch.zeros((4, n, k // 2), dtype=torch.uint8, device=DEV)
    place(x, whole[pick], element == E2M1)
    place(w, w4[wpick], True)
    xs = torch.full((rows, k // 32), 127, dtype=torch.uint8, device=DEV)
    ws = torch.full((4, n, k // 32), 127, dtype=torch.uint8, device=DEV)
    first = rows // 2                                                     # rows of expert 0; the others are expert 3's
    counts = torch.tensor([[0, first, first, first], [0, 0, 0, rows - first]], dtype=torch.int32, device=DEV)
    out = moe.expert_product(x if element == E2M1 else x.view(torch.float8_e4m3fn), xs, w, ws, counts)
    X, V = value[pick], value[wpick]
    want = torch.cat((X[:first] @ V[0].t().contiguous(), X[first:] @ V[3].t().contiguous()))
    assert torch.equal(out, want.to(torch.bfloat16))


@pytest.mark.parametrize("element,k", [(E2M1, 8224), (E4M3, 4112)])
@pytest.mark.parametrize("act", [moe.MOE_ACT_NONE, SWIGLU])
def test_product_of_operands_beyond_4_gib(element, k, act):
    """2^20 rows and more of 4112 bytes, results of as many columns: rows on both sides of the 4 GiB line and at the end
    are those of a call with these rows alone."""
    n, g = 4112 * (1 if act == moe.MOE_ACT_NONE else 2), torch.Generator(DEV).manual_seed(k)
    per = [5, 1 << 20, 0, 777]
    rows, nb = sum(per), -(-k // 32)
    x = _codes(g, (rows, 4112), element)
    w = _codes(g, (4, n, k // 2), E2M1)
    xs = torch.randint(125, 130, (rows, nb), generator=g, device=DEV, dtype=torch.uint8)
    ws = torch.randint(113, 118, (4, n, nb), generator=g, device=DEV, dtype=torch.uint8)
    typed = x if element == E2M1 else x.view(torch.float8_e4m3fn)

    def totals(per):
        a, b, c, d = per
        return torch.tensor([[a, a, a + b, a + b], [c, c, c + d, c + d]], dtype=torch.int32, device=DEV)

    out = moe.expert_product(typed, xs, w, ws, totals(per), act)
    line = (1 << 32) // 4112
    for at, part in ((slice(0, 5), [5, 0, 0, 0]), (slice(5, 100), [0, 95, 0, 0]),
                     (slice(line - 60, line + 60), [0, 120, 0, 0]), (slice(line // 2 - 60, line // 2 + 60), [0, 120, 0, 0]),
                     (slice(rows - 777, rows), [0, 0, 0, 777])):
        small = moe.expert_product(typed[at].contiguous(), xs[at].contiguous(), w, ws, totals(part), act)
        assert torch.equal(small, out[at]), at
    assert torch.isfinite(out[::4097]).all()

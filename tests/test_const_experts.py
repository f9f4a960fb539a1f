"""The gradient of const_x where a const expert has many pairs: lists that are made in several pieces, whose sums are
compared exactly or with the bound of their longest chain, and batches so long that a plain fp32 sum would lose digits."""
import pytest
import torch

import combine_ep_recv_amd as moe
import test_gradients as tg

DEV = "cuda"
U = 2.0 ** -24
PARTS, PART_TOKENS, BLOCK = 64, 32, 1024       # at most so many parts, of so many tokens at least, added 1024 tokens at a time


def parts_of(N):
    return max(1, min(PARTS, -(-N // PART_TOKENS)))


def route(W, bs, epr, K, const, on, seed):
    """K distinct ids of each token, every const expert among them; `on`: part of the pairs that are active."""
    g = torch.Generator(DEV).manual_seed(seed)
    N, E = W * bs, W * epr
    score = torch.rand(N, E + const, generator=g, device=DEV)
    score[:, E:] -= 1
    ids = score.argsort(dim=1)[:, :K]
    # at any place of the token's pairs
    ids = ids.gather(1, torch.rand(N, K, generator=g, device=DEV).argsort(dim=1)).int().contiguous()
    mask = torch.rand(N, K, generator=g, device=DEV) < on if on < 1 else None
    x = torch.zeros((N, 8), dtype=torch.bfloat16, device=DEV)
    _, _, assist, counts = moe.dispatch(x, ids, W, epr, x_active_mask=mask, const_experts=const)
    return g, ids, mask, assist, counts


def gradient(W, bs, epr, K, h, const, dtype, ids, mask, assist, counts, w, g):
    """combine_backward's grad_const_x, of rows of zeros."""
    N = W * bs
    y = torch.zeros(N * K, h, dtype=dtype, device=DEV)
    cx = torch.zeros(const, h, dtype=dtype, device=DEV)
    return moe.combine_backward(g, y, assist, counts, ids, w, W, epr, x_active_mask=mask, const_experts=const, const_x=cx)[2]


def shares(ids, mask, w, E, const):
    """Weight of each const expert in each token, binary64 [const, N] (ids are distinct: one pair at most)."""
    hit = ids[..., None] == E + torch.arange(const, device=DEV)
    if mask is not None:
        hit = hit & mask[..., None]
    return torch.where(hit, w.double()[..., None], 0.0).sum(1).t().contiguous(), hit.any(1)


LONG = [
    # W, bs, epr, K, h, const, active pairs; then pairs in a part, which are listed 256 (1024 above 2048 columns) at a time
    (2, 70000, 1, 1, 40, 1, 1.0),          # 2188, all of them the const expert's: both sides of every list's border
    (2, 70000, 1, 1, 2056, 1, 1.0),
    (4, 5000, 2, 8, 2056, 2, 1.0),         # 2504
    (4, 5000, 2, 8, 2056, 2, 0.6),
    (4, 5000, 2, 8, 264, 3, 0.6),
    (2, 1100, 1, 2, 2049, 2, 0.8),         # 70, in a list that is not full
    (2, 6, 2, 4, 4100, 2, 0.8),            # one part
]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=str)
@pytest.mark.parametrize("shape", LONG, ids=str)
def test_every_pair_of_a_const_expert_counts_once(shape, dtype):
    """Small whole numbers, none of them 0: their sums are exact, so a pair left out or taken twice shows."""
    W, bs, epr, K, h, const, on = shape
    N, E = W * bs, W * epr
    g, ids, mask, *dispatched = route(W, bs, epr, K, const, on, 3)
    whole = lambda *s: torch.tensor([-2, -1, 1, 2], device=DEV)[torch.randint(0, 4, s, generator=g, device=DEV)]
    w, grad = whole(N, K).float(), whole(N, h).to(dtype)
    got = gradient(W, bs, epr, K, h, const, dtype, ids, mask, *dispatched, w, grad)
    share, hit = shares(ids, mask, w, E, const)
    assert (hit.sum(0) >= on * N - 4 * N ** 0.5).all()
    assert torch.equal(got, (share @ grad.double()).to(dtype))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=str)
@pytest.mark.parametrize("shape", LONG + [(2, 700, 4, 6, 264, 4, 0.7)], ids=str)
def test_const_experts_gradient_within_its_longest_chain(shape, dtype):
    """A pair goes through the additions of the pairs behind it among 1024 tokens of a part, of the part's blocks, and of
    the parts, a fused multiply-add each."""
    W, bs, epr, K, h, const, on = shape
    N, E = W * bs, W * epr
    g, ids, mask, *dispatched = route(W, bs, epr, K, const, on, 5)
    w = torch.randn(N, K, generator=g, device=DEV)
    grad = torch.randn(N, h, generator=g, device=DEV).to(dtype)
    got = gradient(W, bs, epr, K, h, const, dtype, ids, mask, *dispatched, w, grad).double()
    share, hit = shares(ids, mask, w, E, const)
    ref, size = share @ grad.double(), share.abs() @ grad.double().abs()
    parts = parts_of(N)
    per = -(-N // parts)
    pad = torch.zeros(parts * per - N, const, dtype=torch.bool, device=DEV)
    most = int(torch.cat((hit, pad)).view(parts, per, const).sum(1).max())
    room = 1.01 * (min(most, BLOCK) + -(-per // BLOCK) + parts) * U * size
    f = torch.finfo(dtype)
    assert ((got - ref).abs() <= room + f.eps / 2 * (ref.abs() + room) + f.tiny * f.eps).all()


@pytest.mark.gpu
def test_a_long_batch_of_like_gradients_loses_no_digits():
    """The longest batch, all of it one const expert's: 2^18 like terms a part. Added one after the other, each sum would be
    off by up to half a unit in the last place, always the same way: 0.35 % in the end, seven of fp16's half steps."""
    W, bs, h, dtype, w = 2, (1 << 23) - 64, 8, torch.float16, 0x121e892 * 2.0 ** -34
    N = W * bs
    ids = torch.full((N, 1), W, dtype=torch.int32, device=DEV)
    x = torch.zeros((N, 8), dtype=torch.bfloat16, device=DEV)
    assist, counts = moe.dispatch(x, ids, W, 1, const_experts=1)[2:4]
    del x
    grad = torch.ones((N, h), dtype=dtype, device=DEV)
    got = gradient(W, bs, 1, 1, h, 1, dtype, ids, None, assist, counts, torch.full((N, 1), w, device=DEV), grad).double()
    ref = N * w
    room = 1.01 * (BLOCK + -(-N // PARTS // BLOCK) + PARTS) * U * ref
    assert ((got - ref).abs() <= room + torch.finfo(dtype).eps / 2 * (ref + room)).all()
    torch.cuda.empty_cache()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=str)
def test_skewed_routing_with_pairs_of_every_special_expert(dtype):
    W, bs, epr, K, h, special, mask, skew = shape = (2, 700, 4, 3, 264, (1, 1, 2), "pair", 0.2)
    ids, _, _, on = tg.route(W, bs, epr, K, sum(special), mask, 5, skew)
    hits = torch.bincount(ids[on].long(), minlength=W * epr + sum(special))
    assert hits[0] > 500 and (hits[W * epr:] > 20).all()
    tg.test_combine_backward(shape, dtype)
    tg.test_dispatch_backward(shape, dtype)

"""The gate where its fp32 choice has to know its own limits, and where one token's result could depend on others.

Ids and weights are held to the definition as in test_gate.py; what must not depend on a token's neighbours or on the
length of the batch must be equal bit for bit.
"""
import pytest
import torch

import combine_ep_recv_amd as moe
from test_gate import DEV, MAX, SIGMOID, SOFTMAX, TOP2, check, draw


@pytest.mark.gpu
@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID])
@pytest.mark.parametrize("N", [300, 1100])
@pytest.mark.parametrize("size", [1e2, 1e3, 1e4])
def test_gate_groups_whose_two_best_cancel(score, N, size):
    """A large bias and its negative in every group: a group's worth is near 1, the terms' rounding that of the bias.
    Groups lie as far apart as that rounding, experts much further. Short batches, and those whose tokens share a
    wavefront."""
    g = torch.Generator().manual_seed(int(size))
    L = torch.randn(1, 1, 2, generator=g).expand(N, 8, 2) + size * 2.0 ** -20 * torch.randn(N, 8, 2, generator=g)
    L = L.reshape(N, 16).contiguous()
    b = (size * (1 + torch.arange(8) / 8))[:, None].mul(torch.tensor([1.0, -1.0])).flatten().float()
    kw = dict(score=score, groups=8, topk_groups=4, group_score=TOP2)
    ids, w = moe.gate(L.to(DEV), 8, bias=b.to(DEV), **kw)
    check(L, ids, w, bias=b, **kw)


@pytest.mark.gpu
@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID])
@pytest.mark.parametrize("N", [40, 1100])
def test_gate_groups_whose_sum_passes_fp32(score, N):
    """Biases near the largest finite ones, both signs: sums of two that are finite in binary64 and infinite in fp32."""
    top = torch.finfo(torch.float32).max
    L = draw(N, 16, torch.float32, 5)
    for b in (torch.tensor([-top] * 12 + [0.0, 0.5, 1.0, 1.5]),
              torch.tensor([-top, 0.75 * -top] * 6 + [0.5 * -top, -top] * 2),
              torch.tensor([top, 0.5 * top] * 4 + [top, 0.75 * top] * 4),
              torch.tensor([0.0, 1.0] * 3 + [float("inf"), 0.0] + [-top] * 8)):
        for keep in (1, 3, 5):
            kw = dict(score=score, groups=8, topk_groups=keep, group_score=TOP2)
            ids, w = moe.gate(L.to(DEV), 2 * keep, bias=b.to(DEV), **kw)
            check(L, ids, w, bias=b, **kw)


@pytest.mark.gpu
@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID])
@pytest.mark.parametrize("renormalize", [True, False])
def test_gate_weights_do_not_depend_on_the_neighbours(score, renormalize):
    """Tokens that share a wavefront with one whose chosen scores lie below e^-80, and without."""
    N, E = 1100, 32
    L = draw(N, E, torch.float32, 7)
    low = L.clone()
    low[1::4, 3:] = -150.0 - torch.arange(E - 3)
    kw = dict(score=score, renormalize=renormalize)
    ids, w = moe.gate(L.to(DEV), 8, **kw)
    ids2, w2 = moe.gate(low.to(DEV), 8, **kw)
    same = torch.arange(N) % 4 != 1
    assert torch.equal(ids[same], ids2[same]) and torch.equal(w[same], w2[same])
    check(low[:60], ids2[:60], w2[:60], **kw)


@pytest.mark.gpu
@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID])
@pytest.mark.parametrize("E,K", [(20, 4), (64, 8), (100, 8), (200, 16), (256, 8), (300, 3), (320, 16)])
def test_gate_weights_do_not_depend_on_the_length_of_the_batch(score, E, K):
    """Tokens alone, in a short batch and in one long enough for several to share a wavefront."""
    N = 33 * E
    L = draw(N, E, torch.float32, E).to(DEV)
    for renormalize in (True, False):
        kw = dict(score=score, renormalize=renormalize)
        ids, w = moe.gate(L, K, **kw)
        for rows in (slice(0, 1), slice(5, 30), slice(N - 200, N)):
            part, pw = moe.gate(L[rows].contiguous(), K, **kw)
            assert torch.equal(part, ids[rows]) and torch.equal(pw, w[rows])

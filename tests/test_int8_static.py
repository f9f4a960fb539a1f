"""The int8 product on dispatch's static rows, with each form of the coefficients: one, which leaves the sum and goes into the
weights' scales, and one a column or one an expert and column, which the weights are divided by before they are quantised."""
import pytest
import torch

import combine_ep_recv_amd as moe

DEV = "cuda"
U = 2.0 ** -24


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=str)
@pytest.mark.parametrize("form", ["one", "columns", "experts and columns"])
def test_int8_product_on_static_rows_is_the_layers(form, dtype):
    W, bs, epr, h, n, K = 4, 20, 3, 272, 134, 3
    N, E = W * bs, W * epr
    g = torch.Generator().manual_seed(23)
    # no product x * c beyond the codes; columns of different size, as smoothing coefficients have
    x = torch.randn(N, h, generator=g).clamp(-4, 4).to(dtype)
    w = torch.randn(E, n, h, generator=g) * h ** -0.5
    ids = torch.rand(N, E, generator=g).argsort(dim=1)[:, :K].int().contiguous()
    c = 30 * 2.0 ** -(4 * torch.rand({"one": (1, 1), "columns": (1, h), "experts and columns": (E, h)}[form], generator=g))
    rows, scales, assist, erc = moe.dispatch(x.to(DEV), ids.to(DEV), W, epr, moe.MOE_QUANT_STATIC, quant_scales=c.flatten().to(DEV))
    assert scales is None
    if form == "one":
        q, s = moe.quantize_int8(w.to(DEV))
        s = s / c.item()
    else:
        q, s = moe.quantize_int8((w / c[..., None, :]).to(DEV))
    out = moe.expert_product(rows, None, q, s, erc, dtype=dtype).cpu().double()

    ends = (erc.cpu()[:, W - 1::W].long() + torch.cat((torch.zeros(1).long(), erc.cpu()[:, -1].long().cumsum(0)[:-1]))[:, None]).flatten()
    expert = torch.searchsorted(ends, torch.arange(N * K), right=True)
    a = assist.cpu().long()
    token = a[:, 0] * bs + a[:, 1]
    X, Wd, C = x.double()[token], w.double()[expert], c.double().expand(E, h)[expert]
    ref = torch.linalg.vecdot(X[:, None], Wd)
    # a code is off by half a one, a weight by half a step of its row; 300 U: the quotients and scales in binary32
    off = 0.5 * (Wd / C[:, None]).abs().sum(2) + rows.cpu().double().abs().sum(1, keepdim=True) * (0.5 + 300 * U) * s.cpu().double()[expert]
    room = off * (1 + 8 * U) + 4 * U * ref.abs()
    f = torch.finfo(dtype)
    assert ((out - ref).abs() <= room + f.eps / 2 * (ref.abs() + room) + f.tiny * f.eps).all()
    # the bound tells: with the coefficients' mean in the scales, as if they could leave the sum, it does not hold
    if form != "one":
        q, s = moe.quantize_int8(w.to(DEV))
        wrong = moe.expert_product(rows, None, q, s / c.mean().item(), erc, dtype=dtype).cpu().double()
        assert ((wrong - ref).abs() > room + f.eps / 2 * (ref.abs() + room)).any()

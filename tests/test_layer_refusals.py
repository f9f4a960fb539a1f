"""Calls of the gate, the microscaled rows and the experts' product that are refused before anything is made or launched.
Tensors on torch's meta device have shapes and no memory."""
import pytest
import torch

import combine_ep_recv_amd as moe
from test_gate import rec  # noqa: F401  (the fixture that records the library's calls)

BIG = 2 ** 32                    # a C int keeps nothing of it


def _meta(*shape, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device="meta")


def _gate(N=4, E=16, K=2, **kw):
    return moe.gate_into(_meta(N, K, dtype=torch.int32), _meta(N, K, dtype=torch.float32), _meta(N, E), **kw)


def _backward(N=4, E=16, K=2, **kw):
    return moe.gate_backward(_meta(N, E), _meta(N, K, dtype=torch.int32), _meta(N, K, dtype=torch.float32),
                             _meta(N, K, dtype=torch.float32), **kw)


def _product(W=2, epr=2, rows=4, k=64, n=32, activation=moe.MOE_ACT_NONE):
    E, nb = W * epr, -(-k // 32)
    u8 = dict(dtype=torch.uint8)
    return moe.expert_product(_meta(rows, k // 2, **u8), _meta(rows, nb, **u8), _meta(E, n, k // 2, **u8),
                              _meta(E, n, nb, **u8), _meta(W, E, dtype=torch.int32), activation)


def test_sizes_that_fit_reach_the_library(rec):  # noqa: F811
    _gate()
    _backward()
    _product()
    moe.quantize_mx(_meta(2, 64))
    moe.dequantize_mx(_meta(2, 32, dtype=torch.uint8), _meta(2, 2, dtype=torch.uint8))
    assert rec.calls == ["moe_gate", "moe_gate_backward", "moe_expert_product", "moe_mx_quantize", "moe_mx_dequantize"]


@pytest.mark.parametrize("call", [
    lambda: _gate(N=BIG + 4), lambda: _gate(E=BIG + 16), lambda: _gate(N=1, E=BIG + 16, K=BIG + 2),
    lambda: _gate(groups=BIG + 1), lambda: _gate(groups=1 - BIG), lambda: _gate(groups=2, topk_groups=BIG + 1),
    lambda: _gate(score=BIG), lambda: _gate(group_score=BIG), lambda: _backward(N=BIG + 4),
    lambda: _backward(E=BIG + 16), lambda: _backward(score=BIG), lambda: _product(rows=BIG + 4),
    lambda: _product(k=BIG + 64), lambda: _product(n=BIG + 32), lambda: _product(activation=BIG),
    lambda: moe.quantize_mx(_meta(BIG + 32)), lambda: moe.quantize_mx(_meta(1, BIG + 32), moe.MOE_MX_E4M3),
    lambda: moe.quantize_mx_into(_meta(1, BIG // 2 + 16, dtype=torch.uint8), _meta(1, BIG // 32 + 1, dtype=torch.uint8),
                                 _meta(1, BIG + 32)),
    lambda: moe.dequantize_mx(_meta(1, BIG + 32, dtype=torch.float8_e4m3fn), _meta(1, BIG // 32 + 1, dtype=torch.uint8)),
])
def test_sizes_beyond_a_c_int_are_refused_not_cut_off(rec, call):  # noqa: F811
    with pytest.raises(moe.MoeError) as e:
        call()
    assert e.value.status == moe.MOE_ERR_SHAPE and rec.calls == []


@pytest.mark.parametrize("topk", [0, -3, 17, 10 ** 12, BIG + 2])
def test_gate_refuses_a_topk_before_it_makes_room_for_it(rec, topk):  # noqa: F811
    with pytest.raises(moe.MoeError) as e:
        moe.gate(torch.zeros(4, 16), topk)
    assert e.value.status == moe.MOE_ERR_SHAPE and rec.calls == []

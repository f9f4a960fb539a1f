"""The limits that the header states for combine's gradient with const experts, taken up to the last one and refused beyond."""
import pytest

import combine_ep_recv_amd as moe

LIMIT = 1 << 24


@pytest.mark.parametrize("bs,h,each", [
    (1, 256, 1),               # one part of the tokens, which count as 1024
    (512, 256, 32),            # a part for each 32 tokens
    (1024, 512, 64),           # 2048 tokens, 64 parts: as many as there can be
    (1 << 20, 512, 64), (1024, 2048, 64 * 4),
    (1024, 4096, 64 * 2),      # 2048 columns a workgroup
])
def test_const_experts_up_to_the_launchs_limit(bs, h, each):
    size = lambda const: moe.combine_backward_workspace_size(2, bs, 2, h, 2, moe.MOE_BF16, const)
    most = (LIMIT - 1 - max(2 * bs, 1024)) // each
    parts = min(64, -(-2 * bs // 32))
    assert size(most) == (most * parts * h * 4 if parts > 1 else 0)
    with pytest.raises(moe.MoeError) as e:
        size(most + 1)
    assert e.value.status == moe.MOE_ERR_SHAPE
    # what the header promises whatever the launch looks like
    promised = (LIMIT - 1 - max(2 * bs, 1024)) // (64 * -(-h // 512))
    assert promised <= most and size(promised) >= 0

"""The backward of many short heads: every key tile has a single query step, so the dK/dV kernel's accumulators
change hands between its warpgroup pairs at every step."""
import pytest
import torch

import flashattention_backward_fa_gb300 as fa
from cross_reference import Reference

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("B,N,H,d", [(40, 40, 16, 64), (60, 64, 8, 128), (25, 1, 32, 64)])
def test_one_step_units(B, N, H, d, dtype):
    g = torch.Generator().manual_seed(3)
    q, k, v, do = (torch.randn((B, N, H, d), generator=g).to(dtype).cuda() for _ in range(4))
    o, lse = fa.attention_forward(q, k, v)
    grads = fa.attention_backward(q, k, v, o, do, lse)
    ref = Reference(q, k, v, do=do)
    for name, x in zip(("dq", "dk", "dv"), grads):
        want = getattr(ref, name)
        assert ((x.cpu().double() - want).abs() <= 5e-3 + 5e-3 * want.abs()).all(), name
    for _ in range(30):
        for a, b in zip(grads, fa.attention_backward(q, k, v, o, do, lse)):
            assert torch.equal(a, b)
    assert fa.fa_get_device_status() == 0

"""Backward of cross attention where few query rows walk long key axes that are cut into splits, some of them empty;
and of few queries a head, whose statistics are padded to whole tiles only."""
import math

import pytest
import torch

import flashattention_backward_fa_gb300 as fa
from cross_reference import Reference

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def make(B, Nq, Nk, Hq, Hk, d, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    return tuple(torch.randn((B, n, h, d), generator=g).to(dtype).cuda()
                 for n, h in ((Nq, Hq), (Nk, Hk), (Nk, Hk), (Nq, Hq)))


def run(q, k, v, do, lens):
    """o, lse, dq, dk, dv with the caller's own workspace: exactly its size, full of NaN, and 256 bytes of it guarded."""
    B, Nq, Hq, d = q.shape
    shape = (B, Nq, k.shape[1], Hq, k.shape[2], d, q.dtype)
    o, lse = fa.cross_attention_forward(q, k, v, k_lens=lens)
    out = [torch.full_like(t, math.nan) for t in (q, k, v)]
    size = fa.fa_cross_bwd_workspace_size(*shape)
    ws = torch.full((size + 256,), 255, dtype=torch.uint8, device="cuda")
    fa.fa_cross_bwd(q, k, v, o, do, lse, *out, ws[:size], k_lens=lens)
    assert fa.fa_get_device_status() == 0 and (ws[size:] == 255).all()
    return [o, lse, *out]


@pytest.mark.parametrize("size, k_lens", [
    ((1, 100, 3000, 2, 2, 64), None),
    ((3, 100, 2500, 2, 2, 128), [2500, 0, 129]),
    ((7, 31, 2049, 8, 2, 64), [1, 128, 129, 256, 257, 1000, 2049]),
    ((1, 64, 9000, 4, 2, 128), [8897]),
    ((44, 70, 1300, 4, 4, 64), [0, 1, 100, 128, 129, 300, 513, 1024, 1025, 1200, 1300] * 4),
    ((2, 1, 700, 4, 2, 64), [700, 3]), ((2, 2, 60, 6, 2, 128), [60, 1]), ((3, 5, 300, 3, 3, 64), [300, 64, 65]),
    ((1, 17, 40, 2, 1, 128), None), ((2, 36, 77, 4, 1, 64), [77, 20]),
])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_backward(size, k_lens, dtype):
    """Results with the bounds; what lies behind the lengths reaches nothing."""
    q, k, v, do = make(*size, dtype)
    lens = None if k_lens is None else torch.tensor(k_lens, dtype=torch.int32, device="cuda")
    clean = run(q, k, v, do, lens)
    ref = Reference(q, k, v, None, lens, None, do)
    ref.check_forward(*clean[:2])
    ref.check_backward(*clean[2:])
    for b, n in enumerate(k_lens or []):
        k[b, n:], v[b, n:] = math.nan, -math.inf
    for a, b in zip(clean, run(q, k, v, do, lens)):
        assert torch.equal(a, b)

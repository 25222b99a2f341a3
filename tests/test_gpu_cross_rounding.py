"""How far cross attention is off in the 2-norm, in units of its results' own rounding (cross_rounding)."""
import pytest
import torch

import flashattention_backward_fa_gb300 as fa
from cross_rounding import CASES, definition, inputs, ratio_of

pytestmark = pytest.mark.gpu


def run(q, k, v, do, k_lens=None):
    """o, dq, dk, dv of the kernels on the CPU."""
    q, k, v, do = (t.cuda() for t in (q, k, v, do))
    lens = None if k_lens is None else torch.tensor(k_lens, dtype=torch.int32, device="cuda")
    o, lse = fa.cross_attention_forward(q, k, v, k_lens=lens)
    grads = fa.cross_attention_backward(q, k, v, o, do, lse, k_lens=lens)
    assert fa.fa_get_device_status() == 0
    return dict(zip(("o", "dq", "dk", "dv"), (x.cpu() for x in (o,) + grads)))


@pytest.mark.parametrize("name", CASES)
def test_case(name):
    c = CASES[name]
    x, lens = inputs(c), c.get("k_lens")
    off = ratio_of(c, run(*x, lens), definition(*x, k_lens=lens))
    assert off < c["most"]

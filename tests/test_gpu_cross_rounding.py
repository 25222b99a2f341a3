"""How far cross attention is off in the 2-norm, in units of its results' own rounding (cross_rounding)."""
import pytest
import torch

import flashattention_backward_fa_gb300 as fa
from cross_rounding import BF16, CASES, F16, activations, definition, inputs, ratio, ratio_of

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


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [3, 17, 64])
def test_padding_does_not_coarsen(n, d, dtype):
    """A short sequence beside a long one has the gradients of a call of its own, up to the order of their sums."""
    g = torch.Generator().manual_seed(n)
    q, do = activations(g, (2, 200, 2, d), dtype), torch.randn((2, 200, 2, d), generator=g).to(dtype)
    k, v = activations(g, (2, 700, 1, d), dtype), activations(g, (2, 700, 1, d), dtype)
    batch = run(q, k, v, do, [n, 700])
    x = q[:1], k[:1, :n], v[:1, :n], do[:1]
    own, ref = run(*(t.contiguous() for t in x)), definition(*x)
    for name in ("dq", "dk", "dv"):
        a, b = batch[name][:1, :ref[name].shape[1]], own[name]
        assert ratio(a, ref[name], dtype) < 1.02 * ratio(b, ref[name], dtype), name

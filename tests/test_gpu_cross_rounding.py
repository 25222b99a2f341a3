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


@pytest.mark.parametrize("Nq,Nk,k_lens", [(5, 6, None), (200, 300, None), (70, 200, [5, 200])])
@pytest.mark.parametrize("d", [64, 128])
def test_large_gradients_in_fp16(d, Nq, Nk, k_lens):
    """dS beyond fp16's largest value, as loss scaling brings it about, where the gradients are within it: each as exact
    as ever. dO V^T is 1e5 to 1e7 here; small queries and keys take dQ and dK back into the range."""
    g = torch.Generator().manual_seed(d)
    B, r = 2, lambda n, s: (torch.randn((B, n, 2, d), generator=g) * s).to(F16)  # noqa: E731
    q, k, v, do = r(Nq, 1e-3), r(Nk, 1e-3), r(Nk, 100.0), r(Nq, 1000.0)
    ref, x = definition(q, k, v, do, k_lens=k_lens), run(q, k, v, do, k_lens)
    for name in ("dq", "dk", "dv"):
        assert ref[name].abs().max() < 65000
        off = ratio(x[name], ref[name], F16)
        assert off < 1.2, name


def test_gradients_of_zero_and_of_the_least_values_in_fp16():
    """Rows, heads and a whole call whose dO or V is zero; the smallest values that fp16 has."""
    g = torch.Generator().manual_seed(1)
    r = lambda n, h: torch.randn((2, n, h, 64), generator=g).to(F16)  # noqa: E731
    q, k, v, do = r(150, 4), r(130, 2), r(130, 2), r(150, 4)
    do[0, 3:9], do[1, :, 1] = 0, 2.0 ** -24
    v[1, :, 1] = 0
    ref, x = definition(q, k, v, do), run(q, k, v, do)
    assert not any(x[n].isnan().any() or x[n].isinf().any() for n in x)
    for n in ("dq", "dk", "dv"):
        assert ratio(x[n], ref[n], F16) < 1.2, n
    assert not x["dq"][0, 3:9].any() and not x["dq"][1, :, 2:].any() and not x["dk"][1, :, 1].any()
    x = run(q, k, v, torch.zeros_like(do))
    assert not any(x[n].any() for n in ("dq", "dk", "dv"))
    x = run(q, k, torch.zeros_like(v), do)
    assert not x["dq"].any() and not x["dk"].any()


def test_infinite_gradients_in_fp16():
    """An infinity in dO spoils its own query's dQ and its key head's dK and dV, and nothing else."""
    g = torch.Generator().manual_seed(2)
    r = lambda n, h: torch.randn((2, n, h, 64), generator=g).to(F16)  # noqa: E731
    q, k, v, do = r(90, 4), r(130, 2), r(130, 2), r(90, 4)
    clean = run(q, k, v, do)
    do[1, 7, 2, 5] = float("inf")
    x = run(q, k, v, do)
    assert not x["dq"][1, 7, 2].isfinite().any() and not x["dk"][1, :, 1].isfinite().any()
    keep = torch.ones(2, 90, 4, dtype=torch.bool)
    keep[1, 7, 2] = False
    assert torch.equal(x["dq"][keep], clean["dq"][keep])
    for n in ("dk", "dv"):
        assert torch.equal(x[n][0], clean[n][0]) and torch.equal(x[n][1, :, 0], clean[n][1, :, 0])

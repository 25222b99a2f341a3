"""The cases of cross_rounding on the CPU: with the kernels' roundings each stays under its limit, and with the rounding
that it is about made coarser it does not."""
import pytest

from cross_rounding import CASES, definition, emulate, inputs, ratio_of


@pytest.mark.parametrize("name", CASES)
def test_case_tells_the_rounding(name):
    c = CASES[name]
    x, lens = inputs(c), c.get("k_lens")
    ref = definition(*x, k_lens=lens)
    fine = ratio_of(c, emulate(*x, k_lens=lens), ref)
    coarse = ratio_of(c, emulate(*x, k_lens=lens, **{c["off"][1]: False}), ref)
    assert fine < c["most"] < coarse

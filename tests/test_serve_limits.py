"""Limits of the norm-and-rotation and cache calls, on the CPU: what is refused, and that sizes up to the
header's limits are not."""
import pytest
import torch

import flashattention_backward_fa_gb300 as fa
from flashattention_backward_fa_gb300 import binding
from test_abi_host import lib  # noqa: F401  (builds the library where it is missing)

P = 1 << 12
EUNSUP = -2


def _attn(lib, T, Hq, H):
    d, page = 64, 128
    cache = binding._Kv8CacheArg(P, P, P, P, 10, page, H, d, fa.FaStrides(page * H * d, d, page * d))
    seqs = binding._Kv8SeqsArg(P, 4096, P, None, 1, 4096)
    st = fa.FaStrides(T * Hq * d, Hq * d, d)
    # a scale that is not finite is refused behind the sizes and in front of the pointers
    return lib.fa_kv8_attn(cache, seqs, P, P, P, T, Hq, 1 << 19, st, st, fa.FA_BF16, float("nan"), 1, 0, None, 0, P,
                           1 << 40, None)


@pytest.mark.parametrize("T,Hq,H", [(32768, 16, 16), (32777, 16, 16), (16385, 64, 1), (1 << 19, 8, 2), (1 << 19, 2048, 8),
                                    (1 << 14, 1 << 16, 1024)])
def test_attention_takes_any_prompt_up_to_the_stated_limits(lib, T, Hq, H):  # noqa: F811
    assert _attn(lib, T, Hq, H) == -1


@pytest.mark.parametrize("T,Hq,H", [((1 << 19) + 1, 8, 2), (1 << 19, 2049, 1), ((1 << 14) + 1, 1 << 16, 1024),
                                    (1, (1 << 16) + 1, 1)])
def test_attention_refuses_more(lib, T, Hq, H):  # noqa: F811
    assert _attn(lib, T, Hq, H) == EUNSUP


@pytest.mark.parametrize("shape", [(4, 64), (2, 4, 64), (1, 2, 4, 8, 64)])
def test_autograd_call_names_what_is_wrong_with_the_shape(shape):
    x = torch.zeros(shape, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        fa.qk_norm_rope_func(x, x)

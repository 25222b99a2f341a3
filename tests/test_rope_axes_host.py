"""Host-only checks of the operators with positions on several axes: bad arguments return the documented codes
before any GPU is touched; the helpers that name the pairs' axes."""
import ctypes
import os
import shutil

import pytest
import torch

import flashattention_backward_fa_gb300 as fa
from flashattention_backward_fa_gb300 import binding

BF16 = fa.FA_BF16
OK, EINVAL, EUNSUP, EALIGN, EWS = 0, -1, -2, -3, -4
P = 0x10000  # a fake, 256-byte-aligned "device" address: validation rejects before any use


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(binding.LIB_PATH):
        if shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"):
            pytest.skip("no nvcc to build the library")
        from flashattention_backward_fa_gb300.build import build_library
        build_library()
    return fa.load_library()


def _calls(lib, ax, rot=128, d=128, dt=BF16, rows=64):
    """The code of each of the three calls for the same axes."""
    st = fa.FaStrides(8 * 4 * d, 4 * d, d)
    yield lib.fa_qk_norm_rope_axes_fwd(P, P, P, P, P, P, P, P, ax, 1, 8, 4, 4, d, rot, 0, rows, st, st, st, st, dt, dt,
                                       1e-6, None)
    yield lib.fa_qk_norm_rope_axes_bwd(P, P, P, P, P, P, P, P, P, P, P, P, ax, 1, 8, 4, 4, d, rot, 0, rows, st, st, st,
                                       st, st, st, dt, dt, 1e-6, P, 1 << 30, None)
    cache = binding._Kv8CacheArg(P, P, P, P, 10, 64, 4, d, fa.FaStrides(64 * 4 * d, d, 64 * d))
    seqs = binding._Kv8SeqsArg(P, 4, P, None, 1, 4)
    yield lib.fa_kv8_norm_rope_axes_append(cache, seqs, P, P, P, P, P, P, P, P, ax, 8, 4, rot, 0, rows, st, st, st, st,
                                           dt, dt, 1e-6, None)


@pytest.mark.parametrize("kw,rot,code", [
    (dict(axes=0), 128, EINVAL), (dict(axes=5), 128, EINVAL), (dict(axes=-1), 128, EINVAL),
    (dict(pair_axis=bytes([3] * 64)), 128, EINVAL), (dict(pair_axis=bytes([0] * 63 + [3])), 128, EINVAL),
    (dict(positions=0), 128, EINVAL), (dict(positions=P + 2), 128, EALIGN),
    (dict(stride_b=-1), 128, EINVAL), (dict(stride_n=-3), 128, EINVAL), (dict(stride_axis=-1), 128, EINVAL),
    (dict(), 0, EINVAL), (dict(), 24, EUNSUP), (dict(), 130, EINVAL),
])
def test_rejects_bad_axes(lib, kw, rot, code):
    a = dict(axes=3, pair_axis=bytes([0] * 20 + [1] * 22 + [2] * 22), positions=P, stride_b=24, stride_n=3, stride_axis=1)
    a.update(kw)
    assert [c for c in _calls(lib, binding._RopeAxes(**a), rot)] == [code] * 3


def test_rejects_missing_axes(lib):
    assert [c for c in _calls(lib, ctypes.POINTER(binding._RopeAxes)())] == [EINVAL] * 3


def test_rope_axes():
    assert fa.rope_axes((2, 3, 1)) == (0, 0, 1, 1, 1, 2)
    assert fa.rope_axes((2, 3, 1), interleaved=True) == (0, 1, 2, 0, 1, 1)
    assert fa.rope_axes((0, 2)) == (1, 1)
    for bad in ((), (0, 0), (1, 2, 3, 4, 5), (-1, 2)):
        with pytest.raises(ValueError):
            fa.rope_axes(bad)


def test_rope_axis_tables():
    """Each axis as a rotation of its own."""
    cos, sin = fa.rope_axis_tables(9, (4, 2, 0, 6), device="cpu")
    assert cos.shape == sin.shape == (9, 12)
    at = 0
    for n in (4, 2, 6):
        c, s = fa.rope_tables(9, 2 * n, device="cpu")
        assert torch.equal(cos[:, at:at + n], c) and torch.equal(sin[:, at:at + n], s)
        at += n

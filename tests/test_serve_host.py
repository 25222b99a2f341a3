"""Host-only checks of the norm-and-rotation and 8-bit cache entry points: bad arguments return the
documented codes before any GPU is touched, the binding refuses what it cannot pass on, and the plain
float64 forms that the GPU tests compare with agree with independent statements of the definitions."""
import ctypes
import math
import os
import shutil

import pytest
import torch

import flashattention_backward_fa_gb300 as fa
from flashattention_backward_fa_gb300 import binding
import serve_reference as ref

F32, F16, BF16 = fa.FA_F32, fa.FA_F16, fa.FA_BF16
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


def _st(N, H, d):
    return fa.FaStrides(N * H * d, H * d, d)


def _rope(lib, *, back=False, q=P, k=P, out=P, qw=P, kw=P, dqw=P, cos=P, sin=P, pos=None, ps=0, B=1, N=8, Hq=4, Hk=2,
          d=128, rot=128, il=0, rows=64, st=None, dt=BF16, wt=None, eps=1e-6, ws=P, ws_bytes=1 << 20):
    qs, ks = st or _st(N, Hq, d), _st(N, Hk, d)
    wt = dt if wt is None else wt
    tail = [cos, sin, pos, ps, B, N, Hq, Hk, d, rot, il, rows]
    if back:
        return lib.fa_qk_norm_rope_bwd(q, k, out, P, P, P, qw, kw, dqw, P, *tail, qs, ks, qs, ks, qs, ks, dt, wt, eps,
                                       ws, ws_bytes, None)
    return lib.fa_qk_norm_rope_fwd(q, k, out, P, qw, kw, *tail, qs, ks, qs, ks, dt, wt, eps, None)


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("kw,code", [
    (dict(B=0), EINVAL), (dict(N=0), EINVAL), (dict(Hq=0), EINVAL), (dict(Hk=0), EINVAL), (dict(d=0), EINVAL),
    (dict(dt=7), EUNSUP), (dict(d=96, rot=96), EUNSUP), (dict(dt=F32, d=129), EUNSUP), (dict(wt=F16), EUNSUP),
    (dict(rot=-2), EINVAL), (dict(rot=130), EINVAL), (dict(rot=31), EINVAL), (dict(rot=24), EUNSUP),
    (dict(rows=0), EINVAL), (dict(eps=0.0), EINVAL), (dict(eps=float("nan")), EINVAL), (dict(eps=float("inf")), EINVAL),
    (dict(q=0), EINVAL), (dict(k=0), EINVAL), (dict(out=0), EINVAL), (dict(cos=0), EINVAL), (dict(sin=0), EINVAL),
    (dict(q=P + 8), EALIGN), (dict(out=P + 2), EALIGN), (dict(cos=P + 4), EALIGN), (dict(pos=P + 2), EALIGN),
    (dict(qw=P + 1), EALIGN), (dict(kw=P + 2, wt=F32), EALIGN), (dict(ps=-1), EINVAL),
    (dict(st=fa.FaStrides(4100, 516, 128)), EALIGN), (dict(st=fa.FaStrides(0, 512, 128)), EINVAL),
    (dict(B=1 << 13, Hq=(1 << 11) + 1), EUNSUP), (dict(N=(1 << 30) + 1), EUNSUP),
])
def test_norm_rope_rejects_bad_arguments(lib, back, kw, code):
    assert _rope(lib, back=back, **kw) == code


def test_norm_rope_backward_rejects_bad_arguments(lib):
    need = fa.fa_qk_norm_rope_bwd_workspace_size(128)
    assert need % 256 == 0 and need > 0
    assert fa.fa_qk_norm_rope_bwd_workspace_size(0) == 0 and fa.fa_qk_norm_rope_bwd_workspace_size(129) == 0
    assert _rope(lib, back=True, ws=0) == EWS
    assert _rope(lib, back=True, ws=P + 128) == EWS
    assert _rope(lib, back=True, ws_bytes=need - 1) == EWS
    assert _rope(lib, back=True, dqw=0) == EINVAL       # a weight without its gradient
    assert _rope(lib, back=True, qw=0) == EINVAL        # a gradient without its weight
    assert _rope(lib, back=True, dqw=P + 2, wt=F32) == EALIGN


def _cache(**kw):
    a = dict(k=P, v=P, k_scale=P, v_scale=P, num_pages=10, page_size=64, H=2, d=128,
             strides=fa.FaStrides(64 * 2 * 128, 128, 64 * 128))
    a.update(kw)
    return binding._Kv8CacheArg(**a)


def _seqs(**kw):
    a = dict(block_table=P, table_stride=4, seq_lens=P, new_lens=None, B=3, max_pages=4)
    a.update(kw)
    return binding._Kv8SeqsArg(**a)


def _calls(lib, c, s, *, T=1, Hq=4, dt=BF16, q=P, k=P, st=None):
    """The code of each of the three cache calls for the same arguments."""
    H, d = c.H, c.d
    ks, qs = st or _st(T, max(H, 1), d), st or _st(T, Hq, d)
    return (lib.fa_kv8_append(c, s, k, P, T, ks, ks, dt, None),
            lib.fa_kv8_norm_rope_append(c, s, q, k, P, P, P, P, P, P, T, Hq, d & ~15, 0, 64, qs, ks, ks, qs, dt, dt,
                                        1e-6, None),
            lib.fa_kv8_attn(c, s, q, P, P, T, Hq, 256, qs, qs, dt, 0.1, 1, 0, None, 0, P, 1 << 30, None))


@pytest.mark.parametrize("cache,seqs,call,code", [
    (dict(k=0), {}, {}, EINVAL), (dict(v_scale=0), {}, {}, EINVAL), (dict(num_pages=0), {}, {}, EINVAL),
    (dict(H=0), {}, {}, EINVAL), (dict(page_size=48), {}, {}, EUNSUP), (dict(page_size=8), {}, {}, EUNSUP),
    (dict(page_size=256), {}, {}, EUNSUP), (dict(d=96), {}, {}, EUNSUP), (dict(H=1025), {}, dict(Hq=1025), EUNSUP),
    (dict(k=P + 8), {}, {}, EALIGN), (dict(k_scale=P + 2), {}, {}, EALIGN),
    (dict(strides=fa.FaStrides(16384, 136, 8192)), {}, {}, EALIGN),
    (dict(strides=fa.FaStrides(0, 128, 8192)), {}, {}, EINVAL),
    (dict(strides=fa.FaStrides(1 << 40, 1 << 28, 128)), {}, {}, EUNSUP),
    ({}, dict(block_table=0), {}, EINVAL), ({}, dict(seq_lens=0), {}, EINVAL), ({}, dict(B=0), {}, EINVAL),
    ({}, dict(max_pages=0), {}, EINVAL), ({}, dict(table_stride=-1), {}, EINVAL), ({}, dict(B=65536), {}, EUNSUP),
    ({}, dict(max_pages=(1 << 24) + 1), {}, EUNSUP), ({}, dict(seq_lens=P + 2), {}, EALIGN),
    ({}, dict(new_lens=P + 1), {}, EALIGN),
    ({}, {}, dict(T=0), EINVAL), ({}, {}, dict(dt=F32), EUNSUP),
    ({}, {}, dict(st=fa.FaStrides(512, 516, 128)), EALIGN), ({}, {}, dict(st=fa.FaStrides(512, 512, 0)), EINVAL),
])
def test_cache_calls_reject_bad_arguments(lib, cache, seqs, call, code):
    assert set(_calls(lib, _cache(**cache), _seqs(**seqs), **call)) == {code}


def test_append_limits_its_tokens(lib):
    a, n, _ = _calls(lib, _cache(), _seqs(), T=(1 << 19) + 1)
    assert (a, n) == (EUNSUP, EUNSUP)


def test_null_structs_and_tensors(lib):
    st = _st(1, 2, 128)
    assert lib.fa_kv8_append(None, _seqs(), P, P, 1, st, st, BF16, None) == EINVAL
    assert lib.fa_kv8_append(_cache(), None, P, P, 1, st, st, BF16, None) == EINVAL
    a, n, t = _calls(lib, _cache(), _seqs(), q=P + 8, k=P)
    assert (n, t) == (EALIGN, EALIGN)
    a, n, _ = _calls(lib, _cache(), _seqs(), k=0)
    assert (a, n) == (EINVAL, EINVAL)


def _attn(lib, *, T=1, Hq=4, msl=256, scale=0.1, window=0, alibi=None, asb=0, lse=P, ws=P, ws_bytes=1 << 30):
    st = _st(T, Hq, 128)
    return lib.fa_kv8_attn(_cache(), _seqs(), P, P, lse, T, Hq, msl, st, st, BF16, scale, 1, window, alibi, asb, ws,
                           ws_bytes, None)


def test_attention_rejects_bad_arguments(lib):
    assert _attn(lib, Hq=3) == EINVAL                # not a multiple of the cache's two heads
    assert _attn(lib, Hq=0) == EINVAL
    assert _attn(lib, msl=0) == EINVAL
    assert _attn(lib, window=-1) == EINVAL
    assert _attn(lib, scale=float("nan")) == EINVAL
    assert _attn(lib, lse=0) == EINVAL
    assert _attn(lib, lse=P + 2) == EALIGN
    assert _attn(lib, alibi=P + 2) == EALIGN
    assert _attn(lib, alibi=P, asb=-1) == EINVAL
    assert _attn(lib, T=(1 << 24) + 1) == EUNSUP
    assert _attn(lib, T=1 << 20) == EUNSUP           # more row tiles than a grid's y extent
    # sequences long enough for the split outputs to need a workspace
    need = fa.fa_kv8_attn_workspace_size(3, 1, 4, 2, 128, 64, 400, 25600)
    assert need > 0 and need % 256 == 0

    def long(ws=P, ws_bytes=1 << 40):
        st = _st(1, 4, 128)
        return lib.fa_kv8_attn(_cache(), _seqs(max_pages=400, table_stride=400), P, P, P, 1, 4, 25600, st, st, BF16,
                               0.1, 1, 0, None, 0, ws, ws_bytes, None)
    assert long(ws=0) == EWS
    assert long(ws=P + 128) == EWS
    assert long(ws_bytes=need - 1) == EWS


def test_attention_workspace_size(lib):
    size = fa.fa_kv8_attn_workspace_size
    assert size(1, 1, 8, 8, 128, 64, 1, 64) == 0       # one block a sequence and head
    # split outputs and their log-sum-exp: a whole number of splits of (d + 1) floats a row
    big = size(1, 1, 32, 8, 128, 64, 2048, 131072)
    assert big > 0 and abs(big / (32 * 129 * 4) - round(big / (32 * 129 * 4))) < 0.02
    # a window bounds the keys, whatever the length
    assert size(1, 1, 32, 8, 128, 64, 2048, 131072, True, 256) < big
    for bad in ((0, 1, 8, 8, 128, 64, 2048, 131072), (1, 1, 9, 8, 128, 64, 2048, 131072),
                (1, 1, 8, 8, 96, 64, 2048, 131072), (1, 1, 8, 8, 128, 48, 2048, 131072),
                (1, 1, 8, 8, 128, 64, 0, 64), (1, 1, 8, 8, 128, 64, 2048, 0)):
        assert size(*bad) == 0


def test_norm_rope_append_rejects_bad_arguments(lib):
    def call(rot=128, rows=64, eps=1e-6, wt=BF16, cos=P, q_out=P, Hq=4):
        qs, ks = _st(1, 4, 128), _st(1, 2, 128)
        return lib.fa_kv8_norm_rope_append(_cache(), _seqs(), P, P, P, q_out, P, P, cos, P, 1, Hq, rot, 0, rows, qs,
                                           ks, ks, qs, BF16, wt, eps, None)
    assert call(rot=24) == EUNSUP
    assert call(rot=256) == EINVAL
    assert call(rows=0) == EINVAL
    assert call(eps=-1.0) == EINVAL
    assert call(wt=F16) == EUNSUP
    assert call(cos=0) == EINVAL
    assert call(cos=P + 4) == EALIGN
    assert call(q_out=0) == EINVAL
    assert call(Hq=0) == EINVAL


def test_binding_refuses_what_it_cannot_pass_on(lib):
    q = torch.zeros(1, 4, 2, 64, dtype=torch.bfloat16)
    cos, sin = fa.rope_tables(8, 64, device="cpu")
    with pytest.raises(ValueError):
        fa.qk_norm_rope_forward(q, q, None, None, cos, sin)        # CPU tensors
    with pytest.raises(ValueError):
        fa.qk_norm_rope_forward(q[0], q[0], None, None, cos, sin)  # three dimensions
    cache = fa.kv8_cache_alloc(2, 16, 2, 64, device="cpu")
    table, lens = torch.zeros(1, 2, dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        fa.kv8_append(cache, q, q, table, lens)
    with pytest.raises(ValueError):
        fa.kv8_attention(q, cache, table, lens, 16)
    with pytest.raises(ValueError):
        fa.rope_tables(0, 64, device="cpu")
    with pytest.raises(ValueError):
        fa.rope_tables(8, 63, device="cpu")


def test_rope_tables_are_exact_far_out():
    cos, sin = fa.rope_tables(70000, 64, 10000.0, device="cpu")
    assert cos.shape == sin.shape == (70000, 32) and cos.dtype == torch.float32
    for pos, i in ((0, 0), (1, 0), (69999, 0), (69999, 1), (65537, 31)):
        a = pos * 10000.0 ** (-2 * i / 64)
        # the table is the fp32 rounding (half a step of values up to 1: 2^-25) of an angle in float64
        assert abs(float(cos[pos, i]) - math.cos(a)) < 2.0 ** -24
        assert abs(float(sin[pos, i]) - math.sin(a)) < 2.0 ** -24


def test_cache_alloc_layout():
    c = fa.kv8_cache_alloc(5, 32, 3, 64, device="cpu")
    assert c.k.shape == (5, 32, 3, 64) and c.k.dtype == torch.float8_e4m3fn and c.k.stride() == c.v.stride()
    assert c.k.stride() == (32 * 3 * 64, 64, 32 * 64, 1)
    assert c.k_scale.shape == (5, 3) and float(c.k_scale.min()) == 1.0


# ---- the plain forms themselves ----
def test_reference_scale_and_rounding():
    for amax, e in ((448.0, 0), (448.5, 1), (1.75, -8), (1.7500001, -7), (0.0, -100), (2.0 ** -120, -100), (896.0, 1)):
        assert ref.scale_of(amax) == 2.0 ** e, amax
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().double()
    codes = codes[codes.isfinite()]
    assert torch.equal(ref.round_e4m3(codes), codes)
    x = torch.linspace(-448, 448, 40001).double()  # fp32 values: torch rounds them once
    assert torch.equal(ref.round_e4m3(x), x.float().to(torch.float8_e4m3fn).float().double())


@pytest.mark.parametrize("interleaved", [False, True])
def test_reference_rotation_is_a_rotation(interleaved):
    g = torch.Generator().manual_seed(3)
    x = torch.randn(2, 5, 3, 64, generator=g, dtype=torch.float64)
    cos, sin = (t.double() for t in fa.rope_tables(16, 32, device="cpu"))
    pos = torch.tensor([[0, 1, 2, 3, 15], [4, 4, 0, 9, 1]])
    y = ref.norm_rope(x, None, cos, sin, pos, 1e-30, interleaved)
    z = x / x.square().mean(-1, keepdim=True).sqrt()
    # tables are rounded to fp32: norms hold to about 2^-24 of each pair
    assert torch.allclose(y.square().sum(-1), z.square().sum(-1), rtol=1e-6, atol=0)
    assert torch.equal(y[..., 32:], z[..., 32:])
    assert torch.equal(y[0, 0], z[0, 0])  # position 0


def test_reference_cache_against_softmax():
    """One sequence through the plain cache and attention equals softmax attention of the values it holds."""
    g = torch.Generator().manual_seed(4)
    cache = fa.kv8_cache_alloc(4, 16, 2, 64, device="cpu")
    r = ref.RefCache(cache)
    k, v = (torch.randn(1, 37, 2, 64, generator=g, dtype=torch.float64) for _ in range(2))
    table, lens = torch.tensor([[2, 0, 3]]), torch.tensor([37])
    r.append(k, v, table, lens, None)
    held = [(r.codes[i][[2, 0, 3]] * r.scales[i][[2, 0, 3]][:, None, :, None]).flatten(0, 1)[:37] for i in (0, 1)]
    # e4m3: half a step is 2^-4 of a value, 2^-10 of the scale below its normal range
    for x, y, s in zip((k, v), held, r.scales):
        assert torch.all((x[0] - y).abs() <= torch.maximum(y.abs() * 2.0 ** -4, s.max() * 2.0 ** -10))
    q = torch.randn(1, 2, 4, 64, generator=g, dtype=torch.float64)
    o, lse = r.attention(q, table, lens, None, 100, 0.125)
    kk, vv = (t.repeat_interleave(2, 1).transpose(0, 1)[None] for t in held)
    mask = torch.arange(37)[None] <= torch.tensor([[35], [36]])
    want = torch.nn.functional.scaled_dot_product_attention(q.transpose(1, 2), kk, vv, attn_mask=mask, scale=0.125)
    assert torch.allclose(o.transpose(1, 2), want, rtol=1e-12, atol=1e-12)
    assert lse.shape == (1, 4, 2)

"""The 8-bit key/value cache on the GPU against the plain float64 form.

Append is exact but for the roundings its definition names, so codes and scales have to be equal.

Attention is compared with the float64 attention over the very values that the cache holds. With
A = max_j scale * sum_i |q_i k_ji| of a row, a score is off by at most (d + 8) * 2^-23 * A (fp32 sums of
exact products, truncated adds counted as whole steps, and the two factors), its exponent by 64 * 2^-24
more (|s - m| < 64 wherever the weight matters, ex2.approx 2^-22): delta in all. Weights are then off
by delta relative and, rounded to f16, by 2^-12 (bf16 outputs) or 2^-22 (f16 outputs, whose rounding
residual is multiplied too); weights below 2^-21 of the largest of their split lose more, at most 2^-32 of
it each, which n keys turn to n * 2^-32. With V = sum_j p_j |v_j| and vmax = max |v| an output is off by
at most half a step of its type + V * (2 delta + 2^-12 or 2^-22 + (n + 64) * 2^-23) + n * 2^-32 * vmax, and
lse by delta + (n + 64) * 2^-23 + 2^-22 (1 + |lse|).
"""
import math

import pytest
import torch

import flashattention_backward_fa_gb300 as fa
import serve_reference as ref

pytestmark = pytest.mark.gpu

HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.bfloat16: 2.0 ** -130, torch.float16: 2.0 ** -25}


def _layout(B, page, max_tokens, g, spare=2):
    """A shuffled block table [B, ceil(max_tokens / page) + 1], its last column unused (-1)."""
    n = -(-max_tokens // page)
    pages = B * n + spare
    table = torch.full((B, n + 1), -1, dtype=torch.int32)
    table[:, :n] = torch.randperm(pages, generator=g)[:B * n].view(B, n).int()
    return pages, table


def _same(cache, want):
    for i, (codes, scale) in enumerate(((cache.k, cache.k_scale), (cache.v, cache.v_scale))):
        assert torch.equal(ref.f64(scale), want.scales[i])
        got = codes.cpu().float().double()
        assert torch.equal(got.isnan(), want.codes[i].isnan())
        assert torch.equal(got.nan_to_num(), want.codes[i].nan_to_num())


def _values(shape, dtype, g, spread=3.0):
    """Values whose size varies from token to token by powers of ten, so that page scales grow."""
    x = torch.randn(shape, generator=g)
    return (x * torch.pow(10.0, spread * (torch.rand(shape[0], shape[1], shape[2], 1, generator=g) - 0.5))).to(dtype)


def _cu(x):
    return None if x is None else torch.as_tensor(x, dtype=torch.int32).cuda()


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("d,dtype", [(64, torch.float16), (128, torch.bfloat16)])
def test_append_in_many_calls(page, d, dtype):
    """Prompts of unequal lengths, single tokens, a longer block, an empty call: after each the codes
    and scales equal the plain form's, earlier tokens requantised where a scale grew."""
    g = torch.Generator().manual_seed(page + d)
    B, H, most = 3, 2, 3 * page + 9
    pages, table = _layout(B, page, most, g)
    cache = fa.kv8_cache_alloc(pages, page, H, d)
    want = ref.RefCache(cache)
    lens = [0] * B
    for T, new in ((page + 5, [page + 5, 1, 0]), (1, None), (1, [1, 0, 1]), (7, [3, 7, 5]), (page, None),
                   (2, [0, 0, 0]), (1, None)):
        n = [T] * B if new is None else new
        lens = [a + b for a, b in zip(lens, n)]
        k, v = _values((B, T, H, d), dtype, g), _values((B, T, H, d), dtype, g)
        fa.kv8_append(cache, k.cuda(), v.cuda(), _cu(table), _cu(lens), _cu(new))
        want.append(ref.f64(k), ref.f64(v), table, lens, new)
        _same(cache, want)
    assert fa.fa_get_device_status() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_append_of_borders_and_non_finite_values(dtype):
    """Largest values at, below and above the border of a scale, zeros, subnormals, infinities, NaN, the
    largest finite value; each in a page of its own and behind an earlier token."""
    d, page = 64, 16
    big = torch.finfo(dtype).max
    tops = [448.0, 449.0 if dtype == torch.float16 else 450.0, 1.75, 1.765625, 0.0, 6e-8, big, float("inf"),
            float("-inf"), float("nan"), 2.0 ** -14, 3.0]
    B = len(tops)
    x = torch.zeros(B, 2, 1, d, dtype=torch.float32)
    x[:, 0, 0, 1] = 2.0 ** -9
    x[:, 1, 0, 3] = torch.tensor(tops)
    x[:, 1, 0, 4:8] = torch.tensor([0.3, -0.01, 1.0, -2.5])
    x = x.to(dtype)
    table = torch.arange(B, dtype=torch.int32)[:, None].contiguous()
    for calls in ((2,), (1, 1)):
        cache = fa.kv8_cache_alloc(B, page, 1, d)
        want = ref.RefCache(cache)
        at = 0
        for T in calls:
            part = x[:, at:at + T].contiguous()
            at += T
            fa.kv8_append(cache, part.cuda(), part.flip(-1).contiguous().cuda(), _cu(table), _cu([at] * B))
            want.append(ref.f64(part), ref.f64(part.flip(-1)), table, [at] * B, None)
        _same(cache, want)


def test_append_skips_what_it_has_no_place_for():
    """Padding rows, tokens past the table, negative positions and pages out of range leave every other
    byte of the cache as it was; a bad page sets its status bit."""
    g = torch.Generator().manual_seed(3)
    page, H, d, dtype = 16, 2, 64, torch.bfloat16
    cache = fa.kv8_cache_alloc(6, page, H, d)
    cache.k.view(torch.uint8).fill_(0x33)
    cache.v.view(torch.uint8).fill_(0x44)
    want = ref.RefCache(cache)
    table = torch.tensor([[0, 1], [2, 3]], dtype=torch.int32)
    k, v = _values((2, 20, H, d), dtype, g), _values((2, 20, H, d), dtype, g)
    # sequence 0: 40 tokens in a table of 32; sequence 1: 7 tokens of which 20 are new (13 negative positions)
    for lens, new in (([40, 7], None), ([5, 2], [5, 2]), ([-4, 0], [0, 0]), ([9, 2 ** 31 - 1], [20, -3])):
        fa.kv8_append(cache, k.cuda(), v.cuda(), _cu(table), _cu(lens), _cu(new))
        want.append(ref.f64(k), ref.f64(v), table, lens, new)
        _same(cache, want)
    assert fa.fa_get_device_status() == 0
    bad = torch.tensor([[6, 4], [-1, 5]], dtype=torch.int32)
    fa.kv8_append(cache, k.cuda(), v.cuda(), _cu(bad), _cu([20, 20]))
    want.append(ref.f64(k), ref.f64(v), bad, [20, 20], None)
    _same(cache, want)
    assert fa.fa_get_device_status(clear=True) == 4


def _strided_cache(pages, page, H, d):
    """A cache whose tokens, heads and pages lie apart in a larger buffer, tokens outermost in a page."""
    sh, sn = d + 16, H * (d + 16) + 32
    sp = page * sn + 48
    halves, bufs = [], []
    for _ in range(2):
        buf = torch.full((pages * sp + 64,), 0x7F, dtype=torch.uint8, device="cuda")
        bufs.append(buf)
        halves.append(buf.view(torch.float8_e4m3fn).as_strided((pages, page, H, d), (sp, sn, sh, 1), 16))
    s = [torch.ones(pages, H, device="cuda") for _ in range(2)]
    return fa.Kv8Cache(*halves, *s), bufs


def test_append_strides_and_guard_bands():
    g = torch.Generator().manual_seed(9)
    B, T, H, d, page, dtype = 2, 21, 3, 64, 16, torch.float16
    pages, table = _layout(B, page, T, g)
    cache, bufs = _strided_cache(pages, page, H, d)
    dense = fa.kv8_cache_alloc(pages, page, H, d)
    qkv = _values((B, T, 3 * H + 1, d), dtype, g).cuda()
    k, v = qkv[:, :, H:2 * H], qkv[:, :, 2 * H:3 * H]
    fa.kv8_append(cache, k, v, _cu(table), _cu([T, T]))
    fa.kv8_append(dense, k.contiguous(), v.contiguous(), _cu(table), _cu([T, T]))
    assert torch.equal(cache.k_scale, dense.k_scale) and torch.equal(cache.v_scale, dense.v_scale)
    for x, y, buf in ((cache.k, dense.k, bufs[0]), (cache.v, dense.v, bufs[1])):
        live = torch.zeros((pages, page), dtype=torch.bool)
        for b in range(B):
            for j in range(T):
                live[table[b, j // page], j % page] = True
        a, c = x.view(torch.uint8).cpu(), y.view(torch.uint8).cpu()
        assert torch.equal(a[live], c[live])
        assert bool((a[~live] == 0x7F).all())  # slots without a token keep what they held
        x.view(torch.uint8).fill_(0x7F)
        assert bool((buf == 0x7F).all())  # nothing between the rows was touched


NRA = [
    # B, T, Hq, H, d, rot, interleaved, page, dtype, weights, lens before, new
    (3, 1, 8, 2, 128, 128, False, 64, torch.bfloat16, "own", [0, 63, 64], None),
    (3, 1, 6, 6, 64, 32, True, 16, torch.float16, "f32", [5, 15, 40], [1, 0, 1]),
    (2, 37, 5, 1, 64, 64, False, 16, torch.bfloat16, None, [0, 11], [37, 20]),
    (2, 50, 4, 4, 128, 96, False, 128, torch.float16, "own", [100, 0], None),
    (1, 130, 2, 1, 128, 128, True, 32, torch.bfloat16, "own", [3], None),
    (1, 9, 2, 2, 128, 0, False, 32, torch.bfloat16, "own", [3], None),
    (1, 150, 3, 2, 128, 64, False, 128, torch.bfloat16, "own", [5], None),       # the largest page, 512 threads
    (2, 600, 27, 9, 64, 64, True, 16, torch.float16, "f32", [3, 40], [600, 333]),  # several heads a block, a short last group
    (2, 600, 27, 9, 128, 128, False, 64, torch.bfloat16, "own", [3, 40], [600, 333]),
    (70, 1, 20, 10, 128, 128, False, 16, torch.bfloat16, "own", list(range(70)), None),
    (3, 5, 13, 1, 64, 32, False, 32, torch.float16, None, [0, 30, 31], [5, 0, 4]),  # q's heads beside each other
]


@pytest.mark.parametrize("case", NRA)
def test_norm_rope_append_equals_the_two_calls(case):
    B, T, Hq, H, d, rot, il, page, dtype, weights, before, new = case
    g = torch.Generator().manual_seed(17)
    most = max(before) + T
    pages, table = _layout(B, page, most, g)
    wd = {"own": dtype, "f32": torch.float32, None: None}[weights]
    wq, wk = (None if wd is None else (1 + 0.3 * torch.randn(d, generator=g)).to(wd).cuda() for _ in range(2))
    cos, sin = fa.rope_tables(most, rot) if rot else (None, None)
    a, b = fa.kv8_cache_alloc(pages, page, H, d), fa.kv8_cache_alloc(pages, page, H, d)
    old = [_values((B, max(max(before), 1), H, d), dtype, g).cuda() for _ in range(2)]
    for c in (a, b):
        fa.kv8_append(c, *old, _cu(table), _cu(before), _cu(before))
    q = _values((B, T, Hq, d), dtype, g).cuda()
    k, v = _values((B, T, H, d), dtype, g).cuda(), _values((B, T, H, d), dtype, g).cuda()
    n = [T] * B if new is None else new
    lens = _cu([x + y for x, y in zip(before, n)])
    qo = fa.kv8_norm_rope_append(a, q, k, v, wq, wk, cos, sin, _cu(table), lens, _cu(new), 1e-5, il)
    pos = _cu([[x + t for t in range(T)] for x in before])
    q2, k2 = fa.qk_norm_rope_forward(q, k, wq, wk, cos, sin, pos, 1e-5, il)
    fa.kv8_append(b, k2, v, _cu(table), lens, _cu(new))
    for x, y in zip(a, b):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    for i, m in enumerate(n):
        assert torch.equal(qo[i, :m], q2[i, :m])
        assert bool((qo[i, m:] == 0).all())
    assert fa.fa_get_device_status() == 0


# ------------------------------------------------------------------ attention
def _filled(pages, page, H, d, g, dtype=torch.float16):
    """A cache filled page by page with values of varying scale."""
    cache = fa.kv8_cache_alloc(pages, page, H, d)
    table = torch.arange(pages, dtype=torch.int32)[:, None].contiguous().cuda()
    k, v = (_values((pages, page, H, d), dtype, g, 1.0).cuda() for _ in range(2))
    fa.kv8_append(cache, k, v, table, _cu([page] * pages))
    return cache


def _check(q, cache, table, lens, new, max_seqlen, dtype, window=0, causal=True, alibi=None, scale=None, o=None,
           lse=None):
    if o is None:
        o, lse = fa.kv8_attention(q, cache, _cu(table), _cu(lens), max_seqlen, _cu(new), scale, causal, window,
                                  None if alibi is None else alibi.cuda())
    d = q.shape[3]
    sc = fa.default_scale(d) if scale is None else scale
    r = ref.RefCache(cache)
    args = (table, lens, new, max_seqlen, sc, causal, window, None if alibi is None else alibi.double())
    wo, wl = r.attention(ref.f64(q), *args)
    r.codes[1] = r.codes[1].abs()
    vabs, _ = r.attention(ref.f64(q), *args)
    n = max(1, min(max(lens), max_seqlen))
    kmax = (r.codes[0].nan_to_num().abs() * r.scales[0][:, None, :, None]).amax((0, 1))  # [H, d]
    G = q.shape[2] // cache.k.shape[2]
    A = abs(sc) * (ref.f64(q).nan_to_num().abs() * kmax.repeat_interleave(G, 0)).sum(-1)  # [B, T, Hq]
    if alibi is not None:
        A = A + alibi.double().abs().max() * n
    delta = (d + 8) * 2.0 ** -23 * A + 64 * 2.0 ** -24
    vmax = float((r.codes[1].nan_to_num() * r.scales[1][:, None, :, None]).max())
    rel = 2 * delta[..., None] + (2.0 ** -12 if dtype == torch.bfloat16 else 2.0 ** -22) + (n + 64) * 2.0 ** -23
    got = ref.f64(o)
    assert torch.equal(got.isnan(), wo.isnan())
    err = (got - wo).abs().nan_to_num()
    bound = (HALF[dtype] * wo.abs() + vabs * rel + n * 2.0 ** -32 * vmax + TINY[dtype]).nan_to_num()
    assert torch.all(err <= bound), float((err / bound.clamp(min=1e-300)).max())
    gl = ref.f64(lse)
    live = wl.isfinite()
    assert torch.equal(gl.isfinite(), live) and bool((gl[wl == -math.inf] == -math.inf).all())
    dl = (delta + (n + 64) * 2.0 ** -23).transpose(1, 2) + 2.0 ** -22 * (1 + wl.abs())
    assert torch.all(((gl - wl).abs() <= dl)[live])
    return o, lse


ATTN = [
    # B, T, Hq, H, d, page, dtype, lens, new, window, causal, alibi
    (3, 1, 4, 4, 128, 16, torch.bfloat16, [1, 17, 0], None, 0, True, False),
    (3, 1, 4, 4, 64, 64, torch.float16, [1, 64, 65], None, 0, True, False),
    (2, 1, 8, 1, 128, 64, torch.bfloat16, [300, 127], None, 0, True, True),
    (2, 1, 12, 4, 64, 32, torch.float16, [257, 31], None, 20, True, False),
    (2, 1, 15, 1, 128, 16, torch.float16, [100, 33], None, 0, True, False),
    (1, 1, 64, 2, 64, 128, torch.bfloat16, [201], None, 0, True, False),
    (2, 5, 2, 2, 128, 32, torch.bfloat16, [70, 5], [5, 2], 0, True, False),
    (2, 5, 6, 2, 64, 16, torch.float16, [70, 3], None, 3, True, True),      # more new tokens than tokens
    (1, 40, 4, 2, 64, 16, torch.bfloat16, [40], None, 0, True, False),      # a whole prompt
    (1, 33, 3, 1, 128, 64, torch.float16, [150], None, 17, True, False),
    (2, 3, 4, 2, 128, 32, torch.bfloat16, [90, 40], [3, 0], 0, False, True),
    (1, 3, 4, 2, 64, 16, torch.float16, [90], None, 30, False, False),
    (1, 1, 2, 2, 128, 64, torch.bfloat16, [5000], None, 0, True, False),
    (1, 2, 16, 2, 64, 16, torch.float16, [3001], None, 0, True, False),
    (2, 5, 4, 4, 64, 32, torch.float16, [900, 333], [3, 4], 500, True, False),  # padding rows in whole steps
    (2, 4, 2, 1, 128, 64, torch.bfloat16, [64, 48], [1, 0], 0, False, False),
    (1, 3, 4, 2, 64, 64, torch.float16, [9000], None, 0, True, True),
    (2, 2, 12, 1, 128, 128, torch.bfloat16, [7001, 13], [2, 1], 6000, True, False),
    (1, 9, 4, 1, 128, 128, torch.bfloat16, [6500], None, 0, False, False),
    (1, 1, 33, 1, 64, 32, torch.bfloat16, [200], None, 0, True, False),     # rows in three blocks of 16
    (40, 1, 16, 16, 64, 16, torch.float16, [(37 * b) % 300 for b in range(40)], None, 0, True, False),
]


@pytest.mark.parametrize("case", ATTN)
def test_attention_against_float64(case):
    B, T, Hq, H, d, page, dtype, lens, new, window, causal, alibi = case
    g = torch.Generator().manual_seed(23)
    pages, table = _layout(B, page, max(lens), g)
    cache = _filled(pages, page, H, d, g)
    q = _values((B, T, Hq, d), dtype, g, 1.0).cuda()
    slopes = (0.02 + 0.3 * torch.rand(B, Hq, generator=g)) if alibi else None
    a = _check(q, cache, table, lens, new, max(lens), dtype, window, causal, slopes)
    b = fa.kv8_attention(q, cache, _cu(table), _cu(lens), max(lens), _cu(new), None, causal, window,
                         None if slopes is None else slopes.cuda())
    for x, y in zip(a, b):
        assert torch.equal(x.view(torch.int16 if x.element_size() == 2 else torch.int32),
                           y.view(torch.int16 if x.element_size() == 2 else torch.int32))  # the same bits again
    if alibi:  # one slope a head for all sequences
        _check(q, cache, table, lens, new, max(lens), dtype, window, causal, slopes[0].contiguous())
    assert fa.fa_get_device_status() == 0


@pytest.mark.parametrize("B,T,Hq,H,d,page,width,dtype", [
    (127, 1, 4, 4, 64, 16, 2048, torch.float16),
    (128, 1, 8, 4, 128, 32, 2048, torch.bfloat16),
    (129, 1, 4, 4, 64, 16, 2048, torch.bfloat16),   # taken in the given order
    (128, 1, 4, 4, 64, 16, 0, torch.bfloat16),      # short blocks, in the given order
    (32, 1, 8, 8, 64, 16, 16384, torch.bfloat16),   # clusters of four blocks a sequence
    (3, 40, 32, 4, 64, 16, 2048, torch.float16),    # twenty row tiles a key head
    (2, 64, 64, 4, 128, 64, 9000, torch.bfloat16),
])
def test_unequal_lengths_in_several_rounds_of_blocks(B, T, Hq, H, d, page, width, dtype):
    # lengths that come several times, that are zero, that pass max_seqlen
    lens = [(29 * b * b + T) % 83 for b in range(B)]
    lens[0], lens[-1] = 0, 200
    g = torch.Generator().manual_seed(29)
    pages, table = _layout(B, page, max(lens), g)
    cache = _filled(pages, page, H, d, g)
    q = _values((B, T, Hq, d), dtype, g, 1.0).cuda()
    limit = max(lens)
    if width:  # a table made for longer sequences
        table = torch.nn.functional.pad(torch.as_tensor(table), (0, width // page - len(table[0])), value=-1)
        limit = width
    else:
        lens[1] = page * len(table[0]) + 7
    _check(q, cache, table, lens, None, limit, dtype)
    assert fa.fa_get_device_status() == 0


@pytest.mark.parametrize("max_seqlen", [40, 100, 4000])
def test_max_seqlen_bounds_the_keys(max_seqlen):
    """Any upper bound gives the same values up to the tolerance (another split); a smaller one ends the keys."""
    g = torch.Generator().manual_seed(29)
    pages, table = _layout(2, 16, 100, g)
    cache = _filled(pages, 16, 2, 128, g)
    q = _values((2, 1, 4, 128), torch.bfloat16, g, 1.0).cuda()
    _check(q, cache, table, [100, 63], None, max_seqlen, torch.bfloat16)
    # with a window that ends before the last key in reach: rows without a key
    o, lse = _check(q, cache, table, [100, 63], None, max_seqlen, torch.bfloat16, window=20)
    assert bool((o[0] == 0).all()) == (max_seqlen == 40) and bool((lse[0] == -math.inf).all()) == (max_seqlen == 40)


def test_nan_reaches_only_the_rows_that_attend_to_it():
    """NaN codes (and whatever unused slots hold) in keys and values: rows that see the token get NaN, all
    others are as without it."""
    g = torch.Generator().manual_seed(37)
    B, T, H, d, page = 1, 6, 2, 64, 16
    pages, table = _layout(B, page, 60, g)
    cache = _filled(pages, page, H, d, g)
    q = _values((B, T, 2 * H, d), torch.float16, g, 1.0).cuda()

    def slot(j):
        return int(table[0, j // page]), j % page

    for x in (cache.k, cache.v):  # behind the last token
        p, s = slot(56)
        x.view(torch.uint8)[p, s + 1:] = 0x7F
    # a value of the third newest token, head 0; a key of the second newest, head 1; a value outside the window
    p, s = slot(54)
    cache.v.view(torch.uint8)[p, s, 0, 5] = 0xFF
    p, s = slot(55)
    cache.k.view(torch.uint8)[p, s, 1, 9] = 0x7F
    p, s = slot(31)
    cache.v.view(torch.uint8)[p, s, :, 3] = 0x7F
    for window in (0, 20):
        o, lse = _check(q, cache, table, [57], None, 57, torch.float16, window)
        assert bool(o.isnan().any()) and not bool(o.isnan().all())
    # newest six tokens (51 .. 56), window 20: token 31 is seen by none but the first (51 - 19 = 32 > 31: none)
    assert not bool(o[0, :3, :2].isnan().any())
    assert bool(o[0, 3:, :2, 5].isnan().all()) and not bool(o[0, 3:, :2, :5].isnan().any())
    assert not bool(o[0, :4, 2:].isnan().any()) and bool(o[0, 4:, 2:].isnan().all())


@pytest.mark.parametrize("length", [200, 3000, 9000])
def test_nan_does_not_reach_padding_rows(length):
    """Keys and values that hold NaN everywhere: padding rows are zeros and -inf all the same, whether one
    block, a cluster or a second kernel writes them; rows with a token are NaN."""
    g = torch.Generator().manual_seed(38)
    pages, table = _layout(1, 64, length, g)
    cache = _filled(pages, 64, 1, 64, g)
    cache.k.view(torch.uint8).fill_(0x7F)
    cache.v.view(torch.uint8).fill_(0xFF)
    q = _values((1, 4, 2, 64), torch.bfloat16, g, 1.0).cuda()
    o, lse = fa.kv8_attention(q, cache, _cu(table), _cu([length]), length, _cu([2]))
    assert bool(o[0, :2].isnan().all()) and bool((o[0, 2:] == 0).all())
    assert bool(lse[0, :, :2].isnan().all()) and bool((lse[0, :, 2:] == -math.inf).all())


def test_nan_weights_do_not_reach_padding():
    """A NaN weight makes the rows with a token NaN and nothing else: padding rows of q stay zeros, and the
    values and the other pages of the cache are untouched."""
    g = torch.Generator().manual_seed(39)
    cache = fa.kv8_cache_alloc(4, 16, 2, 64)
    want = ref.RefCache(cache)
    table = torch.tensor([[0, 1], [2, 3]], dtype=torch.int32)
    q, k, v = (_values((2, 5, h, 64), torch.float16, g, 1.0) for h in (4, 2, 2))
    w = torch.ones(64, dtype=torch.float16)
    w[3] = float("nan")
    cos, sin = fa.rope_tables(32, 32)
    qo = fa.kv8_norm_rope_append(cache, q.cuda(), k.cuda(), v.cuda(), w.cuda(), w.cuda(), cos, sin, _cu(table),
                                 _cu([5, 2]), _cu([5, 2]))
    assert bool((qo[1, 2:] == 0).all()) and bool(qo[1, :2].isnan().any())
    want.append(ref.f64(k), ref.f64(v), table, [5, 2], [5, 2])
    assert torch.equal(cache.v.cpu().float().double(), want.codes[1])
    held = cache.k.cpu().float()
    assert bool(held[0, :5, :, 3].isnan().all()) and bool((held[1] == 0).all()) and bool((held[2, 2:] == 0).all())
    assert bool(held[0, :5, :, 32:].isfinite().all())  # (past the rotated half a NaN weight touches its value alone)


def test_bad_pages_are_not_attended_to():
    g = torch.Generator().manual_seed(41)
    cache = _filled(5, 16, 2, 64, g)
    q = _values((2, 2, 4, 64), torch.bfloat16, g, 1.0).cuda()
    table = torch.tensor([[0, 5, 2], [-1, 7, 2 ** 31 - 1]], dtype=torch.int32)
    o, lse = _check(q, cache, table, [40, 48], None, 48, torch.bfloat16)
    assert bool((o[1] == 0).all()) and bool((lse[1] == -math.inf).all())
    assert fa.fa_get_device_status(clear=True) == 4


def test_page_scales_far_apart():
    """Pages whose key and value scales differ by up to 2^100, in both orders."""
    g = torch.Generator().manual_seed(43)
    page, d = 16, 128
    for order in ([0, 1, 2, 3], [3, 2, 1, 0], [1, 3, 0, 2]):
        cache = fa.kv8_cache_alloc(4, page, 1, d)
        table = torch.tensor([order], dtype=torch.int32)
        size = torch.tensor([2.0 ** -60, 1.0, 2.0 ** 13, 2.0 ** 40]).repeat_interleave(page)
        k = torch.randn(1, 64, 1, d, generator=g).to(torch.bfloat16)
        v = (torch.randn(1, 64, 1, d, generator=g) * size[None, :, None, None]).to(torch.bfloat16)
        fa.kv8_append(cache, k.cuda(), v.cuda(), _cu(table), _cu([64]))
        q = torch.randn(1, 1, 2, d, generator=g).to(torch.bfloat16).cuda()
        _check(q, cache, table, [64], None, 64, torch.bfloat16)
        # only the smallest page is in reach: its values are not lost beside the others' units
        first = order.index(0)
        _check(q, cache, table, [64], None, 64, torch.bfloat16, window=16) if first == 3 else None


def test_large_and_small_queries():
    """bf16 queries of sizes that f16 cannot hold: the power of two goes out of the row and back."""
    g = torch.Generator().manual_seed(47)
    cache = _filled(4, 16, 2, 64, g)
    table = torch.tensor([[3, 1, 0, 2]], dtype=torch.int32)
    for size, scale in ((2.0 ** 60, 2.0 ** -63), (2.0 ** -60, 2.0 ** 57), (2.0 ** 20, 2.0 ** -23)):
        q = (torch.randn(1, 1, 4, 64, generator=g) * size).to(torch.bfloat16).cuda()
        _check(q, cache, table, [60], None, 60, torch.bfloat16, scale=scale)
    q = torch.zeros(1, 1, 4, 64, dtype=torch.bfloat16, device="cuda")
    _check(q, cache, table, [60], None, 60, torch.bfloat16)
    _check(q + 1, cache, table, [60], None, 60, torch.bfloat16, scale=0.0)
    _check(q + 1, cache, table, [60], None, 60, torch.bfloat16, scale=-0.2)


def test_rising_scores():
    """Every next step holds a larger maximum: the running reference moves again and again."""
    d, page = 64, 16
    cache = fa.kv8_cache_alloc(40, page, 1, d)
    table = torch.arange(40, dtype=torch.int32)[None].contiguous()
    g = torch.Generator().manual_seed(51)
    ramp = torch.arange(640).float()
    for sign in (1.0, -1.0):
        k = torch.zeros(1, 640, 1, d)
        k[0, :, 0, 0] = sign * ramp
        v = torch.randn(1, 640, 1, d, generator=g)
        fa.kv8_append(cache, k.half().cuda(), v.half().cuda(), _cu(table), _cu([640]))
        q = torch.zeros(1, 1, 2, d, dtype=torch.float16, device="cuda")
        q[..., 0] = 1.0
        _check(q, cache, table, [640], None, 640, torch.float16, scale=0.7)


def test_strided_cache_queries_and_outputs():
    """A cache with tokens, heads and pages apart (NaN codes between), q as a slice of a projection, o in a
    larger buffer: the dense call's bits, nothing else written."""
    g = torch.Generator().manual_seed(53)
    B, T, Hq, H, d, page = 2, 3, 4, 2, 64, 16
    pages, table = _layout(B, page, 40, g)
    dense = _filled(pages, page, H, d, g)
    cache, _ = _strided_cache(pages, page, H, d)
    cache.k.view(torch.uint8).copy_(dense.k.view(torch.uint8))
    cache.v.view(torch.uint8).copy_(dense.v.view(torch.uint8))
    cache.k_scale.copy_(dense.k_scale)
    cache.v_scale.copy_(dense.v_scale)
    q = _values((B, T, Hq + 3, d), torch.bfloat16, g, 1.0).cuda()[:, :, 1:1 + Hq]
    want = fa.kv8_attention(q.contiguous(), dense, _cu(table), _cu([40, 21]), 40)
    buf = torch.full((B * T * (Hq + 2) * (d + 8) + 16,), 7.0, dtype=torch.bfloat16, device="cuda")
    o = buf.as_strided((B, T, Hq, d), (T * (Hq + 2) * (d + 8), (Hq + 2) * (d + 8), d + 8, 1), 8)
    lse = torch.full((B * Hq * T + 8,), 7.0, device="cuda")
    size = fa.fa_kv8_attn_workspace_size(B, T, Hq, H, d, page, table.shape[1], 40)
    assert size == 0  # no workspace needed: one that is there all the same is left alone
    ws = torch.full((512,), 165, dtype=torch.uint8, device="cuda")
    fa.fa_kv8_attn(q, cache, o, lse[4:-4].view(B, Hq, T), _cu(table), _cu([40, 21]), 40, ws)
    assert torch.equal(o, want[0]) and torch.equal(lse[4:-4].view(B, Hq, T), want[1])
    o.fill_(7.0)
    assert bool((buf == 7.0).all()) and bool((lse[:4] == 7).all()) and bool((lse[-4:] == 7).all())
    assert bool((ws == 165).all())


def test_workspace_is_not_overrun_by_splits():
    g = torch.Generator().manual_seed(59)
    cache = _filled(130, 64, 1, 64, g)
    table = torch.arange(130, dtype=torch.int32)[None].contiguous()
    q = _values((1, 2, 3, 64), torch.float16, g, 1.0).cuda()
    size = fa.fa_kv8_attn_workspace_size(1, 2, 3, 1, 64, 64, 130, 8320)
    assert size > 0  # split
    ws = torch.full((size + 256,), 165, dtype=torch.uint8, device="cuda")
    o, lse = torch.empty_like(q), torch.empty(1, 3, 2, device="cuda")
    fa.fa_kv8_attn(q, cache, o, lse, _cu(table), _cu([8309]), 8320, ws[:size])
    assert bool((ws[size:] == 165).all())
    _check(q, cache, table, [8309], None, 8320, torch.float16, o=o, lse=lse)


def test_offsets_past_32_bits():
    """Pages beyond 2^32 bytes of the cache are written and read in place."""
    d, page, H = 128, 128, 8
    per = page * H * d
    pages = (1 << 32) // per + 40
    buf = [torch.empty(pages * per, dtype=torch.uint8, device="cuda") for _ in range(2)]
    big = fa.Kv8Cache(*(b.view(torch.float8_e4m3fn).view(pages, H, page, d).transpose(1, 2) for b in buf),
                      *(torch.ones(pages, H, device="cuda") for _ in range(2)))
    small = fa.kv8_cache_alloc(40, page, H, d)
    g = torch.Generator().manual_seed(61)
    k, v = (_values((1, 300, H, d), torch.bfloat16, g).cuda() for _ in range(2))
    q = _values((1, 1, 2 * H, d), torch.bfloat16, g, 1.0).cuda()
    table = torch.tensor([[7, 39, 1]], dtype=torch.int32)
    out = []
    for cache, add in ((small, 0), (big, pages - 40)):
        fa.kv8_append(cache, k, v, _cu(table + add), _cu([300]))
        out.append(fa.kv8_attention(q, cache, _cu(table + add), _cu([300]), 300))
    assert torch.equal(out[0][0], out[1][0]) and torch.equal(out[0][1], out[1][1])


def test_shared_prefix_pages():
    """Two sequences read the same pages, a token's page may occur twice in a table that is only read."""
    g = torch.Generator().manual_seed(67)
    cache = _filled(6, 16, 2, 64, g)
    q = _values((2, 1, 4, 64), torch.float16, g, 1.0).cuda()
    table = torch.tensor([[0, 1, 2], [0, 1, 0]], dtype=torch.int32)
    _check(q, cache, table, [40, 47], None, 48, torch.float16)


def test_serving_loop_together_and_captured():
    """A prompt, then tokens one by one: norm + rotation + append, attention; the outputs equal attention over
    everything so far (float64, over the cache's values), and a captured step replayed for every token gives
    the eager loop's bits. Two captured steps on two caches, replayed in turn, do not disturb each other."""
    g = torch.Generator().manual_seed(71)
    B, Hq, H, d, page, dtype, prompt, steps = 2, 4, 2, 64, 16, torch.bfloat16, 21, 14
    most = prompt + steps
    pages, table_h = _layout(B, page, most, g)
    table = _cu(table_h)
    cos, sin = fa.rope_tables(most, d)
    wq, wk = ((1 + 0.2 * torch.randn(d, generator=g)).to(dtype).cuda() for _ in range(2))
    qkv = _values((B, most, Hq + 2 * H, d), dtype, g, 2.0).cuda()

    def step(cache, x, lens, most_now):
        q = fa.kv8_norm_rope_append(cache, x[:, :, :Hq], x[:, :, Hq:Hq + H], x[:, :, Hq + H:], wq, wk, cos, sin, table,
                                    lens)
        return q, fa.kv8_attention(q, cache, table, lens, most_now)

    def fresh():
        c = fa.kv8_cache_alloc(pages, page, H, d)
        lens = _cu([prompt] * B)
        q, out = step(c, qkv[:, :prompt], lens, most)
        _check(q, c, table_h, [prompt] * B, None, most, dtype, o=out[0], lse=out[1])
        return c, lens

    eager, lens = fresh()
    outs = []
    for t in range(prompt, most):
        lens += 1
        q, out = step(eager, qkv[:, t:t + 1], lens, most)
        outs.append(out)
        if t in (prompt, most - 1):
            _check(q, eager, table_h, [t + 1] * B, None, most, dtype, o=out[0], lse=out[1])
    made = []
    for _ in range(2):
        c, ln = fresh()
        x = torch.empty_like(qkv[:, :1])
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            ln += 1
            _, out = step(c, x, ln, most)
        made.append((c, x, graph, out, ln))  # (what a graph reads has to live as long as it)
    for i, t in enumerate(range(prompt, most)):
        for c, x, graph, out, _ in made:
            x.copy_(qkv[:, t:t + 1])
            graph.replay()
        for c, x, graph, out, _ in made:
            assert torch.equal(out[0], outs[i][0]) and torch.equal(out[1], outs[i][1])
    for c, *_ in made:
        for a, b in zip(c, eager):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("length,heads", [(600, 2), (9000, 1)])
def test_attention_captured_and_two_threads(length, heads):
    """Split over a cluster and over a workspace: captured twice and replayed in turn with new queries, and
    called by two host threads on two streams at once, every result equals the lone call's."""
    import threading

    g = torch.Generator().manual_seed(83)
    pages, table_h = _layout(1, 64, length, g)
    cache = _filled(pages, 64, heads, 128, g)
    table, lens = _cu(table_h), _cu([length])
    qs = [_values((1, 1, 4 * heads, 128), torch.bfloat16, g, 1.0).cuda() for _ in range(4)]
    want = [fa.kv8_attention(q, cache, table, lens, length) for q in qs]
    made = []
    for _ in range(2):
        x = torch.empty_like(qs[0])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = fa.kv8_attention(x, cache, table, lens, length)
        made.append((x, graph, out))
    for i in (0, 2):
        for j, (x, graph, _) in enumerate(made):
            x.copy_(qs[i + j])
        for _, graph, _ in made:
            graph.replay()
        for j, (_, _, out) in enumerate(made):
            assert torch.equal(out[0], want[i + j][0]) and torch.equal(out[1], want[i + j][1])
    torch.cuda.synchronize()
    got, errors = {}, []

    def worker(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                got[i] = [fa.kv8_attention(qs[i], cache, table, lens, length) for _ in range(20)]
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # surfaced below
            errors.append(e)

    threads = [threading.Thread(target=worker, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for i in range(2):
        for o, lse in got[i]:
            assert torch.equal(o, want[i][0]) and torch.equal(lse, want[i][1])


def test_captured_with_forked_streams():
    """A step whose append runs on a side stream beside another kernel and is joined before the attention,
    captured into a graph and replayed on new values: the eager results. (The kernels are launched so that
    they may begin early; across streams the events alone order them.)"""
    g = torch.Generator().manual_seed(89)
    B, Hq, H, d, page, tokens = 2, 4, 2, 128, 16, 40
    pages, table_h = _layout(B, page, tokens, g)
    table, lens = _cu(table_h), _cu([tokens] * B)
    made = [_values((B, tokens, h, d), torch.bfloat16, g, 1.0).cuda() for h in (Hq, H, H, Hq, H, H)]
    x = [torch.empty_like(t) for t in made[:3]]
    cache = fa.kv8_cache_alloc(pages, page, H, d)
    cos, sin = fa.rope_tables(tokens, d)
    side = torch.cuda.Stream()

    def step():
        main = torch.cuda.current_stream()
        k, v = x[1] * 1, x[2] * 1
        side.wait_stream(main)
        with torch.cuda.stream(side):
            fa.kv8_append(cache, k, v, table, lens)
        q, _ = fa.qk_norm_rope_forward(x[0], x[1], None, None, cos, sin)
        main.wait_stream(side)
        return fa.kv8_attention(q, cache, table, lens, tokens)

    want = []
    for i in (0, 3):
        for a, b in zip(x, made[i:i + 3]):
            a.copy_(b)
        want.append([t.clone() for t in step()])
        torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for n in (0, 1, 0):
        for a, b in zip(x, made[3 * n:3 * n + 3]):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], want[n][0]) and torch.equal(out[1], want[n][1])


def test_a_row_of_calls_without_waiting():
    """Calls enqueued one behind the other, each reading what the one before wrote (early beginnings must
    not be seen): token by token through append and attention on one stream, against the same calls with
    the GPU waited for after each."""
    g = torch.Generator().manual_seed(97)
    B, Hq, H, d, page, tokens = 3, 8, 2, 128, 32, 70
    pages, table_h = _layout(B, page, tokens, g)
    table = _cu(table_h)
    cos, sin = fa.rope_tables(tokens, d)
    w = (1 + 0.2 * torch.randn(d, generator=g)).to(torch.bfloat16).cuda()
    q, k, v = (_values((B, tokens, h, d), torch.bfloat16, g, 2.0).cuda() for h in (Hq, H, H))
    lens = [_cu([t + 1] * B) for t in range(tokens)]

    def loop(wait):
        cache = fa.kv8_cache_alloc(pages, page, H, d)
        x = q[:, :1].contiguous()
        outs = []
        torch.cuda.synchronize()
        if not wait:
            torch.cuda._sleep(40_000_000)  # so that the calls pile up
        for t in range(tokens):
            # the next query depends on the last output
            x = fa.kv8_norm_rope_append(cache, (q[:, t:t + 1] + x).contiguous(), k[:, t:t + 1], v[:, t:t + 1], w, w, cos,
                                        sin, table, lens[t])
            x, lse = fa.kv8_attention(x, cache, table, lens[t], tokens)
            x, _ = fa.qk_norm_rope_forward(x, x, None, None, cos, sin)
            outs.append((x, lse))
            if wait:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        return outs, cache

    (a, ca), (b, cb) = loop(True), loop(False)
    for (x, l), (y, m) in zip(a, b):
        assert torch.equal(x, y) and torch.equal(l, m)
    for s, t in zip(ca, cb):
        assert torch.equal(s.view(torch.uint8), t.view(torch.uint8))


def test_other_stream():
    """Calls on a side stream take that stream's order: inputs written there just before are seen."""
    g = torch.Generator().manual_seed(73)
    k, v = (_values((1, 600, 2, 64), torch.float16, g).cuda() for _ in range(2))
    q = _values((1, 1, 4, 64), torch.float16, g, 1.0).cuda()
    table, lens = _cu([list(range(5))]), _cu([600])
    a, b = fa.kv8_cache_alloc(5, 128, 2, 64), fa.kv8_cache_alloc(5, 128, 2, 64)
    fa.kv8_append(a, k, v, table, lens)
    want = fa.kv8_attention(q, a, table, lens, 600)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
        k2, v2, q2 = k * 1, v * 1, q * 1
        fa.kv8_append(b, k2, v2, table, lens)
        got = fa.kv8_attention(q2, b, table, lens, 600)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_refusals_on_the_gpu():
    g = torch.Generator().manual_seed(79)
    cache = fa.kv8_cache_alloc(3, 16, 2, 64)
    q, k = (torch.zeros(1, 1, h, 64, dtype=torch.float16, device="cuda") for h in (4, 2))
    table, lens = _cu([[0, 1, 2]]), _cu([1])
    with pytest.raises(ValueError):
        fa.kv8_append(cache, k, k, table.long(), lens)
    with pytest.raises(ValueError):
        fa.kv8_append(cache, k, k, table, lens.cpu())
    with pytest.raises(ValueError):
        fa.kv8_append(cache, k, k, table, _cu([1, 1]))                # another batch size
    with pytest.raises(ValueError):
        fa.kv8_append(cache, k, q, table, lens)                       # v of other heads
    with pytest.raises(ValueError):
        fa.kv8_append(cache, q, q, table, lens)                       # more heads than the cache's
    with pytest.raises(ValueError):
        fa.kv8_append(cache, k.float(), k.float(), table, lens)
    with pytest.raises(ValueError):
        fa.kv8_append(cache, k[..., :32], k[..., :32], table, lens)
    with pytest.raises(ValueError):
        fa.kv8_append(cache, k, k.bfloat16(), table, lens)
    with pytest.raises(ValueError):
        fa.kv8_append(cache._replace(k_scale=cache.k_scale.half()), k, k, table, lens)
    with pytest.raises(ValueError):
        fa.kv8_append(cache._replace(k=cache.k.view(torch.uint8)), k, k, table, lens)
    with pytest.raises(ValueError):
        fa.kv8_append(cache._replace(v=fa.kv8_cache_alloc(4, 16, 2, 64).v), k, k, table, lens)
    with pytest.raises(fa.FaError):
        fa.kv8_attention(q[:, :, :3], cache, table, lens, 16)         # 3 query heads over 2
    with pytest.raises(fa.FaError):
        fa.kv8_attention(q, cache, table, lens, 0)
    o, lse = torch.empty_like(q), torch.empty(1, 4, 1, device="cuda")
    long = _cu([list(range(3)) * 400])
    with pytest.raises(fa.FaError):
        fa.fa_kv8_attn(q, cache, o, lse, long, lens, 16 * 1200, torch.empty(0, dtype=torch.uint8, device="cuda"))
    with pytest.raises(fa.FaError):
        fa.fa_kv8_attn(q, cache, o, lse, long, lens, 16 * 1200, None)
    with pytest.raises(ValueError):
        fa.fa_kv8_attn(q, cache, o, lse[:, :2], table, lens, 16, torch.empty(256, dtype=torch.uint8, device="cuda"))
    other = fa.kv8_cache_alloc(3, 16, 2, 64, device="cpu")
    with pytest.raises(ValueError):
        fa.kv8_append(other, k, k, table, lens)

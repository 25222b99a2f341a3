"""Attention over the 8-bit cache where pages hold values of very different sizes, held to each row's own
output (only the keys that the row attends to enter the bound), against float64.

With p_j the exact weights of a row, v_j its values and A = max_j |scale| sum_i |q_i k_ji|: a score is off
by (d + 8) * 2^-23 * A (fp32 sums) + 64 * 2^-24 (ex2.approx, |s - m| < 64 where a weight matters) + what the
query's e4m3 pieces leave, at most 2^-21 (bf16, two pieces) or 2^-25 (f16, three) of its largest value:
Q = |scale| * max|q| * max_j sum_i |k_ji| of it. Together delta; a weight is off by 2 delta relative (its
own, and the sum's). Its product with the page's scale s_j is rounded to f16 (half a step: 2^-11 relative,
with its residual 2^-22; bf16 has the residual up to eight rows a key head) in units in which the largest p_j s_j of a warp is at least 2^7, so products below 2^-14 of
the unit lose up to 2^-25 of it: 2^-32 of the largest p_j s_j, times a code of at most 448. n keys are
summed in fp32: (n + 64) * 2^-23. The output is rounded to its type.
"""
import math

import pytest
import torch

import flashattention_backward_fa_gb300 as fa
import serve_reference as ref

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16
HALF = {BF16: 2.0 ** -8, F16: 2.0 ** -11}     # half a step of the type, relative to the value
TINY = {BF16: 2.0 ** -126, F16: 2.0 ** -25}   # half a step of f16's subnormals; fp32's may count as zero
RESIDUAL_ROWS = {BF16: 8, F16: 1 << 30}       # most rows (tokens x query heads) of a key head with the residual
PIECES = {BF16: 2.0 ** -21, F16: 2.0 ** -25}


def _cu(x):
    return torch.as_tensor(x, dtype=torch.int32).cuda()


def _check(q, cache, table, lens, new=None, scale=1.0, causal=True, window=0):
    """One call against float64, row by row; the (o, lse) that it gave."""
    dtype = q.dtype
    B, T, Hq, d = q.shape
    H, page = cache.k.shape[2], cache.k.shape[1]
    o, lse = fa.kv8_attention(q, cache, _cu(table), _cu(lens), max(lens), None if new is None else _cu(new), scale,
                              causal, window)
    got, got_lse, q64 = ref.f64(o), ref.f64(lse), ref.f64(q)
    codes = [ref.f64(x.float()) for x in (cache.k, cache.v)]
    scales = [ref.f64(x) for x in (cache.k_scale, cache.v_scale)]
    for b in range(B):
        n, count = lens[b], T if new is None else new[b]
        at = torch.as_tensor(table[b][:-(-n // page)]).long()
        k, v = ((codes[i][at] * scales[i][at][:, None, :, None]).flatten(0, 1)[:n] for i in (0, 1))
        unit = scales[1][at].repeat_interleave(page, 0)[:n]
        i, j = torch.arange(n - count, n)[:, None], torch.arange(n)
        hide = (j > i) if causal else torch.zeros(count, n, dtype=torch.bool)
        if window:
            hide = hide | (j <= i - window)
        assert bool((got[b, count:] == 0).all())
        for hq in range(Hq):
            h = hq // (Hq // H)
            qr = q64[b, :count, hq]
            s = (qr @ k[:, h].T * scale).masked_fill(hide, -math.inf)
            p = s.softmax(-1)
            A = (qr.abs() @ k[:, h].abs().T * abs(scale)).masked_fill(hide, 0).amax(-1)
            Q = abs(scale) * qr.abs().amax(-1) * k[:, h].abs().sum(-1).masked_fill(hide, 0).amax(-1)
            delta = (d + 8) * 2.0 ** -23 * A + 64 * 2.0 ** -24 + PIECES[dtype] * Q
            want, size = p @ v[:, h], p @ v[:, h].abs()
            most = (p * unit[:, h]).amax(-1)
            weight = 2.0 ** -22 if T * (Hq // H) <= RESIDUAL_ROWS[dtype] else 2.0 ** -11
            rel = 2 * delta + weight + (n + 64) * 2.0 ** -23
            bound = HALF[dtype] * want.abs() * (1 + 2.0 ** -6) + size * rel[:, None] + \
                (n * 448 * 2.0 ** -32 * most)[:, None] + TINY[dtype]
            err = (got[b, :count, hq] - want).abs()
            assert bool((err <= bound).all()), (b, hq, float((err / bound).nan_to_num(nan=math.inf).max()))
            wl = s.logsumexp(-1)
            dl = delta + (n + 64) * 2.0 ** -23 + 2.0 ** -22 * (1 + wl.abs())
            assert bool(((got_lse[b, hq, :count] - wl).abs() <= dl).all())
    assert fa.fa_get_device_status() == 0
    return o, lse


def _cache(k, v, page, table):
    """A cache that holds k, v [B, n, H, d] in the table's pages."""
    B, n, H, d = k.shape
    cache = fa.kv8_cache_alloc(int(table.max()) + 1, page, H, d)
    fa.kv8_append(cache, k.cuda(), v.cuda(), _cu(table), _cu([n] * B))
    return cache


def test_sums_survive_pages_of_zeros_behind_a_scale_of_one():
    """Values of 400 (scale 1.0, which is also the first unit of the sums) with weights that rise by 2^7.9
    in the second step of each warp, then pages of zeros, whose scale is 2^-100; keys not split."""
    B, H, d, page, n = 15, 16, 64, 16, 384
    k = torch.zeros(B, n, H, d, dtype=BF16)
    k[:, 128:, :, 0] = 5.5
    v = torch.full((B, n, H, d), 400.0, dtype=BF16)
    v[:, 256:] = 0.0
    table = torch.arange(B * n // page, dtype=torch.int32).view(B, -1)
    cache = _cache(k, v, page, table)
    assert float(cache.v_scale[0, 0]) == 1.0 and float(cache.v_scale[n // page - 1, 0]) == 2.0 ** -100
    q = torch.zeros(B, 1, H, d, dtype=BF16, device="cuda")
    q[..., 0] = 1.0
    o, _ = _check(q, cache, table, [n] * B)
    assert bool(o.isfinite().all())


# (page, log2 of the small page's size under the large one's)
FAR = [(16, 9, F16), (16, 20, F16), (16, 26, F16), (16, 26, BF16), (16, 30, BF16), (16, 60, BF16), (16, 100, BF16)]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page,ratio,dtype", FAR)
def test_weight_on_the_page_of_smaller_values(page, ratio, dtype, d):
    """Two pages in one step of 32 keys: nearly all the weight is on the one with the small values, the
    other one's is e^-80."""
    g = torch.Generator().manual_seed(71)
    top = 10 if dtype == F16 else 0
    for small in (0, 1):
        k = torch.randn(1, 2 * page, 1, d, generator=g) * 0.1
        k[..., 0] = 0.0
        k[0, (1 - small) * page:(2 - small) * page, 0, 0] = -10.0
        size = torch.full((2 * page,), 2.0 ** top)
        size[small * page:(small + 1) * page] = 2.0 ** (top - ratio)
        v = torch.randn(1, 2 * page, 1, d, generator=g) * size[None, :, None, None]
        table = torch.tensor([[1, 0]], dtype=torch.int32)
        cache = _cache(k.to(dtype), v.to(dtype), page, table)
        q = (torch.randn(1, 1, 3, d, generator=g) * 0.1).to(dtype)
        q[..., 0] = 8.0
        _check(q.cuda(), cache, table, [2 * page])


@pytest.mark.parametrize("dtype,ratio", [(F16, 20), (F16, 28), (BF16, 28), (BF16, 40), (BF16, 110)])
@pytest.mark.parametrize("page,length,T", [(16, 17, 2), (16, 40, 25), (32, 33, 2), (64, 200, 12)])
def test_large_values_that_a_row_does_not_see(page, length, T, dtype, ratio):
    """The last tokens' values are far larger than those before: rows before them must not notice."""
    g = torch.Generator().manual_seed(73)
    d, Hq, H = 64, 6, 2
    n = -(-length // page)
    top = 12 if dtype == F16 else 0
    size = torch.full((length,), 2.0 ** (top - ratio))
    size[(length - 1) // page * page:] = 2.0 ** top
    k = torch.randn(1, length, H, d, generator=g).to(dtype)
    v = (torch.randn(1, length, H, d, generator=g) * size[None, :, None, None]).to(dtype)
    table = torch.randperm(n, generator=g)[None].int()
    cache = _cache(k, v, page, table)
    q = torch.randn(1, T, Hq, d, generator=g).to(dtype).cuda()
    _check(q, cache, table, [length], scale=0.125)
    _check(q, cache, table, [length], scale=0.125, window=min(20, length))


@pytest.mark.parametrize("weight", [-18, -24, -30])
def test_small_weights_on_large_values(weight):
    """A page with 2^weight of the others' weights and values 2^40 times theirs makes the output; its
    weights must not be rounded as if they did not matter. Steps of one warp and of several."""
    g = torch.Generator().manual_seed(79)
    d, page = 128, 16
    for n, large in ((32, 1), (32, 0), (640, 33), (640, 0)):
        k = torch.zeros(1, n, 1, d)
        k[0, large * page:(large + 1) * page, 0, 0] = weight * math.log(2.0)
        size = torch.ones(n)
        size[large * page:(large + 1) * page] = 2.0 ** 40
        v = torch.randn(1, n, 1, d, generator=g) * size[None, :, None, None]
        table = torch.randperm(n // page, generator=g)[None].int()
        cache = _cache(k.to(BF16), v.to(BF16), page, table)
        q = torch.zeros(1, 1, 1, d, dtype=BF16, device="cuda")
        q[..., 0] = 1.0
        _check(q, cache, table, [n])


@pytest.mark.parametrize("order", [[0, 1, 2, 3], [3, 2, 1, 0], [1, 3, 0, 2], [2, 0, 3, 1]])
@pytest.mark.parametrize("T,window", [(1, 0), (3, 16), (20, 16), (50, 40)])
def test_pages_of_four_sizes(order, T, window):
    """Every step holds two sizes; rows reach different pages of the four."""
    g = torch.Generator().manual_seed(83)
    page, d, n = 16, 128, 64
    size = torch.tensor([2.0 ** -60, 1.0, 2.0 ** 13, 2.0 ** 40])[order].repeat_interleave(page)
    k = torch.randn(2, n, 2, d, generator=g).to(BF16)
    v = (torch.randn(2, n, 2, d, generator=g) * size[None, :, None, None]).to(BF16)
    table = torch.randperm(8, generator=g).view(2, 4).int()
    cache = _cache(k, v, page, table)
    q = torch.randn(2, T, 4, d, generator=g).to(BF16).cuda()
    _check(q, cache, table, [n, n], scale=0.1, window=window)
    _check(q, cache, table, [n, n - 11], [T, max(T - 2, 0)], scale=0.1, window=window)


@pytest.mark.parametrize("size", [2.0 ** -110, 2.0 ** -95, 2.0 ** 100, 2.0 ** 124])
def test_values_of_one_extreme_size(size):
    """Scales near both ends of the range, alone and beside pages of zeros."""
    g = torch.Generator().manual_seed(89)
    page, d, n = 16, 64, 400
    k = torch.randn(1, n, 1, d, generator=g).to(BF16)
    v = (torch.randn(1, n, 1, d, generator=g).clamp(-3, 3) * size).to(BF16)
    v[:, 16:48] = 0.0
    table = torch.randperm(n // page, generator=g)[None].int()
    cache = _cache(k, v, page, table)
    q = torch.randn(1, 2, 2, d, generator=g).to(BF16).cuda()
    _check(q, cache, table, [n], scale=0.2)


def test_scales_that_are_no_powers_of_two():
    """A cache filled by its user: any positive scales, V's also 0 (the page stands for zeros)."""
    g = torch.Generator().manual_seed(97)
    pages, page, H, d = 9, 16, 2, 128
    cache = fa.kv8_cache_alloc(pages, page, H, d)
    for x in (cache.k, cache.v):
        x.copy_((torch.randn(x.shape, generator=g) * 60).clamp(-440, 440))
    cache.k_scale.copy_(0.003 * (0.5 + torch.rand(pages, H, generator=g)))
    cache.v_scale.copy_(torch.pow(10.0, 6 * torch.rand(pages, H, generator=g) - 4))
    cache.v_scale[4, 0] = 0.0
    table = torch.randperm(pages, generator=g)[None].int()
    for dtype in (BF16, F16):
        q = torch.randn(1, 3, 4, d, generator=g).to(dtype).cuda()
        _check(q, cache, table, [pages * page - 5], scale=0.1)


def test_rising_and_falling_scores_with_changing_scales():
    """The running maximum and the pages' scales move against each other from step to step."""
    g = torch.Generator().manual_seed(101)
    page, d, n = 16, 64, 1280
    for sign in (1.0, -1.0):
        for dtype in (BF16, F16):
            ramp = torch.arange(n) / n
            k = torch.zeros(1, n, 1, d)
            k[0, :, 0, 0] = sign * 40 * ramp
            e = torch.randint(-8, 9, (n // page,), generator=g).repeat_interleave(page) - sign * 30 * (ramp - 0.5) / 2
            v = torch.randn(1, n, 1, d, generator=g).clamp(-3, 3) * torch.exp2(e / 2)[None, :, None, None]
            table = torch.randperm(n // page, generator=g)[None].int()
            cache = _cache(k.to(dtype), v.to(dtype), page, table)
            q = torch.zeros(1, 2, 2, d, dtype=dtype, device="cuda")
            q[..., 0] = 1.0
            _check(q, cache, table, [n])


@pytest.mark.parametrize("Hq,T", [(1, 1), (4, 2), (8, 1), (4, 5)])
@pytest.mark.parametrize("n", [2, 16, 100, 3000])
def test_values_that_cancel(n, Hq, T):
    """Outputs far smaller than the values: a weight's rounding to f16 alone would show beside the output's."""
    g = torch.Generator().manual_seed(109)
    page, d = 16, 128
    sign = torch.ones(n) - 2 * (torch.arange(n) % 2)
    for dtype in (BF16, F16):
        k = torch.randn(1, n, 1, d, generator=g)
        v = sign[None, :, None, None] * (1 + torch.randint(0, 2, (1, n, 1, d), generator=g) / 8)
        table = torch.randperm(-(-n // page), generator=g)[None].int()
        cache = _cache(k.to(dtype), v.to(dtype), page, table)
        q = (torch.randn(1, T, Hq, d, generator=g) * 0.02).to(dtype).cuda()
        _check(q, cache, table, [n], new=[min(T, n)], scale=0.3)


@pytest.mark.parametrize("outlier", [2.0 ** 6, 2.0 ** 12, 2.0 ** 16])
def test_an_outlier_channel_of_the_queries(outlier):
    """One channel of q far above the others, where the keys are small: what the pieces of the others lose
    stays within the stated share of the largest."""
    g = torch.Generator().manual_seed(107)
    page, d, n = 32, 128, 300
    table = torch.randperm(10, generator=g)[None].int()
    for dtype in (BF16, F16):
        k = torch.randn(1, n, 2, d, generator=g)
        k[..., 77] *= 2.0 ** -9
        q = torch.randn(1, 2, 8, d, generator=g)
        q[..., 77] = outlier * 0.9 * torch.sign(q[..., 77])
        cache = _cache(k.to(dtype), torch.randn(1, n, 2, d, generator=g).to(dtype), page, table)
        _check(q.to(dtype).cuda(), cache, table, [n], scale=0.09)


@pytest.mark.parametrize("T,Hq,H,window", [(32777, 16, 16, 40), (16385, 64, 1, 33)])
def test_more_row_tiles_than_16_bits_count(T, Hq, H, window):
    """A whole prompt's queries in one call: 65556 and 65540 row tiles; rows at both ends and between."""
    g = torch.Generator().manual_seed(103)
    page, d, n = 128, 64, T + 5
    pages = -(-n // page)
    k, v = (torch.randn(1, n, H, d, generator=g).to(BF16) for _ in range(2))
    table = torch.randperm(pages, generator=g)[None].int()
    cache = _cache(k, v, page, table)
    q = torch.randn(1, T, Hq, d, generator=g).to(BF16)
    o, lse = fa.kv8_attention(q.cuda(), cache, _cu(table), _cu([n]), n, scale=0.1, window=window)
    o, lse = ref.f64(o), ref.f64(lse)
    at = table[0].long()
    k, v = ((ref.f64(c.float())[at] * ref.f64(s)[at][:, None, :, None]).flatten(0, 1)
            for c, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)))
    for t in [0, 1, 15, 16, 17, T // 3, T // 2 + 1, T - 18, T - 17, T - 2, T - 1]:
        i = n - T + t
        keys = slice(max(0, i - window + 1), i + 1)
        for hq in (0, Hq // 2, Hq - 1):
            h = hq // (Hq // H)
            kk, vv, qq = k[keys, h], v[keys, h], ref.f64(q[0, t, hq])
            s = kk @ qq * 0.1
            p = s.softmax(0)
            delta = (d + 8) * 2.0 ** -23 * 0.1 * float((kk.abs() @ qq.abs()).max()) + 64 * 2.0 ** -24 + \
                2.0 ** -21 * 0.1 * float(qq.abs().max() * kk.abs().sum(-1).max())
            want, size = p @ vv, p @ vv.abs()
            bound = 2.0 ** -8 * want.abs() * (1 + 2.0 ** -6) + size * (2 * delta + 2.0 ** -11 + 128 * 2.0 ** -23)
            assert bool(((o[0, t, hq] - want).abs() <= bound).all()), (t, hq)
            assert abs(float(lse[0, hq, t] - s.logsumexp(0))) <= delta + 2.0 ** -16 + 2.0 ** -22 * 8

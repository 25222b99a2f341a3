"""Attention over the 8-bit cache where pages hold values of very different sizes, held to each row's own
output (only the keys that the row attends to enter the bound), against float64.

With p_j the exact weights of a row, v_j its values and A = max_j |scale| sum_i |q_i k_ji|: a score is off
by (d + 8) * 2^-23 * A (fp32 sums) + 64 * 2^-24 (ex2.approx, |s - m| < 64 where a weight matters) + what the
query's e4m3 pieces leave, at most 2^-21 (bf16, two pieces) or 2^-25 (f16, three) of its largest value:
Q = |scale| * max|q| * max_j sum_i |k_ji| of it. Together delta; a weight is off by 2 delta relative (its
own, and the sum's). Its product with the page's scale s_j is rounded to f16 (half a step: 2^-11 relative,
with its residual 2^-22) in units in which the largest p_j s_j of a warp is at least 2^7, so products below 2^-14 of
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
WEIGHT = {BF16: 2.0 ** -11, F16: 2.0 ** -22}
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
            rel = 2 * delta + WEIGHT[dtype] + (n + 64) * 2.0 ** -23
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

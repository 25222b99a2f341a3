"""Norm and rotation of rows with infinities on the GPU: what is not finite reaches the values that the
definition gives it to, and no others. Which values are finite has to be equal to the formula's in float64;
the finite ones are compared as in test_gpu_norm_rope.py (80 * 2^-24 of the terms, half a step of the type).
"""
import pytest
import torch

import flashattention_backward_fa_gb300 as fa
import serve_reference as ref

pytestmark = pytest.mark.gpu

HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
INF = float("inf")

CASES = [
    # d, rot, interleaved, dtype
    (128, 0, False, torch.bfloat16),
    (128, 32, False, torch.bfloat16),
    (128, 64, True, torch.float16),
    (64, 16, False, torch.float16),
    (64, 16, True, torch.bfloat16),
    (128, 128, False, torch.bfloat16),
    (64, 64, True, torch.float32),
    (64, 32, False, torch.float32),
    (80, 20, False, torch.float32),
]


def _rotate(y, cos, sin, interleaved, back=False):
    half = cos.shape[1]
    a = torch.arange(half) * (2 if interleaved else 1)
    b = a + (1 if interleaved else half)
    c, s = cos[None, :, None], (-sin if back else sin)[None, :, None]
    out = y.clone()
    out[..., a] = y[..., a] * c - y[..., b] * s
    out[..., b] = y[..., b] * c + y[..., a] * s
    return out


def _same(got, want, size, dtype):
    got = ref.f64(got)
    assert torch.equal(got.isnan(), want.isnan())
    big = want.isinf()
    assert torch.equal(got.isinf(), big) and torch.equal(got[big], want[big])
    ok = want.isfinite()
    bound = HALF[dtype] * want.abs() + 80 * 2.0 ** -24 * size + 2.0 ** -25
    assert bool(((got - want).abs() <= bound)[ok].all())


@pytest.mark.parametrize("d,rot,interleaved,dtype", CASES)
def test_infinities_stay_with_their_values(d, rot, interleaved, dtype):
    """One infinity a row, in every place of the row in turn: among the inputs, then in the gradient."""
    g = torch.Generator().manual_seed(5)
    N, H = d, 2
    x = torch.randn(1, N, H, d, generator=g).to(dtype)
    dout = torch.randn(1, N, H, d, generator=g).to(dtype)
    w = (1 + 0.3 * torch.randn(d, generator=g)).to(dtype)
    cos, sin = fa.rope_tables(N, rot) if rot else (None, None)
    c64, s64 = (ref.f64(t) if rot else torch.zeros(N, 0, dtype=torch.float64) for t in (cos, sin))
    place = torch.arange(N)
    x_inf, dout_inf = x.clone(), dout.clone()
    x_inf[0, place, 0, place] = INF
    dout_inf[0, place, 0, place] = -INF
    eps = 1e-6
    for xs, ds in ((x_inf, dout), (x, dout_inf)):
        dev = [t.cuda() for t in (xs, ds, w)]
        out, _ = fa.qk_norm_rope_forward(dev[0], dev[0], dev[2], dev[2], cos, sin, None, eps, interleaved)
        dx, _, dw, _ = fa.qk_norm_rope_backward(dev[0], dev[0], dev[1], dev[1], dev[2], dev[2], cos, sin, None, eps,
                                                interleaved)
        x64, d64, w64 = ref.f64(xs), ref.f64(ds), ref.f64(w)
        root = (x64.square().mean(-1, keepdim=True) + eps).sqrt()
        xn = x64 / root
        y = xn * w64
        _same(out, _rotate(y, c64, s64, interleaved), y.nan_to_num(posinf=0, neginf=0).abs().amax(-1, keepdim=True) * 2,
              dtype)
        dy = _rotate(d64, c64, s64, interleaved, back=True)
        gy = dy * w64
        want = (gy - xn * (gy * xn).mean(-1, keepdim=True)) / root
        plain = gy.nan_to_num(posinf=0, neginf=0).abs().amax(-1, keepdim=True)
        size = plain * (1 + xn.nan_to_num().abs().amax(-1, keepdim=True) ** 2) / root * 2
        _same(dx, want, size, dtype)
        terms = dy * xn
        dw_want = terms.flatten(0, 2).sum(0)
        # (each weight's gradient holds its own column's infinity; in the other columns the sums are finite)
        dw_got = ref.f64(dw)
        assert torch.equal(dw_got.isfinite(), dw_want.isfinite())
        ok = dw_want.isfinite()
        size = terms.nan_to_num(posinf=0, neginf=0).abs().flatten(0, 2).sum(0)
        bound = HALF[dtype] * dw_want.abs() + (N * H + 128) * 2.0 ** -24 * 2 * size
        assert bool(((dw_got - dw_want).abs() <= bound)[ok].all())
        if xs is x and rot < d and dtype is not torch.float32:
            assert bool(ok[rot:].logical_not().all())


@pytest.mark.parametrize("interleaved", [False, True])
def test_infinities_on_their_way_into_the_cache(interleaved):
    """The fused call with infinities and a partial rotation: the two calls' results, NaN for NaN."""
    g = torch.Generator().manual_seed(7)
    B, T, Hq, H, d, page, rot = 2, 40, 4, 2, 128, 16, 32
    q, k, v = (torch.randn(B, T, h, d, generator=g).half() for h in (Hq, H, H))
    for x in (q, k):
        x[0, torch.arange(T), 0, torch.arange(T) * 3] = INF
    q, k, v = q.cuda(), k.cuda(), v.cuda()
    cos, sin = fa.rope_tables(T, rot)
    w = (1 + 0.3 * torch.randn(d, generator=g)).half().cuda()
    table = torch.arange(6, dtype=torch.int32).view(2, 3).cuda()
    lens = torch.tensor([T, T], dtype=torch.int32).cuda()
    one, two = (fa.kv8_cache_alloc(6, page, H, d) for _ in range(2))
    qo = fa.kv8_norm_rope_append(one, q, k, v, w, w, cos, sin, table, lens, interleaved=interleaved)
    q2, k2 = fa.qk_norm_rope_forward(q, k, w, w, cos, sin, interleaved=interleaved)
    fa.kv8_append(two, k2, v, table, lens)
    assert torch.equal(qo.isnan(), q2.isnan()) and torch.equal(qo.nan_to_num(), q2.nan_to_num())
    assert torch.equal(one.k.view(torch.uint8), two.k.view(torch.uint8))
    assert torch.equal(one.k_scale, two.k_scale)
    # one NaN a row where the infinity is not rotated, a pair of them where it is
    assert int(qo[0, :, 0].isnan().sum()) == T + sum(3 * t < rot for t in range(T))

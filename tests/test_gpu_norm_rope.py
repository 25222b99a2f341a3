"""Per-head norm and rotation on the GPU against the plain float64 form.

Tolerances. Outputs are rounded once, so each is off by at most half a step of its type relative to
its size, plus what fp32 arithmetic leaves: the sum of squares of d <= 128 values in any order is off
by at most 128 * 2^-24 relative, its root by half of that, and each of the about six further fp32
operations of an output by 2^-24 of the terms, whose size is at most |y_a| + |y_b|, the pair's. So
|error| <= half_step * |out| + 80 * 2^-24 * (|y_a| + |y_b|). For dx the terms are r |g| and
r |xn| mean|g xn|; for dw, a sum of `rows` products, sqrt-growth is not relied on: the bound is
(rows + 128) * 2^-24 * sum |dy xn|.
"""
import pytest
import torch

import flashattention_backward_fa_gb300 as fa
import serve_reference as ref

pytestmark = pytest.mark.gpu

EPS32 = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}  # half a step, upper bound
TINY = {torch.float32: 2.0 ** -140, torch.bfloat16: 2.0 ** -130, torch.float16: 2.0 ** -25}  # half a subnormal step


def _make(shape, dtype, g, device="cuda"):
    return (torch.randn(shape, generator=g) * (0.2 + 2 * torch.rand(shape[-1], generator=g))).to(dtype).to(device)


def _reference(q, k, wq, wk, cos, sin, pos, eps, il, dq=None, dk=None):
    """Outputs, gradients by float64 autograd of the plain form, and the scales of the terms."""
    B, N = q.shape[:2]
    p = torch.arange(N).expand(B, N) if pos is None else pos.cpu().long().expand(B, N)
    if cos is not None:
        p = p.clamp(0, cos.shape[0] - 1)
    out = []
    for x, w, d in ((q, wq, dq), (k, wk, dk)):
        x64 = ref.f64(x).requires_grad_()
        w64 = (torch.ones(x.shape[-1], dtype=torch.float64) if w is None else ref.f64(w)).requires_grad_()
        y = ref.norm_rope(x64, w64, ref.f64(cos), ref.f64(sin), p, eps, il)
        pair = (ref.norm_rope(x64, w64, None, None, p, eps, il).abs()).amax(-1, keepdim=True) * 2  # >= |y_a| + |y_b|
        if d is None:
            out.append((y.detach(), pair.detach()))
        else:
            d64 = ref.f64(d)
            dx, dw = torch.autograd.grad(y, (x64, w64), d64)
            x64 = x64.detach()
            r = 1 / (x64.square().mean(-1, keepdim=True) + eps).sqrt()
            g = (d64.abs().amax(-1, keepdim=True) * 2) * w64.detach().abs().amax()
            size = r * g * (1 + (x64 * r).abs().amax(-1, keepdim=True) * (x64 * r).abs().mean(-1, keepdim=True))
            rows = x64.flatten(0, 2)
            wsum = (2 * d64.abs().amax(-1).flatten()[:, None] * (rows * r.flatten()[:, None]).abs()).sum(0)
            out.append((y.detach(), pair.detach(), dx, size, dw, wsum, rows.shape[0]))
    return out


def _near(got, want, size, dtype):
    err = (ref.f64(got) - want).abs()
    bound = HALF[dtype] * want.abs() + 80 * EPS32 * size + TINY[dtype]
    bad = ~(err <= bound)
    assert not bad.any(), (int(bad.sum()), float((err / bound).max()))


CASES = [
    # B, N, Hq, Hk, d, rot, interleaved, dtype, weights, positions
    (1, 1, 1, 1, 64, 64, False, torch.bfloat16, "own", None),
    (2, 37, 5, 3, 128, 128, False, torch.bfloat16, "own", None),
    (2, 37, 5, 3, 128, 128, True, torch.float16, "f32", "rows"),
    (3, 50, 8, 2, 64, 32, False, torch.float16, "own", "batch"),
    (3, 50, 8, 2, 64, 16, True, torch.bfloat16, None, "batch"),
    (1, 65, 7, 7, 128, 96, False, torch.bfloat16, "f32", None),
    (1, 9, 2, 1, 128, 0, False, torch.bfloat16, "own", None),
    (1, 128, 1, 1, 64, 64, False, torch.float32, "own", None),
    (2, 33, 3, 2, 128, 128, True, torch.float32, "own", "batch"),
    (2, 19, 3, 2, 80, 20, False, torch.float32, "own", "batch"),
    (2, 19, 3, 2, 37, 36, True, torch.float32, None, None),
    (1, 5, 2, 2, 1, 0, False, torch.float32, "own", None),
]


def _inputs(case, seed):
    B, N, Hq, Hk, d, rot, il, dtype, weights, positions = case
    g = torch.Generator().manual_seed(seed)
    q, k = _make((B, N, Hq, d), dtype, g), _make((B, N, Hk, d), dtype, g)
    wd = {"own": dtype, "f32": torch.float32, None: None}[weights]
    wq, wk = (None if wd is None else (1 + 0.3 * torch.randn(d, generator=g)).to(wd).cuda() for _ in range(2))
    cos, sin = fa.rope_tables(200, rot) if rot else (None, None)
    pos = None
    if positions == "rows":
        pos = torch.randint(0, 200, (N,), generator=g, dtype=torch.int32).cuda()
    elif positions == "batch":  # some out of the tables' range: clamped
        pos = torch.randint(-3, 203, (B, N), generator=g, dtype=torch.int32).cuda()
    return q, k, wq, wk, cos, sin, pos


@pytest.mark.parametrize("case", CASES)
def test_forward_and_backward_against_float64(case):
    dtype, il, eps = case[7], case[6], 1e-5
    q, k, wq, wk, cos, sin, pos = _inputs(case, 11)
    g = torch.Generator().manual_seed(12)
    dq, dk = _make(q.shape, dtype, g), _make(k.shape, dtype, g)
    want = _reference(q, k, wq, wk, cos, sin, pos, eps, il, dq, dk)
    out = fa.qk_norm_rope_forward(q, k, wq, wk, cos, sin, pos, eps, il)
    grads = fa.qk_norm_rope_backward(q, k, dq, dk, wq, wk, cos, sin, pos, eps, il)
    for i, w in enumerate(want):
        _near(out[i], w[0], w[1], dtype)
        _near(grads[i], w[2], w[3], dtype)
        if wq is None:
            assert grads[2 + i] is None
        else:
            wt = grads[2 + i].dtype
            err = (ref.f64(grads[2 + i]) - w[4]).abs()
            assert torch.all(err <= HALF[wt] * w[4].abs() + (w[6] + 128) * EPS32 * w[5] + TINY[wt])
    again = fa.qk_norm_rope_backward(q, k, dq, dk, wq, wk, cos, sin, pos, eps, il)
    for a, b in zip(grads, again):
        assert a is b is None or torch.equal(a, b)
    assert fa.fa_get_device_status() == 0


@pytest.mark.parametrize("dtype,d", [(torch.bfloat16, 128), (torch.float32, 64), (torch.float32, 50)])
def test_strides_and_guard_bands(dtype, d):
    """Inputs and outputs as slices of larger buffers with rows apart: the values of dense ones, and
    nothing outside the outputs changes."""
    B, N, Hq, Hk = 2, 21, 3, 2
    unit = 8 if dtype != torch.float32 else (4 if d == 64 else 3)
    g = torch.Generator().manual_seed(5)
    cos, sin = fa.rope_tables(N, 16)
    dense = [_make((B, N, H, d), dtype, g) for H in (Hq, Hk, Hq, Hk)]
    w = _make((d,), dtype, g)

    def strided(t, fill):
        B_, N_, H, _ = t.shape
        sh, off = d + unit, 16
        sn = H * sh + 2 * unit
        sb = N_ * sn + 3 * unit
        buf = torch.full((off + B_ * sb + 64,), fill, dtype=dtype, device="cuda")
        view = buf.as_strided(t.shape, (sb, sn, sh, 1), off)
        return buf, view

    ins = []
    for t in dense:
        _, v = strided(t, float("nan"))
        v.copy_(t)
        ins.append(v)
    want = fa.qk_norm_rope_forward(dense[0], dense[1], w, w, cos, sin)
    wantg = fa.qk_norm_rope_backward(*dense, w, w, cos, sin)
    bufs = [strided(t, 7.0) for t in (dense[0], dense[1], dense[0], dense[1])]
    fa.fa_qk_norm_rope_fwd(ins[0], ins[1], bufs[0][1], bufs[1][1], w, w, cos, sin)
    ws = torch.empty(fa.fa_qk_norm_rope_bwd_workspace_size(d) + 256, dtype=torch.uint8, device="cuda").fill_(165)
    dw = [torch.empty_like(w) for _ in range(2)]
    fa.fa_qk_norm_rope_bwd(*ins, bufs[2][1], bufs[3][1], *dw, ws[:-256], w, w, cos, sin)
    assert torch.equal(dw[0], wantg[2]) and torch.equal(dw[1], wantg[3])
    for (buf, view), t in zip(bufs, (*want, *wantg[:2])):
        assert torch.equal(view, t)
        view.fill_(7.0)
        assert bool((buf == 7.0).all())
    assert bool((ws[-256:] == 165).all())


def test_finite_differences():
    """The gradients against central differences of the float32 forward: sum(out o R) has curvature of
    order one, so a step of 2^-7 is off by about 2^-14 relative, and fp32 rounding of the sum by less."""
    g = torch.Generator().manual_seed(8)
    B, N, Hq, Hk, d = 1, 3, 2, 1, 64
    q, k = (torch.randn((B, N, H, d), generator=g).cuda() for H in (Hq, Hk))
    w = [(1 + 0.3 * torch.randn(d, generator=g)).cuda() for _ in range(2)]
    rq, rk = (torch.randn(t.shape, generator=g).cuda() for t in (q, k))
    cos, sin = fa.rope_tables(N, 32)

    def loss(*a):
        o = fa.qk_norm_rope_forward(a[0], a[1], a[2], a[3], cos, sin)
        return float((o[0].double() * rq).sum() + (o[1].double() * rk).sum())

    grads = fa.qk_norm_rope_backward(q, k, rq, rk, *w, cos, sin)
    args = [q, k, *w]
    h = 2.0 ** -7
    for i, gr in enumerate(grads):
        for _ in range(3):
            u = torch.randn(args[i].shape, generator=g).cuda()
            u /= u.norm()
            hi, lo = (args[:i] + [args[i] + s * h * u] + args[i + 1:] for s in (1, -1))
            num = (loss(*hi) - loss(*lo)) / (2 * h)
            assert abs(num - float((gr.double() * u).sum())) <= 2.0 ** -10 * float(gr.double().norm())


def test_extreme_rows():
    """Zero rows, rows of the smallest and of large values, and a NaN that stays in its row."""
    d = 128
    q = torch.zeros(1, 4, 2, d, dtype=torch.bfloat16, device="cuda")
    q[0, 1] = 1e15
    q[0, 2] = 1e-30
    q[0, 3, 0, 5] = float("nan")
    q[0, 3, 1] = 1.0
    cos, sin = fa.rope_tables(4, d)
    o, _ = fa.qk_norm_rope_forward(q, q, None, None, cos, sin, eps=1e-6)
    assert bool((o[0, 0] == 0).all()) and bool(o[0, 3, 0].isnan().all())
    want = ref.norm_rope(ref.f64(q), None, ref.f64(cos), ref.f64(sin), torch.arange(4)[None], 1e-6, False)
    err = (ref.f64(o) - want).abs()
    for n, h in ((1, 0), (2, 0), (3, 1)):
        assert torch.all(err[0, n, h] <= 2.0 ** -8 * want[0, n, h].abs() + 160 * EPS32 * want[0, n, h].abs().max() + 2.0 ** -130)


def test_autograd_with_attention_and_broadcast_gradients():
    """qk_norm_rope_func feeds flash_attn_func; gradients of all leaves equal the chained calls', also
    from a gradient that is a broadcast (strides of zero), and leave no trace in the inputs."""
    B, N, H, d = 2, 70, 3, 64
    g = torch.Generator().manual_seed(21)
    q, k, v, do = (_make((B, N, H, d), torch.bfloat16, g) for _ in range(4))
    w = [(1 + 0.2 * torch.randn(d, generator=g)).to(torch.bfloat16).cuda() for _ in range(2)]
    cos, sin = fa.rope_tables(N, d)
    leaves = [t.clone().requires_grad_() for t in (q, k, v, *w)]
    qr, kr = fa.qk_norm_rope_func(leaves[0], leaves[1], leaves[3], leaves[4], cos, sin)
    o = fa.flash_attn_func(qr, kr, leaves[2], causal=True)
    grads = torch.autograd.grad(o, leaves, do)
    q2, k2 = fa.qk_norm_rope_forward(q, k, *w, cos, sin)
    o2, lse = fa.attention_forward(q2, k2, v, causal=True)
    dq2, dk2, dv2 = fa.attention_backward(q2, k2, v, o2, do, lse, causal=True)
    want = fa.qk_norm_rope_backward(q, k, dq2, dk2, *w, cos, sin)
    assert torch.equal(o, o2)
    for a, b in zip(grads, (want[0], want[1], dv2, want[2], want[3])):
        assert torch.equal(a, b)
    qr, kr = fa.qk_norm_rope_func(leaves[0], leaves[1], leaves[3], leaves[4], cos, sin)
    got = torch.autograd.grad(qr.sum() + 0 * kr.sum(), (leaves[0], leaves[3]))
    ones = torch.ones_like(q)
    want = fa.qk_norm_rope_backward(q, k, ones, torch.zeros_like(k), *w, cos, sin)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[2])


def test_side_stream_graph_and_two_graphs():
    """On another stream and captured: replays on new inputs give the eager calls' bits, two graphs
    replayed in turn do not disturb each other."""
    g = torch.Generator().manual_seed(31)
    cos, sin = fa.rope_tables(64, 128)
    made = []
    for H in (3, 2):
        x = [_make((2, 40, h, 128), torch.bfloat16, g) for h in (H, 1, H, 1)]
        w = _make((128,), torch.bfloat16, g)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            fa.qk_norm_rope_backward(*x, w, w, cos, sin)
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = (*fa.qk_norm_rope_forward(x[0], x[1], w, w, cos, sin),
                   *fa.qk_norm_rope_backward(*x, w, w, cos, sin))
        made.append((x, w, graph, out))
    for x, w, graph, out in made:
        for t in x:
            t.copy_(_make(t.shape, t.dtype, g))
    for _ in range(2):
        for x, w, graph, out in made:
            graph.replay()
    torch.cuda.synchronize()
    for x, w, graph, out in made:
        want = (*fa.qk_norm_rope_forward(x[0], x[1], w, w, cos, sin), *fa.qk_norm_rope_backward(*x, w, w, cos, sin))
        for a, b in zip(out, want):
            assert torch.equal(a, b)


def test_one_weight_alone():
    """A weight on one side only: the other side is normed with ones and has no weight gradient."""
    g = torch.Generator().manual_seed(41)
    x = [_make((2, 9, h, 64), torch.float16, g) for h in (3, 2, 3, 2)]
    w = (1 + 0.3 * torch.randn(64, generator=g)).half().cuda()
    ones = torch.ones_like(w)
    cos, sin = fa.rope_tables(9, 32)
    for a, b in ((w, None), (None, w)):
        full = (w, ones) if b is None else (ones, w)
        got = fa.qk_norm_rope_forward(x[0], x[1], a, b, cos, sin)
        for u, v in zip(got, fa.qk_norm_rope_forward(x[0], x[1], *full, cos, sin)):
            assert torch.equal(u, v)
        got = fa.qk_norm_rope_backward(*x, a, b, cos, sin)
        want = fa.qk_norm_rope_backward(*x, *full, cos, sin)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert (got[2] is None) == (a is None) and (got[3] is None) == (b is None)
        assert torch.equal(got[2] if b is None else got[3], want[2] if b is None else want[3])


def test_autograd_captured_into_a_graph():
    """Forward and backward of qk_norm_rope_func captured with leaves of their own: a replay on new values
    gives the eager gradients."""
    g = torch.Generator().manual_seed(43)
    q, k = (_make((1, 30, h, 128), torch.bfloat16, g).requires_grad_() for h in (4, 2))
    w = [(1 + 0.2 * torch.randn(128, generator=g)).to(torch.bfloat16).cuda().requires_grad_() for _ in range(2)]
    dq, dk = _make((1, 30, 4, 128), torch.bfloat16, g), _make((1, 30, 2, 128), torch.bfloat16, g)
    cos, sin = fa.rope_tables(30, 128)

    def step():
        out = fa.qk_norm_rope_func(q, k, *w, cos, sin)
        return torch.autograd.grad(out, (q, k, *w), (dq, dk))

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    with torch.no_grad():
        q.copy_(_make(q.shape, q.dtype, g))
        w[0].mul_(1.5)
    graph.replay()
    for a, b in zip(out, step()):
        assert torch.equal(a, b)


def test_many_rows_a_group():
    """Enough rows that every row group takes several, with heads that do not divide the span: against the
    same rows in small calls."""
    g = torch.Generator().manual_seed(47)
    B, N, Hq, Hk, d = 3, 2100, 23, 5, 64
    q, k, dq, dk = (_make((B, N, h, d), torch.bfloat16, g) for h in (Hq, Hk, Hq, Hk))
    w = [(1 + 0.2 * torch.randn(d, generator=g)).cuda() for _ in range(2)]
    cos, sin = fa.rope_tables(N, d)
    out = fa.qk_norm_rope_forward(q, k, *w, cos, sin)
    grads = fa.qk_norm_rope_backward(q, k, dq, dk, *w, cos, sin)
    sums = [torch.zeros(d, dtype=torch.float64, device="cuda") for _ in range(2)]
    for b in range(B):
        for n in range(0, N, 700):
            at = (slice(b, b + 1), slice(n, n + 700))
            pos = torch.arange(n, n + 700, dtype=torch.int32, device="cuda")
            o = fa.qk_norm_rope_forward(q[at], k[at], *w, cos, sin, pos)
            gr = fa.qk_norm_rope_backward(q[at], k[at], dq[at], dk[at], *w, cos, sin, pos)
            for x, y in zip((*o, *gr[:2]), (*out, *grads[:2])):
                assert torch.equal(x, y[at])
            for s, y in zip(sums, gr[2:]):
                s += y.double()
    for s, y, x, dd in zip(sums, grads[2:], (q, k), (dq, dk)):
        # two orders of the same fp32 sums of `rows` products of up to about 2 max|dout| max|xn|
        rows = x[..., 0].numel()
        assert torch.all((s - y.double()).abs() <= rows * EPS32 * (2 * dd.float().abs().amax() * 2 * rows ** 0.5).double())


def test_large_offsets():
    """Rows past 2^31 elements of one buffer (a stride that reaches there) are read and written in place."""
    d, far = 128, (1 << 31) + 128 * 8
    buf = torch.empty(far + 4 * d, dtype=torch.bfloat16, device="cuda")
    q = buf.as_strided((2, 2, 1, d), (far, d, d, 1))
    g = torch.Generator().manual_seed(2)
    q.copy_(_make((2, 2, 1, d), torch.bfloat16, g))
    out = torch.empty_like(buf).as_strided((2, 2, 1, d), (far, d, d, 1))
    cos, sin = fa.rope_tables(2, d)
    kk = q.contiguous()
    ko = torch.empty_like(kk)
    fa.fa_qk_norm_rope_fwd(q, kk, out, ko, None, None, cos, sin)
    assert torch.equal(out, ko)


def test_refusals_on_the_gpu():
    q = torch.randn(1, 4, 2, 64, device="cuda").to(torch.bfloat16)
    cos, sin = fa.rope_tables(8, 64)
    with pytest.raises(ValueError):
        fa.qk_norm_rope_forward(q, q.float(), None, None, cos, sin)          # another dtype
    with pytest.raises(ValueError):
        fa.qk_norm_rope_forward(q, q[:, :2], None, None, cos, sin)           # another length
    with pytest.raises(ValueError):
        fa.qk_norm_rope_forward(q, q, torch.ones(32, device="cuda"), None, cos, sin)
    with pytest.raises(ValueError):
        fa.qk_norm_rope_forward(q, q, None, None, cos, sin.cpu())
    with pytest.raises(ValueError):
        fa.qk_norm_rope_forward(q, q, None, None, cos, None)
    with pytest.raises(ValueError):
        fa.qk_norm_rope_forward(q, q, None, None, cos, sin, positions=torch.arange(4, device="cuda"))  # int64
    with pytest.raises(ValueError):
        fa.qk_norm_rope_forward(q, q, None, None, *fa.rope_tables(8, 128))   # more than the head holds
    with pytest.raises(fa.FaError):
        fa.qk_norm_rope_forward(q, q, None, None, *fa.rope_tables(8, 8))     # 16-bit: multiples of 16
    with pytest.raises(fa.FaError):
        fa.qk_norm_rope_forward(q[..., :32], q[..., :32], None, None, *fa.rope_tables(8, 32))  # d = 32
    host = torch.zeros(64, pin_memory=True)
    lib = fa.load_library()
    st = fa.FaStrides(512, 128, 64)
    rc = lib.fa_qk_norm_rope_fwd(q.data_ptr(), q.data_ptr(), q.data_ptr(), q.data_ptr(), host.data_ptr(), None,
                                 cos.data_ptr(), sin.data_ptr(), None, 0, 1, 4, 2, 2, 64, 64, 0, 8, st, st, st, st,
                                 fa.FA_BF16, fa.FA_F32, 1e-6, None)
    assert rc == -1  # a host pointer is refused, nothing is launched

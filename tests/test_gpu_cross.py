"""Cross attention (fa_cross_fwd, fa_cross_bwd) against its definition in float64, with the bounds of
cross_reference."""
import math

import pytest
import torch

import flashattention_backward_fa_gb300 as fa
from cross_reference import Reference

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def make(B, Nq, Nk, Hq, Hk, d, dtype, seed=0, sharp=1.0):
    g = torch.Generator().manual_seed(seed)
    r = lambda n, h: torch.randn((B, n, h, d), generator=g)  # noqa: E731
    q, k, v, do = (r(Nq, Hq) * sharp).to(dtype), r(Nk, Hk).to(dtype), r(Nk, Hk).to(dtype), r(Nq, Hq).to(dtype)
    return tuple(t.cuda() for t in (q, k, v, do))


def ints(x):
    return None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda")


def run(q, k, v, do, q_lens=None, k_lens=None, scale=None, **kw):
    ql, kl = ints(q_lens), ints(k_lens)
    o, lse = fa.cross_attention_forward(q, k, v, ql, kl, scale)
    grads = fa.cross_attention_backward(q, k, v, o, do, lse, ql, kl, scale)
    ref = Reference(q, k, v, ql, kl, scale, do)
    ref.check_forward(o, lse)
    ref.check_backward(*grads)
    assert fa.fa_get_device_status() == 0
    return (o, lse) + grads


# B, Nq, Nk, Hq, Hk, d
SIZES = [
    (1, 1, 1, 1, 1, 64), (1, 1, 2, 1, 1, 128), (2, 1, 77, 4, 2, 64), (3, 2, 129, 3, 1, 128), (1, 7, 1000, 8, 1, 64),
    (2, 5, 300, 12, 4, 128), (1, 33, 65, 2, 2, 64), (2, 64, 64, 2, 1, 128), (1, 65, 128, 3, 1, 64),
    (1, 127, 127, 2, 2, 128), (1, 128, 256, 2, 1, 128), (2, 129, 255, 2, 2, 64), (1, 257, 383, 4, 2, 64),
    (1, 300, 513, 2, 1, 128), (1, 16, 2100, 2, 2, 64), (1, 1030, 40, 2, 1, 64), (5, 40, 3, 2, 2, 64),
]


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("size", SIZES)
def test_sizes(size, dtype):
    run(*make(*size, dtype))


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("size,q_lens,k_lens", [
    ((8, 520, 300, 16, 8, 64), None, None),
    ((9, 300, 400, 16, 4, 128), [300, 0, 1, 129, 200, 300, 64, 257, 300], [400, 400, 129, 0, 1, 256, 300, 128, 399]),
    ((40, 70, 130, 8, 8, 64), None, [(37 * b) % 131 for b in range(40)]),
    # one query step a key tile, several tiles a block: accumulators change hands at every step
    ((2, 40, 4000, 16, 16, 64), None, None), ((3, 33, 3000, 16, 8, 128), [33, 1, 20], [3000, 2999, 1300]),
    ((1, 70, 2600, 32, 32, 128), None, None), ((40, 130, 100, 8, 4, 64), [(29 * b) % 131 for b in range(40)], None),
])
def test_many_units_a_block(size, q_lens, k_lens, dtype):
    """More units of work than the GPU has places, some of them empty, so that blocks go from one to the next. The
    same bits again and again."""
    q, k, v, do = make(*size, dtype)
    first = run(q, k, v, do, q_lens, k_lens)
    ql, kl = ints(q_lens), ints(k_lens)
    for _ in range(20):
        o, lse = fa.cross_attention_forward(q, k, v, ql, kl)
        for a, b in zip(first, (o, lse) + fa.cross_attention_backward(q, k, v, o, do, lse, ql, kl)):
            assert torch.equal(a, b)
    assert fa.fa_get_device_status() == 0


FEW = [
    # few rows a key head: one block, clusters of two to eight, shares through the workspace, several row tiles
    ((1, 1, 5000, 2, 1, 128), None), ((1, 1, 9001, 1, 1, 64), None), ((2, 3, 4111, 4, 2, 64), [4111, 17]),
    ((3, 1, 700, 32, 8, 128), [700, 1, 0]), ((40, 1, 333, 16, 8, 64), [(53 * b) % 334 for b in range(40)]),
    ((2, 17, 1500, 2, 2, 64), None), ((1, 31, 900, 4, 2, 128), None), ((1, 64, 600, 3, 3, 64), [599]),
    ((1, 1, 40, 64, 1, 128), None), ((100, 1, 60, 8, 8, 64), None), ((1, 2, 6000, 8, 1, 128), [5999]),
    ((1, 5, 5000, 3, 1, 64), [129]),
    # several rounds of long blocks, longest sequences first; equal lengths, none
    ((70, 1, 2100, 8, 8, 128), [(1000 + 700 * b) % 2101 for b in range(70)]),
    ((128, 1, 2048, 4, 4, 64), [2048, 0, 5] * 42 + [7, 7]),
]


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("size,k_lens", FEW)
def test_few_rows(size, k_lens, dtype):
    """Forward of single and few new tokens, with the bounds; what lies behind the lengths reaches nothing."""
    q, k, v, _ = make(*size, dtype)
    o, lse = fa.cross_attention_forward(q, k, v, k_lens=ints(k_lens))
    Reference(q, k, v, None, ints(k_lens)).check_forward(o, lse)
    if k_lens is not None:
        for b, n in enumerate(k_lens):
            k[b, n:], v[b, n:] = math.nan, math.inf
        o2, lse2 = fa.cross_attention_forward(q, k, v, k_lens=ints(k_lens))
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
    assert fa.fa_get_device_status() == 0


@pytest.mark.parametrize("size, k_lens", [
    ((1, 100, 3000, 2, 2, 64), None),
    ((3, 100, 2500, 2, 2, 128), [2500, 0, 129]),
    ((7, 31, 2049, 8, 2, 64), [1, 128, 129, 256, 257, 1000, 2049]),
    ((1, 64, 9000, 4, 2, 128), [8897]),
    ((44, 70, 1300, 4, 4, 64), [0, 1, 100, 128, 129, 300, 513, 1024, 1025, 1200, 1300] * 4),
])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_one_row_tile(size, k_lens, dtype):
    """Up to 128 query rows a key head and keys enough to share out: even and odd key blocks, some without a block."""
    q, k, v, do = make(*size, dtype)
    lens = None if k_lens is None else ints(k_lens)
    o, lse = fa.cross_attention_forward(q, k, v, k_lens=lens)
    Reference(q, k, v, None, lens).check_forward(o, lse)


@pytest.mark.parametrize("d", [1, 17, 63, 96, 128])
def test_fp32_head_dimensions(d):
    run(*make(2, 70, 45, 4, 2, d, F32))


LENS = [
    # B, Nq, Nk, Hq, Hk, d, q_lens, k_lens
    (4, 70, 90, 2, 1, 64, [0, 1, 70, 69], [90, 0, 1, 64]),
    (3, 200, 300, 4, 2, 128, [200, 129, 64], [257, 300, 128]),
    (3, 1, 500, 8, 2, 64, None, [500, 3, 0]),
    (3, 3, 1000, 8, 1, 128, [3, 0, 2], [999, 1000, 17]),
    (2, 513, 80, 2, 2, 64, [512, 130], [80, 33]),
    (2, 10, 20, 2, 2, 64, [-5, 99], [1 << 30, -1]),  # clamped into the tensors
    (2, 260, 140, 6, 2, 128, [255, 260], [0, 0]),
]


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("case", LENS)
@pytest.mark.parametrize("fill", [math.nan, math.inf])
def test_padding_reaches_nothing(case, dtype, fill):
    """Lengths of each sequence; what lies behind them is NaN or infinite."""
    *size, q_lens, k_lens = case
    q, k, v, do = make(*size, dtype)
    B, Nq, Nk = size[:3]
    clean = run(q, k, v, do, q_lens, k_lens)
    for b in range(B):
        n = Nq if q_lens is None else min(max(q_lens[b], 0), Nq)
        m = Nk if k_lens is None else min(max(k_lens[b], 0), Nk)
        q[b, n:], do[b, n:], k[b, m:], v[b, m:] = fill, fill, fill, -fill
    o, lse = fa.cross_attention_forward(q, k, v, ints(q_lens), ints(k_lens))
    grads = fa.cross_attention_backward(q, k, v, o, do, lse, ints(q_lens), ints(k_lens))
    for name, a, b in zip(("o", "lse", "dq", "dk", "dv"), clean, (o, lse) + grads):
        assert torch.equal(a, b), name


def test_nan_of_one_head_or_sequence_stays_there():
    q, k, v, do = make(3, 9, 150, 6, 2, 64, BF16)
    clean = run(q, k, v, do)
    q[1, 4, 2], k[2, 7, 1], v[0, 3, 0], do[1, 0, 5] = (math.nan,) * 4
    o, lse = fa.cross_attention_forward(q, k, v)
    grads = fa.cross_attention_backward(q, k, v, o, do, lse)
    # (sequence, query heads) whose rows may differ: the key heads' groups of three
    hit_rows = {(1, 2), (2, 3), (2, 4), (2, 5), (0, 0), (0, 1), (0, 2), (1, 5)}
    hit_keys = {(1, 0), (2, 1), (0, 0), (1, 1)}
    for name, a, b in zip(("o", "lse", "dq", "dk", "dv"), clean, (o, lse) + grads):
        a, b = (a.transpose(1, 2), b.transpose(1, 2)) if name != "lse" else (a, b)
        for s in range(a.shape[0]):
            for h in range(a.shape[1]):
                if (s, h) not in (hit_keys if name in ("dk", "dv") else hit_rows):
                    assert torch.equal(a[s, h], b[s, h]), (name, s, h)
    assert o[1, 4, 2].isnan().all() and o[2, :, 3:].isnan().all() and o[0, :, :3].isnan().all()
    assert not o[1, :4, 2].isnan().any()


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_sharp_and_large_scores(dtype):
    run(*make(2, 130, 200, 2, 1, 64, dtype, sharp=8.0))
    run(*make(1, 3, 400, 4, 2, 128, dtype, sharp=20.0))
    run(*make(1, 150, 70, 2, 2, 64, dtype), scale=3.0)
    run(*make(1, 150, 70, 2, 2, 64, dtype), scale=1e-4)


def test_rising_scores_move_the_reference():
    """Keys in the order of rising scores: the running maximum moves at every step."""
    q, k, v, do = make(1, 140, 900, 2, 1, 64, BF16)
    k[0, :, 0] = q[0, :, 0].float().mean(0) * torch.linspace(0, 6, 900, device="cuda")[:, None]
    q[0] = q[0, :, :1].float().mean(0, keepdim=True)[:, :1].expand(140, 2, 64).to(BF16) + q[0] * 0.25
    run(q, k, v, do)


def test_scores_of_minus_infinity():
    """A query whose scores are all -inf has no keys; a key at -inf has no weight."""
    q, k, v, _ = make(1, 4, 5, 1, 1, 64, F32)
    q.abs_()
    k[0, 2] = -math.inf
    o, lse = fa.cross_attention_forward(q, k, v)
    keep = [0, 1, 3, 4]
    ref = Reference(q, k[:, keep].contiguous(), v[:, keep].contiguous())
    ref.check_forward(o, lse)
    k[0] = -math.inf
    o, lse = fa.cross_attention_forward(q, k, v)
    assert (o == 0).all() and (lse == -math.inf).all()


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_strides(dtype):
    """q a slice of a packed projection, k and v of another, heads before positions, a gradient transposed."""
    B, Nq, Nk, H, d = 2, 150, 90, 3, 64
    g = torch.Generator(device="cuda").manual_seed(1)
    r = lambda *s: torch.randn(s, generator=g, device="cuda").to(dtype)  # noqa: E731
    q = r(B, Nq, 3 * H, d)[:, :, H:2 * H]
    kv = r(B, H, Nk, 2 * d)
    k, v = kv[..., :d].transpose(1, 2), kv[..., d:].transpose(1, 2)
    do = r(H, B, Nq, d).permute(1, 2, 0, 3)
    assert not any(t.is_contiguous() for t in (q, k, v, do))
    out = run(q, k, v, do)
    same = run(*(t.contiguous() for t in (q, k, v, do)))
    for a, b in zip(out, same):
        assert torch.equal(a, b)


@pytest.mark.parametrize("Nq", [1, 520])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_offsets_past_32_bits(Nq, dtype):
    """Rows 2^22 values apart, all tensors in one buffer: places beyond 2^31 values have the bits of packed tensors."""
    Nk, H, d, apart = 520, 2, 64, 1 << 22
    packed = make(1, Nq, Nk, H, H, d, dtype)
    want = run(*packed)
    room = torch.empty(519 * apart + 8 * H * d, dtype=dtype, device="cuda")
    at = lambda i, N: room.as_strided((1, N, H, d), (Nk * apart, apart, d, 1), i * H * d)  # noqa: E731
    q, k, v, do, o, dq, dk, dv = (at(i, N) for i, N in enumerate((Nq, Nk, Nk, Nq, Nq, Nq, Nk, Nk)))
    for t, x in zip((q, k, v, do), packed):
        t.copy_(x)
    lse = torch.empty((1, H, Nq), device="cuda")
    size = (1, Nq, Nk, H, H, d, dtype)
    ws = [torch.empty(max(n(*size), 1), dtype=torch.uint8, device="cuda")
          for n in (fa.fa_cross_fwd_workspace_size, fa.fa_cross_bwd_workspace_size)]
    fa.fa_cross_fwd(q, k, v, o, lse, ws[0])
    fa.fa_cross_bwd(q, k, v, o, do, lse, dq, dk, dv, ws[1])
    for a, b in zip(want, (o, lse, dq, dk, dv)):
        assert torch.equal(a, b)


def test_outputs_of_the_caller():
    """The C entry points fill what they are given, with its strides, and nothing beside it."""
    q, k, v, do = make(2, 100, 70, 4, 2, 64, BF16)
    want = run(q, k, v, do)
    ws = torch.full((max(1, fa.fa_cross_fwd_workspace_size(2, 100, 70, 4, 2, 64, BF16)),), 255, dtype=torch.uint8,
                    device="cuda")
    wb = torch.full((fa.fa_cross_bwd_workspace_size(2, 100, 70, 4, 2, 64, BF16),), 255, dtype=torch.uint8,
                    device="cuda")
    wide = [torch.full((2, t.shape[1] + 2, t.shape[2] + 1, 64 + 8), 7.0, dtype=BF16, device="cuda")
            for t in (q, q, k, k)]
    o, dq, dk, dv = (w[:, 1:-1, :-1, :64] for w in wide)
    lse = torch.empty((2, 4, 100), device="cuda")
    fa.fa_cross_fwd(q, k, v, o, lse, ws)
    fa.fa_cross_bwd(q, k, v, o, do, lse, dq, dk, dv, wb)
    for a, b in zip(want, (o, lse, dq, dk, dv)):
        assert torch.equal(a, b)
    for w in wide:
        w[:, 1:-1, :-1, :64] = 7.0
        assert (w == 7.0).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_autograd(dtype):
    q, k, v, do = make(2, 70, 50, 4, 2, 64, dtype)
    kl = ints([50, 13])
    leaves = [t.clone().requires_grad_() for t in (q, k, v)]
    o = fa.cross_attn_func(*leaves, k_lens=kl)
    o.backward(do)
    ref = Reference(q, k, v, None, kl, None, do)
    ref.check_backward(*(t.grad for t in leaves))
    # states shared by the whole batch, and a gradient of one value
    k1, v1 = (t[:1].clone().requires_grad_() for t in (k, v))
    o = fa.cross_attn_func(q, k1.expand(2, -1, -1, -1), v1.expand(2, -1, -1, -1))
    o.sum().backward()
    ref = Reference(q, k[:1].expand(2, -1, -1, -1), v[:1].expand(2, -1, -1, -1), do=torch.ones_like(q))
    for x, r, t in ((k1, ref.dk, ref.dk_tol), (v1, ref.dv, ref.dv_tol)):
        tol = t.sum(0) + 2 * torch.finfo(dtype).eps * r.abs().sum(0)
        assert ((x.grad[0].cpu().double() - r.sum(0)).abs() <= tol).all()


def test_gradient_against_differences():
    q, k, v, do = make(1, 9, 13, 2, 1, 32, F32)
    o, lse = fa.cross_attention_forward(q, k, v)
    grads = fa.cross_attention_backward(q, k, v, o, do, lse)
    g = torch.Generator(device="cuda").manual_seed(5)
    for x, gx in zip((q, k, v), grads):
        step = torch.randn(x.shape, generator=g, device="cuda")
        h = 2.0 ** -7
        lo, hi = ((fa.cross_attention_forward(*(t + s * h * step if t is x else t for t in (q, k, v)))[0].double()
                   * do.double()).sum() for s in (-1, 1))
        want, got = (hi - lo) / (2 * h), (gx.double() * step.double()).sum()
        # fp32 sums of about 600 terms over 2 h, and the third derivative's h^2 / 6
        assert abs(want - got) <= 600 * 2.0 ** -22 / (2 * h) + 600 * h * h, (float(want), float(got))


def test_same_bits_again():
    q, k, v, do = make(1, 50, 3000, 8, 2, 128, BF16)
    first = run(q, k, v, do)
    for _ in range(3):
        o, lse = fa.cross_attention_forward(q, k, v)
        for a, b in zip(first, (o, lse) + fa.cross_attention_backward(q, k, v, o, do, lse)):
            assert torch.equal(a, b)


@pytest.mark.parametrize("size", [(2, 1, 700, 8, 2, 64), (1, 200, 300, 2, 2, 128), (1, 2000, 60, 2, 1, 64)])
def test_captured_and_replayed(size):
    """A captured forward and backward, replayed on new inputs and lengths, while an eager graph of the same leaves
    lives; on a stream of its own beside other calls."""
    q, k, v, do = make(*size, BF16)
    kl = ints([size[2]] * size[0])
    leaves = [t.clone().requires_grad_() for t in (q, k, v)]
    eager = fa.cross_attn_func(*leaves, k_lens=kl.clone())
    o, lse = fa.cross_attention_forward(q, k, v, k_lens=kl)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        go, gl = fa.cross_attention_forward(q, k, v, k_lens=kl)
        gg = fa.cross_attention_backward(q, k, v, go, do, gl, k_lens=kl)
    for seed in (1, 2):
        for a, b in zip((q, k, v, do), make(*size, BF16, seed=seed)):
            a.copy_(b)
        kl.fill_(size[2] - 3 * seed)
        graph.replay()
        fa.cross_attention_forward(q, k, v)  # another call right behind
        ref = Reference(q, k, v, None, kl, None, do)
        ref.check_forward(go, gl)
        ref.check_backward(*gg)
    eager.sum().backward()
    assert all(t.grad.isfinite().all() for t in leaves)


def test_calls_on_two_streams():
    sets = [make(1, 30, 4000, 4, 2, 64, BF16, seed=s) for s in range(2)]
    want = [run(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [None, None]
    for _ in range(5):
        for i, (st, (q, k, v, do)) in enumerate(zip(streams, sets)):
            with torch.cuda.stream(st):
                o, lse = fa.cross_attention_forward(q, k, v)
                got[i] = (o, lse) + fa.cross_attention_backward(q, k, v, o, do, lse)
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        for a, b in zip(w, g):
            assert torch.equal(a, b)


def test_refuses_what_it_cannot_take():
    q, k, v, do = make(1, 8, 9, 4, 2, 64, BF16)
    f = fa.cross_attention_forward
    for bad in (lambda: f(q, k, v[:, :8]), lambda: f(q, k.float(), v), lambda: f(q, k[..., :32], v),
                lambda: f(q, k, v, k_lens=torch.ones(1, device="cuda")), lambda: f(q, k, v, k_lens=ints([1, 2])),
                lambda: f(q.cpu(), k, v), lambda: f(q, k.cpu(), v), lambda: f(q[0], k, v),
                lambda: f(q.transpose(2, 3), k, v), lambda: fa.fa_cross_fwd(q, k, v, q, torch.empty(3, device="cuda"))):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: f(q[:, :, :3].contiguous(), k, v), lambda: f(q, k, v, scale=0.0),
                lambda: f(q, k, v, scale=math.nan), lambda: f(q, k[:, :0], v[:, :0]),
                lambda: f(q, k.expand(1, 9, 2, 64).as_strided((1, 9, 2, 64), (1152, 0, 64, 1)), v)):
        with pytest.raises(fa.FaError):
            bad()
    assert fa.fa_get_device_status() == 0

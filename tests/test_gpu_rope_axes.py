"""Norm and rotation by positions on several axes. A token's cos and sin are columns of several table rows; with
these columns gathered into a table of its own row, the one-axis operators have to give the same bits, and
those are held to float64 by their own tests. One case is compared with float64 here too (bounds: half a step of
the result and 80 * 2^-24 of the pair's two values, as derived there)."""
import pytest
import torch

import flashattention_backward_fa_gb300 as fa

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
MAX_POS = 90

CASES = [
    # B, N, Hq, Hk, d, sections, in turn, neighbouring pairs, dtype, weights, positions
    (1, 1, 1, 1, 64, (10, 11, 11), False, False, BF16, "own", "rows"),
    (2, 37, 5, 3, 128, (16, 24, 24), False, False, BF16, "own", "batch"),
    (2, 37, 5, 3, 128, (24, 20, 20), True, False, F16, "f32", "rows"),
    (2, 33, 3, 2, 128, (20, 22, 22), True, True, BF16, "own", "batch"),
    (3, 50, 8, 2, 64, (6, 5, 5), True, True, F16, "own", "batch"),
    (3, 50, 8, 2, 64, (3, 5, 8), False, True, F16, None, "axis first"),
    (2, 21, 4, 4, 128, (7, 1, 24, 16), False, False, BF16, "own", "axis first"),
    (1, 65, 7, 7, 128, (24, 24), True, False, BF16, "f32", "rows"),
    (2, 20, 6, 1, 64, (32,), False, False, F16, "own", "batch"),
    (1, 40, 2, 2, 64, (0, 8, 0, 8), False, False, BF16, "own", "rows"),
    (1, 128, 1, 1, 64, (12, 10, 10), False, False, F32, "own", "rows"),
    (2, 33, 3, 2, 128, (21, 21, 22), True, True, F32, "own", "batch"),
    (2, 19, 3, 2, 80, (3, 4, 3), False, False, F32, "own", "axis first"),
    (2, 19, 3, 2, 37, (9, 9), True, True, F32, None, "batch"),
]


def ids(c):
    return f"{c[0]}x{c[1]}x{c[2]}-{c[3]}x{c[4]}-{'.'.join(map(str, c[5]))}-{c[6]:d}{c[7]:d}-{str(c[8])[6:]}"


def make(case, seed=0):
    B, N, Hq, Hk, d, sections, turn, il, dtype, weights, positions = case
    g = torch.Generator().manual_seed(seed)
    q, k, dq, dk = (torch.randn((B, N, h, d), generator=g).to(dtype).cuda() for h in (Hq, Hk, Hq, Hk))
    wt = {"own": dtype, "f32": F32, None: None}[weights]
    wq, wk = (None if wt is None else (1 + 0.3 * torch.randn(d, generator=g)).to(wt).cuda() for _ in range(2))
    axes = fa.rope_axes(sections, turn)
    cos, sin = fa.rope_tables(MAX_POS, 2 * len(axes)) if turn else fa.rope_axis_tables(MAX_POS, sections)
    assert cos.shape == (MAX_POS, sum(sections)) and len(axes) == sum(sections)
    A = len(sections)
    if positions == "rows":  # [N, A], some outside the tables: clamped
        pos = torch.randint(-4, MAX_POS + 4, (N, A), generator=g, dtype=torch.int32).cuda()
    elif positions == "batch":
        pos = torch.randint(-4, MAX_POS + 4, (B, N, A), generator=g, dtype=torch.int32).cuda()
    else:  # [A, B, N] seen as [B, N, A]
        pos = torch.randint(0, MAX_POS, (A, B, N), generator=g, dtype=torch.int32).cuda().permute(1, 2, 0)
    return q, k, dq, dk, wq, wk, cos, sin, pos, axes


def gathered(cos, sin, pos, axes, B, N):
    """Tables with a row for each token, and the tokens' rows as positions [B, N]."""
    p = pos.expand(B, N, pos.shape[-1]).long().clamp(0, cos.shape[0] - 1)[..., list(axes)]
    col = torch.arange(len(axes), device=p.device)
    rows = torch.arange(B * N, dtype=torch.int32, device=p.device).view(B, N)
    return cos[p, col].flatten(0, 1).contiguous(), sin[p, col].flatten(0, 1).contiguous(), rows


@pytest.mark.parametrize("case", CASES, ids=ids)
def test_equals_gathered_tables(case):
    q, k, dq, dk, wq, wk, cos, sin, pos, axes = make(case)
    il = case[7]
    c2, s2, rows = gathered(cos, sin, pos, axes, *q.shape[:2])
    out = fa.qk_norm_rope_forward(q, k, wq, wk, cos, sin, pos, 1e-5, il, axes=axes)
    want = fa.qk_norm_rope_forward(q, k, wq, wk, c2, s2, rows, 1e-5, il)
    grads = fa.qk_norm_rope_backward(q, k, dq, dk, wq, wk, cos, sin, pos, 1e-5, il, axes=axes)
    wantg = fa.qk_norm_rope_backward(q, k, dq, dk, wq, wk, c2, s2, rows, 1e-5, il)
    for a, b in zip(out + grads, want + wantg):
        assert a is b is None or torch.equal(a, b)
    assert fa.fa_get_device_status() == 0


def test_many_tokens_and_spans():
    """Row groups with several tokens and ragged ends, of both tensors."""
    for B, N, Hq, Hk, d in ((1, 3001, 3, 1, 128), (2, 1777, 16, 4, 64)):
        case = (B, N, Hq, Hk, d, (8, 12, 12), False, False, BF16, "own", "batch")
        q, k, dq, dk, wq, wk, cos, sin, pos, axes = make(case, 3)
        c2, s2, rows = gathered(cos, sin, pos, axes, B, N)
        args, want_args = (wq, wk, cos, sin, pos), (wq, wk, c2, s2, rows)
        for a, b in zip(fa.qk_norm_rope_forward(q, k, *args, axes=axes) +
                        fa.qk_norm_rope_backward(q, k, dq, dk, *args, axes=axes),
                        fa.qk_norm_rope_forward(q, k, *want_args) + fa.qk_norm_rope_backward(q, k, dq, dk, *want_args)):
            assert torch.equal(a, b)


def test_against_float64():
    case = (2, 30, 4, 2, 64, (5, 6, 5), True, False, F32, "own", "batch")
    q, k, dq, dk, wq, wk, cos, sin, pos, axes = make(case, 7)
    out = fa.qk_norm_rope_forward(q, k, wq, wk, cos, sin, pos, 1e-5, axes=axes)
    for x, w, got in ((q, wq, out[0]), (k, wk, out[1])):
        x, w, got = x.cpu().double(), w.cpu().double(), got.cpu().double()
        y = x / (x.square().mean(-1, keepdim=True) + 1e-5).sqrt() * w
        want = y.clone()
        for i, a in enumerate(axes):
            at = pos[..., a].cpu().long().clamp(0, MAX_POS - 1)
            c, s = cos.cpu().double()[at, i][..., None], sin.cpu().double()[at, i][..., None]
            want[..., i] = y[..., i] * c - y[..., i + 16] * s
            want[..., i + 16] = y[..., i + 16] * c + y[..., i] * s
        size = y.abs().amax(-1, keepdim=True) * 2
        assert ((got - want).abs() <= 2.0 ** -24 * want.abs() + 80 * 2.0 ** -24 * size).all()


def test_same_position_on_every_axis_is_one_axis():
    q, k, *_ = make(CASES[1])
    cos, sin = fa.rope_tables(MAX_POS, 128)
    pos = torch.arange(37, dtype=torch.int32, device="cuda")
    axes = fa.rope_axes((16, 24, 24))
    a = fa.qk_norm_rope_forward(q, k, None, None, cos, sin, pos)
    b = fa.qk_norm_rope_forward(q, k, None, None, cos, sin, pos[:, None].expand(37, 3), axes=axes)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_autograd_and_captured():
    q, k, dq, dk, wq, wk, cos, sin, pos, axes = make(CASES[3])
    leaves = [t.clone().requires_grad_() for t in (q, k, wq, wk)]

    def step():
        out = fa.qk_norm_rope_func(*leaves, cos, sin, pos, 1e-5, True, axes=list(axes))
        return torch.autograd.grad(out, leaves, (dq, dk))

    for a, b in zip(step(), fa.qk_norm_rope_backward(q, k, dq, dk, wq, wk, cos, sin, pos, 1e-5, True, axes=axes)):
        assert torch.equal(a, b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    pos.sub_(3)
    graph.replay()
    for a, b in zip(got, step()):
        assert torch.equal(a, b)


APPEND = [
    # B, T, Hq, H, d, page, sections, in turn, neighbouring pairs, dtype, positions
    (3, 1, 8, 2, 128, 64, (16, 24, 24), False, False, BF16, "batch"),
    (2, 1, 3, 1, 64, 16, (11, 11, 10), True, True, F16, "batch"),
    (2, 40, 4, 2, 128, 32, (24, 20, 20), True, False, BF16, "rows"),
    (2, 70, 2, 2, 64, 128, (5, 6, 5), False, True, F16, "axis first"),
    (1, 150, 6, 3, 128, 128, (8, 8, 16), False, False, F16, "batch"),
    (4, 5, 4, 4, 64, 16, (16, 16), True, False, BF16, "rows"),
]


def caches(pages, page, H, d, g):
    one = fa.kv8_cache_alloc(pages, page, H, d)
    for t in (one.k, one.v):
        t.view(torch.uint8).copy_(torch.randint(0, 0x70, t.shape, generator=g, dtype=torch.uint8))
    for t in (one.k_scale, one.v_scale):
        t.copy_(torch.exp2(torch.randint(-12, -6, t.shape, generator=g).float()))
    return one, fa.Kv8Cache(*(t.clone(memory_format=torch.preserve_format) for t in one))


@pytest.mark.parametrize("case", APPEND)
def test_append_equals_the_two_calls(case):
    """Codes, scales and q of the fused call against the rotation by itself and the append of its result."""
    B, T, Hq, H, d, page, sections, turn, il, dtype, positions = case
    q, k, _, _, wq, wk, cos, sin, pos, axes = make((B, T, Hq, H, d, sections, turn, il, dtype, "own", positions), 5)
    g = torch.Generator().manual_seed(2)
    v = torch.randn((B, T, H, d), generator=g).to(dtype).cuda()
    lens = torch.tensor([T + 7 * b + 3 for b in range(B)], dtype=torch.int32, device="cuda")
    new = torch.tensor([max(1, T - 2 * b) for b in range(B)], dtype=torch.int32, device="cuda")
    per = -(-int(lens.max()) // page)
    table = torch.randperm(B * per, generator=g).int().view(B, per).cuda()
    one, two = caches(B * per, page, H, d, g)
    qo = fa.kv8_norm_rope_append(one, q, k, v, wq, wk, cos, sin, table, lens, new, 1e-5, il, pos, axes)
    q2, k2 = fa.qk_norm_rope_forward(q, k, wq, wk, cos, sin, pos, 1e-5, il, axes=axes)
    fa.kv8_append(two, k2, v, table, lens, new)
    for a, b in zip(one, two):
        assert torch.equal(a.view(torch.uint8) if a.dtype is torch.float8_e4m3fn else a,
                           b.view(torch.uint8) if b.dtype is torch.float8_e4m3fn else b)
    for b in range(B):
        n = int(new[b])
        assert torch.equal(qo[b, :n], q2[b, :n]) and (qo[b, n:] == 0).all()
    assert fa.fa_get_device_status() == 0


def test_append_at_given_positions_without_axes():
    """Positions [T] and [B, T]: the places in the sequences give the plain call's bits, others the rotation's."""
    B, T, Hq, H, d, page = 2, 6, 4, 2, 64, 16
    q, k, _, _, wq, wk, cos, sin, _, _ = make((B, T, Hq, H, d, (32,), False, False, BF16, "own", "rows"), 5)
    v = k.flip(1).contiguous()
    lens = torch.tensor([10, 22], dtype=torch.int32, device="cuda")
    table = torch.arange(4, dtype=torch.int32, device="cuda").view(2, 2)
    places = lens[:, None] - T + torch.arange(T, dtype=torch.int32, device="cuda")
    runs = []
    for kw in ({}, dict(positions=places.int()), dict(positions=places.int()[1])):
        cache, _ = caches(4, page, H, d, torch.Generator().manual_seed(2))
        runs.append((fa.kv8_norm_rope_append(cache, q, k, v, wq, wk, cos, sin, table, lens, **kw), cache))
    as_bytes = lambda c: [t.view(torch.uint8) for t in c]  # noqa: E731
    assert torch.equal(runs[0][0], runs[1][0])
    assert all(torch.equal(a, b) for a, b in zip(as_bytes(runs[0][1]), as_bytes(runs[1][1])))
    assert torch.equal(runs[0][0][1], runs[2][0][1]) and not torch.equal(runs[0][0][0], runs[2][0][0])


def test_rotated_step_and_attention_captured():
    """A decode step as a vision-language model runs it: positions that differ from the places in the cache,
    advanced on the device, captured and replayed; equal to the eager steps."""
    B, Hq, H, d, page, steps = 2, 4, 2, 64, 16, 5
    g = torch.Generator().manual_seed(9)
    xs = [[torch.randn((B, 1, h, d), generator=g).to(BF16).cuda() for h in (Hq, H, H)] for _ in range(steps)]
    cos, sin = fa.rope_tables(MAX_POS, d)
    axes = fa.rope_axes((12, 10, 10), True)
    table = torch.arange(8, dtype=torch.int32, device="cuda").view(2, 4)

    def run(captured):
        cache, _ = caches(8, page, H, d, torch.Generator().manual_seed(2))
        lens = torch.tensor([14, 30], dtype=torch.int32, device="cuda")
        pos = torch.tensor([[[5, 5, 5]], [[17, 17, 17]]], dtype=torch.int32, device="cuda")
        x = [t.clone() for t in xs[0]]

        def step():
            lens.add_(1)
            pos.add_(1)
            qo = fa.kv8_norm_rope_append(cache, *x, None, None, cos, sin, table, lens, positions=pos, axes=axes)
            return fa.kv8_attention(qo, cache, table, lens, 64)

        graph = None
        if captured:
            keep = [t.clone() for t in (*cache, lens, pos)]
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                step()
            torch.cuda.current_stream().wait_stream(side)
            for t, was in zip((*cache, lens, pos), keep):
                t.copy_(was)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                out = step()
        outs = []
        for new in xs:
            for t, n in zip(x, new):
                t.copy_(n)
            if graph:
                graph.replay()
            else:
                out = step()
            outs.append([t.clone() for t in out])
        return outs

    for a, b in zip(run(False), run(True)):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_refusals():
    q, k, dq, dk, wq, wk, cos, sin, pos, axes = make(CASES[1])
    f = lambda **kw: fa.qk_norm_rope_forward(q, k, wq, wk, **{**dict(cos=cos, sin=sin, positions=pos, axes=axes), **kw})  # noqa: E731
    for kw in (dict(positions=None), dict(positions=pos.long()), dict(positions=pos.cpu()), dict(axes=axes[:-1]),
               dict(axes=(4,) * 64), dict(axes=(-1,) * 64), dict(axes=()), dict(positions=pos[..., :2]),
               dict(positions=pos[:, :-1]), dict(positions=pos[:1].repeat(3, 1, 1)), dict(cos=None, sin=None),
               dict(axes=None), dict(axes=(0.5,) * 64)):
        with pytest.raises(ValueError):
            f(**kw)
    with pytest.raises(ValueError):
        fa.qk_norm_rope_backward(q, k, dq, dk, wq, wk, cos, sin, None, axes=axes)

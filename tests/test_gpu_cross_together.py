"""Cross attention and the rotation by several axes as they are used together: a block of a model whose tokens lie on a
grid and attend to a text (training), and a decoder's step over its 8-bit cache and an encoder's states (serving)."""
import math

import pytest
import torch

import flashattention_backward_fa_gb300 as fa
from cross_reference import Reference

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def grid_positions(*sizes):
    """[tokens, axes] places of a grid's tokens."""
    at = torch.meshgrid(*(torch.arange(n, dtype=torch.int32) for n in sizes), indexing="ij")
    return torch.stack([a.reshape(-1) for a in at], -1).cuda()


def block_inputs(dtype, d=64, B=2, H=4, Hk=2, Nk=13):
    g = torch.Generator().manual_seed(3)
    draw = lambda *s: torch.randn(s, generator=g).to(dtype).cuda()  # noqa: E731
    pos = grid_positions(2, 3, 4)
    N = pos.shape[0]
    q, k, v, do = (draw(B, N, H, d) for _ in range(4))
    weights = [(1 + 0.1 * torch.randn(d, generator=g)).cuda() for _ in range(2)]
    return [q, k, v, draw(B, Nk, Hk, d), draw(B, Nk, Hk, d), *weights], do, pos


SECTIONS = (8, 12, 12)


def block(q, k, v, ks, vs, wq, wk, cos, sin, pos, k_lens):
    q, k = fa.qk_norm_rope_func(q, k, wq, wk, cos, sin, pos, axes=fa.rope_axes(SECTIONS))
    return fa.cross_attn_func(fa.flash_attn_func(q, k, v), ks, vs, k_lens=k_lens)


def block_plain(q, k, v, ks, vs, wq, wk, cos, sin, pos, k_lens):
    """The same from the definitions."""
    which = torch.tensor(fa.rope_axes(SECTIONS))
    rows = pos.cpu().long()[:, which]  # [N, pairs]
    c, s = (t.cpu().double()[rows, torch.arange(len(which))][None, :, None] for t in (cos, sin))

    def turned(x, w):
        x = x * (x.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * w
        a, b = x.chunk(2, -1)
        return torch.cat([a * c - b * s, b * c + a * s], -1)

    def attend(q, k, v, lens=None):
        k, v = (t.repeat_interleave(q.shape[2] // t.shape[2], 2) for t in (k, v))
        x = torch.einsum("bihd,bjhd->bhij", q, k) / math.sqrt(q.shape[-1])
        if lens is not None:
            x = x.masked_fill((torch.arange(k.shape[1]) >= lens[:, None])[:, None, None], -math.inf)
        return torch.einsum("bhij,bjhd->bihd", x.softmax(-1), v)

    return attend(attend(turned(q, wq), turned(k, wk), v), ks, vs, k_lens.cpu())


def test_block_against_float64():
    """In fp32. Each stage's sums are off by at most about (d + N) 2^-24 = 2^-17.4 of their terms' magnitudes; a
    softmax passes twice its scores' error on, and |scores| <= sqrt(d) (1.3)^2 = 14 of normed queries and keys, and
    there are three stages and their backwards: 6 * 2 * 14 * 2^-17.4 = 2^-10 of the largest value."""
    leaves, do, pos = block_inputs(F32)
    cos, sin = fa.rope_tables(16, 64)
    lens = torch.tensor([13, 5], dtype=torch.int32, device="cuda")
    leaves = [t.requires_grad_() for t in leaves]
    o = block(*leaves, cos, sin, pos, lens)
    o.backward(do)
    plain = [t.detach().cpu().double().requires_grad_() for t in leaves]
    want = block_plain(*plain, cos, sin, pos, lens)
    want.backward(do.cpu().double())
    pairs = [(o, want)] + [(t.grad, p.grad) for t, p in zip(leaves, plain)]
    for i, (x, ref) in enumerate(pairs):
        off = (x.detach().cpu().double() - ref.detach()).abs().max() / ref.abs().max()
        assert off <= 2.0 ** -10, (i, float(off))


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_block_is_its_stages(dtype):
    """Forward and gradients have the bits of the stages' calls one by one, and the attention to the text, which reads
    what the stage before it wrote, is right."""
    leaves, do, pos = block_inputs(dtype)
    q, k, v, ks, vs, wq, wk = leaves
    cos, sin = fa.rope_tables(16, 64)
    lens = torch.tensor([0, 9], dtype=torch.int32, device="cuda")
    axes = fa.rope_axes(SECTIONS)
    copies = [t.clone().requires_grad_() for t in leaves]
    o = block(*copies, cos, sin, pos, lens)
    got = torch.autograd.grad(o, copies, do)
    q1, k1 = fa.qk_norm_rope_forward(q, k, wq, wk, cos, sin, pos, axes=axes)
    o1, l1 = fa.attention_forward(q1, k1, v)
    o2, l2 = fa.cross_attention_forward(o1, ks, vs, k_lens=lens)
    do1, dks, dvs = fa.cross_attention_backward(o1, ks, vs, o2, do, l2, k_lens=lens)
    dq1, dk1, dv = fa.attention_backward(q1, k1, v, o1, do1, l1)
    dq, dk, dwq, dwk = fa.qk_norm_rope_backward(q, k, dq1, dk1, wq, wk, cos, sin, pos, axes=axes)
    assert torch.equal(o, o2)
    for a, b in zip(got, (dq, dk, dv, dks, dvs, dwq, dwk)):
        assert torch.equal(a, b)
    ref = Reference(o1, ks, vs, None, lens, None, do)
    ref.check_forward(o2, l2)
    ref.check_backward(do1, dks, dvs)
    assert (dks[0] == 0).all() and (dq[0] == 0).all()  # (nothing attends there)


def test_block_captured_as_a_training_step():
    leaves, do, pos = block_inputs(BF16)
    cos, sin = fa.rope_tables(16, 64)
    lens = torch.tensor([13, 6], dtype=torch.int32, device="cuda")
    copies = [t.clone().requires_grad_() for t in leaves]

    def step():
        o = block(*copies, cos, sin, pos, lens)
        return (o.detach(), *torch.autograd.grad(o, copies, do))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for n in (4, 13):
        lens.fill_(n)
        with torch.no_grad():
            copies[3].mul_(1.25)
        graph.replay()
        for a, b in zip(got, step()):
            assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_decoder_step_captured(dtype):
    """One token a step: normed, rotated and appended, attention over the cache, then over an encoder's states of its
    sequence's length. Captured and replayed with the eager steps' bits, two captured steps on one set of states in
    turn; the last attention against the definition at every step."""
    B, Hq, H, d, page, steps = 3, 4, 2, 64, 16, 4
    g = torch.Generator().manual_seed(11)
    draw = lambda *s: torch.randn(s, generator=g).to(dtype).cuda()  # noqa: E731
    xs = [[draw(B, 1, h, d) for h in (Hq, H, H)] for _ in range(steps)]
    ks, vs = draw(B, 700, H, d), draw(B, 700, H, d)
    klens = torch.tensor([700, 0, 133], dtype=torch.int32, device="cuda")
    cos, sin = fa.rope_tables(64, d)
    axes = fa.rope_axes((12, 10, 10), True)
    table = torch.arange(2 * B, dtype=torch.int32, device="cuda").view(B, 2)

    def decoder():
        cache = fa.kv8_cache_alloc(2 * B, page, H, d)
        for t in cache:
            t.zero_()
        lens = torch.zeros(B, dtype=torch.int32, device="cuda")
        pos = torch.full((B, 1, 3), 7, dtype=torch.int32, device="cuda")
        x = [t.clone() for t in xs[0]]

        def step():
            lens.add_(1)
            pos.add_(1)
            q = fa.kv8_norm_rope_append(cache, *x, None, None, cos, sin, table, lens, positions=pos, axes=axes)
            o, _ = fa.kv8_attention(q, cache, table, lens, 2 * page)
            return o, *fa.cross_attention_forward(o, ks, vs, k_lens=klens)

        def restart():
            for t in cache:
                t.zero_()
            lens.zero_()
            pos.fill_(7)

        return x, step, restart

    x, step, _ = decoder()
    want = []
    for new in xs:
        for t, n in zip(x, new):
            t.copy_(n)
        want.append([t.clone() for t in step()])
        o, c, lse = want[-1]
        Reference(o, ks, vs, None, klens).check_forward(c, lse)
    captured = []
    for _ in range(2):
        x, step, restart = decoder()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.current_stream().wait_stream(side)
        restart()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step()
        captured.append((x, graph, out, step))  # (the step keeps its cache and lengths)
    for new, w in zip(xs, want):
        for x, graph, *_ in captured:
            for t, n in zip(x, new):
                t.copy_(n)
            graph.replay()
        for _, _, out, _ in captured:
            for a, b in zip(out, w):
                assert torch.equal(a, b)


def test_on_another_stream_than_the_inputs():
    """Inputs made on one stream, used on another that waits for it, and their memory given back at once."""
    leaves, do, pos = block_inputs(BF16)
    cos, sin = fa.rope_tables(16, 64)
    lens = torch.tensor([13, 6], dtype=torch.int32, device="cuda")

    def step(leaves):
        o = block(*leaves, cos, sin, pos, lens)
        return (o.detach(), *torch.autograd.grad(o, leaves, do))

    want = step([t.clone().requires_grad_() for t in leaves])
    side = torch.cuda.Stream()
    for _ in range(3):
        copies = [t.clone().requires_grad_() for t in leaves]
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            got = step(copies)
        for t in copies:
            t.record_stream(side)
        del copies
        torch.cuda.current_stream().wait_stream(side)
        for a, b in zip(got, want):
            assert torch.equal(a, b)

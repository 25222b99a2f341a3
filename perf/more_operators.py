"""Timed cases of cross attention and of rotation by positions on several axes.

Three operators, each as a user's program calls it:

* ``cross``   attention of queries over the states of another sequence of another length, with shared
              key heads and the real lengths of padded batches (``cross_attention_forward``); with
              ``grad`` its backward pass too (``cross_attention_backward``);
* ``rotate``  per-head RMS norm of queries and keys and their rotation by positions with several axes
              (``qk_norm_rope_forward`` with ``axes``); with ``grad`` its backward pass too
              (``qk_norm_rope_backward``);
* ``step``    the same norm and rotation of new queries and keys, keys and values into the paged e4m3
              cache (``kv8_norm_rope_append`` with ``positions`` and ``axes``).

With ``own`` false, ``run`` computes them from elementary torch operations in 32 bits.

Definitions. Cross attention: query head h reads key head h // (Hq / Hk); o = softmax(q k^T / sqrt(d)) v
over the first ``k_lens`` keys, lse the natural log of the sum; queries from ``q_lens`` on, and queries
without keys, get o = 0, lse = -inf and no part in any gradient; gradients of shared key heads are summed
over their query heads. Rotation: y = w * x / sqrt(mean(x^2) + eps); pair i of the first ``rot`` values of
y, (a, b), becomes (a cos - b sin, b cos + a sin) with column i of the tables' row pos[axis of pair i],
the partners being ``rot / 2`` apart, or neighbours where ``interleaved``. Cache: page p, token slot t,
head h hold e4m3 codes of x / scale[p, h] with scale = 2^e, e the least integer with amax <= 448 * 2^e
(amax: largest magnitude of the tokens that a call brings to the page), and never less than the page's
former scale when the page holds earlier tokens, which are rounded anew to the larger scale.
"""
import math

import torch

own = False

EPS = 1e-6
E_MIN = -100  # least scale exponent
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ---------------------------------------------------------------- cases
def listed():
    return [
        # One new token of a decoder over an encoder's states, one sequence: nothing but latency.
        dict(name="token_f16_1x16_1499x64", op="cross", grad=False, B=1, Nq=1, Nk=1499, Hq=16, Hkv=16, d=64,
             dtype="f16", q_ragged=False, k_ragged=False),
        # The same for a serving batch with shared key heads and long states of unequal lengths.
        dict(name="token_bf16_32x32_4096x128", op="cross", grad=False, B=32, Nq=1, Nk=4096, Hq=32, Hkv=8, d=128,
             dtype="bf16", q_ragged=False, k_ragged=True),
        # A few learned queries that sum up one long sequence of states.
        dict(name="latents_bf16_1x16_64x16383x128", op="cross", grad=False, B=1, Nq=64, Nk=16383, Hq=16, Hkv=16,
             d=128, dtype="bf16", q_ragged=False, k_ragged=False),
        # Image tokens that read a text's states, texts of unequal lengths: answering.
        dict(name="image_bf16_4x16_4096x512x128", op="cross", grad=False, B=4, Nq=4096, Nk=512, Hq=16, Hkv=16, d=128,
             dtype="bf16", q_ragged=False, k_ragged=True),
        # The benchmark's training batch over such texts, with the backward pass.
        dict(name="grad_bf16_4x16_2048x512x128", op="cross", grad=True, B=4, Nq=2048, Nk=512, Hq=16, Hkv=16, d=128,
             dtype="bf16", q_ragged=False, k_ragged=True),
        # A short text with an odd number of tokens, shared key heads, padded batch on both sides.
        dict(name="grad_f16_2x16_4095x77x64", op="cross", grad=True, B=2, Nq=4095, Nk=77, Hq=16, Hkv=4, d=64,
             dtype="f16", q_ragged=True, k_ragged=True),
        # A long document's decoder over its encoder, shared key heads: the largest.
        dict(name="grad_bf16_1x32_8192x4096x128", op="cross", grad=True, B=1, Nq=8192, Nk=4096, Hq=32, Hkv=8, d=128,
             dtype="bf16", q_ragged=False, k_ragged=False),
        # A toy-sized training step in single precision.
        dict(name="grad_f32_1x2_128x77x64", op="cross", grad=True, B=1, Nq=128, Nk=77, Hq=2, Hkv=2, d=64,
             dtype="f32", q_ragged=False, k_ragged=False),
        # The benchmark's headline shape as a video of 8 frames of 32 x 32 patches, before its attention.
        dict(name="rotate_bf16_1x32x8192x128", op="rotate", grad=False, B=1, N=8192, Hq=32, Hkv=32, d=128,
             sections="16,24,24", spread=False, interleaved=False, dtype="bf16", packed=False, each=False),
        # Training on texts with images in them: shared key heads, an odd length, axes in turn over half of the
        # head, neighbouring pairs, q and k as slices of one packed projection, positions of each sequence.
        dict(name="rotate_grad_f16_2x16x4095x64", op="rotate", grad=True, B=2, N=4095, Hq=16, Hkv=4, d=64,
             sections="6,5,5", spread=True, interleaved=True, dtype="f16", packed=True, each=True),
        # One new token for each of 32 sequences with images behind them.
        dict(name="step_bf16_token_32x32x128", op="step", B=32, T=1, L=4097, Hq=32, Hkv=8, d=128,
             sections="16,24,24", spread=False, interleaved=False, page=64, dtype="bf16", ragged=True),
        # A prompt of 2048 tokens, images among them, for each of 4 sequences.
        dict(name="step_bf16_prompt_4x16x2048x128", op="step", B=4, T=2048, L=2048, Hq=16, Hkv=16, d=128,
             sections="24,20,20", spread=True, interleaved=False, page=64, dtype="bf16", ragged=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def _sections(rng, pairs):
    """Pairs of two or three axes, unequal, all of them used."""
    n = rng.choice([2, 3, 3])
    first = max(1, pairs // n - rng.choice([0, 1, 2]))
    left = pairs - first
    return ",".join(map(str, [first, left] if n == 2 else [first, left // 2, left - left // 2]))


def draw(rng):
    op = rng.choice(["cross", "cross", "cross", "cross", "rotate", "rotate", "step"])
    d = rng.choice([64, 128])
    dtype = rng.choice(["bf16", "bf16", "f16"])
    Hkv = rng.choice([1, 2, 4, 8, 16])
    Hq = Hkv * rng.choice([1, 1, 2, 3, 4, 8])
    if op == "cross":
        grad = rng.random() < 0.5
        if rng.random() < 0.12:
            dtype = "f32"
        B = _log(rng, 1, 32)
        # no more products and no more states than the largest listed cases, in single precision a 16th of them
        part = 16 if dtype == "f32" else 1
        if not grad and rng.random() < 0.5:
            Nq = rng.choice([1, 1, 1, 2, 3, 5, 8])
        else:
            Nq = _log(rng, 1, max(1, min(8192, 8192 * 32 * 128 // (B * Hq * d * part))))
        most = min(32768, 32 * 4096 * 8 * 128 // (B * Hkv * d * part),
                   32 * 8192 * 4096 * 128 // (B * Hq * Nq * d * part))
        least = 4 if grad else 1  # (over one key the gradient of q is zero, and what is computed of it noise)
        return dict(op=op, grad=grad, B=B, Nq=Nq, Nk=_log(rng, least, max(least, most)), Hq=Hq, Hkv=Hkv, d=d,
                    dtype=dtype, q_ragged=rng.random() < 0.25, k_ragged=rng.random() < 0.6)
    rot = rng.choice([d, d, d // 2])
    if op == "rotate":
        B = _log(rng, 1, 8)
        N = _log(rng, 1, max(1, 8192 * 32 * 64 // (B * (Hq + Hkv) * d)))
        return dict(op=op, grad=rng.random() < 0.5, B=B, N=min(N, 16384), Hq=Hq, Hkv=Hkv, d=d,
                    sections=_sections(rng, rot // 2), spread=rng.random() < 0.5, interleaved=rng.random() < 0.3,
                    dtype=rng.choice([dtype, dtype, dtype, "f32"]), packed=rng.random() < 0.5, each=rng.random() < 0.5)
    B = _log(rng, 1, 64)
    T = 1 if rng.random() < 0.5 else min(2048, _log(rng, 1, max(1, 8192 * 16 // (B * Hq))))
    return dict(op=op, B=B, T=T, L=T + _log(rng, 1, 4000), Hq=Hq, Hkv=Hkv, d=d, sections=_sections(rng, rot // 2),
                spread=rng.random() < 0.5, interleaved=rng.random() < 0.3, page=rng.choice([16, 32, 64, 128]),
                dtype=dtype, ragged=rng.random() < 0.5)


def _spread(n, most, part, at):
    """n lengths between (1 - part) * most and most, spread evenly in a fixed order."""
    return [max(1, most - int(part * most * math.modf(at * b)[0])) for b in range(n)]


def _cross_lengths(c):
    """(queries, keys) of each sequence."""
    q = _spread(c["B"], c["Nq"], 0.3, 0.381966) if c["q_ragged"] else [c["Nq"]] * c["B"]
    k = _spread(c["B"], c["Nk"], 0.9, 0.618034) if c["k_ragged"] else [c["Nk"]] * c["B"]
    return q, k


def _step_lengths(c):
    """(tokens of each sequence with the new ones, new tokens of each)."""
    B, T, L = c["B"], c["T"], c["L"]
    if not c["ragged"]:
        return [L] * B, [T] * B
    new = _spread(B, T, 0.4, 0.381966)
    return [max(n, m) for n, m in zip(_spread(B, L, 0.95, 0.618034), new)], new


# ---------------------------------------------------------------- inputs
def _activations(g, shape, dtype):
    """Values as a projection gives them: unit spread, a few channels much larger than the rest."""
    x = torch.randn(shape, generator=g, device="cuda")
    x *= 1 + 3 * (torch.rand(shape[-1], generator=g, device="cuda") < 0.03)
    return x.to(dtype)


def _axes(c):
    """The axis of each pair: the sections one after the other, or in turn while they last."""
    left = [int(n) for n in c["sections"].split(",")]
    if not c["spread"]:
        return tuple(a for a, n in enumerate(left) for _ in range(n))
    out = []
    while any(left):
        for a, n in enumerate(left):
            if n:
                out.append(a)
                left[a] -= 1
    return tuple(out)


def _tables(c, rows):
    """cos and sin [rows, pairs]: an axis has frequencies of its own where its pairs lie side by side, else the
    axes share one row of frequencies."""
    parts = [int(n) for n in c["sections"].split(",")]
    e = [torch.arange(n, device="cuda", dtype=torch.float64) / n for n in ([sum(parts)] if c["spread"] else parts)]
    ang = torch.arange(rows, device="cuda", dtype=torch.float64)[:, None] * torch.pow(10000.0, -torch.cat(e))
    return ang.cos().float(), ang.sin().float()


def _grid(n, axes, start):
    """Positions [n, axes] of tokens `start` .. of frames of 32 x 32 patches (two axes: of images side by side)."""
    i = torch.arange(start, start + n, device="cuda")
    p = torch.stack([i // 1024, i // 32 % 32, i % 32], -1)
    return (p if axes == 3 else torch.stack([i // 32, i % 32], -1)).int()


def _text(n, axes, start):
    """Positions [n, axes] of text tokens: the same on every axis."""
    return torch.arange(start, start + n, device="cuda", dtype=torch.int32)[:, None].expand(n, axes)


def _pow2_scale(amax):
    m, x = torch.frexp(amax)
    return torch.exp2(torch.where(amax > 0, x - 9 + (m > 0.875).int(), x * 0 + E_MIN).clamp(min=E_MIN).float())


def _new_cache(g, pages, page, H, d):
    """A filled cache, [pages, page, H, d] e4m3 codes stored head by head, and its scales [pages, H]."""
    x = torch.randn((pages, H, page, d), generator=g, device="cuda")
    x *= 0.5 + torch.rand((pages, H, 1, 1), generator=g, device="cuda")
    scale = _pow2_scale(x.abs().amax((2, 3)))
    return (x / scale[:, :, None, None]).to(torch.float8_e4m3fn).transpose(1, 2), scale


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt, d, Hq, Hkv, B = DTYPES[c["dtype"]], c["d"], c["Hq"], c["Hkv"], c["B"]
    s = dict(case=c)
    ints = lambda v: torch.tensor(v, device="cuda", dtype=torch.int32)  # noqa: E731
    if c["op"] == "cross":
        ql, kl = _cross_lengths(c)
        s["q"] = _activations(g, (B, c["Nq"], Hq, d), dt)
        s["k"], s["v"] = _activations(g, (B, c["Nk"], Hkv, d), dt), _activations(g, (B, c["Nk"], Hkv, d), dt)
        s["q_lens"] = ints(ql) if c["q_ragged"] else None
        s["k_lens"] = ints(kl) if c["k_ragged"] else None
        if c["grad"]:
            s["do"] = torch.randn((B, c["Nq"], Hq, d), generator=g, device="cuda").to(dt)
        return s
    s["axes"] = _axes(c)
    axes = max(s["axes"]) + 1
    s["wq"] = (1 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(dt)
    s["wk"] = (1 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(dt)
    if c["op"] == "rotate":
        N = c["N"]
        s["cos"], s["sin"] = _tables(c, max(N, 64))
        half = N // 2  # each sequence a text, then images
        s["pos"] = _grid(N, axes, 0) if not c["each"] else torch.stack(
            [torch.cat([_text(half, axes, b), half // 2 + _grid(N - half, axes, 32 * b)]) for b in range(B)])
        s["pos"].clamp_(max=max(N, 64) - 1)
        if c["packed"]:  # q, k and v side by side in one projection's output
            qkv = _activations(g, (B, N, Hq + 2 * Hkv, d), dt)
            s["q"], s["k"] = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv]
        else:
            s["q"], s["k"] = _activations(g, (B, N, Hq, d), dt), _activations(g, (B, N, Hkv, d), dt)
        if c["grad"]:
            s["dq"] = torch.randn((B, N, Hq, d), generator=g, device="cuda").to(dt)
            s["dk"] = torch.randn((B, N, Hkv, d), generator=g, device="cuda").to(dt)
        return s
    lens, new = _step_lengths(c)
    page, T = c["page"], c["T"]
    s["cos"], s["sin"] = _tables(c, c["L"] + 64)
    # a single token is text behind images, which take fewer positions than tokens; a prompt begins with an image
    s["pos"] = torch.stack([_text(T, axes, lens[b] * 3 // 4) if T == 1 else
                            torch.cat([_grid(T // 2, axes, 0), _text(T - T // 2, axes, 40 + b)]) for b in range(B)])
    s["pos"].clamp_(max=c["L"] + 63)
    need = [-(-n // page) for n in lens]
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=g, device="cuda", dtype=torch.int32)
    table = torch.full((B, max(need)), -1, device="cuda", dtype=torch.int32)
    table[torch.arange(max(need), device="cuda")[None] < ints(need)[:, None]] = order[:sum(need)]
    s["k_cache"], s["k_scale"] = _new_cache(g, pages, page, Hkv, d)
    s["v_cache"], s["v_scale"] = _new_cache(g, pages, page, Hkv, d)
    s["table"], s["lens"], s["new"] = table, ints(lens), ints(new) if c["ragged"] else None
    s["k"], s["v"] = _activations(g, (B, T, Hkv, d), dt), _activations(g, (B, T, Hkv, d), dt)
    s["q"] = _activations(g, (B, T, Hq, d), dt)
    return s


# ---------------------------------------------------------------- plain forms
def _cross(s):
    c, dt = s["case"], s["q"].dtype
    B, Nq, Hq, d = s["q"].shape
    Nk, H = s["k"].shape[1:3]
    G, scale = Hq // H, 1 / math.sqrt(d)
    rows = lambda x: x.float().view(B, Nq, H, G, d).permute(0, 2, 3, 1, 4).flatten(2, 3)  # noqa: E731  [B, H, G Nq, d]
    back = lambda x: x.unflatten(2, (G, Nq)).permute(0, 3, 1, 2, 4).reshape(B, Nq, Hq, d).to(dt)  # noqa: E731
    q, k, v = rows(s["q"]), s["k"].float().transpose(1, 2), s["v"].float().transpose(1, 2)
    sc = (q @ k.transpose(2, 3)).mul_(scale)
    keep = None
    if s["k_lens"] is not None:
        keep = (torch.arange(Nk, device=q.device) < s["k_lens"][:, None])[:, None, None]
    if s["q_lens"] is not None:
        live = (torch.arange(Nq, device=q.device) < s["q_lens"][:, None]).repeat(1, G)[:, None, :, None]
        keep = live if keep is None else keep & live
    if keep is not None:
        sc.masked_fill_(~keep, -math.inf)
    m = sc.amax(-1, keepdim=True).clamp(min=-1e30)
    p = sc.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    p = p.div_(torch.where(l > 0, l, 1))
    o = p @ v
    out = back(o), (m + l.log())[..., 0].view(B, Hq, Nq)
    if not c["grad"]:
        return out
    do = rows(s["do"])
    if s["q_lens"] is not None:
        do = do * live
    dv = p.transpose(2, 3) @ do
    ds = (do @ v.transpose(2, 3)).sub_((do * o).sum(-1, keepdim=True)).mul_(p).mul_(scale)
    dk = ds.transpose(2, 3) @ q
    return out + (back(ds @ k), dk.transpose(1, 2).to(dt), dv.transpose(1, 2).to(dt))


def _pairs(y, rot, interleaved):
    if interleaved:
        return y[..., 0:rot:2], y[..., 1:rot:2]
    return y[..., :rot // 2], y[..., rot // 2:rot]


def _join(a, b, rest, interleaved):
    if interleaved:
        return torch.cat([torch.stack([a, b], -1).flatten(-2), rest], -1)
    return torch.cat([a, b, rest], -1)


def _angles(s):
    """cos and sin [B or 1, N, 1, pairs] of the tokens."""
    pos = s["pos"].long()
    at = pos[..., torch.tensor(s["axes"], device=pos.device)]  # [.., N, pairs]
    if at.dim() == 2:
        at = at[None]
    col = torch.arange(at.shape[-1], device=pos.device)
    return s["cos"][at, col][:, :, None], s["sin"][at, col][:, :, None]


def _norm_rope(x, w, cos, sin, interleaved):
    rot = 2 * cos.shape[-1]
    x = x.float()
    y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.float()
    a, b = _pairs(y, rot, interleaved)
    return _join(a * cos - b * sin, b * cos + a * sin, y[..., rot:], interleaved)


def _norm_rope_grad(x, dout, w, cos, sin, interleaved):
    rot = 2 * cos.shape[-1]
    x, dout, w = x.float(), dout.float(), w.float()
    a, b = _pairs(dout, rot, interleaved)
    dy = _join(a * cos + b * sin, b * cos - a * sin, dout[..., rot:], interleaved)
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    xn = x * r
    gy = dy * w
    dx = r * (gy - xn * (gy * xn).mean(-1, keepdim=True))
    return dx, (dy * xn).flatten(0, -2).sum(0)


def _write(x, cache, scale, s):
    """New values [B, T, H, d] into one half of the cache."""
    page, T = s["case"]["page"], x.shape[1]
    new = s["new"] if s["new"] is not None else torch.full_like(s["lens"], T)
    t = torch.arange(T, device=x.device)
    start = (s["lens"] - new).long()
    pos = (start[:, None] + t).clamp(max=s["table"].shape[1] * page - 1)
    live = t < new[:, None]
    at = s["table"].gather(1, pos // page).long()[live]
    slot = (pos % page)[live]
    x = x.float()[live]
    # largest new magnitude of each (page, head); pages that hold earlier tokens keep their scale at least
    most = torch.full_like(scale, -1).index_reduce_(0, at, x.abs().amax(-1), "amax")
    grown = _pow2_scale(most.clamp(min=0))
    first = s["table"].gather(1, (start // page).clamp(max=s["table"].shape[1] - 1)[:, None])[:, 0].long().clamp(min=0)
    old = torch.full_like(scale, -1)
    old[first] = torch.where((start % page != 0)[:, None], scale[first], old[first])
    fresh = torch.where(most >= 0, torch.maximum(grown, old), scale)
    # earlier tokens of the page in which the new ones begin
    kept = (torch.arange(page, device=x.device) < (start % page)[:, None])[:, :, None, None]
    was = cache[first]
    again = (was.float() * (scale[first] / fresh[first])[:, None, :, None]).to(cache.dtype)
    cache.view(torch.uint8)[first] = torch.where(kept, again.view(torch.uint8), was.view(torch.uint8))
    cache.view(torch.uint8)[at, slot] = (x / fresh[at][:, :, None]).to(cache.dtype).view(torch.uint8)
    scale.copy_(fresh)


def run(state):
    s, c = state, state["case"]
    if own:
        return _run_own(s, c)
    if c["op"] == "cross":
        return _cross(s)
    cos, sin = _angles(s)
    dt, il = s["q"].dtype, c["interleaved"]
    q, k = (_norm_rope(s[x], s[w], cos, sin, il).to(dt) for x, w in (("q", "wq"), ("k", "wk")))
    if c["op"] == "rotate":
        if not c["grad"]:
            return q, k
        dq, dwq = _norm_rope_grad(s["q"], s["dq"], s["wq"], cos, sin, il)
        dk, dwk = _norm_rope_grad(s["k"], s["dk"], s["wk"], cos, sin, il)
        return q, k, dq.to(dt), dk.to(dt), dwq.to(dt), dwk.to(dt)
    if s["new"] is not None:
        q = q.masked_fill((torch.arange(c["T"], device=q.device) >= s["new"][:, None])[:, :, None, None], 0)
    _write(k, s["k_cache"], s["k_scale"], s)
    _write(s["v"], s["v_cache"], s["v_scale"], s)
    return s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], q


def _run_own(s, c):
    import flashattention_backward_fa_gb300 as fa

    if c["op"] == "cross":
        lens = dict(q_lens=s["q_lens"], k_lens=s["k_lens"])
        o, lse = fa.cross_attention_forward(s["q"], s["k"], s["v"], **lens)
        if not c["grad"]:
            return o, lse
        return (o, lse) + tuple(fa.cross_attention_backward(s["q"], s["k"], s["v"], o, s["do"], lse, **lens))
    how = dict(eps=EPS, interleaved=c["interleaved"], positions=s["pos"], axes=s["axes"])
    if c["op"] == "rotate":
        args = (s["wq"], s["wk"], s["cos"], s["sin"])
        q, k = fa.qk_norm_rope_forward(s["q"], s["k"], *args, **how)
        if not c["grad"]:
            return q, k
        return (q, k) + tuple(fa.qk_norm_rope_backward(s["q"], s["k"], s["dq"], s["dk"], *args, **how))
    cache = fa.Kv8Cache(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"])
    q = fa.kv8_norm_rope_append(cache, s["q"], s["k"], s["v"], s["wq"], s["wk"], s["cos"], s["sin"], s["table"],
                                s["lens"], new_lens=s["new"], **how)
    return cache.k, cache.v, cache.k_scale, cache.v_scale, q


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    c = case
    size, d, Hq, Hkv = (4 if c["dtype"] == "f32" else 2), c["d"], c["Hq"], c["Hkv"]
    if c["op"] == "cross":
        ql, kl = _cross_lengths(c)
        q, k = sum(ql) * Hq * d * size, sum(kl) * Hkv * d * size
        pairs = sum(a * b for a, b in zip(ql, kl))
        # q, k, v in, o out; with the backward pass the gradient of o in, those of q, k, v out
        return dict(bytes=2 * q + 2 * k + 4 * sum(ql) * Hq + (2 * q + 2 * k if c["grad"] else 0),
                    flops=(14 if c["grad"] else 4) * pairs * Hq * d)
    pairs = sum(int(n) for n in c["sections"].split(","))
    axes = c["sections"].count(",") + 1
    if c["op"] == "rotate":
        tokens = c["B"] * c["N"]
        rows = tokens * (Hq + Hkv)
        # the rows of the tables that are read are few: one for each place on each axis
        small = 4 * axes * (tokens if c["each"] else c["N"]) + 2 * d * size
        return dict(bytes=(4 if c["grad"] else 2) * rows * d * size + small, flops=(27 if c["grad"] else 9) * rows * d)
    tokens = sum(_step_lengths(c)[1])
    return dict(bytes=2 * tokens * Hkv * d * (size + 1) + 2 * tokens * Hq * d * size + 4 * axes * tokens + 8 * pairs,
                flops=6 * tokens * Hkv * d + 9 * tokens * (Hq + Hkv) * d)


# ---------------------------------------------------------------- the definitions in 64 bits
def _exact_cross(c, s):
    ql, kl = _cross_lengths(c)
    B, Nq, Hq, d = s["q"].shape
    G = Hq // c["Hkv"]
    zeros = lambda x: torch.zeros(x.shape, device="cuda", dtype=torch.float64)  # noqa: E731
    o, lse = zeros(s["q"]), torch.full((B, Hq, Nq), -math.inf, device="cuda", dtype=torch.float64)
    dq, dk, dv = zeros(s["q"]), zeros(s["k"]), zeros(s["v"])
    for b, (n, m) in enumerate(zip(ql, kl)):
        for h in range(Hq):
            q, k, v = s["q"][b, :n, h].double(), s["k"][b, :m, h // G].double(), s["v"][b, :m, h // G].double()
            sc = torch.einsum("id,jd->ij", q, k) / math.sqrt(d)
            lse[b, h, :n] = sc.logsumexp(-1)
            p = sc.softmax(-1)
            o[b, :n, h] = p @ v
            if not c["grad"]:
                continue
            do = s["do"][b, :n, h].double()
            dv[b, :m, h // G] += p.T @ do
            dp = do @ v.T
            ds = p * (dp - (p * dp).sum(-1, keepdim=True)) / math.sqrt(d)
            dq[b, :n, h] = ds @ k
            dk[b, :m, h // G] += ds.T @ q
    return (o, lse, dq, dk, dv) if c["grad"] else (o, lse)


def _exact_rotated(x, w, pos, s, interleaved):
    """x [.., n, H, d], pos [n, axes]: pair by pair."""
    x = x.double()
    y = x / (x.square().mean(-1, keepdim=True) + EPS).sqrt() * w.double()
    out = y.clone()
    pairs = len(s["axes"])
    for i, axis in enumerate(s["axes"]):
        ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + pairs)
        at = pos[:, axis].long()
        cos, sin = s["cos"][at, i].double()[:, None], s["sin"][at, i].double()[:, None]
        out[..., ia] = y[..., ia] * cos - y[..., ib] * sin
        out[..., ib] = y[..., ib] * cos + y[..., ia] * sin
    return out


def _round_e4m3(x):
    """Nearest e4m3 value (ties to even), for |x| <= 448."""
    _, e = torch.frexp(x)
    step = torch.exp2((e - 1).clamp(min=-6).double() - 3)
    return (x / step).round() * step


def exact(case, seed):
    c, s = case, prepare(case, seed)
    dt, il = DTYPES[c["dtype"]], c["interleaved"] if c["op"] != "cross" else False
    if c["op"] == "cross":
        return _exact_cross(c, s)
    if c["op"] == "rotate":
        leaf = {n: s[n].double().requires_grad_(c["grad"]) for n in ("q", "k", "wq", "wk")}
        out = []
        for x, w in (("q", "wq"), ("k", "wk")):
            out.append(torch.stack([_exact_rotated(leaf[x][b], leaf[w], s["pos"][b] if c["each"] else s["pos"], s, il)
                                    for b in range(c["B"])]))
        if not c["grad"]:
            return tuple(out)
        return tuple(o.detach() for o in out) + torch.autograd.grad(out, tuple(leaf.values()),
                                                                    (s["dq"].double(), s["dk"].double()))
    lens, new = _step_lengths(c)
    page, H = c["page"], c["Hkv"]
    out = {}
    q, k = torch.zeros(s["q"].shape, device="cuda", dtype=torch.float64), s["k"].double()
    for b, w in enumerate(new):
        q[b, :w] = _exact_rotated(s["q"][b, :w], s["wq"], s["pos"][b, :w], s, il)
        k[b, :w] = _exact_rotated(s["k"][b, :w], s["wk"], s["pos"][b, :w], s, il).to(dt).double()
    for name, x in (("k", k), ("v", s["v"].double())):
        codes, scale = s[name + "_cache"].double(), s[name + "_scale"].double()
        for b, (n, w) in enumerate(zip(lens, new)):
            # the pages that the new tokens reach, as rows [pages, page, H, d], earlier tokens by their values
            p0, p1 = (n - w) // page, -(-n // page)
            at = s["table"][b, p0:p1].long()
            rows = torch.zeros(((p1 - p0) * page, H, c["d"]), device="cuda", dtype=torch.float64)
            head = (n - w) - p0 * page
            rows[head:head + w] = x[b, :w]
            amax = rows.unflatten(0, (-1, page)).abs().amax((1, 3))
            e = torch.log2(amax.clamp(min=2.0 ** (E_MIN + 8)) / 448).round()
            e = torch.where(448 * torch.exp2(e) < amax, e + 1, e)  # a logarithm alone may miss the border
            e = torch.where(448 * torch.exp2(e - 1) >= amax, e - 1, e).clamp(min=E_MIN)
            sc = torch.exp2(e)
            if head:
                sc[0] = torch.maximum(sc[0], scale[at[0]])
                rows[:head] = codes[at[0], :head] * scale[at[0]][:, None]
            fresh = _round_e4m3(rows.unflatten(0, (-1, page)) / sc[:, None, :, None]).flatten(0, 1)
            was = codes[at].flatten(0, 1)
            was[:head + w] = fresh[:head + w]
            codes[at] = was.unflatten(0, (-1, page))
            scale[at] = sc
        out[name] = codes, scale
    return out["k"][0], out["v"][0], out["k"][1], out["v"][1], q

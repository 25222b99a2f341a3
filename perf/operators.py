"""Timed cases of the query/key norm-and-rotation operators and of the 8-bit key/value cache.

Five operators, each as a user's program calls it:

* ``norm_rope``        per-head RMS norm of queries and keys and their rotation by position
                       (``qk_norm_rope_forward``);
* ``norm_rope_grad``   the same with its backward pass: outputs, gradients of q, k and of the two
                       weight vectors (``qk_norm_rope_forward`` + ``qk_norm_rope_backward``);
* ``append``           new keys and values into the paged e4m3 cache (``kv8_append``);
* ``step``             norm and rotation of new queries and keys, keys and values into the cache
                       (``kv8_norm_rope_append``);
* ``attention``        attention of the newest tokens over the cache (``kv8_attention``).

With ``own`` false, ``run`` computes them from elementary torch operations in 32 bits.

Definitions. Norm and rotation: y = w * x / sqrt(mean(x^2) + eps); pairs (a, b) of the first
``rot`` values of y become (a cos - b sin, b cos + a sin), the pair partners being ``rot / 2``
apart, or neighbours where ``interleaved``. Cache: page p, token slot t, head h hold e4m3 codes of
x / scale[p, h] with scale = 2^e, e the least integer with amax <= 448 * 2^e (amax: largest finite
magnitude of the tokens that a call brings to the page), and never less than the page's former
scale when the page holds earlier tokens, which are rounded anew to the larger scale. A sequence's
``seq_lens`` entry counts the call's new tokens, the last ``new_lens`` of it.
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
        # A toy-sized single-precision training step: nothing but latency.
        dict(name="norm_rope_f32_1x1x128x64", op="norm_rope", B=1, N=128, Hq=1, Hkv=1, d=64, rot=64,
             interleaved=False, dtype="f32", packed=False),
        # The benchmark's headline attention shape, before its forward.
        dict(name="norm_rope_bf16_1x32x8192x128", op="norm_rope", B=1, N=8192, Hq=32, Hkv=32, d=128, rot=128,
             interleaved=False, dtype="bf16", packed=False),
        # The benchmark's training batch, with its backward.
        dict(name="grad_bf16_4x16x2048x128", op="norm_rope_grad", B=4, N=2048, Hq=16, Hkv=16, d=128, rot=128,
             interleaved=False, dtype="bf16", packed=False),
        # Shared key heads, an odd length, rotation of half the head in neighbouring pairs, q and k as
        # slices of one packed projection.
        dict(name="grad_f16_2x16x4095x64_partial", op="norm_rope_grad", B=2, N=4095, Hq=16, Hkv=4, d=64, rot=32,
             interleaved=True, dtype="f16", packed=True),
        # A long prompt going into the cache.
        dict(name="append_bf16_prompt_1x32x8192x128", op="append", B=1, T=8192, L=8192, Hq=32, Hkv=32, d=128, page=64,
             dtype="bf16", ragged=False),
        # A batch of prompts of unequal lengths, each behind a prefix that ends inside a page.
        dict(name="append_f16_ragged_6x4x777x64", op="append", B=6, T=777, L=1999, Hq=4, Hkv=4, d=64, page=16,
             dtype="f16", ragged=True),
        # One new token for each of 32 sequences: what a serving loop does before each attention.
        dict(name="step_bf16_token_32x32x128", op="step", B=32, T=1, L=4097, Hq=32, Hkv=8, d=128, rot=128,
             interleaved=False, page=64, dtype="bf16", ragged=True),
        # A prompt of 2048 tokens for each of 4 sequences.
        dict(name="step_bf16_prompt_4x16x2048x128", op="step", B=4, T=2048, L=2048, Hq=16, Hkv=16, d=128, rot=128,
             interleaved=False, page=64, dtype="bf16", ragged=False),
        # The start of an answer: one sequence, a hundred tokens.
        dict(name="attn_bf16_token_1x16_len100", op="attention", B=1, T=1, L=100, Hq=16, Hkv=16, d=128, page=16,
             dtype="bf16", ragged=False, window=0),
        # One sequence with a very long context, shared key heads.
        dict(name="attn_bf16_token_1x32_len131071", op="attention", B=1, T=1, L=131071, Hq=32, Hkv=8, d=128, page=64,
             dtype="bf16", ragged=False, window=0),
        # A serving batch of unequal lengths.
        dict(name="attn_bf16_token_32x32_len16384", op="attention", B=32, T=1, L=16384, Hq=32, Hkv=8, d=128, page=64,
             dtype="bf16", ragged=True, window=0),
        # Five drafted tokens checked at once, sliding window, no shared heads, small head dimension.
        dict(name="attn_f16_draft5_16x16_len4097_window", op="attention", B=16, T=5, L=4097, Hq=16, Hkv=16, d=64,
             page=32, dtype="f16", ragged=True, window=1024),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["norm_rope", "norm_rope_grad", "append", "step", "attention", "attention"])
    d = rng.choice([64, 128])
    dtype = rng.choice(["bf16", "bf16", "f16"])
    Hkv = rng.choice([1, 2, 4, 8, 16])
    Hq = Hkv * rng.choice([1, 2, 3, 4, 8])
    if op in ("norm_rope", "norm_rope_grad"):
        B = _log(rng, 1, 8)
        N = _log(rng, 1, max(1, 8192 * 32 * 64 // (B * (Hq + Hkv) * d)))
        return dict(op=op, B=B, N=min(N, 16384), Hq=Hq, Hkv=Hkv, d=d, rot=rng.choice([d, d, d // 2, 16]),
                    interleaved=rng.random() < 0.3, dtype=rng.choice([dtype, dtype, dtype, "f32"]),
                    packed=rng.random() < 0.5)
    page = rng.choice([16, 32, 64, 128])
    if op == "append":
        B = _log(rng, 1, 32)
        T = _log(rng, 1, max(1, 8192 * 16 // (B * Hkv)))
        T = min(T, 8192)
        return dict(op=op, B=B, T=T, L=T + _log(rng, 1, 2000), Hq=Hkv, Hkv=Hkv, d=d, page=page, dtype=dtype,
                    ragged=rng.random() < 0.5)
    if op == "step":
        B = _log(rng, 1, 64)
        T = 1 if rng.random() < 0.5 else min(2048, _log(rng, 1, max(1, 8192 * 16 // (B * Hq))))
        return dict(op=op, B=B, T=T, L=T + _log(rng, 1, 4000), Hq=Hq, Hkv=Hkv, d=d, rot=rng.choice([d, d, d // 2]),
                    interleaved=rng.random() < 0.3, page=page, dtype=dtype, ragged=rng.random() < 0.5)
    B = _log(rng, 1, 64)
    T = rng.choice([1, 1, 1, 1, 2, 3, 4, 8])
    # no more cached bytes and no more products than the largest listed cases
    L = _log(rng, 8, max(9, min(131072, 16 * 16384 * 8 * 128 // (B * Hkv * d), 16 * 16384 * 32 * 128 // (B * T * Hq * d))))
    return dict(op=op, B=B, T=T, L=max(L, T), Hq=Hq, Hkv=Hkv, d=d, page=page, dtype=dtype, ragged=rng.random() < 0.5,
                window=_log(rng, 16, 4096) if rng.random() < 0.2 else 0)


def _lengths(c):
    """(tokens of each sequence with the new ones, new tokens of each): a fixed spread over the range."""
    B, T, L = c["B"], c["T"], c["L"]
    if not c["ragged"]:
        return [L] * B, [T] * B
    new = [T - int(0.4 * T * math.modf(0.381966 * b)[0]) for b in range(B)]
    lens = [max(n, int(L * (1 - 0.95 * math.modf(0.618034 * b)[0]))) for b, n in enumerate(new)]
    return lens, new


# ---------------------------------------------------------------- inputs
def _tables(rows, rot):
    ang = torch.arange(rows, device="cuda", dtype=torch.float64)[:, None] * torch.pow(
        10000.0, -torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
    return ang.cos().float(), ang.sin().float()


def _activations(g, shape, dtype):
    """Values as a projection gives them: unit spread, a few channels much larger than the rest."""
    x = torch.randn(shape, generator=g, device="cuda")
    x *= 1 + 3 * (torch.rand(shape[-1], generator=g, device="cuda") < 0.03)
    return x.to(dtype)


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
    dt, d, Hq, Hkv = DTYPES[c["dtype"]], c["d"], c["Hq"], c["Hkv"]
    s = dict(case=c)
    if "rot" in c:
        rows = c["N"] if "N" in c else c["L"]
        s["cos"], s["sin"] = _tables(rows, c["rot"])
        s["wq"] = (1 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(dt)
        s["wk"] = (1 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(dt)
    if c["op"] in ("norm_rope", "norm_rope_grad"):
        B, N = c["B"], c["N"]
        if c["packed"]:  # q, k and v side by side in one projection's output
            qkv = _activations(g, (B, N, Hq + 2 * Hkv, d), dt)
            s["q"], s["k"] = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv]
        else:
            s["q"], s["k"] = _activations(g, (B, N, Hq, d), dt), _activations(g, (B, N, Hkv, d), dt)
        if c["op"] == "norm_rope_grad":
            s["dq"] = torch.randn((B, N, Hq, d), generator=g, device="cuda").to(dt)
            s["dk"] = torch.randn((B, N, Hkv, d), generator=g, device="cuda").to(dt)
        return s
    lens, new = _lengths(c)
    page, B, T = c["page"], c["B"], c["T"]
    need = [-(-n // page) for n in lens]
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=g, device="cuda", dtype=torch.int32)
    table = torch.full((B, max(need)), -1, device="cuda", dtype=torch.int32)
    at = torch.tensor(need, device="cuda")
    held = torch.arange(max(need), device="cuda")[None] < at[:, None]
    table[held] = order[:sum(need)]
    s["k_cache"], s["k_scale"] = _new_cache(g, pages, page, Hkv, d)
    s["v_cache"], s["v_scale"] = _new_cache(g, pages, page, Hkv, d)
    s["table"] = table
    s["lens"] = torch.tensor(lens, device="cuda", dtype=torch.int32)
    s["new"] = torch.tensor(new, device="cuda", dtype=torch.int32) if c["ragged"] else None
    if c["op"] in ("append", "step"):
        s["k"], s["v"] = _activations(g, (B, T, Hkv, d), dt), _activations(g, (B, T, Hkv, d), dt)
    if c["op"] in ("step", "attention"):
        s["q"] = _activations(g, (B, T, Hq, d), dt)
    return s


# ---------------------------------------------------------------- plain forms
def _pairs(y, rot, interleaved):
    if interleaved:
        return y[..., 0:rot:2], y[..., 1:rot:2]
    return y[..., :rot // 2], y[..., rot // 2:rot]


def _join(a, b, rest, interleaved):
    if interleaved:
        return torch.cat([torch.stack([a, b], -1).flatten(-2), rest], -1)
    return torch.cat([a, b, rest], -1)


def _norm_rope(x, w, cos, sin, rot, interleaved):
    """x [B, N, H, d], cos / sin [B or 1, N, 1, rot / 2]: the rotated values in fp32."""
    x = x.float()
    y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.float()
    a, b = _pairs(y, rot, interleaved)
    return _join(a * cos - b * sin, b * cos + a * sin, y[..., rot:], interleaved)


def _norm_rope_grad(x, dout, w, cos, sin, rot, interleaved):
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
    amax = torch.where(x.isfinite(), x.abs(), 0).amax(-1)
    # largest new magnitude of each (page, head); pages that hold earlier tokens keep their scale at least
    most = torch.full_like(scale, -1).index_reduce_(0, at, amax, "amax")
    grown = _pow2_scale(most.clamp(min=0))
    first = s["table"].gather(1, (start // page).clamp(max=s["table"].shape[1] - 1)[:, None])[:, 0].long().clamp(min=0)
    old = torch.full_like(scale, -1)
    begun = (start % page != 0)[:, None]
    old[first] = torch.where(begun, scale[first], old[first])
    grown = torch.maximum(grown, old)
    fresh = torch.where(most >= 0, grown, scale)
    # earlier tokens of the page in which the new ones begin
    kept = (torch.arange(page, device=x.device) < (start % page)[:, None])[:, :, None, None]
    was = cache[first]
    again = (was.float() * (scale[first] / fresh[first])[:, None, :, None]).to(cache.dtype)
    cache.view(torch.uint8)[first] = torch.where(kept, again.view(torch.uint8), was.view(torch.uint8))
    cache.view(torch.uint8)[at, slot] = (x / fresh[at][:, :, None]).to(cache.dtype).view(torch.uint8)
    scale.copy_(fresh)


def _attention(s):
    c, q = s["case"], s["q"].float()
    B, T, Hq, d = q.shape
    H, table, lens = c["Hkv"], s["table"].clamp(min=0).long(), s["lens"].long()
    k = (s["k_cache"][table].float() * s["k_scale"][table][:, :, None, :, None]).flatten(1, 2)
    v = (s["v_cache"][table].float() * s["v_scale"][table][:, :, None, :, None]).flatten(1, 2)
    new = s["new"].long() if s["new"] is not None else torch.full_like(lens, T)
    i = ((lens - new)[:, None] + torch.arange(T, device=q.device))[:, :, None]
    j = torch.arange(k.shape[1], device=q.device)
    keep = (j <= i) & (torch.arange(T, device=q.device)[:, None] < new[:, None, None])
    if c["window"]:
        keep = keep & (j > i - c["window"])
    keep = keep[:, None, None]  # [B, 1, 1, T, keys]
    qg = q.view(B, T, H, Hq // H, d).permute(0, 2, 3, 1, 4)
    sc = (qg.flatten(2, 3) @ k.permute(0, 2, 3, 1)).unflatten(2, (Hq // H, T)) / math.sqrt(d)
    sc = sc.masked_fill(~keep, -math.inf)
    m = sc.amax(-1, keepdim=True).clamp(min=-1e30)
    p = (sc - m).exp()
    l = p.sum(-1, keepdim=True)
    o = (p.flatten(2, 3) @ v.permute(0, 2, 1, 3)).unflatten(2, (Hq // H, T)) / torch.where(l > 0, l, 1)
    lse = (m + l.log())[..., 0]
    return o.permute(0, 3, 1, 2, 4).reshape(B, T, Hq, d).to(s["q"].dtype), lse.reshape(B, Hq, T)


def _positions(s):
    """Positions [B, T] of new tokens and which rows hold one."""
    c = s["case"]
    t = torch.arange(c["T"], device="cuda")
    new = s["new"] if s["new"] is not None else torch.full_like(s["lens"], c["T"])
    live = t < new[:, None]
    return torch.where(live, (s["lens"] - new)[:, None] + t, 0).long(), live


def run(state):
    s, c = state, state["case"]
    if own:
        return _run_own(s, c)
    if c["op"] in ("norm_rope", "norm_rope_grad"):
        N, rot, il, dt = c["N"], c["rot"], c["interleaved"], s["q"].dtype
        cos, sin = s["cos"][None, :N, None], s["sin"][None, :N, None]
        q, k = (_norm_rope(s[x], s[w], cos, sin, rot, il).to(dt) for x, w in (("q", "wq"), ("k", "wk")))
        if c["op"] == "norm_rope":
            return q, k
        dq, dwq = _norm_rope_grad(s["q"], s["dq"], s["wq"], cos, sin, rot, il)
        dk, dwk = _norm_rope_grad(s["k"], s["dk"], s["wk"], cos, sin, rot, il)
        return q, k, dq.to(dt), dk.to(dt), dwq.to(dt), dwk.to(dt)
    if c["op"] == "attention":
        return _attention(s)
    q, k = None, s.get("k")
    if c["op"] == "step":
        pos, live = _positions(s)
        cos, sin = s["cos"][pos][:, :, None], s["sin"][pos][:, :, None]
        q, k = (_norm_rope(s[x], s[w], cos, sin, c["rot"], c["interleaved"]).to(s["k"].dtype)
                for x, w in (("q", "wq"), ("k", "wk")))
        q = q.masked_fill(~live[:, :, None, None], 0)
    _write(k, s["k_cache"], s["k_scale"], s)
    _write(s["v"], s["v_cache"], s["v_scale"], s)
    out = (s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"])
    return out if q is None else out + (q,)


def _run_own(s, c):
    import flashattention_backward_fa_gb300 as fa

    if c["op"] in ("norm_rope", "norm_rope_grad"):
        args = (s["wq"], s["wk"], s["cos"], s["sin"])
        q, k = fa.qk_norm_rope_forward(s["q"], s["k"], *args, eps=EPS, interleaved=c["interleaved"])
        if c["op"] == "norm_rope":
            return q, k
        return (q, k) + tuple(fa.qk_norm_rope_backward(s["q"], s["k"], s["dq"], s["dk"], *args, eps=EPS,
                                                       interleaved=c["interleaved"]))
    cache = fa.Kv8Cache(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"])
    if c["op"] == "attention":
        return fa.kv8_attention(s["q"], cache, s["table"], s["lens"], c["L"], new_lens=s["new"], window=c["window"])
    if c["op"] == "append":
        fa.kv8_append(cache, s["k"], s["v"], s["table"], s["lens"], new_lens=s["new"])
        return cache.k, cache.v, cache.k_scale, cache.v_scale
    q = fa.kv8_norm_rope_append(cache, s["q"], s["k"], s["v"], s["wq"], s["wk"], s["cos"], s["sin"], s["table"],
                                s["lens"], new_lens=s["new"], eps=EPS, interleaved=c["interleaved"])
    return cache.k, cache.v, cache.k_scale, cache.v_scale, q


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    c = case
    size, d, Hq, Hkv = (4 if c["dtype"] == "f32" else 2), c["d"], c["Hq"], c["Hkv"]
    if c["op"] in ("norm_rope", "norm_rope_grad"):
        rows = c["B"] * c["N"] * (Hq + Hkv)
        table = c["N"] * c["rot"] * 4
        if c["op"] == "norm_rope":
            return dict(bytes=2 * rows * d * size + table + 2 * d * size, flops=9 * rows * d)
        # forward: x in, out out; backward: x and dout in, dx out (x counted once over both)
        return dict(bytes=4 * rows * d * size + table + 4 * d * size, flops=27 * rows * d)
    lens, new = _lengths(c)
    if c["op"] == "attention":
        keys = sum(min(n, c["window"] + w - 1) if c["window"] else n for n, w in zip(lens, new))
        pages = sum(-(-n // c["page"]) for n in lens)
        rows = sum(new) * Hq
        pairs = sum(sum(min(n - w + t + 1, c["window"] or n) for t in range(w)) for n, w in zip(lens, new))
        return dict(bytes=2 * keys * Hkv * d + 8 * pages * Hkv + 4 * pages + 2 * rows * d * size + 4 * rows,
                    flops=4 * pairs * Hq * d)
    tokens = sum(new)
    b = 2 * tokens * Hkv * d * (size + 1)
    f = 2 * 3 * tokens * Hkv * d
    if c["op"] == "step":
        b += 2 * tokens * Hq * d * size + tokens * c["rot"] * 4
        f += 9 * tokens * (Hq + Hkv) * d
    return dict(bytes=b, flops=f)


# ---------------------------------------------------------------- the definitions in 64 bits
def _round_e4m3(x):
    """Nearest e4m3 value (ties to even), for |x| <= 448."""
    _, e = torch.frexp(x)
    step = torch.exp2((e - 1).clamp(min=-6).double() - 3)
    return (x / step).round() * step


def _exact_rotated(x, w, ang_rows, c, dt, s):
    x = x.double()
    y = x / (x.square().mean(-1, keepdim=True) + EPS).sqrt() * w.double()
    h = c["rot"] // 2
    cos, sin = s["cos"].double()[ang_rows].unsqueeze(-2), s["sin"].double()[ang_rows].unsqueeze(-2)
    ia = torch.arange(h, device=x.device) * (2 if c["interleaved"] else 1)
    ib = ia + (1 if c["interleaved"] else h)
    out = y.clone()
    out[..., ia] = y[..., ia] * cos - y[..., ib] * sin
    out[..., ib] = y[..., ib] * cos + y[..., ia] * sin
    return out


def exact(case, seed):
    c, s = case, prepare(case, seed)
    dt = DTYPES[c["dtype"]]
    if c["op"] in ("norm_rope", "norm_rope_grad"):
        rows = torch.arange(c["N"], device="cuda")
        q, k, wq, wk = (s[n].double().requires_grad_(c["op"] == "norm_rope_grad") for n in ("q", "k", "wq", "wk"))
        out = _exact_rotated(q, wq, rows, c, dt, s), _exact_rotated(k, wk, rows, c, dt, s)
        if c["op"] == "norm_rope":
            return out
        return tuple(o.detach() for o in out) + torch.autograd.grad(out, (q, k, wq, wk),
                                                                    (s["dq"].double(), s["dk"].double()))
    lens, new = _lengths(c)
    page, H = c["page"], c["Hkv"]
    if c["op"] == "attention":
        o = torch.zeros(s["q"].shape, device="cuda", dtype=torch.float64)
        lse = torch.full((c["B"], c["Hq"], c["T"]), -math.inf, device="cuda", dtype=torch.float64)
        for b, (n, w) in enumerate(zip(lens, new)):
            at = s["table"][b, :-(-n // page)].long()
            k, v = ((s[x + "_cache"][at].double() * s[x + "_scale"][at].double()[:, None, :, None]).flatten(0, 1)[:n]
                    for x in ("k", "v"))
            j = torch.arange(n, device="cuda")
            i = torch.arange(n - w, n, device="cuda")[:, None]
            hide = j > i
            if c["window"]:
                hide = hide | (j <= i - c["window"])
            for h in range(H):
                for hq in range(h * (c["Hq"] // H), (h + 1) * (c["Hq"] // H)):
                    sc = (s["q"][b, :w, hq].double() @ k[:, h].T / math.sqrt(c["d"])).masked_fill(hide, -math.inf)
                    lse[b, hq, :w] = sc.logsumexp(-1)
                    o[b, :w, hq] = sc.softmax(-1) @ v[:, h]
        return o, lse
    out = {}
    q, k = None, s["k"].double()
    if c["op"] == "step":
        q = torch.zeros(s["q"].shape, device="cuda", dtype=torch.float64)
        for b, (n, w) in enumerate(zip(lens, new)):
            rows = torch.arange(n - w, n, device="cuda")
            q[b, :w] = _exact_rotated(s["q"][b, :w], s["wq"], rows, c, dt, s)
            k[b, :w] = _exact_rotated(s["k"][b, :w], s["wk"], rows, c, dt, s).to(dt).double()
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
    res = (out["k"][0], out["v"][0], out["k"][1], out["v"][1])
    return res if q is None else res + (q,)

"""Cross attention with chosen roundings of its operands, and the 2-norm in which they show.

Elementwise bounds (cross_reference) add every operand's largest rounding up without regard to sign, so they allow
ten times what roundings do in earnest, and an operand held coarser than the kernels promise passes them.
Here an output's distance from the definition is measured in units of what rounding the exact output to its
type costs: ``ratio`` = |x - ref| / |round(ref) - ref|, 1 where the output alone is rounded.

What the ratio is. Rounding errors are independent of each other and of the values' signs. The terms of
sum_j P_ij V_j, of random signs, have squares that add up to about the square of the sum; so an operand that is
rounded once to the outputs' type moves the sum about as much as rounding the sum does: ratio sqrt(1 + 1) = 1.41.
With its residual an operand has 16 bits or more and moves nothing: 1. Where terms cancel (a row's dS add up
to 0 and meet the keys' mean, channels that share a large spread) a rounded operand costs more, and so does D =
rowsum(dO o O) of a rounded O. The limits of the tests lie between the two values of the rounding that a case is
about, and test_cross_rounding_host.py holds each case to that with the operands rounded as the kernels do and
with that rounding made coarser.
"""
import math

import torch

BF16, F16 = torch.bfloat16, torch.float16


def activations(g, shape, dtype, big=4.0, shared=False):
    """Unit spread, a few channels (three in a hundred, two at least; shared: the first) `big` times as large."""
    x, n = torch.randn(shape, generator=g), max(2, shape[-1] * 3 // 100)
    x[..., torch.arange(n) if shared else torch.randperm(shape[-1], generator=g)[:n]] *= big
    return x.to(dtype)


# What a case is about: an output, the switch of `emulate` that makes it coarser, and the limit between, which the
# kernels stay under; then the inputs.
CASES = {
    # dQ takes dS with its residual
    "dq_channels": dict(off=("dq", "split_dq"), most=1.3, dtype=BF16, B=1, Nq=700, Nk=160, Hq=2, Hk=1, d=128),
    "dq_channels_f16": dict(off=("dq", "split_dq"), most=1.3, dtype=F16, B=1, Nq=700, Nk=160, Hq=2, Hk=1, d=128),
    # dK and dV take the residuals of dS and P: where a row is made up of a few keys, over some hundreds, and over many
    # of even weight
    "dk_hundreds": dict(off=("dk", "split_kv"), most=1.2, dtype=BF16, B=1, Nq=500, Nk=300, Hq=2, Hk=1, d=128),
    "dv_hundreds": dict(off=("dv", "split_kv"), most=1.2, dtype=F16, B=1, Nq=500, Nk=300, Hq=2, Hk=2, d=64),
    "dk_even": dict(off=("dk", "split_kv"), most=1.2, dtype=BF16, B=1, Nq=300, Nk=3000, Hq=2, Hk=2, d=64, sharp=0.2),
    "dv_even": dict(off=("dv", "split_kv"), most=1.15, dtype=F16, B=1, Nq=200, Nk=3000, Hq=2, Hk=1, d=128, sharp=0.2),
    "dk_sharp": dict(off=("dk", "split_kv"), most=1.2, dtype=BF16, B=1, Nq=300, Nk=64, Hq=2, Hk=2, d=64,
                     sharp=4.0),
    "dv_sharp": dict(off=("dv", "split_kv"), most=1.15, dtype=BF16, B=1, Nq=300, Nk=64, Hq=2, Hk=2, d=64,
                     sharp=4.0),
    # the forward multiplies P's residual: few rows a key head, tiles of them, tiles over split keys
    "few_rows": dict(off=("o", "split_o"), most=1.2, dtype=BF16, B=2, Nq=3, Nk=1000, Hq=4, Hk=2, d=128),
    "few_rows_f16": dict(off=("o", "split_o"), most=1.15, dtype=F16, B=2, Nq=1, Nk=1499, Hq=8, Hk=8, d=64),
    "tiles": dict(off=("o", "split_o"), most=1.15, dtype=BF16, B=2, Nq=300, Nk=512, Hq=2, Hk=2, d=128,
                  k_lens=[512, 77]),
    "tiles_f16": dict(off=("o", "split_o"), most=1.15, dtype=F16, B=1, Nq=200, Nk=300, Hq=4, Hk=1, d=64),
    "tiles_long": dict(off=("o", "split_o"), most=1.15, dtype=BF16, B=1, Nq=128, Nk=9000, Hq=2, Hk=2, d=64),
    # D comes from the scores, not from the rounded o: over few keys, alone or padded to many, where q, k and v share
    # large channels, and where a row is nearly all one key
    "d_of_short": dict(off=("dq", "d_scores"), most=1.35, dtype=BF16, B=4, Nq=300, Nk=512, Hq=2, Hk=2, d=64,
                       k_lens=[4, 8, 24, 60]),
    "d_of_short_f16": dict(off=("dq", "d_scores"), most=1.25, dtype=F16, B=4, Nq=150, Nk=300, Hq=2, Hk=1,
                           d=128, k_lens=[4, 8, 24, 40]),
    "d_of_short_only": dict(off=("dq", "d_scores"), most=1.3, dtype=BF16, B=3, Nq=300, Nk=40, Hq=2, Hk=1,
                            d=128, k_lens=[4, 8, 30]),
    "d_shared": dict(off=("dq", "d_scores"), most=1.3, dtype=BF16, B=2, Nq=260, Nk=1500, Hq=2, Hk=1, d=128,
                     k_lens=[1500, 333], shared=True),
    "d_shared_f16": dict(off=("dq", "d_scores"), most=1.3, dtype=F16, B=1, Nq=100, Nk=4000, Hq=2, Hk=2,
                         d=64, shared=True),
    "d_sharp": dict(off=("dk", "d_scores"), most=1.3, dtype=BF16, B=1, Nq=300, Nk=200, Hq=2, Hk=2, d=64,
                    sharp=8.0),
    # fp16: dS of small upstream gradients over many keys, and P of many keys, below fp16's normal values
    "dq_small": dict(off=("dq", "scaled"), most=1.3, dtype=F16, B=1, Nq=200, Nk=4096, Hq=2, Hk=1, d=128,
                     do=1e-3),
    "dk_small": dict(off=("dk", "scaled"), most=1.3, dtype=F16, B=1, Nq=200, Nk=4096, Hq=2, Hk=1, d=128,
                     do=1e-3),
    "dq_tiny": dict(off=("dq", "scaled"), most=1.3, dtype=F16, B=2, Nq=70, Nk=5000, Hq=2, Hk=2, d=64,
                    do=1e-4, k_lens=[5000, 4097]),
    "dk_tiny": dict(off=("dk", "scaled"), most=1.3, dtype=F16, B=2, Nq=70, Nk=5000, Hq=2, Hk=2, d=64,
                    do=1e-4, k_lens=[5000, 4097]),
    "dv_long": dict(off=("dv", "scaled"), most=1.3, dtype=F16, B=1, Nq=130, Nk=40000, Hq=1, Hk=1, d=64,
                    sharp=0.1),
    # rows of unlike upstream gradients: each row of dQ by itself
    "dq_rows_apart": dict(off=("dq", "scaled"), most=1.5, rows=True, dtype=F16, B=1, Nq=64, Nk=64, Hq=4,
                          Hk=4, d=64, spread=13),
}


def inputs(case, seed=0):
    c, g = case, torch.Generator().manual_seed(seed)
    B, Nq, Nk, Hq, Hk, d, t = (c[n] for n in ("B", "Nq", "Nk", "Hq", "Hk", "d", "dtype"))
    shared = c.get("shared", False)
    q = (activations(g, (B, Nq, Hq, d), torch.float32, shared=shared) * c.get("sharp", 1.0)).to(t)
    k, v = (activations(g, (B, Nk, Hk, d), t, shared=shared) for _ in range(2))
    do = torch.randn((B, Nq, Hq, d), generator=g) * c.get("do", 1.0)
    if "spread" in c:  # the first row's as it is, the last one's 2^-spread of it
        do = do * torch.exp2(-torch.linspace(0, c["spread"], Nq))[:, None, None]
    return q, k, v, do.to(t)


def short(x, dtype):
    """Rounded to the type, as a float64."""
    return x.float().to(dtype).double()


def operand(x, dtype, split):
    hi = short(x, dtype)
    return hi + short(x - hi, dtype) if split else hi


def exponent(bound):
    """e with bound * 2^e in [2^14, 2^15)."""
    return 14 - torch.floor(torch.log2(torch.clamp(bound, min=2.0 ** -100)))


def heads(q, k, q_lens, k_lens):
    G = q.shape[2] // k.shape[2]
    for b in range(q.shape[0]):
        n = q.shape[1] if q_lens is None else int(q_lens[b])
        m = k.shape[1] if k_lens is None else int(k_lens[b])
        if n and m:
            for h in range(q.shape[2]):
                yield b, n, m, h, h // G


def softmax(q, k, scale):
    s = scale * q @ k.T
    return torch.softmax(s, -1)


def definition(q, k, v, do, q_lens=None, k_lens=None):
    """o, dq, dk, dv in float64, on the inputs' device."""
    q, k, v, do = (x.double() for x in (q, k, v, do))
    scale = 1 / math.sqrt(q.shape[-1])
    out = dict(o=torch.zeros_like(q), dq=torch.zeros_like(q), dk=torch.zeros_like(k), dv=torch.zeros_like(v))
    for b, n, m, h, j in heads(q, k, q_lens, k_lens):
        qq, kk, vv, g = q[b, :n, h], k[b, :m, j], v[b, :m, j], do[b, :n, h]
        p = softmax(qq, kk, scale)
        dp = g @ vv.T
        ds = p * (dp - (p * dp).sum(-1, keepdim=True))
        out["o"][b, :n, h] = p @ vv
        out["dq"][b, :n, h] = scale * ds @ kk
        out["dk"][b, :m, j] += scale * ds.T @ qq
        out["dv"][b, :m, j] += p.T @ g
    return out


def emulate(q, k, v, do, q_lens=None, k_lens=None, split_o=True, split_kv=True, split_dq=True, d_scores=True,
            scaled=True):
    """The same with operands in the tensors' type (split: with their residual), D from the scores or from the
    rounded o, and (fp16, scaled) operands brought into the type's range by powers of two: dS for dQ by row, dS
    for dK by key head, P for dV by 2^15."""
    t = q.dtype
    q, k, v, do = (x.double() for x in (q, k, v, do))
    scale = 1 / math.sqrt(q.shape[-1])
    out = dict(o=torch.zeros_like(q), dq=torch.zeros_like(q), dk=torch.zeros_like(k), dv=torch.zeros_like(v))
    scaled &= t is F16
    for b, n, m, h, j in heads(q, k, q_lens, k_lens):
        qq, kk, vv, g = q[b, :n, h], k[b, :m, j], v[b, :m, j], do[b, :n, h]
        p = softmax(qq, kk, scale)
        dp = g @ vv.T
        top = p.amax(-1, keepdim=True)
        o = short(operand(p / top, t, split_o) @ vv * top, t)
        D = (p * dp).sum(-1, keepdim=True) if d_scores else (g * o).sum(-1, keepdim=True)
        ds = p * (dp - D)
        bound = 2 * g.norm(dim=-1, keepdim=True) * vv.norm(dim=-1).max()
        row = torch.exp2(exponent(bound)) if scaled else 1.0
        all_ = torch.exp2(exponent(bound.max())) if scaled else 1.0
        one = 2.0 ** 15 if scaled else 1.0
        out["o"][b, :n, h] = o
        out["dq"][b, :n, h] = scale * operand(ds * row, t, split_dq) @ kk / row
        out["dk"][b, :m, j] += scale * operand(ds * all_, t, split_kv).T @ qq / all_
        out["dv"][b, :m, j] += operand(p * one, t, split_kv).T @ g / one
    return {n: short(x, t) for n, x in out.items()}


def ratio_of(case, x, ref):
    name = case["off"][0]
    return ratio(x[name], ref[name], case["dtype"], case.get("rows", False))


def ratio(x, ref, dtype, rows=False):
    """|x - ref| / |round(ref) - ref|; rows: the largest of the rows' (dim 1) own."""
    x = x.double()
    if rows:
        norm = lambda y: y.transpose(0, 1).flatten(1).norm(dim=1)  # noqa: E731
        return float((norm(x - ref) / norm(short(ref, dtype) - ref)).max())
    return float((x - ref).norm() / (short(ref, dtype) - ref).norm())

"""Cross attention in float64 on the CPU, from its definition, with bounds on what the kernels may be off by.

Bounds. u is half a step of the tensors' type (eps / 2). What is computed differs from the definition by

* the rounding of each result: u of it, and where it is subnormal in its type half a step of those (fp16 results
  below 2^-14 are multiples of 2^-24: 2^-25; bf16 and fp32 2^-126 has them at 2^-134 and less);
* P and dS as operands of a product in 16 bits: u of each (the kernels round finer where a probability is
  large, which only helps), and in fp16 half a step of its subnormals, 2^-25, where they are below 2^-14;
* fp32: a sum of n products is off by at most n 2^-24 of the sum of their magnitudes (a chain of n roundings;
  tensor cores add in no more steps), so a score by n 2^-24 scale sum |q k|, n = d + 8, and P by that much of
  itself and 2^-21 (exp2, log2 and the division, each a few 2^-24); sums over keys or queries by their number;
* the backward's D = rowsum(dO o O) takes the O that the forward rounded: off by u sum |dO O|, and by the
  fp32 sum's share; with 16-bit tensors of up to 64 keys it is sum P dP instead, off by what P and dP are and
  the fp32 sum's share.
"""
import math

import torch


def lengths(lens, B, N):
    return [N] * B if lens is None else [min(max(int(x), 0), N) for x in lens.tolist()]


class Reference:
    """Values and elementwise bounds of one call; gradients where `do` is given."""

    def __init__(self, q, k, v, q_lens=None, k_lens=None, scale=None, do=None):
        B, Nq, Hq, d = q.shape
        Nk, Hk = k.shape[1:3]
        G, scale = Hq // Hk, 1 / math.sqrt(d) if scale is None else scale
        f16 = q.dtype is torch.float16
        u = torch.finfo(q.dtype).eps / 2
        up = u if q.dtype is not torch.float32 else 0.0  # rounding of P and dS as operands
        sub = 2.0 ** -25 if f16 else 0.0
        q, k, v = (t.detach().cpu().double() for t in (q, k, v))
        do = None if do is None else do.detach().cpu().double()
        zeros = lambda t: torch.zeros(t.shape, dtype=torch.float64)  # noqa: E731
        self.o, self.lse = zeros(q), torch.full((B, Hq, Nq), -math.inf, dtype=torch.float64)
        self.o_tol, self.lse_tol = zeros(q), zeros(self.lse)
        self.dq, self.dk, self.dv, self.dq_tol, self.dk_tol, self.dv_tol = (zeros(t) for t in (q, k, v, q, k, v))
        e = 2.0 ** -24
        for b, (n, m) in enumerate(zip(lengths(q_lens, B, Nq), lengths(k_lens, B, Nk))):
            if n == 0 or m == 0:
                continue
            for h in range(Hq):
                qh, kh, vh = q[b, :n, h], k[b, :m, h // G], v[b, :m, h // G]
                s = scale * qh @ kh.T
                top = s.amax(-1, keepdim=True)
                p = (s - top).exp()
                total = p.sum(-1, keepdim=True)
                p = p / total
                self.lse[b, h, :n] = (top + total.log())[:, 0]
                self.o[b, :n, h] = p @ vh
                s_err = (d + 8) * e * scale * (qh.abs() @ kh.abs().T)
                p_rel = 2 * s_err.amax(-1, keepdim=True) + 2.0 ** -21  # its own score's error and the sum's
                self.lse_tol[b, h, :n] = p_rel[:, 0] + 2.0 ** -22 * (1 + self.lse[b, h, :n].abs())
                self.o_tol[b, :n, h] = u * self.o[b, :n, h].abs() + (up + p_rel + (m + 16) * e) * (p @ vh.abs()) + \
                    sub * vh.abs().sum(0)
                if do is None:
                    continue
                g = do[b, :n, h]
                dp = g @ vh.T
                D = (p * dp).sum(-1, keepdim=True)
                ds = p * (dp - D)
                self.dv[b, :m, h // G] += p.T @ g
                self.dq[b, :n, h] = scale * ds @ kh
                self.dk[b, :m, h // G] += scale * ds.T @ qh
                dp_err = (d + 8) * e * (g.abs() @ vh.abs().T)
                if up and Nk <= 64:
                    go = (p * dp_err + (p_rel + (Nk + 16) * e) * p * dp.abs()).sum(-1, keepdim=True)
                else:
                    go = (g.abs() * self.o_tol[b, :n, h]).sum(-1, keepdim=True) + \
                        (d + 8) * e * (g.abs() * self.o[b, :n, h].abs()).sum(-1, keepdim=True)
                ds_err = p * (go + dp_err) + ds.abs() * (up + p_rel) + sub
                rows, keys = (m + 16) * e, (n * G + 16) * e
                self.dq_tol[b, :n, h] = scale * (ds_err + rows * ds.abs()) @ kh.abs() + u * self.dq[b, :n, h].abs()
                self.dk_tol[b, :m, h // G] += scale * (ds_err + keys * ds.abs()).T @ qh.abs()
                self.dv_tol[b, :m, h // G] += ((up + p_rel + keys) * p + sub).T @ g.abs()
        self.dk_tol += u * self.dk.abs()
        self.dv_tol += u * self.dv.abs()

    def check_forward(self, o, lse):
        close("o", o, self.o, self.o_tol)
        close("lse", lse, self.lse, self.lse_tol)

    def check_backward(self, dq, dk, dv):
        for name, x in (("dq", dq), ("dk", dk), ("dv", dv)):
            close(name, x, getattr(self, name), getattr(self, name + "_tol"))


def close(name, x, ref, tol):
    tiny = 2.0 ** -25 if x.dtype is torch.float16 else 2.0 ** -126  # half a step of subnormal results
    x = x.detach().cpu().double()
    assert x.shape == ref.shape, name
    same = x == ref  # (infinities too)
    bad = ~same & ~((x - ref).abs() <= tol + tiny)
    if bad.any():
        at = tuple(bad.nonzero()[0].tolist())
        raise AssertionError(f"{name}: {int(bad.sum())} of {x.numel()} off, first at {at}: {x[at]} against {ref[at]}, "
                             f"tolerance {tol[at]}")

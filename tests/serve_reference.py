"""Plain float64 forms of the norm-and-rotation operators and of the 8-bit key/value cache, written
from their definitions with loops, on the CPU. The GPU tests compare with them."""
import math

import torch

E4M3_MAX = 448.0
MIN_EXP = -100


def f64(t):
    return None if t is None else t.detach().cpu().double()


def norm_rope(x, w, cos, sin, positions, eps, interleaved):
    """x [B, N, H, d] float64, positions [B, N] (long): norm, then rotation by the position's table row."""
    y = x / (x.square().mean(-1, keepdim=True) + eps).sqrt()
    if w is not None:
        y = y * w
    if cos is None or cos.shape[1] == 0:
        return y
    half = cos.shape[1]
    c, s = cos[positions][:, :, None], sin[positions][:, :, None]
    first = torch.arange(half) * 2 if interleaved else torch.arange(half)
    second = first + 1 if interleaved else first + half
    a, b = y[..., first], y[..., second]
    out = y.clone()
    out[..., first] = a * c - b * s
    out[..., second] = b * c + a * s
    return out


def round_e4m3(x):
    """Nearest e4m3 value of a finite x with |x| <= 448 (ties to even), as float64."""
    _, e = torch.frexp(x)
    step = torch.exp2((e - 1).clamp(min=-6).double() - 3)
    return (x / step).round() * step


def scale_of(amax):
    """Least power of two s >= 2^-100 with amax <= 448 s."""
    e = MIN_EXP
    if amax > E4M3_MAX * 2.0 ** MIN_EXP:
        e = math.frexp(amax / E4M3_MAX)[1] - 1
        while amax > E4M3_MAX * 2.0 ** e:
            e += 1
    return 2.0 ** e


class RefCache:
    """Codes (their values, float64) and scales, updated one new token page at a time."""

    def __init__(self, cache):
        self.codes = [f64(cache.k.cpu().float()), f64(cache.v.cpu().float())]
        self.scales = [f64(cache.k_scale), f64(cache.v_scale)]

    def append(self, k, v, table, seq_lens, new_lens):
        pages, page, H, _ = self.codes[0].shape
        B, T = k.shape[:2]
        for side, x in enumerate((k, v)):
            codes, scales = self.codes[side], self.scales[side]
            for b in range(B):
                n = T if new_lens is None else min(max(int(new_lens[b]), 0), T)
                start = int(seq_lens[b]) - n
                by_page = {}
                for t in range(n):
                    pos = start + t
                    if pos >= 0 and pos // page < table.shape[1]:
                        by_page.setdefault(pos // page, []).append((pos % page, t))
                for ordinal, tokens in by_page.items():
                    pid = int(table[b, ordinal])
                    if not 0 <= pid < pages:
                        continue
                    first = tokens[0][0]
                    for h in range(H):
                        rows = x[b, [t for _, t in tokens], h]
                        finite = rows[rows.isfinite()].abs()
                        s = scale_of(float(finite.max()) if finite.numel() else 0.0)
                        if first > 0:
                            s = max(s, float(scales[pid, h]))
                            codes[pid, :first, h] = round_e4m3(codes[pid, :first, h] * (float(scales[pid, h]) / s))
                        scales[pid, h] = s
                        q = torch.where(rows.isfinite(), rows / s, float("nan"))
                        codes[pid, [slot for slot, _ in tokens], h] = torch.where(
                            q.isnan(), q, round_e4m3(q.nan_to_num()))

    def attention(self, q, table, seq_lens, new_lens, max_seqlen, scale, causal=True, window=0, alibi=None):
        pages, page, H, d = self.codes[0].shape
        B, T, Hq, _ = q.shape
        o = torch.zeros(q.shape, dtype=torch.float64)
        lse = torch.full((B, Hq, T), -math.inf, dtype=torch.float64)
        for b in range(B):
            n = T if new_lens is None else min(max(int(new_lens[b]), 0), T)
            total = max(int(seq_lens[b]), 0)
            keys = min(total, max_seqlen, table.shape[1] * page)
            ids = table[b, :-(-keys // page)].long() if keys else table[b, :0].long()
            ok = ((ids >= 0) & (ids < pages)).repeat_interleave(page)[:keys]
            at = ids.clamp(0, pages - 1)
            k, v = ((self.codes[i][at] * self.scales[i][at][:, None, :, None]).flatten(0, 1)[:keys] for i in (0, 1))
            j = torch.arange(keys)
            for t in range(n):
                i = total - n + t
                if i < 0:
                    continue
                keep = ok.clone()
                if causal:
                    keep &= j <= i
                if window > 0:
                    keep &= j > i - window
                if not keep.any():
                    continue
                for hq in range(Hq):
                    h = hq // (Hq // H)
                    s = k[keep, h] @ q[b, t, hq] * scale
                    if alibi is not None:
                        m = float(alibi[hq] if alibi.dim() == 1 else alibi[b, hq])
                        s = s - m * (i - j[keep]).abs()
                    lse[b, hq, t] = s.logsumexp(0)
                    o[b, t, hq] = s.softmax(0) @ v[keep, h]
        return o, lse

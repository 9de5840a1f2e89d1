"""The 8-bit key/value cache in 64 bits, from its definition: plain torch on whatever device
its tensors are on, one sequence and one block at a time.  Shares no code with the library."""
from __future__ import annotations

import math

import numpy as np
import torch

BLOCK = 16
TOP = {"e4m3": 448.0, "int8": 127.0}
MIN_EXP = -100


def code_values(fmt: str) -> torch.Tensor:
    """The number that each of the 256 codes stands for (the two e4m3 NaN codes: nan)."""
    u = np.arange(256)
    if fmt == "int8":
        return torch.tensor(np.where(u < 128, u, u - 256).astype(np.float64))
    e, m = (u >> 3) & 15, u & 7
    mag = np.where(e == 0, m / 512.0, (8 + m) * 2.0 ** (e - 10.0))
    mag[[127, 255]] = np.nan
    return torch.tensor(np.where(u < 128, mag, -mag))


def nearest_code(y: torch.Tensor, fmt: str) -> torch.Tensor:
    """Codes of the representable numbers next to y (float64, in range), ties to the even one."""
    if fmt == "int8":
        return torch.round(y).to(torch.int64) % 256
    grid = code_values(fmt)[:127].to(y.device)
    a = y.abs().contiguous()
    hi = torch.searchsorted(grid, a).clamp(1, 126)
    lo = hi - 1
    up, down = grid[hi] - a, a - grid[lo]
    pick = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return pick + 128 * torch.signbit(y).to(torch.int64)


def scale_exp(amax: float, fmt: str) -> int:
    """The smallest e >= -100 with amax <= top * 2^e."""
    e = MIN_EXP
    if amax > 0:
        e = max(e, math.frexp(amax / TOP[fmt])[1] - 2)
    while amax > math.ldexp(TOP[fmt], e):
        e += 1
    return e


class RefCache:
    """codes uint8 and scales float64 as plain tensors, names as the library's wrapper."""

    def __init__(self, k, v, k_scale, v_scale, fmt):
        self.codes = {"k": k.clone(), "v": v.clone()}
        self.scales = {"k": k_scale.double().clone(), "v": v_scale.double().clone()}
        self.fmt = fmt
        self.page = k.shape[2]

    def append(self, table, lens, offsets, k, v):
        """k, v float64 [T, hkv, d]; table, lens, offsets: nested lists / arrays of ints."""
        of = code_values(self.fmt).to(k.device)
        for b in range(len(lens)):
            n = int(offsets[b + 1]) - int(offsets[b])
            first = int(lens[b]) - n
            if n == 0:
                continue
            for blk in range(first // BLOCK, (int(lens[b]) - 1) // BLOCK + 1):
                p0 = blk * BLOCK
                pg, at = int(table[b][p0 // self.page]), p0 % self.page
                lo, hi = max(first, p0), min(int(lens[b]), p0 + BLOCK)
                rows = slice(int(offsets[b]) + lo - first, int(offsets[b]) + hi - first)
                for name, x in (("k", k[rows]), ("v", v[rows])):
                    for h in range(x.shape[1]):
                        y = x[:, h]
                        fin = y[torch.isfinite(y)]
                        e = scale_exp(float(fin.abs().max()) if fin.numel() else 0.0, self.fmt)
                        sc, c = self.scales[name], self.codes[name]
                        if lo > p0:
                            old = float(sc[pg, h, at // BLOCK])
                            e = max(e, int(math.log2(old)))
                            if 2.0 ** e > old:
                                part = c[pg, h, at:at + lo - p0]
                                part[:] = nearest_code(of[part.long()] * (old / 2.0 ** e), self.fmt).to(torch.uint8)
                        sc[pg, h, at // BLOCK] = 2.0 ** e
                        y = torch.nan_to_num(y, nan=0.0, posinf=math.inf, neginf=-math.inf)
                        y = (y / 2.0 ** e).clamp(-TOP[self.fmt], TOP[self.fmt])
                        c[pg, h, at + lo - p0:at + hi - p0] = nearest_code(y, self.fmt).to(torch.uint8)

    def values(self, table_row, n):
        """Positions 0 .. n - 1 of one sequence: k, v float64 [n, hkv, d], and the scales [n, hkv]."""
        dev = self.codes["k"].device
        pos = torch.arange(n, device=dev)
        pg = torch.as_tensor(table_row, device=dev).long()[pos // self.page]
        of, out = code_values(self.fmt).to(dev), []
        for name in ("k", "v"):
            c = of[self.codes[name][pg, :, pos % self.page].long()]
            s = self.scales[name][pg, :, pos % self.page // BLOCK]
            out += [c * s[..., None], s]
        return out[0], out[2], out[3]

    def attention(self, table, lens, offsets, q, scale=None):
        """(out, bound) float64 [T, hq, d]: the definition, and how far the library's bf16 result
        may be from it.  The bound counts, relative to sum_i p_i |v_i|: the weights' rounding to
        fp16 (2^-11); twice (numerator and normaliser) the scores' error, which is 2^-19 of
        sum_d |q_d k_d| (fp32 sums of exact products, 16 steps of at most 2^-23) and a few fp32
        roundings of |s| + 128 (2^-22), and the exponential's (2^-21); fp32 sums over the
        positions ((n / 128 + 64) steps of 2^-23).  Weights under 2^-14 of the largest one lose up to 2^-25
        of it, times the largest value scale.  Then one rounding to bf16, 2^-8 of the result."""
        t, hq, d = q.shape
        out, bound = torch.zeros_like(q), torch.zeros_like(q)
        scale = 1 / math.sqrt(d) if not scale else scale
        for b in range(len(lens)):
            n, r0 = int(lens[b]), int(offsets[b])
            w = int(offsets[b + 1]) - r0
            if n == 0 or w == 0:
                continue
            k, v, vs = self.values(table[b], n)
            hkv = k.shape[1]
            see = n - w + 1 + torch.arange(w, device=q.device)
            hide = torch.arange(n, device=q.device)[None] >= see[:, None]
            for h in range(hq):
                g = h // (hq // hkv)
                qh = q[r0:r0 + w, h]
                s = (qh @ k[:, g].T * scale).masked_fill(hide, -math.inf)
                p = torch.softmax(s, dim=-1)
                p = torch.where(see[:, None] > 0, p, 0.0)
                o = p @ v[:, g]
                pv = p @ v[:, g].abs()
                a = (qh.abs() @ k[:, g].abs().T).amax(-1, keepdim=True) * scale * math.log2(math.e)
                score = 2.0 ** -19 * a + 2.0 ** -22 * (a + 128) + 2.0 ** -21
                small = 2.0 ** -25 * float(vs[:, g].max()) * (v[:, g].abs() / vs[:, g, None]).sum(0)
                out[r0:r0 + w, h] = o
                bound[r0:r0 + w, h] = ((2.0 ** -11 + 2 * math.log(2) * score + (n / 128 + 64) * 2.0 ** -23) * pv +
                                       small + 2.0 ** -8 * o.abs() + 1e-30)
        return out, bound


def rope(x: torch.Tensor, pos, inv_freq, axis_of, rotary: int) -> torch.Tensor:
    """x float64 [T, heads, d], pos int [axes, T] -> rotated, float64."""
    out, half = x.clone(), rotary // 2
    for j in range(half):
        angle = torch.as_tensor(pos, device=x.device)[axis_of[j]].double() * float(inv_freq[j])
        c, s = angle.cos()[:, None], angle.sin()[:, None]
        out[:, :, j] = x[:, :, j] * c - x[:, :, j + half] * s
        out[:, :, j + half] = x[:, :, j + half] * c + x[:, :, j] * s
    return out

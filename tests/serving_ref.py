"""Window and prefix attention, head norms and page tables in 64 bits (or whole numbers), from
their definitions.  Shares no code with the library."""
from __future__ import annotations

import math

import torch


def attention(ref, table, lens, offsets, q, scale=None, window=None, sinks=0):
    """(out, bound) float64 [T, hq, d] over a kv8_ref.RefCache: the definition, and how far the
    library's bf16 result may be from it, by the count of kv8_ref.RefCache.attention.  Joining the
    two sums of a shared prefix adds four fp32 roundings to each weight, 2^-21, which twice
    (numerator and normaliser) is counted in the 64 steps of 2^-23 there."""
    t, hq, d = q.shape
    out, bound = torch.zeros_like(q), torch.zeros_like(q)
    scale = 1 / math.sqrt(d) if not scale else scale
    for b in range(len(lens)):
        n, r0 = int(lens[b]), int(offsets[b])
        w = int(offsets[b + 1]) - r0
        if n == 0 or w == 0:
            continue
        k, v, vs = ref.values(table[b], n)
        hkv = k.shape[1]
        p = (n - w + torch.arange(w, device=q.device))[:, None]
        i = torch.arange(n, device=q.device)[None]
        see = i <= p
        if window is not None:
            see &= (i > p - window) | (i < sinks)
        some = see.any(0)
        vmax = torch.where(some[:, None], vs, 0.0).amax(0)
        for h in range(hq):
            g = h // (hq // hkv)
            qh = q[r0:r0 + w, h]
            s = (qh @ k[:, g].T * scale).masked_fill(~see, -math.inf)
            pr = torch.softmax(s, dim=-1)
            pr = torch.where(see.any(1, keepdim=True), pr, 0.0)
            o, pv = pr @ v[:, g], pr @ v[:, g].abs()
            a = (qh.abs() @ k[:, g].abs().T).masked_fill(~see, 0.0).amax(-1, keepdim=True) * scale * math.log2(math.e)
            score = 2.0 ** -19 * a + 2.0 ** -22 * (a + 128) + 2.0 ** -21
            small = 2.0 ** -25 * float(vmax[g]) * (v[some][:, g].abs() / vs[some][:, g, None]).sum(0)
            out[r0:r0 + w, h] = o
            bound[r0:r0 + w, h] = ((2.0 ** -11 + 2 * math.log(2) * score + (n / 128 + 64) * 2.0 ** -23) * pv +
                                   small + 2.0 ** -8 * o.abs() + 1e-30)
    return out, bound


def norm_rope(x, weight, eps, offset, pos, inv_freq, axis_of, rotary):
    """x float64 [T, heads, d] -> (out, bound).  The bound: a head's factor is off by 2^-20 (16 + 3 sums
    of squares, halved by the root, the reciprocal root's 2 ulp, three products), which the rotation
    adds up over its two elements with 2^-20 of its own, and one rounding to bf16, 2^-8 (at least half
    of its smallest number)."""
    y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    y = torch.where(x.abs().amax(-1, keepdim=True) == 0, 0.0, y)
    if weight is not None:
        y = y * (weight.double() + offset)
    out, mag, half = y.clone(), y.abs(), rotary // 2
    for j in range(half):
        angle = pos[axis_of[j]].double() * float(inv_freq[j])
        c, s = angle.cos()[:, None], angle.sin()[:, None]
        out[:, :, j] = y[:, :, j] * c - y[:, :, j + half] * s
        out[:, :, j + half] = y[:, :, j + half] * c + y[:, :, j] * s
        mag[:, :, j] = mag[:, :, j + half] = y[:, :, j].abs() + y[:, :, j + half].abs()
    return out, 2.0 ** -8 * out.abs() + 2.0 ** -19 * mag + 2.0 ** -134


class Pages:
    """The pool as Python lists.  `missing` tells whether a page was wanted and not there."""

    def __init__(self, table, free, n_free, lens, held, page):
        self.table, self.free = [list(r) for r in table], list(free)
        self.n_free, self.lens, self.held, self.page = n_free, list(lens), list(held), page

    def step(self, new, keep=None, borrowed=None):
        n = len(self.lens)
        keep = list(self.lens) if keep is None else keep
        after = [-(-(k + m) // self.page) for k, m in zip(keep, new)]
        stack = self.free[:self.n_free]
        for b in range(n):
            stack += self.table[b][max(after[b], borrowed[b] if borrowed else 0):self.held[b]]
        missing = False
        for b in range(n):
            got = self.held[b]
            for j in range(self.held[b], after[b]):
                self.table[b][j] = stack.pop() if stack else -1
                got += self.table[b][j] >= 0
            missing |= got < after[b]
            self.held[b] = min(after[b], got)
        self.free[:len(stack)] = stack
        self.n_free = len(stack)
        offsets, positions, slots = [0], [], []
        for b in range(n):
            for p in range(keep[b], keep[b] + new[b]):
                id = self.table[b][p // self.page]
                positions.append(p)
                slots.append(id * self.page + p % self.page if id >= 0 else -1)
            offsets.append(offsets[-1] + new[b])
            self.lens[b] = keep[b] + new[b]
        return offsets, positions, slots, missing

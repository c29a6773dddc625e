"""64-bit definitions of the paged cache operators, and the error bounds they are held to.

Everything here runs on the CPU in float64, one sequence and one kv head at a time.
"""
from __future__ import annotations

import dataclasses
import math

import torch

F64 = torch.float64
EPS = {torch.bfloat16: 2.0 ** -7, torch.float16: 2.0 ** -10}  # finfo.eps: a rounding errs by half


@dataclasses.dataclass
class Pages:
    """A pool on the CPU in float64, in the order [n_pages][Hkv][page_size][D]."""
    k: torch.Tensor
    v: torch.Tensor

    @property
    def page_size(self):
        return self.k.shape[2]

    def gather(self, table, pos):
        """K, V [Hkv][len(pos)][D]; a table entry that names no page reads as zeros."""
        ps, n = self.page_size, self.k.shape[0]
        page = table[pos // ps].long()
        ok = ((page >= 0) & (page < n))
        page = page.clamp(0, n - 1)
        out = []
        for x in (self.k, self.v):
            g = x[page, :, pos % ps]
            out.append(torch.where(ok[:, None, None], g, torch.zeros_like(g)).transpose(0, 1))
        return out


def rotate(x, pos, theta):
    """Rotate-half RoPE of x [rows][heads][D] at integer positions pos [rows]."""
    D = x.shape[-1]
    if theta == 0:
        return x.clone()
    w = torch.tensor([theta ** (-2.0 * i / D) for i in range(D // 2)], dtype=F64)
    a = pos.to(F64)[:, None] * w
    c, s = torch.cos(a)[:, None], torch.sin(a)[:, None]
    lo, hi = x[..., :D // 2], x[..., D // 2:]
    return torch.cat([lo * c - hi * s, hi * c + lo * s], -1)


def rotate_bound(ref, x, dtype):
    """Half a step of the output type, and cosines and sines that are off by at most 2^-21
    each (a fraction of a turn rounded to fp32 is off by 2^-25, times 2 pi; sincospif 2^-23;
    the two products and their sum 3 * 2^-24 of their size)."""
    D = x.shape[-1]
    a = x[..., :D // 2].abs() + x[..., D // 2:].abs()
    return EPS[dtype] / 2 * ref.abs() + 2.0 ** -21 * torch.cat([a, a], -1) + 2.0 ** -25


def seq_positions(segs, cap):
    """Sorted positions of the union of two (start, len) segments inside [0, cap)."""
    pos = set()
    for st, n in segs:
        pos |= set(range(max(st, 0), min(st + max(n, 0), cap)))
    return torch.tensor(sorted(pos), dtype=torch.long)


def attention(pages, q, row_start, table, segs, row_limit=None, scale=None, groups=None,
              dtype=torch.bfloat16):
    """Returns {row: (out [Hq][D], lse [Hq], bound of out, bound of lse)} of every row that
    belongs to a sequence.  groups: (seq_start, table, len) or None.

    The bounds: a score is a sum of D products in fp32, off by at most D * 2^-23 of the sum of
    their sizes B (a tensor core may cut each addition instead of rounding it), which shifts a
    probability by that factor, and the normaliser by as much; the exponential and the sums add
    at most 2^-16.  Each probability is rounded to the cache's type once (half a step), and so
    is the output; fp16 probabilities below 2^-14 are off by up to 2^-25 each, the sum of
    probabilities being at least one."""
    D = q.shape[-1]
    hkv = pages.k.shape[1]
    g = q.shape[1] // hkv
    scale = D ** -0.5 if not scale else scale
    e = EPS[dtype]
    res = {}
    for s in range(len(row_start) - 1):
        r0, r1 = row_start[s], row_start[s + 1]
        if r1 <= r0:
            continue
        own = seq_positions(segs[s], table.shape[1] * pages.page_size)
        k, v = pages.gather(table[s], own)
        pre = 0
        if groups is not None:
            for i in range(len(groups[0]) - 1):
                if groups[0][i] <= s < groups[0][i + 1]:
                    pp = torch.arange(min(max(groups[2][i], 0), groups[1].shape[1] * pages.page_size))
                    pk, pv = pages.gather(groups[1][i], pp)
                    k, v, pre = torch.cat([pk, k], 1), torch.cat([pv, v], 1), len(pp)
        qs = q[r0:r1].to(F64).reshape(r1 - r0, hkv, g, D)
        seen = torch.ones(r1 - r0, k.shape[1], dtype=torch.bool)
        if row_limit is not None:
            seen[:, pre:] = own[None] < torch.tensor(row_limit[r0:r1])[:, None]
        n = seen.sum(1)
        for h in range(hkv):
            if k.shape[1]:
                x = torch.einsum("rgd,kd->rgk", qs[:, h], k[h]) * scale
                B = (torch.einsum("rgd,kd->rgk", qs[:, h].abs(), k[h].abs()) * scale)
                x = torch.where(seen[:, None], x, -math.inf)
                B = torch.where(seen[:, None], B, torch.zeros_like(B)).amax(2)
                z = torch.logsumexp(x, 2)
                w = torch.where(torch.isfinite(z)[..., None], torch.exp(x - z[..., None]),
                                torch.zeros_like(x))
                w = torch.where(seen[:, None], w, torch.zeros_like(w))
                vh = torch.where(seen.any(0)[:, None], v[h], torch.zeros_like(v[h]))
                o = torch.einsum("rgk,kd->rgd", w, vh)
                A = torch.einsum("rgk,kd->rgd", w, vh.abs())
                vmax = vh.abs().amax() if vh.numel() else torch.zeros((), dtype=F64)
            else:
                z = torch.full((r1 - r0, g), -math.inf, dtype=F64)
                o = torch.zeros(r1 - r0, g, D, dtype=F64)
                A, B, vmax = o, torch.zeros(r1 - r0, g, dtype=F64), torch.zeros((), dtype=F64)
            sub = n[:, None, None] * 2.0 ** -25 * vmax if dtype == torch.float16 else 0.0
            shift = 2 * D * 2.0 ** -23 * B + 2.0 ** -16
            tol = e / 2 * o.abs() + (e / 2 + shift[..., None]) * A * (1 + e) + sub + 2.0 ** -25
            for i in range(r1 - r0):
                item = res.setdefault(r0 + i, ([], [], [], []))
                for lst, val in zip(item, (o[i], z[i], tol[i], shift[i])):
                    lst.append(val)
    return {r: tuple(torch.cat(x) for x in it) for r, it in res.items()}

"""Plain model of the paged cache (include/hils.h, hils_cache_t), on the CPU.

What the cache holds is defined by float32 operations in a given order, so the
model repeats them and the tests ask for equal bits; summaries and attention
are computed from the held values in float64.
"""
from __future__ import annotations

import math

import torch

MAX_CODE = {torch.int8: 127.0, torch.float8_e4m3fn: 448.0}
TINY = 2.0 ** -110


def rotate(x, cos, sin, interleaved):
    """Rows x [n, heads, d] in their type, angles [n, rot / 2] float32: each product and sum rounded to float32."""
    r = 2 * cos.shape[1]
    y = x.float().clone()
    co, si = cos[:, None], sin[:, None]
    a, c = (y[..., 0:r:2].clone(), y[..., 1:r:2].clone()) if interleaved else (y[..., :r // 2].clone(), y[..., r // 2:r].clone())
    ra, rc = a * co - c * si, c * co + a * si
    if interleaved:
        y[..., 0:r:2], y[..., 1:r:2] = ra, rc
    else:
        y[..., :r // 2], y[..., r // 2:r] = ra, rc
    return y.to(x.dtype)


def encode(block, code_type):
    """(codes, scale) of one block [S, d]."""
    m, x = MAX_CODE[code_type], block.float()
    if not torch.isfinite(x).all():
        return torch.zeros_like(x).to(code_type), math.nan
    top = x.abs().max()
    if top < TINY:
        return torch.zeros_like(x).to(code_type), 0.0
    one, m32 = torch.tensor(1.0), torch.tensor(m)
    y = (x * ((one / top) * m32)).clamp(-m, m)
    return (y.round() if code_type is torch.int8 else y).to(code_type), float(top * (one / m32))


class RefCache:
    """pool, scale and tail of keys and values, as plain tensors; code_type None: a native cache."""

    def __init__(self, B, Hkv, S, d, dtype, table, num_pages, code_type=None, fill=0.0):
        self.B, self.Hkv, self.S, self.d, self.dtype, self.code, self.table = B, Hkv, S, d, dtype, code_type, table
        new = lambda *s, t: torch.full(s, fill, dtype=torch.float32).to(t)  # noqa: E731
        self.pool = [new(num_pages, Hkv, S, d, t=code_type or dtype) for _ in range(2)]
        self.scale = [new(num_pages, Hkv, t=torch.float32) for _ in range(2)]
        self.tail = [new(B, 2, Hkv, S, d, t=dtype) for _ in range(2)]

    def append(self, lens, news, k, v):
        """Rows k, v [n, Hkv, d], already rotated, sequence after sequence; lens counts them."""
        S, row = self.S, 0
        for b, (L, n) in enumerate(zip(lens, news)):
            first = L - n
            for x, rows in enumerate((k, v)):
                # whole chunks are put together first: the tail holds the last two chunks only
                slots = self.tail[x][b].clone()
                for c in range(first // S, (L - 1) // S + 1 if n else 0):
                    lo, hi = max(first, c * S), min(L, c * S + S)
                    part = rows[row + lo - first:row + hi - first].transpose(0, 1)
                    page = int(self.table[b, c])
                    if self.code is None:
                        self.pool[x][page, :, lo - c * S:hi - c * S] = part
                        continue
                    block = self.tail[x][b, c & 1].clone() if c == first // S else torch.zeros_like(self.tail[x][b, 0])
                    block[:, lo - c * S:hi - c * S] = part
                    if c >= (L - 1) // S - 1:
                        slots[c & 1, :, lo - c * S:hi - c * S] = part
                    if hi == c * S + S:
                        for g in range(self.Hkv):
                            codes, scale = encode(block[g], self.code)
                            self.pool[x].view(torch.uint8 if self.code is not torch.int8 else torch.int8)[page, g] = (
                                codes if self.code is torch.int8 else codes.view(torch.uint8))
                            self.scale[x][page, g] = scale
                self.tail[x][b] = slots
            row += n

    def values(self, x, b, L):
        """What the cache holds of keys (0) or values (1) of sequence b: float64 [Hkv, L, d]."""
        out = torch.empty((self.Hkv, L, self.d), dtype=torch.float64)
        for c in range(-(-L // self.S)):
            lo, hi = c * self.S, min(L, c * self.S + self.S)
            page = int(self.table[b, c])
            if self.code is None:
                t = self.pool[x][page].double()
            elif hi - lo < self.S:
                t = self.tail[x][b, c & 1].double()
            else:
                t = self.pool[x][page].float().double() * self.scale[x][page].double()[:, None, None]
            out[:, lo:hi] = t[:, :hi - lo]
        return out


def summaries(k, q_lmk, scale):
    """k [Hkv, C, S, d], q_lmk [Hq, C, d] float64 -> k_sum [Hq, C, d], b_sum [Hq, C], sum p |k|, and
    (largest p) sum |k|."""
    G = q_lmk.shape[0] // k.shape[0]
    kk = k.repeat_interleave(G, dim=0)
    p = torch.softmax(torch.einsum("hcd,hcsd->hcs", q_lmk, kk) * scale, dim=-1)
    return (torch.einsum("hcs,hcsd->hcd", p, kk), torch.special.entr(p).sum(dim=-1),
            torch.einsum("hcs,hcsd->hcd", p, kk.abs()), p.amax(dim=-1, keepdim=True) * kk.abs().sum(dim=2))


def attend(q, k, v, lists, s_sel, S, W, scale):
    """One token: q [Hq, d], k, v [Hkv, L, d], lists [Hkv][..] of chunks (with -1), s_sel [Hq, K], all float64.
    -> out [Hq, d], sum w |v| [Hq, d], sum (largest w of the chunk) |v|, and the largest sum |q_e k_e| scale and
    max |q| sum |k_e| scale over the keys it reads."""
    Hq, Hkv, L = q.shape[0], k.shape[0], k.shape[1]
    G, first = Hq // Hkv, max(0, (L - 1) // S - W // S + 1) * S
    out, mag, low, big = torch.empty_like(q), torch.empty_like(q), torch.zeros_like(q), 0.0
    wide = 0.0
    for h in range(Hq):
        g = h // G
        logit = k[g] @ q[h] * scale
        w = [logit[first:]]
        vals = [v[g, first:]]
        keys = [k[g, first:]]
        for slot, c in enumerate(lists[g]):
            if c < 0:
                continue
            s = logit[c * S:c * S + S]
            w.append(s - torch.logsumexp(s, 0) + s_sel[h, slot])
            vals.append(v[g, c * S:c * S + S])
            keys.append(k[g, c * S:c * S + S])
        w = torch.softmax(torch.cat(w), 0)
        vals = torch.cat(vals)
        out[h] = w @ vals
        mag[h] = w @ vals.abs()
        own = L - first
        edges = list(range(0, own, S)) + list(range(own, len(w) + 1, S))
        for a, z in zip(edges, edges[1:]):
            low[h] += w[a:z].max() * vals[a:z].abs().sum(dim=0)
        keys = torch.cat(keys).abs()
        big = max(big, float((keys @ q[h].abs()).max() * scale))
        wide = max(wide, float(keys.sum(dim=1).max() * q[h].abs().max() * scale))
    return out, mag, low, big, wide

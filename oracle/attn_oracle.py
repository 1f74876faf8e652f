"""The attention half's operators in plain form: the packed linear product and
attention in 64 bits over explicitly dequantised values, and the page operations
of the 4-bit cache as sequential loops over Python lists.  Test infrastructure
only; shares no code with the HIP path.
"""
from __future__ import annotations

import math

import numpy as np

from oracle import moe_oracle as orc

ACT = {
    "none": lambda v: v,
    "silu": lambda v: v / (1.0 + np.exp(-v)),
    "gelu": lambda v: 0.5 * v * np.array([math.erfc(-t / math.sqrt(2.0)) for t in np.ravel(v)]).reshape(v.shape),
    "relu": lambda v: np.maximum(v, 0.0),
}


def linear(x, codes, scale, bias=None, act="none", residual=None):
    """act(x W^T + bias) + residual, W = codes * scale, all in float64."""
    v = x.astype(np.float64) @ (codes.astype(np.float64) * scale.astype(np.float64)[:, None]).T
    if bias is not None:
        v = v + bias
    y = ACT[act](v)
    return y if residual is None else y + residual


def cache_values(x):
    """What the cache holds for fp32 rows [..., D]: (float32 codes * scale, as
    fp32 products).  NaN rows stay NaN."""
    rows = np.ascontiguousarray(x, np.float32).reshape(-1, x.shape[-1])
    q, s = orc.quantize_rows(rows, 4)
    with np.errstate(invalid="ignore"):
        return (q.astype(np.float32) * s[:, None]).reshape(x.shape)


def attention(q, k, v, pos0, scale, window=0):
    """Queries q [m, H, D] at positions pos0 .. pos0+m-1 over keys and values
    [L, Hk, D] at positions 0 .. L-1 (float64; negative positions see nothing).
    Returns out, lse, and per (row, head) the data an error bound needs: the sum
    of p |v| over p per column, and the largest scale * sum |q||k|."""
    m, H, D = q.shape
    L, Hk = k.shape[0], k.shape[1]
    out, mag = np.zeros((m, H, D)), np.zeros((m, H, D))
    lse, dots = np.full((m, H), -np.inf), np.zeros((m, H))
    for i in range(m):
        pos = pos0 + i
        lo, hi = (max(0, pos - window + 1) if window else 0), min(pos + 1, L)
        if hi <= lo:
            continue
        for h in range(H):
            kk, vv = k[lo:hi, h // (H // Hk)], v[lo:hi, h // (H // Hk)]
            z = kk @ q[i, h] * scale
            p = np.exp(z - z.max())
            out[i, h] = p @ vv / p.sum()
            mag[i, h] = p @ np.abs(vv) / p.sum()
            lse[i, h] = z.max() + math.log(p.sum())
            dots[i, h] = (np.abs(kk) @ np.abs(q[i, h])).max() * abs(scale)
    return out, lse, mag, dots


class Pages:
    """The page tables of a cache on the host; the rules one step at a time."""

    def __init__(self, n_pages, page_tokens, n_seqs, max_pages):
        self.pt, self.max_pages = page_tokens, max_pages
        self.ref = [0] * n_pages
        self.len = [0] * n_seqs
        self.table = [[] for _ in range(n_seqs)]
        self.copies = []                          # (from, to) of the last call

    def _count(self, n):
        return -(-n // self.pt)

    def reserve(self, n_new):
        granted, stopped = [0] * len(self.len), False
        self.copies = []
        for s, n in enumerate(n_new):
            n = max(n, 0)
            if n == 0 or self._count(self.len[s] + n) > self.max_pages:
                continue
            have, want = self._count(self.len[s]), self._count(self.len[s] + n)
            copy = self.len[s] % self.pt != 0 and self.ref[self.table[s][-1]] > 1
            free = [p for p, r in enumerate(self.ref) if r == 0]
            if stopped or want - have + copy > len(free):
                stopped = True
                continue
            if copy:
                p = free.pop(0)
                self.copies.append((self.table[s][-1], p))
                self.ref[self.table[s][-1]] -= 1
                self.ref[p] = 1
                self.table[s][-1] = p
            for _ in range(have, want):
                p = free.pop(0)
                self.ref[p] = 1
                self.table[s].append(p)
            self.len[s] += n
            granted[s] = n
        return granted

    def fork(self, src, dst, n_tokens=None):
        ok, named = [0] * len(src), set()
        old_len, old = list(self.len), [list(t) for t in self.table]
        for i, (a, b) in enumerate(zip(src, dst)):
            first = b not in named
            named.add(b)
            if not (0 <= a < len(self.len) and 0 <= b < len(self.len)) or not first or old_len[b] != 0:
                continue
            n = old_len[a] if n_tokens is None else n_tokens[i]
            if n < 0 or n > old_len[a]:
                continue
            self.table[b] = old[a][:self._count(n)]
            self.len[b] = n
            for p in self.table[b]:
                self.ref[p] += 1
            ok[i] = 1
        return ok

    def truncate(self, new_len):
        for s, n in enumerate(new_len):
            if 0 <= n < self.len[s]:
                for p in self.table[s][self._count(n):]:
                    self.ref[p] -= 1
                self.table[s] = self.table[s][:self._count(n)]
                self.len[s] = n

    def compact(self):
        live = sum(r > 0 for r in self.ref)
        remap = [p if r > 0 else -1 for p, r in enumerate(self.ref)]
        holes = [p for p in range(live) if self.ref[p] == 0]
        self.copies = []
        for p in range(live, len(self.ref)):
            if self.ref[p] > 0:
                h = holes.pop(0)
                remap[p] = h
                self.ref[h], self.ref[p] = self.ref[p], 0
                self.copies.append((p, h))
        self.table = [[remap[p] for p in t] for t in self.table]
        return remap, live

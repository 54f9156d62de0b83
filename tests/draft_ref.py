"""Plain forms, in 64 bits and on the host, of the operators around drafted
tokens and the pages of the cache: trees and what their nodes see, attention
under any mask with entry-wise bounds, verification, and the pages' book."""

import numpy as np
import torch

from gpu_util import EXP_ERR, U, gamma
from window_ref import AB


# ------------------------------------------------------------------ trees --

def depths(parent):
    d = []
    for p in parent:
        d.append(0 if p < 0 else d[p] + 1)
    return d


def tree_mask(parent, ctx, window, sinks):
    """[n, n] truth values: node i sees node a."""
    n, d = len(parent), depths(parent)
    m = np.zeros((n, n), dtype=bool)
    for i in range(n):
        a = i
        while a >= 0:
            m[i, a] = not window or d[i] - d[a] < window or ctx + d[a] < sinks
            a = parent[a]
    return m


def pack(mask, words):
    """int32 [n, words], bit a % 32 of word a / 32."""
    n = mask.shape[1]
    full = np.zeros((mask.shape[0], 32 * words), dtype=np.uint8)
    full[:, :n] = mask
    return np.packbits(full, axis=1, bitorder="little").view("<u4").astype(np.uint32).view(np.int32)


def masked(q, k, v, keep, scale, dtype):
    """Attention of one head, q [n, D], k and v [m, D] in fp64 under keep [n, m]:
    O, lse and their bounds.  The bounds are those of window_ref: u = half a step
    of the type, scores off by gamma(D) scale sum |q||k| and 2^-23 of themselves,
    P rounded to the type, sums in fp32."""
    n, D = q.shape
    u, ab = U[dtype], AB[dtype]
    s = ((q @ k.T) * scale).masked_fill(~keep, float("-inf"))
    lse = torch.logsumexp(s, -1)
    P = torch.exp(s - lse[:, None].masked_fill(torch.isinf(lse)[:, None], 0.0)).masked_fill(~keep, 0.0)
    O = P @ v
    mags = (q.abs() @ k.abs().T) * scale * keep
    mags = torch.cat([mags, torch.zeros(n, 1, dtype=mags.dtype, device=q.device)], 1)
    es = (gamma(D) * mags).amax(-1, keepdim=True) + 2.0 ** -23 * mags.amax(-1, keepdim=True)
    ep = u + 2 * es + 4 * EXP_ERR
    cnt = keep.sum(-1, keepdim=True)
    eO = u * O.abs() + (ep + gamma(1) + cnt * 2.0 ** -22) * (P @ v.abs()) + ab * (keep.double() @ v.abs()) + ab
    el = 2 * es[:, 0] + 8 * EXP_ERR + 2.0 ** -22 * (lse.abs().nan_to_num(posinf=0.0) + 1) + cnt[:, 0] * 2.0 ** -22
    return O, eO, lse, el


# ----------------------------------------------------------- verification --

def verify(target, draft, tokens, parent, accept, sample):
    """One sequence, rows in fp64 numpy: (path, token)."""
    n, V = target.shape
    path, node = [0], 0
    while True:
        r, s = np.where(target[node] > 0, target[node], 0.0), 1.0
        first, taken = target[node], None
        for a in range(node + 1, n):
            if parent[a] != node or not 0 <= tokens[a] < V:
                continue
            x = tokens[a]
            q = 1.0 if draft is None else draft[node][x]
            have = first[x] if s == 1.0 and r is not None and first is target[node] else r[x]
            if float(accept[a]) * q * s < have:
                taken = a
                break
            if draft is None:
                r = r.copy()
                r[x] = 0.0
            else:
                d = r - s * draft[node]
                r = np.where(d > 0, d, 0.0)
            first = r
            s = float(r.sum())
        if taken is None:
            break
        node = taken
        path.append(node)
    if r.sum() <= 0:
        r = np.where(target[node] > 0, target[node], 0.0)
    if r.sum() <= 0:
        return path, -1
    run = np.cumsum(r)
    at = int(np.searchsorted(run, float(sample) * run[-1], side="right"))
    return path, min(at, int(np.nonzero(r)[0][-1]))


# ------------------------------------------------------------------ pages --

class Book:
    """The pages' book as lists, entry after entry."""

    def __init__(self, n_pages, n_seq, max_pages, page):
        self.refs, self.page = [0] * n_pages, page
        self.table = [[-1] * max_pages for _ in range(n_seq)]
        self.kv = [0] * n_seq

    def held(self, n):
        return -(-n // self.page)

    def free(self):
        for row, n in zip(self.table, self.kv):
            for j in range(self.held(n), len(row)):
                if row[j] >= 0:
                    self.refs[row[j]] -= 1
                row[j] = -1

    def fork(self, parent):
        table, kv = [list(r) for r in self.table], list(self.kv)
        for s, p in enumerate(parent):
            if p == s:
                continue
            for x in table[s]:
                if x >= 0:
                    self.refs[x] -= 1
            new = [-1] * len(table[s]) if p < 0 else [x if j < self.held(kv[p]) else -1 for j, x in enumerate(table[p])]
            for x in new:
                if x >= 0:
                    self.refs[x] += 1
            self.table[s], self.kv[s] = new, 0 if p < 0 else kv[p]

    def reserve(self, want):
        """(src, dst, whether the pages sufficed)"""
        items = [(s, j) for s, (n, w) in enumerate(zip(self.kv, want)) if w > n for j in range(n // self.page, self.held(w))]
        holders, ask = list(self.refs), {}
        for s, j in items:
            if self.table[s][j] >= 0:
                ask.setdefault(self.table[s][j], []).append((s, j))
        give = []
        for s, j in items:
            x = self.table[s][j]
            if x < 0 or (holders[x] > 1 and not (len(ask[x]) == holders[x] and ask[x][0] == (s, j))):
                give.append((s, j))
        for s, j in give:
            if self.table[s][j] >= 0:
                self.refs[self.table[s][j]] -= 1
        free = [x for x, n in enumerate(self.refs) if n == 0]
        src, dst = [-1] * len(want), [-1] * len(want)
        for i, (s, j) in enumerate(give):
            x = self.table[s][j]
            if i >= len(free):
                if x >= 0:
                    self.refs[x] += 1
                continue
            self.table[s][j] = free[i]
            self.refs[free[i]] = 1
            if x >= 0 and j == self.kv[s] // self.page and self.kv[s] % self.page:
                src[s], dst[s] = x, free[i]
        return src, dst, len(give) <= len(free)

    def compact(self):
        live = sum(n > 0 for n in self.refs)
        high = [x for x in range(live, len(self.refs)) if self.refs[x] > 0]
        low = [x for x in range(live) if self.refs[x] <= 0]
        to = dict(zip(high, low))
        for a, b in to.items():
            self.refs[b], self.refs[a] = self.refs[a], 0
        self.table = [[to.get(x, x) for x in row] for row in self.table]
        rest = [-1] * (len(self.refs) // 2 - len(high))
        return high + rest, low + rest

    def agrees(self):
        count = [0] * len(self.refs)
        for row in self.table:
            for x in row:
                if x >= 0:
                    count[x] += 1
        return count == self.refs

"""CPU oracles for speculative decoding over a paged KV cache -- TEST
INFRASTRUCTURE ONLY (tests and ``smoke()``; the product library never imports
it).  Plain numpy in fp64 and Python lists, written from the definitions in
``include/cache.h`` and ``include/tree.h``:

  tree_attention  one tree against one sequence's K and V
  verify_drafts   the walk and the draw over one tree
  Pages           the page bookkeeping and the rows, one sequence at a time

Pinned by ``tests/test_tree_oracle.py`` (closed forms, the single-token oracle,
and the distribution that verification must leave unchanged).
"""
from __future__ import annotations

import numpy as np


def ancestors(parent) -> np.ndarray:
    """sees[i, j]: node j is node i or an ancestor of it; padding (-2) sees nothing."""
    n = len(parent)
    sees = np.zeros((n, n), bool)
    for i in range(n):
        j = i
        while j >= 0 and parent[i] != -2:
            sees[i, j] = True
            j = parent[j]
    return sees


def tree_attention(q, k_old, v_old, k_new, v_new, parent, scale=None):
    """(o [n, Hq, D], weighted |v| [n, Hq, D], sum of |v| seen [n, Hq, D], largest
    sum |q k| scale [n, Hq]) in fp64, the last three for error bounds.  q [n, Hq, D],
    k_old, v_old [L, Hkv, D], k_new, v_new [n, Hkv, D]."""
    n, Hq, D = q.shape
    G = Hq // k_new.shape[1]
    scale = 1.0 / np.sqrt(D) if scale is None else scale
    sees = ancestors(parent)
    o, wv, av = np.zeros((n, Hq, D)), np.zeros((n, Hq, D)), np.zeros((n, Hq, D))
    big = np.zeros((n, Hq))
    for i in range(n):
        if parent[i] == -2:
            continue
        k = np.concatenate([k_old, k_new[sees[i]]])
        v = np.concatenate([v_old, v_new[sees[i]]])
        for h in range(Hq):
            g = h // G
            s = scale * (k[:, g] @ q[i, h])
            p = np.exp(s - s.max())
            p /= p.sum()
            o[i, h] = p @ v[:, g]
            wv[i, h] = p @ np.abs(v[:, g])
            av[i, h] = np.abs(v[:, g]).sum(0)
            big[i, h] = scale * (np.abs(k[:, g]) @ np.abs(q[i, h])).max()
    return o, wv, av, big


def verify_drafts(p, q, tokens, parent, u_accept, u_sample):
    """(path, next token) of one tree; p [n, V], q [n, V] or None."""
    p = np.asarray(p, np.float64)
    cur, path, S, R = 0, [0], 1.0, p[0].copy()
    for j in range(1, len(parent)):
        if parent[j] != cur:
            continue
        x = int(tokens[j])
        qx = 1.0 if q is None else float(q[cur][x])
        if float(u_accept[j]) * S * qx < R[x]:
            path.append(j)
            cur, S, R = j, 1.0, p[j].copy()
        elif q is None:
            S, R[x] = S - R[x], 0.0
        else:
            R = np.maximum(R - S * np.asarray(q[cur], np.float64), 0.0)
            S = R.sum()
    if not R.sum() > 0:
        R = p[cur]
    c = np.cumsum(R)
    t = int(np.searchsorted(c, float(u_sample) * c[-1], side="right"))
    return path, min(t, int(np.flatnonzero(R)[-1]))


class Pages:
    """A paged cache: k, v [layers, pages, page, heads, dim], refs, table, lens as numpy arrays (changed in place)."""

    def __init__(self, k, v, refs, table, lens):
        self.k, self.v, self.refs, self.table, self.lens = k, v, refs, table, lens
        self.page = k.shape[2]

    def _blocks(self, n):
        return -(-n // self.page)

    def trim(self, slot, new):
        for j in range(self._blocks(new), self._blocks(int(self.lens[slot]))):
            self.refs[self.table[slot, j]] -= 1
            self.table[slot, j] = -1
        self.lens[slot] = new

    def append(self, jobs):
        """jobs: (slot, k rows [layers, n, heads, dim], v rows) in the call's order."""
        free = iter(np.flatnonzero(self.refs == 0).tolist())
        shared = {s: self.lens[s] % self.page != 0 and self.refs[self.table[s, self.lens[s] // self.page]] > 1
                  for s, kr, _ in jobs if kr.shape[1]}
        plan = []
        for s, kr, vr in jobs:
            L, n = int(self.lens[s]), kr.shape[1]
            if n and shared[s]:
                old, new = self.table[s, L // self.page], next(free)
                plan.append((s, L // self.page, new, old, L % self.page))
            for j in range(self._blocks(L), self._blocks(L + n)):
                plan.append((s, j, next(free), -1, 0))
        for s, j, new, old, rows in plan:
            self.table[s, j] = new
            self.refs[new] = 1
            if old >= 0:
                self.refs[old] -= 1
                self.k[:, new, :rows] = self.k[:, old, :rows]
                self.v[:, new, :rows] = self.v[:, old, :rows]
        for s, kr, vr in jobs:
            for i in range(kr.shape[1]):
                pos = int(self.lens[s]) + i
                at = self.table[s, pos // self.page], pos % self.page
                self.k[:, at[0], at[1]] = kr[:, i]
                self.v[:, at[0], at[1]] = vr[:, i]
            self.lens[s] += kr.shape[1]

    def fork(self, pairs):
        free = iter(np.flatnonzero(self.refs == 0).tolist())
        for s, d in pairs:
            full, rest = divmod(int(self.lens[s]), self.page)
            self.table[d, :full] = self.table[s, :full]
            np.add.at(self.refs, self.table[s, :full], 1)
            if rest:
                new, old = next(free), self.table[s, full]
                self.table[d, full] = new
                self.refs[new] = 1
                self.k[:, new, :rest] = self.k[:, old, :rest]
                self.v[:, new, :rest] = self.v[:, old, :rest]
            self.lens[d] = self.lens[s]

    def rows(self, slot, layer=0):
        """K and V rows of a sequence, in order."""
        L = int(self.lens[slot])
        t = self.table[slot, :self._blocks(L)]
        return tuple(a[layer][t].reshape(-1, *a.shape[3:])[:L] for a in (self.k, self.v))

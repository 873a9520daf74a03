"""fp64 oracle of the 8-bit paged cache and of attention over it
(include/qcache.h), written from the formulas."""
from __future__ import annotations

import numpy as np

from oracle.tree import Pages


def nearest(x):
    """The e4m3 value nearest to x (ties to the even code), beyond 448 the largest; NaN and infinity give NaN."""
    x = np.asarray(x, np.float64)
    a = np.where(np.isfinite(x), np.abs(x), 0.0)
    e = np.floor(np.log2(np.maximum(a, 2.0 ** -6)))
    step = 2.0 ** (e - 3)
    y = np.minimum(np.round(a / step) * step, 448.0)
    return np.where(np.isfinite(x), np.copysign(y, x), np.nan)


def scale_of(most):
    """2^e, e the least whole number from -100 on with most <= 448 * 2^e."""
    e = -100
    if most > 0:
        e = max(e, int(np.frexp(most)[1]) - 11)  # 448 < 2^9, most < 2^exponent
        while most > 448.0 * 2.0 ** e:
            e += 1
    return 2.0 ** e


class QPages(Pages):
    """Pages whose k, v hold e4m3 values, with ks, vs [layers, pages, heads]."""

    def __init__(self, k, v, ks, vs, refs, table, lens):
        super().__init__(k, v, refs, table, lens)
        self.ks, self.vs = ks, vs

    def append(self, jobs):
        before = {s: int(self.lens[s]) for s, _, _ in jobs}
        old_page = {s: int(self.table[s, n // self.page]) for s, n in before.items() if n % self.page}
        old_rows = {s: [a[:, p].copy() for a in (self.k, self.v, self.ks, self.vs)] for s, p in old_page.items()}
        codes, (self.k, self.v) = (self.k, self.v), (self.k.copy(), self.v.copy())
        super().append(jobs)  # tables and holders; the rows are put right below
        self.k, self.v = codes
        for s, kr, vr in jobs:
            i = 0
            while i < kr.shape[1]:
                pos = before[s] + i
                page, at = int(self.table[s, pos // self.page]), pos % self.page
                n = min(self.page - at, kr.shape[1] - i)
                for pool, scales, rows, which in ((self.k, self.ks, kr, 0), (self.v, self.vs, vr, 1)):
                    for l in range(pool.shape[0]):
                        for h in range(pool.shape[3]):
                            x = rows[l, i:i + n, h]
                            new = scale_of(np.max(np.abs(x[np.isfinite(x)]), initial=0.0))
                            if at:
                                was = old_rows[s][2 + which][l, h]
                                new = max(new, was)
                                pool[l, page, :at, h] = nearest(old_rows[s][which][l, :at, h] * (was / new))
                            scales[l, page, h] = new
                            pool[l, page, at:at + n, h] = nearest(x / new)
                i += n

    def fork(self, pairs):
        super().fork(pairs)
        for s, d in pairs:
            full, rest = divmod(int(self.lens[s]), self.page)
            if rest:
                new, old = self.table[d, full], self.table[s, full]
                self.ks[:, new], self.vs[:, new] = self.ks[:, old], self.vs[:, old]

    def values(self, slot, layer=0):
        """K and V values of a sequence, in order."""
        L = int(self.lens[slot])
        t = self.table[slot, :self._blocks(L)]
        return tuple((a[layer][t] * sc[layer][t][:, None, :, None]).reshape(-1, *a.shape[3:])[:L]
                     for a, sc in ((self.k, self.ks), (self.v, self.vs)))


def attend(q, k, v, scale=None):
    """Causal attention of the last rows: q [n, Hq, D] at positions L - n .. L - 1 of k, v [L, Hkv, D].  Returns o,
    sum p |v| and max over the positions of sum |q k| scale, each of o's leading shape (or o's)."""
    n, Hq, D = q.shape
    L, Hkv, _ = k.shape
    G = Hq // Hkv
    scale = 1.0 / np.sqrt(D) if scale is None else scale
    o, mass, most = np.zeros((n, Hq, D)), np.zeros((n, Hq, D)), np.zeros((n, Hq))
    for i in range(n):
        sees = L - n + i + 1
        if sees <= 0:
            continue
        for h in range(Hq):
            kk, vv = k[:sees, h // G], v[:sees, h // G]
            s = kk @ q[i, h] * scale
            p = np.exp(s - s.max())
            p /= p.sum()
            o[i, h], mass[i, h] = p @ vv, p @ np.abs(vv)
            most[i, h] = (np.abs(kk) @ np.abs(q[i, h])).max() * scale
    return o, mass, most

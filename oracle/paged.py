"""The paged 8-bit cache in float64: block quantisation, attention over what the codes stand
for, and the page management (tables, reference counts, lowest-first allocation)."""
from __future__ import annotations

import math

import numpy as np

MIN_MAX = 2.0 ** -100


def round_e4m3(y: np.ndarray) -> np.ndarray:
    """Nearest e4m3 value (half to even), |y| <= 448."""
    step = np.exp2(np.floor(np.log2(np.maximum(np.abs(y), 2.0 ** -6))) - 3)
    return np.rint(y / step) * step


def block_values(x: np.ndarray, code: str):
    """A block's entries -> (what they are stored as, times the scale; the scale)."""
    x = np.asarray(x, np.float64)
    fin = np.isfinite(x)
    a = float(np.max(np.abs(np.where(fin, x, 0.0)))) if x.size else 0.0
    if a < MIN_MAX:
        return np.zeros_like(x), 0.0
    if code == "int8":
        s = float(np.float32(a) / np.float32(127.0))
        c = np.rint(127.0 * np.where(fin, x, 0.0) / a)
        top = 127.0
    else:
        m, e = math.frexp(a)
        s = 2.0 ** (e - 9 if m <= 0.875 else e - 8)
        c = round_e4m3(np.where(fin, x, 0.0) / s)
        top = 448.0
    c = np.where(np.isposinf(x), top, np.where(np.isneginf(x), -top, c))
    return c * s, s


def cached_values(x: np.ndarray, code: str, page: int) -> np.ndarray:
    """One sequence's tokens [T, H, d] as the cache holds them."""
    out = np.zeros(x.shape, np.float64)
    for t in range(0, x.shape[0], page):
        for h in range(x.shape[1]):
            out[t:t + page, h] = block_values(x[t:t + page, h], code)[0]
    return out


def attention(q, k, v, causal: bool, scale: float):
    """q [n, Hq, d] over k, v [T, Hkv, d]: (out, lse [n, Hq], mass [n, Hq, d] = sum p |v|,
    reach [n, Hq] = the largest scale * sum_j |q_j k_j| over the visible tokens)."""
    n, Hq, d = q.shape
    T, Hkv, _ = k.shape
    G = Hq // Hkv
    out, mass = np.zeros((n, Hq, d)), np.zeros((n, Hq, d))
    lse, reach = np.full((n, Hq), -np.inf), np.zeros((n, Hq))
    for i in range(n):
        vis = max(0, min(T, T - n + i + 1)) if causal else T
        if vis == 0:
            continue
        for hq in range(Hq):
            kk, vv = k[:vis, hq // G], v[:vis, hq // G]
            s = scale * (kk @ q[i, hq])
            m = s.max()
            p = np.exp(s - m)
            l = p.sum()
            out[i, hq], mass[i, hq] = p @ vv / l, p @ np.abs(vv) / l
            lse[i, hq] = m + math.log(l)
            reach[i, hq] = (abs(scale) * (np.abs(kk) @ np.abs(q[i, hq]))).max()
    return out, lse, mass, reach


class PagedModel:
    """Tokens, page tables and reference counts of a cache; sequences keep their raw tokens."""

    def __init__(self, Hkv, d, pages, slots, max_pages, page, code, layers=1):
        self.Hkv, self.d, self.page, self.code, self.layers = Hkv, d, page, code, layers
        self.max_pages = max_pages
        self.ref = [0] * pages
        self.table = [[] for _ in range(slots)]
        self.tok = [[(np.zeros((0, Hkv, d)),) * 2 for _ in range(layers)] for _ in range(slots)]
        self.len = [0] * slots

    def _take(self, n):
        free = [p for p, r in enumerate(self.ref) if r == 0]
        if len(free) < n:
            raise RuntimeError("pages")
        for p in free[:n]:
            self.ref[p] = 1
        return free[:n]

    def append(self, slot, KV):
        """KV: per layer (K [n, Hkv, d], V)."""
        n = KV[0][0].shape[0]
        need = -(-(self.len[slot] + n) // self.page) - len(self.table[slot])
        self.table[slot] += self._take(need)
        for l in range(self.layers):
            self.tok[slot][l] = tuple(np.concatenate([a, b]) for a, b in zip(self.tok[slot][l], KV[l]))
        self.len[slot] += n

    def values(self, slot, layer=0):
        return tuple(cached_values(t, self.code, self.page) for t in self.tok[slot][layer])

    def fork(self, a, b, share=True):
        assert self.len[b] == 0 and not self.table[b]
        full = self.len[a] // self.page if share else 0
        for p in self.table[a][:full]:
            self.ref[p] += 1
        self.table[b] = self.table[a][:full] + self._take(len(self.table[a]) - full)
        self.tok[b], self.len[b] = [t for t in self.tok[a]], self.len[a]

    def free(self, s):
        for p in self.table[s]:
            self.ref[p] -= 1
        self.table[s], self.len[s] = [], 0
        self.tok[s] = [(np.zeros((0, self.Hkv, self.d)),) * 2 for _ in range(self.layers)]

    def compact(self):
        live = sum(r > 0 for r in self.ref)
        holes = [p for p in range(live) if self.ref[p] == 0]
        high = [p for p in range(live, len(self.ref)) if self.ref[p] > 0]
        to = dict(zip(high, holes))
        for a, b in to.items():
            self.ref[b], self.ref[a] = self.ref[a], 0
        self.table = [[to.get(p, p) for p in t] for t in self.table]

"""Plain float64 forms of the serving operators, for their tests: the 8-bit cache's number format, its write, the
attention over it, the weight of prompt keys and the eviction, each from its definition."""
import math

import numpy as np

PAGE = 64
QMAX = {"int8": 127.0, "e4m3": 448.0}

# the finite e4m3 numbers of codes 0 .. 0x7E (sign 0): 4 exponent bits (bias 7), 3 mantissa bits
E4M3 = np.array([(m / 8.0) * 2.0 ** -6 if e == 0 else (1 + m / 8.0) * 2.0 ** (e - 7)
                 for e in range(16) for m in range(8)][:127])


def scale_rule(amax, code):
    """0 for 0, else the smallest 2^e >= amax / Qmax with e >= -126, by exact search."""
    if amax == 0:
        return 0.0
    e = -126
    if amax > 0 and math.isfinite(amax):
        e = max(-126, math.frexp(amax / QMAX[code])[1] - 2)
    while math.ldexp(QMAX[code], e) < amax:
        e += 1
    return math.ldexp(1.0, e)


def encode(y, code):
    """Values in units of their scale -> the values that their codes stand for (still in those units)."""
    y = np.clip(np.where(np.isnan(y), 0.0, y), -QMAX[code], QMAX[code])
    if code == "int8":
        return np.rint(y)
    a = np.abs(y)
    hi = np.minimum(np.searchsorted(E4M3, a), 126)   # first number >= a
    lo = np.maximum(hi - 1, 0)
    up, down = E4M3[hi] - a, a - E4M3[lo]
    pick = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    pick = np.where(E4M3[hi] == a, hi, pick)
    return np.copysign(E4M3[pick], y)


def finite_max(x):
    f = np.where(np.isfinite(x), np.abs(x), 0.0)
    return float(f.max()) if f.size else 0.0


class Cache:
    """values[b][h]: list of slots in code units with one scale per block, as float64."""

    def __init__(self, B, H_kv, D, max_pages, code):
        self.code, self.D, self.max_pages = code, D, max_pages
        self.units = {n: np.zeros((B, H_kv, max_pages, PAGE, D)) for n in "kv"}
        self.scale = {n: np.zeros((B, H_kv, max_pages)) for n in "kv"}
        self.weight = np.zeros((B, H_kv, max_pages * PAGE))
        self.pos = np.zeros((B, H_kv, max_pages * PAGE), np.int64)

    def append(self, k, v, start, count=None, row=None):
        B, n_new = k.shape[:2]
        for b in range(B):
            c = n_new if count is None else min(max(int(count[b]), 0), n_new)
            s0 = int(start[b])
            for blk in range(self.max_pages):
                slots = np.arange(blk * PAGE, blk * PAGE + PAGE)
                t = slots - s0
                fresh, old = (t >= 0) & (t < c), t < 0
                if not fresh.any():
                    continue
                for name, x in (("k", k), ("v", v)):
                    for h in range(x.shape[2]):
                        new = x[b, t[fresh], h]
                        was = self.scale[name][b, h, blk] if old.any() else 0.0
                        s = max(was, scale_rule(finite_max(new), self.code))
                        u = self.units[name][b, h, blk]
                        with np.errstate(all="ignore"):
                            if s > 0:
                                u[fresh] = encode(new / s, self.code)
                                if s != was:
                                    u[old] = encode(u[old] * (was / s), self.code)
                            else:
                                u[fresh] = 0.0
                        self.scale[name][b, h, blk] = s
                self.weight[b, :, slots[fresh]] = 0.0
                self.pos[b, :, slots[fresh]] = ((s0 if row is None else int(row[b])) + t[fresh])[:, None]

    def values(self, name, b, h):
        return (self.units[name][b, h] * self.scale[name][b, h][:, None, None]).reshape(-1, self.D)

    def evict(self, dst, lens, budget, recent):
        """Into dst, another Cache; returns the new lengths."""
        new_len = np.minimum(lens, budget)
        for b in range(len(lens)):
            for h in range(self.weight.shape[1]):
                n = int(lens[b])
                if n <= budget:
                    kept = np.arange(n)
                else:
                    w = self.weight[b, h, :n - recent]
                    key = np.where(np.isnan(w), np.inf, w)  # NaN counts as the largest: above an infinity
                    order = sorted(range(n - recent), key=lambda i: (not np.isnan(w[i]), -key[i], i))
                    kept = np.concatenate([np.sort(np.array(order[:budget - recent], np.int64)),
                                           np.arange(n - recent, n)]).astype(np.int64)
                for name in "kv":
                    x = self.values(name, b, h)[kept]
                    for blk in range(-(-len(kept) // PAGE)):
                        part = x[blk * PAGE:(blk + 1) * PAGE]
                        s = scale_rule(finite_max(part), self.code)
                        dst.scale[name][b, h, blk] = s
                        dst.units[name][b, h, blk] = 0.0
                        if s > 0:
                            dst.units[name][b, h, blk, :len(part)] = encode(part / s, self.code)
                dst.weight[b, h, :len(kept)] = self.weight[b, h, kept]
                dst.pos[b, h, :len(kept)] = self.pos[b, h, kept]
        return new_len


def seen(j, i, vecs, n_k, causal):
    """[len(i), len(j)]: key of row index j is unmasked for row i.  vecs: four int arrays [n_k] or None each."""
    j, i = np.asarray(j)[None, :], np.asarray(i)[:, None]
    ok = np.ones((i.shape[0], j.shape[1]), bool)
    if causal:
        ok &= j <= i
    if vecs is not None and any(v is not None for v in vecs):
        inside = (j >= 0) & (j < n_k)
        at = np.clip(j, 0, n_k - 1)
        big = np.iinfo(np.int32).max
        lts, lte, uts, ute = (np.full(n_k, d, np.int64)[at] if v is None else np.asarray(v, np.int64)[at]
                              for v, d in zip(vecs, (big, big, 0, 0)))
        ok &= ~(inside & (((lts <= i) & (i < lte)) | ((uts <= i) & (i < ute))))
    return ok


def attention(q, K, V, ok, scale):
    """q [R, D], K, V [n, D], ok [R, n] -> O, LSE, weights [R, n], and the sums of |terms| that error bounds need:
    sum_d |q_d k_d| * scale [R, n] and sum_j p_j |v_j| [R, D]."""
    s = scale * (q @ K.T)
    s = np.where(ok, s, -np.inf)
    with np.errstate(all="ignore"):
        m = s.max(-1, initial=-np.inf)
        p = np.where(ok, np.exp(s - np.where(np.isfinite(m), m, 0.0)[:, None]), 0.0)
        total = p.sum(-1)
        p = np.where(total[:, None] > 0, p / np.where(total > 0, total, 1.0)[:, None], 0.0)
        lse = np.where(total > 0, m + np.log(np.where(total > 0, total, 1.0)), -np.inf)
    return p @ V, lse, p, scale * (np.abs(q) @ np.abs(K).T), p @ np.abs(V)

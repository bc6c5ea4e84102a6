"""Plain 64-bit statements of the KV cache operators, one token, key or page at a time (test infrastructure)."""
import math

import numpy as np

U = 2.0 ** -24          # half a step of fp32, relative


def cu_of(ns):
    return np.concatenate([[0], np.cumsum(ns)]).astype(np.int32)


def rope(x, heads, d, rot, adjacent, pos, axis, freq):
    """x [ntok][heads * d] fp32 -> (values, error bounds)."""
    ntok = x.shape[0]
    x = x.astype(np.float64).reshape(ntok, heads, d)
    y, e = x.copy(), np.zeros_like(x)
    half = rot // 2
    for i in range(half):
        ia, ib = (2 * i, 2 * i + 1) if adjacent else (i, half + i)
        # the angle of a position in whole turns, by exact integer arithmetic on the fp64 frequency
        ang = np.array([math.remainder(int(p) * float(freq[i]), 2 * math.pi) for p in pos[axis[i]]])
        c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
        a, b = x[..., ia], x[..., ib]
        y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
        # angle to fp32 (2^-24 of at most pi), sincospi (2 ulps), two products and a sum: at most 10 half steps;
        # the fp64 angle itself: 2^-51 of it
        far = 2.0 ** -51 * np.abs(pos[axis[i]] * float(freq[i]))[:, None]
        e[..., ia] = e[..., ib] = (np.abs(a) + np.abs(b)) * (10 * U + far)
    return y.reshape(ntok, -1), e.reshape(ntok, -1)


def quant(x, s):
    """fp32 values / an fp32 scale, rounded to nearest even in 64 bits (exact up to the border: |x/s| <= 127.01, 53 bits)."""
    if not (s > 0):
        return np.zeros(x.shape, np.int8)
    return np.clip(np.rint(x.astype(np.float64) / np.float64(s)), -127, 127).astype(np.int8)


class Cache:
    """Host copy of an lq_kv8 pool."""

    def __init__(self, n_pages, n_kv, page, d, rng=None):
        self.n_pages, self.n_kv, self.page, self.d = n_pages, n_kv, page, d
        sh = (n_pages, n_kv)
        if rng is None:
            self.k, self.v = np.zeros(sh + (page, d), np.int8), np.zeros(sh + (d, page), np.int8)
            self.ks, self.vs = np.zeros(sh, np.float32), np.zeros(sh, np.float32)
        else:
            self.k = np.clip(np.rint(rng.standard_normal(sh + (page, d)) * 40), -127, 127).astype(np.int8)
            self.v = np.clip(np.rint(rng.standard_normal(sh + (d, page)) * 40), -127, 127).astype(np.int8)
            self.ks = np.exp(rng.standard_normal(sh) - 3.5).astype(np.float32)
            self.vs = np.exp(rng.standard_normal(sh) - 3.5).astype(np.float32)

    def append(self, table, start, cu, k, v):
        P = self.page
        with np.errstate(all="ignore"):
            for s in range(len(start)):
                n = int(cu[s + 1] - cu[s])
                at, end = max(int(start[s]), 0), int(start[s]) + n
                while at < end:
                    pj = at // P
                    to = min(end, (pj + 1) * P)
                    page = table[s][pj] if pj < table.shape[1] else -1
                    if 0 <= page < self.n_pages:
                        r = int(cu[s]) + at - int(start[s])
                        self._page(page, at - pj * P, k[r:r + to - at].reshape(to - at, self.n_kv, self.d),
                                   v[r:r + to - at].reshape(to - at, self.n_kv, self.d))
                    at = to

    def _page(self, page, slot, k, v):
        m = k.shape[0]
        for h in range(self.n_kv):
            for codes, scales, x in ((self.k[page, h], self.ks, k[:, h]), (self.v[page, h].T, self.vs, v[:, h])):
                was = scales[page, h] if slot > 0 else np.float32(0)
                mine = np.abs(x).max() * (np.float32(1) / np.float32(127)) if np.isfinite(x).all() else np.float32(np.nan)
                now = was if np.isnan(was) or was >= mine else mine
                good = np.isfinite(now) and now > 0
                if good and slot > 0 and now > was:
                    codes[:slot] = quant(codes[:slot].astype(np.float32) * was, now)
                codes[slot:slot + m] = quant(x, now) if good else 0
                scales[page, h] = now


def attn(c, table, start, cu, q, n_q, scale, softcap=0.0, window=0, prefix=None, slopes=None):
    """q [ntok][n_q * d] -> (out, bound)."""
    ntok, d, g = q.shape[0], c.d, n_q // c.n_kv
    out, bound = np.zeros((ntok, n_q, d)), np.zeros((ntok, n_q, d))
    q = q.astype(np.float64).reshape(ntok, n_q, d)
    P = c.page
    for s in range(len(start)):
        n = int(cu[s + 1] - cu[s])
        L = int(start[s]) + n
        if n == 0 or L <= 0:
            continue
        pages = [int(table[s][j]) if j < table.shape[1] else -1 for j in range(-(-L // P))]
        held = np.repeat([0 <= p < c.n_pages for p in pages], P)[:L]
        pages = [p if 0 <= p < c.n_pages else 0 for p in pages]
        for h in range(n_q):
            hk = h // g
            K = (c.k[pages, hk].astype(np.float64) * c.ks[pages, hk].astype(np.float64)[:, None, None]).reshape(-1, d)[:L]
            V = (c.v[pages, hk].astype(np.float64) * c.vs[pages, hk].astype(np.float64)[:, None, None]) \
                .transpose(0, 2, 1).reshape(-1, d)[:L]
            j = np.arange(L)
            for i in range(n):
                p = int(start[s]) + i
                if p < 0:
                    continue
                sees = (j <= p) & ((window == 0) | (p - j < window))
                if prefix is not None:
                    sees = sees | (j < prefix[s])
                sees = sees & held
                if not sees.any():
                    continue
                qi, Ks, Vs, js = q[cu[s] + i, h], K[sees], V[sees], j[sees]
                t = scale * (Ks @ qi)
                # the score: pieces of q (2^-21 of its largest value against |k|), d / 16 + 4 sums, the scales
                et = abs(scale) * (2.0 ** -21 * np.abs(qi).max() * np.abs(Ks).sum(1) + (d / 8 + 8) * U * (np.abs(Ks) @ np.abs(qi)))
                if softcap:
                    t = softcap * np.tanh(t / softcap)
                    et = et + 8 * U * np.abs(t)
                if slopes is not None:
                    b = np.float64(slopes[h]) * np.abs(p - js)
                    t = t - b
                    et = et + 3 * U * b
                et = et + 4 * U * np.abs(t)                      # to powers of two
                w = np.exp(t - t.max())
                w = w / w.sum()
                out[cu[s] + i, h] = w @ Vs
                # weights: e^(2 et) - 1 over the row; the pieces of the weights and the sums over the keys; a floor
                # where a weight next to the largest of the row leaves fp16
                mag = w @ np.abs(Vs)
                rel = 2 * np.expm1((w * et).sum() + et[w > 1e-9].max()) + 2.0 ** -20 + (len(js) / 8 + 64) * U
                bound[cu[s] + i, h] = mag * rel + 2.0 ** -36 * np.abs(Vs).max() * len(js) + 1e-30
    return out.reshape(ntok, -1), bound.reshape(ntok, -1)


# ---- pages


class Pages:
    def __init__(self, n_rows, max_pages, n_pages, page):
        self.page, self.n_pages = page, n_pages
        self.table = np.full((n_rows, max_pages), -1, np.int32)
        self.ref = np.zeros(n_pages, np.int32)
        self.lens = np.zeros(n_rows, np.int32)

    def _free(self):
        return [int(p) for p in np.flatnonzero(self.ref == 0)]

    def reserve(self, start, cu):
        want = []
        for s in range(len(start)):
            n = int(cu[s + 1] - cu[s])
            a, e = max(int(start[s]), 0), int(start[s]) + n
            if n <= 0 or e <= a:
                continue
            if (e - 1) // self.page >= self.table.shape[1]:
                return (0, 1)
            miss = [j for j in range(a // self.page, (e - 1) // self.page + 1) if self.table[s, j] < 0]
            if miss and len(miss) != (e - 1) // self.page + 1 - miss[0]:
                return (0, 1)
            want += [(s, j) for j in miss]
        free = self._free()
        if len(free) < len(want):
            return (len(want) - len(free), 0)
        for (s, j), p in zip(want, free):
            self.table[s, j] = p
            self.ref[p] = 1
        return (0, 0)

    def fork(self, parent, child):
        n = len(parent)
        tails = [int(self.lens[p]) % self.page > 0 for p in parent]
        free = self._free()
        src, dst = np.full(n, -1, np.int32), np.full(n, -1, np.int32)
        if sum(tails) > len(free):
            return src, dst, (sum(tails) - len(free), 0)
        it = iter(free)
        for i in range(n):
            p, c = int(parent[i]), int(child[i])
            full = int(self.lens[p]) // self.page
            self.table[c] = -1
            self.table[c, :full] = self.table[p, :full]
            for x in self.table[p, :full]:
                self.ref[x] += 1
            if tails[i]:
                src[i], dst[i] = self.table[p, full], next(it)
                self.table[c, full] = dst[i]
                self.ref[dst[i]] = 1
            self.lens[c] = self.lens[p]
        return src, dst, (0, 0)

    def release(self, rows):
        for r in rows:
            for p in self.table[r]:
                if p >= 0:
                    self.ref[p] -= 1
            self.table[r] = -1
            self.lens[r] = 0

    def compact(self):
        u = int((self.ref > 0).sum())
        high = [p for p in range(u, self.n_pages) if self.ref[p] > 0]
        low = [p for p in range(u) if self.ref[p] <= 0]
        m = np.array([p if self.ref[p] > 0 else -1 for p in range(self.n_pages)], np.int32)
        src, dst = np.full(self.n_pages // 2, -1, np.int32), np.full(self.n_pages // 2, -1, np.int32)
        for i, (a, b) in enumerate(zip(high, low)):
            src[i], dst[i], m[a] = a, b, b
            self.ref[b], self.ref[a] = self.ref[a], 0
        self.table = np.where(self.table >= 0, m[np.maximum(self.table, 0)], -1).astype(np.int32)
        return m, src, dst, len(high)

"""CPU oracle of what a paged cache's pages hold -- TEST INFRASTRUCTURE ONLY.

The operators of include/cachedata.h, one row at a time on numpy arrays, in 64
bits but where the header fixes 32-bit steps. It shares nothing with the CUDA
library. Pools are [pages, tokens, heads, width] here (scales without the
width): tests hand over transposed views of the other order.
"""

from __future__ import annotations

import numpy as np

OK, INVALID = 0, 1
KEEP_ALL = 0xFFFFFFFF
LARGEST = {"e4m3": 448.0, "i8": 127.0}
MAX_NODES = 1024


def _e4m3_values() -> np.ndarray:
    """The value of each 8-bit code (code 127 and 255 are NaN)."""
    v = np.zeros(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = m * 2.0**-9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        v[c] = np.nan if c & 127 == 127 else (-x if c & 128 else x)
    return v


E4M3 = _e4m3_values()


def e4m3_code(x) -> np.ndarray:
    """Nearest codes (ties to the even one) of finite float32 values, saturated."""
    x = np.asarray(x, np.float32).astype(np.float64)
    mags = E4M3[:127]
    a = np.minimum(np.abs(x), 448.0)
    hi = np.clip(np.searchsorted(mags, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    up, down = mags[hi] - a, a - mags[lo]
    code = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return (code | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def quantise(row, kind):
    """(codes as bytes, scale) of one row of float32 values."""
    row = np.asarray(row, np.float32)
    if not np.isfinite(row).all():
        return np.zeros(row.size, np.uint8), np.float32(np.nan)
    top, full = np.abs(row).max(), np.float32(LARGEST[kind])
    with np.errstate(divide="ignore", over="ignore", under="ignore"):
        by, scale = np.float32(full / top), np.float32(top / full)
    if scale == 0 or np.isinf(by):
        return np.zeros(row.size, np.uint8), np.float32(0)
    x = (row * by).astype(np.float32)
    if kind == "e4m3":
        return e4m3_code(x), scale
    return np.clip(np.rint(x), -127, 127).astype(np.int8).view(np.uint8), scale


class Batch:
    """Requests of a batch on tables: table [n_seqs, columns], length, n_pages, T tokens a page."""

    def __init__(self, table, length, n_pages, T, seq, start, rows, fresh, max_tokens=None):
        self.table, self.length, self.n_pages, self.T = np.asarray(table), np.asarray(length), n_pages, T
        self.requests, self.status = [], []
        self.broken = False
        for i in range(len(seq)):
            s, a, b = int(seq[i]), int(start[i]), int(start[i + 1])
            ok = 0 <= s < self.table.shape[0] and 0 <= a <= b <= rows
            n = int(self.length[s]) & 0xFFFFFFFF if ok else 0
            ok = ok and n < 1 << 31 and n <= self.table.shape[1] * T and not (fresh and b - a > n)
            ok = ok and (max_tokens is None or b - a <= max_tokens)
            self.status.append(OK if ok else INVALID)
            self.requests.append((s, a, b - a, n) if ok else None)

    def counters(self):
        return [sum(r[2] for r in self.requests if r), sum(r is None for r in self.requests), 0, 8 if self.broken else 0]

    def place(self, s, position):
        """(page, slot), or None where the table names no page."""
        page = int(self.table[s, position // self.T])
        if not 0 <= page < self.n_pages:
            self.broken = True
            return None
        return page, position % self.T


def write(b: Batch, rows, pool, scale, kind, narrow):
    """rows [rows, heads, width] of float32 values into pool (bytes or 16-bit) and scale, in place.
    narrow(x): float32 values as a 16-bit cache holds them."""
    for r in b.requests:
        if r is None:
            continue
        s, first, m, n = r
        for j in range(m):
            at = b.place(s, n - m + j)
            if at is None:
                continue
            for h in range(rows.shape[1]):
                if kind in LARGEST:
                    pool[at][h], scale[at][h] = quantise(rows[first + j, h], kind)
                else:
                    pool[at][h] = narrow(rows[first + j, h])


def values(pool, scale):
    """Cached values in 64 bits: pool of numbers (codes' values), scale or None."""
    with np.errstate(invalid="ignore"):
        return pool.astype(np.float64) * (1.0 if scale is None else scale.astype(np.float64)[..., None])


def read(b: Batch, first, vals, out):
    """out [rows, heads, width] gets positions first[i] on; vals [pages, tokens, heads, width]."""
    for i, r in enumerate(b.requests):
        if r is None:
            continue
        s, row, m, n = r
        for j in range(m):
            position = (int(first[i]) & 0xFFFFFFFF if first is not None else 0) + j
            at = b.place(s, position) if position < n else None
            out[row + j] = 0 if at is None else vals[at]


def attend(b: Batch, q, keys, vals, scale, mask=None):
    """(out, lse, spread, size): spread is sum of weights times |v|, over their sum, which bounds what roundings of
    the weights do; size the largest sum of |q_d k_d| scale of a row, which bounds what those of scores do. mask
    [rows, words] of 32-bit words. Rows of no valid request are NaN."""
    rows, q_heads, width = q.shape
    group = q_heads // keys.shape[2]
    out, spread = np.full((2,) + q.shape, np.nan)
    lse, size = np.full((2, rows, q_heads), np.nan)
    for r in b.requests:
        if r is None:
            continue
        s, first, m, n = r
        places = [b.place(s, x) for x in range(n)]
        there = np.array([p is not None for p in places], bool)
        at = np.array([p if p is not None else (0, 0) for p in places], np.int64).reshape(n, 2)
        k, v = keys[at[:, 0], at[:, 1]].astype(np.float64), vals[at[:, 0], at[:, 1]].astype(np.float64)
        own = np.arange(n) - (n - m)
        for j in range(m):
            if mask is None:
                sees = own <= j
            else:
                bits = [(int(mask[first + j, o // 32]) >> (o % 32)) & 1 for o in range(m)]
                sees = np.concatenate([np.ones(n - m, bool), np.array(bits, bool)])
            sees = sees & there
            for x in range(q_heads):
                where = (first + j, x)
                if not sees.any():
                    out[where], lse[where], spread[where], size[where] = 0, -np.inf, 0, 0
                    continue
                kk, vv, qq = k[sees, x // group], v[sees, x // group], q[where].astype(np.float64)
                with np.errstate(invalid="ignore", over="ignore"):
                    sc = (kk @ qq) * scale
                    size[where] = np.nanmax(np.abs(kk) @ np.abs(qq)) * abs(scale)
                    top = sc.max()
                    if top == -np.inf:
                        out[where], lse[where], spread[where] = 0, -np.inf, 0
                        continue
                    w = np.exp(sc - top)
                    out[where] = (w @ vv) / w.sum()
                    spread[where] = (w @ np.abs(vv)) / w.sum()
                    lse[where] = top + np.log(w.sum())
    return out, lse, spread, size


ONE = 1 << 44


def _uniform(u) -> float:
    """A random number as the call takes it: in [0, 1), NaN as 0."""
    return 0.0 if np.isnan(u) else float(np.float32(min(max(float(u), 0.0), 1 - 2.0**-24)))


def verify(start, rows, parent, token, p, q, u, vocab):
    """(path, accepted, next, status) of the trees; p, q float32 [rows, vocab]. Weights are 32-bit floats and
    sums of them integers, as the header says."""
    n = len(start) - 1
    path, accepted, following, status = np.full(rows, -7, np.int64), [], [], []

    def clean(x):
        x = np.asarray(x, np.float32)
        return np.where(np.isnan(x), np.float32(0), np.clip(x, np.float32(0), np.float32(1))).astype(np.float32)

    def fixed(w):
        return np.rint(w.astype(np.float64) * ONE).astype(np.int64)

    for i in range(n):
        a, e = int(start[i]), int(start[i + 1])
        placed = 0 <= a <= e <= rows
        m = e - a if placed else 0
        ok = 0 < m <= MAX_NODES and all(
            0 <= parent[a + j] < j and 0 <= token[a + j] < vocab for j in range(1, m))
        if not ok:
            path[a:a + m] = -1
            accepted.append(0), following.append(-1), status.append(INVALID)
            continue
        here, way, W, refused = 0, [0], 1.0, set()
        target = clean(p[a])
        w = target.copy()
        for j in range(1, m):
            if parent[a + j] != here:
                continue
            t = int(token[a + j])
            by = float(clean(q[a + here])[t]) if q is not None else 1.0
            if _uniform(u[a + j]) * by * W < float(w[t]):
                here, W, refused = j, 1.0, set()
                way.append(j)
                target = clean(p[a + j])
                w = target.copy()
            elif q is not None:
                inv = np.float32(1.0 / W) if W > 0 else np.float32(1)
                d = clean(q[a + here]).astype(np.float64)
                # one rounding of the product less q (a fused multiply-add) or two: see fused below
                w = np.maximum(fused(w, inv, d), np.float32(0))
                W = float(fixed(w).sum()) / ONE
            else:
                W -= float(w[t])
                w[t] = 0
        x = fixed(w)
        total = int(x.sum())
        if total == 0:
            x = fixed(target)
            total = int(x.sum())
        path[a:a + m] = -1
        path[a:a + len(way)] = way
        accepted.append(len(way)), status.append(OK)
        if total == 0:
            following.append(-1)
            continue
        goal = (total * int(_uniform(u[a]) * 2.0**64)) >> 64
        following.append(int(np.searchsorted(np.cumsum(x), goal, side="right")))
    return path, np.array(accepted, np.int64), np.array(following, np.int64), status


def fused(w, inv, q):
    """w * inv - q in 32 bits, rounded once (the product of two 32-bit floats is exact in 64 bits, and the
    difference rounded to 64 bits before 32 differs from one rounding in none of the tests' values)."""
    return (w.astype(np.float64) * float(inv) - q).astype(np.float32)


def keep(b: Batch, path, accepted, pool):
    """The accepted tokens move together in pool [planes, pages, tokens, ...], in place; the cuts."""
    cut = []
    for i, r in enumerate(b.requests):
        s = None if r is None else r[0]
        if r is not None:
            _, first, m, n = r
            a = int(accepted[i]) & 0xFFFFFFFF
            way = [int(x) for x in path[first:first + min(a, m)]]
            if a > m or any(not 0 <= x < m for x in way) or any(x >= y for x, y in zip(way, way[1:])):
                b.status[i], b.requests[i] = INVALID, None
                r = None
        cut.append([s, KEEP_ALL if r is None else n - m + a])
        if r is None:
            continue
        for k, x in enumerate(way):
            if x == k:
                continue
            src, dst = b.place(s, n - m + x), b.place(s, n - m + k)
            if src is not None and dst is not None:
                pool[(slice(None),) + dst] = pool[(slice(None),) + src]
    return cut

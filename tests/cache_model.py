"""A plain model of the paged 4-bit cache in NumPy float64, written from the definitions.

The model keeps each sequence as a list of pages and each page as arrays of held values; it shares
no code with the package or the oracle."""

import math

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def e4m3_grid():
    """The 127 finite non-negative e4m3 values by code: 2^(e-7) (1 + m/8), m/8 2^-6 where e = 0."""
    c = np.arange(127)
    e, m = c >> 3, c & 7
    return np.where(e > 0, 2.0 ** (e - 7.0) * (1 + m / 8), m / 8 * 2.0 ** -6)


E4M3 = e4m3_grid()


def nearest(x, grid):
    """Index of the grid value nearest to x >= 0 (saturating), ties to the even index."""
    x = np.asarray(x, np.float64)
    hi = np.clip(np.searchsorted(grid, x), 1, len(grid) - 1)
    lo = hi - 1
    with np.errstate(invalid="ignore"):
        up, down = grid[hi] - x, x - grid[lo]
    pick = np.where(up < down, hi, np.where(down < up, lo, np.where(lo % 2 == 0, lo, hi)))
    return np.where(x >= grid[-1], len(grid) - 1, pick)


def quantise(x, exp=0):
    """(codes, scale codes) of x [..., d]: codes [..., d] in 0..15, scale codes [..., d / 16] (127: NaN)."""
    y = np.asarray(x, np.float64) * 2.0 ** -exp
    g = y.reshape(y.shape[:-1] + (-1, 16))
    nan = np.isnan(g).any(-1)
    a = np.abs(np.where(np.isnan(g), 0, g)).max(-1)
    s = nearest(np.minimum(a / 6, 448.0), E4M3)
    step = E4M3[s]
    with np.errstate(divide="ignore", invalid="ignore"):
        r = np.where(step[..., None] > 0, np.abs(g) / step[..., None], 0.0)
    c = nearest(np.where(np.isnan(r), 0, r), E2M1) + 8 * np.signbit(g)
    c = np.where((step[..., None] > 0) & ~nan[..., None], c, 0)
    return c.reshape(y.shape), np.where(nan, 127, s)


def values(codes, scales, exp=0):
    step = np.append(E4M3, np.nan)[scales]
    v = E2M1[codes & 7] * np.where(codes >= 8, -1.0, 1.0)
    return v * np.repeat(step, 16, -1) * 2.0 ** exp


def pack(codes):
    return (codes[..., 0::2] + 16 * codes[..., 1::2]).astype(np.uint8)


class Model:
    def __init__(self, pages, seqs, blocks, heads, d, chunk, k_exp=0, v_exp=0):
        self.np, self.ns, self.nb, self.h, self.d, self.chunk = pages, seqs, blocks, heads, d, chunk
        self.exp = (k_exp, v_exp)
        self.refs = np.zeros(pages, np.int64)
        self.table = np.full((seqs, blocks), -1, np.int64)
        self.lengths = np.zeros(seqs, np.int64)
        self.codes = [np.zeros((pages, heads, chunk, d), np.int64) for _ in "kv"]
        self.scales = [np.zeros((pages, heads, chunk, d // 16), np.int64) for _ in "kv"]
        self.mean = np.zeros((pages, heads, d))

    def held(self, x, page):
        return values(self.codes[x][page], self.scales[x][page], self.exp[x])

    def reserve(self, upto):
        want = []
        for i, u in enumerate(upto):
            have = int((self.table[i] >= 0).sum())
            want += [(i, j) for j in range(have, -(-int(u) // self.chunk))]
        free = np.flatnonzero(self.refs == 0)
        if len(free) < len(want):
            return False
        for (i, j), p in zip(want, free):
            self.table[i, j] = p
            self.refs[p] = 1
        return True

    def append(self, k, v, cu, start):
        """k, v float64 [n, heads, d]; returns the held values."""
        held = [np.zeros_like(k), np.zeros_like(v)]
        for i in range(self.ns):
            for r in range(cu[i], cu[i + 1]):
                t = int(start[i]) + r - cu[i]
                p, o = self.table[i, t // self.chunk], t % self.chunk
                for x, y in enumerate((k, v)):
                    c, s = quantise(y[r], self.exp[x])
                    self.codes[x][p, :, o], self.scales[x][p, :, o] = c, s
                    held[x][r] = values(c, s, self.exp[x])
                if o == self.chunk - 1:
                    self.mean[p] = self.held(0, p).mean(1)
            if cu[i + 1] > cu[i]:
                self.lengths[i] = start[i] + cu[i + 1] - cu[i]
        return held

    def fork(self, src, dst):
        free = np.flatnonzero(self.refs == 0)
        if (self.lengths[src] % self.chunk > 0).sum() > len(free):
            return False
        at = 0
        for a, b in zip(src, dst):
            n = int(self.lengths[a])
            for j in range(n // self.chunk):
                self.table[b, j] = self.table[a, j]
                self.refs[self.table[a, j]] += 1
            if n % self.chunk:
                p, old, m = free[at], self.table[a, n // self.chunk], n % self.chunk
                at += 1
                self.table[b, n // self.chunk] = p
                self.refs[p] = 1
                for x in (0, 1):
                    self.codes[x][p, :, :m] = self.codes[x][old, :, :m]
                    self.scales[x][p, :, :m] = self.scales[x][old, :, :m]
            self.lengths[b] = n
        return True

    def free(self, seqs):
        for i in seqs:
            for p in self.table[i]:
                if p >= 0:
                    self.refs[p] -= 1
            self.table[i] = -1
            self.lengths[i] = 0

    def compact(self, into):
        live = np.flatnonzero(self.refs > 0)
        if len(live) > into.np:
            return False
        name = {int(p): n for n, p in enumerate(live)}
        for p, n in name.items():
            for x in (0, 1):
                into.codes[x][n], into.scales[x][n] = self.codes[x][p], self.scales[x][p]
            into.mean[n] = self.mean[p]
        into.refs[:] = 0
        into.refs[:len(live)] = self.refs[live]
        into.table[:] = np.vectorize(lambda p: name.get(int(p), -1))(self.table)
        into.lengths[:] = self.lengths
        return True

    def decode(self, q, topk, scale=None):
        """out [seqs, hq, d], lse [hq, seqs], and per row: the smallest gap between the score of the last
        block taken and the best one left, over the largest sum |q mean| of a block (inf where all are taken),
        sum p |v| and the largest sum |q k| per key (for error bounds).  q float64."""
        hq, d = q.shape[1], self.d
        scale = scale or 1 / math.sqrt(d)
        out, lse = np.zeros(q.shape), np.full((hq, self.ns), -np.inf)
        gap, pv, qk = np.full((self.ns, hq), np.inf), np.zeros(q.shape), np.zeros((self.ns, hq))
        for i in range(self.ns):
            n = int(self.lengths[i])
            if not n:
                continue
            own = (n - 1) // self.chunk
            for h in range(hq):
                g = h // (hq // self.h)
                take = list(range(own + 1))
                if topk and own > topk - 1:
                    s = self.mean[self.table[i, :own], g] @ q[i, h]
                    order = np.lexsort((np.arange(own), -s))
                    take = sorted(order[:topk - 1]) + [own]
                    if topk > 1:
                        size = (np.abs(self.mean[self.table[i, :own], g]) @ np.abs(q[i, h])).max()
                        gap[i, h] = (s[order[topk - 2]] - s[order[topk - 1]]) / max(size, 1e-300)
                ks, vs = [], []
                for j in take:
                    m = n - own * self.chunk if j == own else self.chunk
                    ks.append(self.held(0, self.table[i, j])[g, :m])
                    vs.append(self.held(1, self.table[i, j])[g, :m])
                ks, vs = np.concatenate(ks), np.concatenate(vs)
                z = scale * (ks @ q[i, h])
                top = z.max()
                p = np.exp(z - top)
                out[i, h] = p @ vs / p.sum()
                lse[h, i] = top + math.log(p.sum())
                pv[i, h] = p @ np.abs(vs) / p.sum()
                qk[i, h] = scale * (np.abs(ks) @ np.abs(q[i, h])).max()
        return out, lse, gap, pv, qk

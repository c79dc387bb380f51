"""The 4-bit paged cache in plain numpy and 64 bits: the oracle of tests/test_gpu_pages.py.

Shares no code with the library: format and page table rules are written out here from their
definition in include/kvs.h, row by row.
"""

import numpy as np

PAGE = 32
HALVES = np.arange(0x7c00, dtype=np.uint16).view(np.float16).astype(np.float64)   # finite, ascending


def page_bytes(d):
    return 36 * d + 128


def quantise(x):
    """(codes 0..15, half scales) of rows x [..., d]."""
    x = np.asarray(x, np.float64)
    y = x.reshape(*x.shape[:-1], -1, 32)
    top = np.abs(y).max(-1)
    bad = ~(top <= 7 * 65504.0)
    top = np.where(bad, 0.0, top)
    s = HALVES[np.searchsorted(7 * HALVES, top)]
    q = np.where(bad[..., None], 0.0, y) / np.where(s == 0, 1.0, s)[..., None]
    code = (np.rint(q) + 8).astype(np.uint8)                      # rint: ties to even
    return code.reshape(x.shape), np.where(bad, np.nan, s).astype(np.float16)


def value(code, s):
    y = (code.astype(np.float64) - 8).reshape(*code.shape[:-1], -1, 32)
    return (y * s.astype(np.float64)[..., None]).reshape(code.shape)


def held(x):
    """What rows x stand for once they are held in 4 bits."""
    return value(*quantise(x))


def _offsets(d, r):
    """Byte offsets, in the order of the channels or blocks, of row r of a page."""
    nb = d // 32
    k = [b * 512 + r * 16 + i for b in range(nb) for i in range(16)]
    v = [16 * d + b * 512 + (r // 2) * 32 + i * 4 + (r % 2) * 2 + j
         for b in range(nb) for i in range(8) for j in range(2)]
    ks = [32 * d + (r * nb + b) * 2 for b in range(nb)]
    vs = [34 * d + (b * 32 + r) * 2 for b in range(nb)]
    return k, v, ks, vs, 36 * d + 4 * r


def put_row(pages, slot, k, v, logn):
    """Quantise one row into pages [P, page_bytes] (uint8)."""
    d = len(k)
    pg = pages[slot // PAGE]
    ko, vo, kso, vso, _ = _offsets(d, slot % PAGE)
    for x, codes, scales in ((k, ko, kso), (v, vo, vso)):
        c, s = quantise(x)
        pg[codes] = c[0::2] | (c[1::2] << 4)
        bits = s.view(np.uint16).copy()
        bits[np.isnan(s)] = 0x7fff
        for o, h in zip(scales, bits):
            pg[o], pg[o + 1] = h & 255, h >> 8
    put_logn(pages, slot, logn)


def put_logn(pages, slot, logn):
    pg = pages[slot // PAGE]
    at = len(pg) - 4 * PAGE + 4 * (slot % PAGE)
    pg[at:at + 4] = np.frombuffer(np.float32(logn).tobytes(), np.uint8)


def get_row(pages, slot, d):
    """(k, v, logn) of a slot as 64-bit values."""
    pg = pages[slot // PAGE]
    ko, vo, kso, vso, lo = _offsets(d, slot % PAGE)
    out = []
    for codes, scales in ((ko, kso), (vo, vso)):
        c = np.empty(d, np.uint8)
        c[0::2], c[1::2] = pg[codes] & 15, pg[codes] >> 4
        s = np.array([int(pg[o]) | int(pg[o + 1]) << 8 for o in scales], np.uint16).view(np.float16)
        out.append(value(c, s))
    return out[0], out[1], float(np.frombuffer(pg[lo:lo + 4].tobytes(), np.float32)[0])


def rows_of(pages, table, n, d):
    """Rows 0 .. n - 1 of the unit with this page table."""
    if n == 0:
        return np.zeros((0, d)), np.zeros((0, d)), np.zeros(0)
    k, v, ln = zip(*(get_row(pages, int(table[t // PAGE]) * PAGE + t % PAGE, d) for t in range(n)))
    return np.array(k), np.array(v), np.array(ln)


def value_scales(pages, table, n, d):
    """The scales [n, d / 32] of the values of rows 0 .. n - 1."""
    out = np.zeros((n, d // 32))
    for t in range(n):
        pg = pages[int(table[t // PAGE])]
        at = _offsets(d, t % PAGE)[3]
        out[t] = np.array([int(pg[o]) | int(pg[o + 1]) << 8 for o in at], np.uint16).view(np.float16)
    return out


def weights(q, k, logn):
    x = q @ k.T / np.sqrt(q.shape[1]) + logn
    p = np.exp(x - x.max(-1, keepdims=True))
    return p / p.sum(-1, keepdims=True)


def attend(q, k, v, logn):
    """(out, size): softmax attention of queries q [G, d], and sum_t p_t |v_t|, which errors of
    the weights scale with. Nothing to attend: zeros."""
    if len(k) == 0 or np.all(logn == -np.inf):
        return np.zeros_like(q), np.zeros_like(q)
    p = weights(q, k, logn)
    return p @ v, p @ np.abs(v)


class Tables:
    """Page tables, free stack and slot maps, one page at a time."""

    def __init__(self, units, max_pages, free):
        self.table = -np.ones((units, max_pages), np.int64)
        self.held = [0] * units
        self.free = list(free)

    def assign(self, rows):
        """False (and nothing changed) when the free pages do not suffice."""
        max_pages = self.table.shape[1]
        want = [(r + PAGE - 1) // PAGE if 0 <= r <= max_pages * PAGE else h
                for r, h in zip(rows, self.held)]
        need = sum(max(0, w - h) for w, h in zip(want, self.held))
        if need > len(self.free) + sum(max(0, h - w) for w, h in zip(want, self.held)):
            return False
        for u, w in enumerate(want):
            for j in range(w, self.held[u]):
                self.free.append(int(self.table[u, j]))
                self.table[u, j] = -1
        taken = self.free[len(self.free) - need:]
        del self.free[len(self.free) - need:]
        for u, w in enumerate(want):
            for j in range(self.held[u], w):
                self.table[u, j] = taken.pop(0)
        self.held = want
        return True

    def slots(self, rows, begin, stride):
        out = -np.ones((len(rows), stride), np.int64)
        for u, r in enumerate(rows):
            for i in range(stride):
                t = begin[u] + i
                if 0 <= t < r and t // PAGE < self.held[u]:
                    out[u, i] = self.table[u, t // PAGE] * PAGE + t % PAGE
        return out

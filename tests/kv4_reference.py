"""The paged 4-bit cache in 64 bits and in plain loops: format, attention and page bookkeeping.

Written from the definitions in include/dg.h, with numpy only; used by the tests.
"""
import numpy as np

PAGE = 64
LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def scale_value(byte):
    """ue5m3: 5 exponent bits (bias 15), 3 mantissa bits; exponent 31 is infinite (mantissa 0) or NaN."""
    byte = np.asarray(byte).astype(np.int64)
    e, m = byte >> 3, byte & 7
    v = np.where(e > 0, (8 + m) * np.exp2(e - 18.0), m * 2.0 ** -17)
    v = np.where(byte == 248, np.inf, v)
    return np.where(byte > 248, np.nan, v)


def nearest(x, grid):
    """Index of the grid value nearest to x, ties to the even index."""
    up = np.clip(np.searchsorted(grid, x), 1, len(grid) - 1)
    low, high = x - grid[up - 1], grid[up] - x
    return np.where((low < high) | ((low == high) & (up % 2 == 1)), up - 1, up)


def quantise(x):
    """x float64 [..., dh] -> codes uint8 [..., dh], scale bytes uint8 [..., dh / 16]."""
    b = x.reshape(x.shape[:-1] + (-1, 16))
    amax = np.abs(b).max(-1)             # NaN if one is NaN
    scales = scale_value(np.arange(227))  # up to 10240
    with np.errstate(invalid="ignore"):
        byte = np.where(np.isnan(amax), 255, nearest(np.where(np.isnan(amax), 0, np.minimum(amax / 6, 1e9)), scales))
    s = scale_value(byte)[..., None]
    with np.errstate(invalid="ignore", divide="ignore"):
        y = np.where(s > 0, np.abs(b) / s, 0.0)
    code = nearest(np.minimum(np.nan_to_num(y, nan=0.0, posinf=9.0), 9.0), LEVELS)
    code = code + 8 * (b < 0)
    return code.astype(np.uint8).reshape(x.shape), byte.astype(np.uint8)


def value(code, byte):
    s = np.repeat(scale_value(byte), 16, axis=-1)
    with np.errstate(invalid="ignore"):
        return np.where(code >= 8, -1.0, 1.0) * LEVELS[code & 7] * s


def k_place(pos, ch, dh):
    """(byte, shift) of a K code in its block, and the byte of its scale."""
    h, t, rest = dh // 64, ch // (dh // 4), ch % (dh // 4)
    jh, j = rest // 16, rest % 16 // 4
    word = ((pos // 16 * h + jh) * 32 + pos % 8 * 4 + t) * 4 + j
    byte = 4 * word + 2 * (rest % 4 // 2) + pos // 8 % 2
    return byte, 4 * (ch % 2), 64 * dh + (pos % 8 * 4 + t) * 8 * h + pos // 8 * h + jh


def v_place(pos, ch, dh):
    h, g, rest, t = dh // 64, ch // (dh // 8), ch % (dh // 8), pos % 8 // 2
    jh, j = rest // 8, rest % 8 // 2
    word = ((pos // 16 * h + jh) * 32 + g * 4 + t) * 4 + j
    byte = 32 * dh + 4 * word + 2 * (pos // 8 % 2) + ch % 2
    return byte, 4 * (pos % 2), 68 * dh + ((ch // 16 * 4 + t) * 4 + pos // 16) * 4 + 2 * (pos // 8 % 2) + pos % 2


_GRIDS = {}


def grids(dh):
    if dh not in _GRIDS:
        pos, ch = np.meshgrid(np.arange(PAGE), np.arange(dh), indexing="ij")
        _GRIDS[dh] = k_place(pos, ch, dh), v_place(pos, ch, dh)
    return _GRIDS[dh]


def read_block(block, dh):
    """block uint8 [..., 72 dh] -> K, V float64 [..., 64, dh]."""
    out = []
    for byte, shift, scale in grids(dh):
        code = block[..., byte] >> shift.astype(np.uint8) & 15
        s = scale_value(block[..., scale])
        with np.errstate(invalid="ignore"):
            out.append(np.where(code >= 8, -1.0, 1.0) * LEVELS[code & 7] * s)
    return out


def write_row(block, pos, k, v, dh):
    """Quantised rows k, v float64 [dh] into block uint8 [72 dh] at position pos."""
    for place, x in ((k_place, k), (v_place, v)):
        code, byte = quantise(x)
        for c in range(dh):
            at, shift, scale = place(pos, c, dh)
            block[at] = (int(block[at]) & ~(15 << shift) | int(code[c]) << shift) & 255
            block[scale] = byte[c // 16]


def attention(q, k, v, limits, scale):
    """q [rows, n_q, dh], k, v [n_kv, positions, dh], limits [rows]: o, lse and, for tolerances, sum p |v| / sum p and the
    largest sum |q k| scale of a row, and the sum of |v| that a row sees."""
    rows, n_q, dh = q.shape
    group = n_q // k.shape[0]
    o, absum, vsum = np.zeros(q.shape), np.zeros(q.shape), np.zeros(q.shape)
    lse, reach = np.full((rows, n_q), -np.inf), np.zeros((rows, n_q))
    for h in range(n_q):
        s = q[:, h] @ k[h // group].T * scale
        s = np.where(np.arange(s.shape[1])[None] < np.asarray(limits)[:, None], s, -np.inf)
        some = np.asarray(limits) > 0
        if not some.any():
            continue
        top = s[some].max(1, keepdims=True)
        p = np.exp(s[some] - top)
        den = p.sum(1, keepdims=True)
        o[some, h] = p @ v[h // group] / den
        absum[some, h] = p @ np.abs(v[h // group]) / den
        vsum[some, h] = (p > 0) @ np.abs(v[h // group])
        lse[some, h] = (top + np.log(den))[:, 0]
        reach[some, h] = (np.abs(q[some, h]) @ np.abs(k[h // group]).T * scale).max(1)
    return o, lse, absum, reach, vsum


class Book:
    """Lengths, tables and reference counts, by the rules of the header; every call says whether it was carried out."""

    def __init__(self, n_seq, n_pages, max_pages):
        self.n_seq, self.n_pages, self.max_pages = n_seq, n_pages, max_pages
        self.lens = [0] * n_seq
        self.refs = [0] * n_pages
        self.table = [[-1] * max_pages for _ in range(n_seq)]

    def pages(self, s):
        return -(-self.lens[s] // PAGE)

    def extend(self, counts):
        """None, or the list of page copies (from, to)."""
        need, moves = [], []
        for s, n in enumerate(counts):
            if n < 0 or self.lens[s] + n > self.max_pages * PAGE:
                return None
            copy = n > 0 and self.lens[s] % PAGE > 0 and self.refs[self.table[s][self.pages(s) - 1]] > 1
            need.append((copy, -(-(self.lens[s] + n) // PAGE) - self.pages(s)))
        free = [p for p in range(self.n_pages) if not self.refs[p]]
        if sum(c + n for c, n in need) > len(free):
            return None
        for s, (copy, n) in enumerate(need):
            have = self.pages(s)
            if copy:
                old, new = self.table[s][have - 1], free.pop(0)
                moves.append((old, new))
                self.refs[old] -= 1
                self.refs[new] = 1
                self.table[s][have - 1] = new
            for i in range(n):
                self.table[s][have + i] = free.pop(0)
                self.refs[self.table[s][have + i]] = 1
            self.lens[s] += counts[s]
        return moves

    def fork(self, src, dst):
        if len(set(dst)) < len(dst) or set(dst) & set(src) or any(self.lens[d] for d in dst):
            return False
        for a, b in zip(src, dst):
            self.table[b], self.lens[b] = list(self.table[a]), self.lens[a]
            for i in range(self.pages(a)):
                self.refs[self.table[a][i]] += 1
        return True

    def free(self, slots):
        if len(set(slots)) < len(slots):
            return False
        for s in slots:
            for i in range(self.pages(s)):
                self.refs[self.table[s][i]] -= 1
            self.table[s], self.lens[s] = [-1] * self.max_pages, 0
        return True

    def compact(self):
        live = sum(r > 0 for r in self.refs)
        src = [p for p in range(live, self.n_pages) if self.refs[p]]
        dst = [p for p in range(live) if not self.refs[p]]
        for a, b in zip(src, dst):
            self.refs[b], self.refs[a] = self.refs[a], 0
            self.table = [[b if p == a else p for p in row] for row in self.table]
        return list(zip(src, dst))

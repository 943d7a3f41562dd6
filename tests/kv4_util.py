"""The 4-bit KV cache in plain numpy, 64 bits, from the format's definition:
the reference of the GPU tests."""
import numpy as np

GROUP, BLOCK = 16, 32
MAG = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
# the non-negative finite e4m3 values, by code
E4M3 = np.array([m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
                 for e in range(16) for m in range(8)][:127])


def page_bytes(heads, dim, page):
    return heads * page * (dim + dim // 8)


def _nearest(x, grid):
    """Index of the grid value nearest to each x >= 0, halves to the even index."""
    up = np.clip(np.searchsorted(grid, x), 1, len(grid) - 1)
    a, b = np.abs(x - grid[up - 1]), np.abs(grid[up] - x)
    return np.where((b < a) | ((b == a) & (up % 2 == 0)), up, up - 1)


def quantize(x, log2=0):
    """Rows x [..., dim] -> (codes [..., dim], scale bytes [..., dim / 16])."""
    x = np.asarray(x, dtype=np.float64)
    g = x.reshape(*x.shape[:-1], -1, GROUP) * 2.0 ** -log2
    bad = ~np.isfinite(g).all(-1)
    g = np.where(np.isfinite(g), g, 0.0)
    scale = _nearest(np.minimum(np.abs(g).max(-1) / 6, 448.0), E4M3)
    s = E4M3[scale][..., None]
    y = np.where(s > 0, np.minimum(np.abs(g) / np.where(s > 0, s, 1.0), 6.0), 0.0)
    code = _nearest(y, MAG) + 8 * (g < 0)
    code = np.where(bad[..., None], 0, code)
    scale = np.where(bad, 0x7F, scale)
    return code.reshape(x.shape).astype(np.uint8), scale.astype(np.uint8)


def values(codes, scales, log2=0):
    s = np.where(scales & 0x7F == 0x7F, np.nan, E4M3[np.minimum(scales & 0x7F, 126)])
    v = np.where(codes >= 8, -1.0, 1.0) * MAG[codes & 7]
    return v * np.repeat(s, GROUP, -1) * 2.0 ** log2


class Plain:
    """A cache in numpy: pool bytes, table, and rows by (sequence, slot)."""

    def __init__(self, n_seq, heads, dim, page, pages_per_seq, seed=0, n_pages=None, k_log2=0, v_log2=0,
                 fill=None):
        rng = np.random.default_rng(seed)
        self.n_seq, self.heads, self.dim, self.page, self.pps = n_seq, heads, dim, page, pages_per_seq
        self.log2 = (k_log2, v_log2)
        n_pages = n_pages or n_seq * pages_per_seq
        self.table = rng.permutation(n_pages)[:n_seq * pages_per_seq].reshape(n_seq, pages_per_seq).astype(np.int32)
        self.pool = np.zeros((n_pages, page_bytes(heads, dim, page)), np.uint8)
        if fill is not None:
            self.pool[:] = fill
        self.capacity = page * pages_per_seq

    def _at(self, s, slot, head):
        d, size = self.dim, BLOCK * (self.dim + self.dim // 8)
        base = (head * (self.page // BLOCK) + slot % self.page // BLOCK) * size
        row = slot % BLOCK
        half = BLOCK * (d // 2 + d // GROUP)
        return self.table[s, slot // self.page], [
            (base + w * half + row * (d // 2), base + w * half + BLOCK * (d // 2) + row * (d // GROUP))
            for w in (0, 1)]

    def write(self, s, slot, k, v):
        """k, v [heads][dim] into one slot."""
        for head in range(self.heads):
            page, at = self._at(s, slot, head)
            for w, x in enumerate((k[head], v[head])):
                c, sc = quantize(x, self.log2[w])
                a, b = at[w]
                self.pool[page, a:a + self.dim // 2] = c[0::2] | c[1::2] << 4
                self.pool[page, b:b + self.dim // GROUP] = sc

    def read(self, s, n):
        """k, v [n][heads][dim] of slots 0..n-1."""
        out = np.zeros((2, n, self.heads, self.dim))
        for slot in range(n):
            for head in range(self.heads):
                page, at = self._at(s, slot, head)
                for w in (0, 1):
                    a, b = at[w]
                    raw = self.pool[page, a:a + self.dim // 2]
                    c = np.stack((raw & 15, raw >> 4), -1).reshape(-1)
                    out[w, slot, head] = values(c, self.pool[page, b:b + self.dim // GROUP], self.log2[w])
        return out[0], out[1]

    def fill_random(self, lens, seed=1, size=1.0):
        """Random codes and scales in every slot of lens (fast: no rounding)."""
        rng = np.random.default_rng(seed)
        half = BLOCK * (self.dim // 2 + self.dim // GROUP)
        blocks = self.pool.reshape(self.pool.shape[0], self.heads, self.page // BLOCK, 2, half)
        for s, n in enumerate(lens):
            for lp in range(-(-n // self.page)):
                b = blocks[self.table[s, lp]]
                codes = rng.integers(0, 256, b[..., :BLOCK * self.dim // 2].shape, dtype=np.uint8)
                b[..., :BLOCK * self.dim // 2] = codes
                # scales whose rows have values around `size`
                e = int(np.round(np.log2(size / 3))) + 7
                b[..., BLOCK * self.dim // 2:] = (rng.integers(e - 1, e + 2, b[..., BLOCK * self.dim // 2:].shape) * 8
                                                  + rng.integers(0, 8, b[..., BLOCK * self.dim // 2:].shape))


# A probability enters the products as fp16, 2^11 to 2^15 at the row's maximum:
# far below it the type's step is fixed, 2^-24 / 2^11 = 2^-35 of the maximum at
# most, and the rounding half of that, however small the probability.  In units
# of the smallest relative error that a bound multiplies the mass with (2^-18,
# _bound): 2^-18.
TINY = 2.0 ** -18


def attend(q, k, v, scale, group):
    """q [T][Hq][d], k, v [n][H][d] -> out [T][Hq][d], weights [H][n], and for
    the error bound the sums of p |v| and the largest scale * sum |q||k|."""
    T, Hq, d = q.shape
    n, H = k.shape[0], k.shape[1]
    out, mass, reach = np.zeros(q.shape), np.zeros(q.shape), np.zeros((T, Hq))
    w = np.zeros((H, n))
    for i in range(T):
        m = n - T + i + 1
        if m <= 0:
            continue
        for h in range(Hq):
            g = h // group
            x = scale * (k[:m, g] @ q[i, h])
            p = np.exp(x - x.max()) if np.isfinite(x).all() else np.full(m, np.nan)
            p = p / p.sum()
            # what has no weight still carries a NaN or infinity
            out[i, h] = p @ v[:m, g]
            # with what fp16's fixed step adds for small weights (TINY)
            mass[i, h] = (p + TINY * p.max()) @ np.abs(v[:m, g])
            reach[i, h] = scale * (np.abs(k[:m, g]) @ np.abs(q[i, h])).max()
            w[g, :m] += p
    return out, w, mass, reach

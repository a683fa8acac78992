"""Plain fp64 references of the cache of 4 bits, rotary positions, a step's plan
and the attention over the cache, with bounds for what fp32 sums and roundings
may differ (numpy, CPU)."""
import numpy as np

from ref64 import HALF_BF16, HALF_F32, depth

LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
MIDDLES = (LEVELS[:-1] + LEVELS[1:]) / 2
HALF, PAIRS = 0, 1


def hold(x):
    """x [..., D] -> (codes [..., D] 0..15, scale bytes [..., D / 32])."""
    x = np.asarray(x, np.float64)
    b = x.reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    bad = ~np.isfinite(b).all(-1)
    fine = np.where(np.isfinite(b), b, 0.0)
    top = np.abs(fine).max(-1)
    m, e = np.frexp(np.where(top > 0, top, 1.0))         # top = m 2^e, m in [0.5, 1)
    e = np.where(top > 0, e - 3 + (m >= 0.875), -125)
    e = np.clip(e, -125, 125)
    a = np.abs(fine) * np.exp2(-e.astype(np.float64))[..., None]
    low = np.searchsorted(MIDDLES, a, "left")            # a tie goes down ...
    high = np.searchsorted(MIDDLES, a, "right")          # ... or up
    code = np.where(low % 2 == 0, low, high)
    code = np.where(np.signbit(fine), code + 8, code)
    return code.reshape(x.shape).astype(np.uint8), np.where(bad, 255, e + 127).astype(np.uint8)


def value(codes, bytes_):
    """What codes and scale bytes stand for, fp64."""
    s = np.where(bytes_ == 255, np.nan, np.exp2(bytes_.astype(np.float64) - 127))
    v = LEVELS[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    return v * np.repeat(s, 32, -1)


def rotate(x, positions, freqs, layout, scale=1.0):
    """x [T][H][D] with the first 2 len(freqs) channels of each head rotated."""
    y = np.array(x, np.float64)
    n = len(freqs)
    t = positions.astype(np.float64)[:, None, None] * freqs
    c, s = np.cos(t) * scale, np.sin(t) * scale
    a, b = (slice(0, n), slice(n, 2 * n)) if layout == HALF else (slice(0, 2 * n, 2), slice(1, 2 * n, 2))
    xa, xb = x[..., a].astype(np.float64), x[..., b].astype(np.float64)
    y[..., a], y[..., b] = xa * c - xb * s, xb * c + xa * s
    return y


class Cache:
    """A cache in numpy, in the library's layout."""

    def __init__(self, pages, heads, D, P, rng):
        self.pages, self.heads, self.D, self.P = pages, heads, D, P
        # what nothing has written yet is anything, NaN among it
        self.codes = {n: rng.integers(0, 256, (pages, heads, P, D // 2), dtype=np.uint8) for n in "kv"}
        self.scales = {n: rng.choice(np.array([255, 130, 1], np.uint8), (pages, heads, D // 32, P)) for n in "kv"}

    def write(self, name, slots, x):
        """x [T][heads][D] into the slots that lie in the cache."""
        codes, bytes_ = hold(x)
        for t, slot in enumerate(slots):
            if 0 <= slot < self.pages * self.P:
                page, at = divmod(int(slot), self.P)
                self.codes[name][page, :, at] = codes[t, :, 0::2] | codes[t, :, 1::2] << 4
                self.scales[name][page, :, :, at] = bytes_[t]

    def read(self, name, slots):
        out = np.zeros((len(slots), self.heads, self.D))
        for t, slot in enumerate(slots):
            if 0 <= slot < self.pages * self.P:
                page, at = divmod(int(slot), self.P)
                b = self.codes[name][page, :, at]
                codes = np.stack((b & 15, b >> 4), -1).reshape(self.heads, self.D)
                out[t] = value(codes, self.scales[name][page, :, :, at])
        return out


def attention(q, cache, table, q_start, kv_len, scale, window=0, p_round=HALF_BF16):
    """-> (y [T][Hq][D], bound of its error before its rounding, lse, bound); rows
    of no request stay NaN.

    Bounds.  A score is an fp32 sum of D exact products and two products more; an
    exponential of base 2 is off by a step or two and by its argument's rounding;
    an output's sum passes through as many roundings as a sum of n + D terms does.
    A probability is off by p_round in the second product."""
    T, Hq, D = q.shape
    G, P = Hq // cache.heads, cache.P
    y, lse = np.full((T, Hq, D), np.nan), np.full((T, Hq), np.nan)
    ye, le = np.zeros((T, Hq, D)), np.zeros((T, Hq))
    for b in range(len(kv_len)):
        n, t0, t1 = int(kv_len[b]), int(q_start[b]), int(q_start[b + 1])
        key = np.arange(n)
        page = table[b][key // P].astype(np.int64) if n else key
        there = (page >= 0) & (page < cache.pages)
        slots = np.where(there, page * P + key % P, -1)
        k, v = cache.read("k", slots), cache.read("v", slots)
        for t in range(t0, t1):
            p = n - (t1 - t)
            sees = there & (key <= p) & ((key > p - window) if window else True)
            ks, vs = k[sees], v[sees]
            for h in range(Hq):
                if not sees.any():
                    y[t, h], lse[t, h] = 0.0, -np.inf
                    continue
                z = scale * (ks[:, h // G] @ q[t, h])
                top = z.max()
                w = np.exp(z - top)
                total = w.sum()
                w = w / total
                y[t, h] = w @ vs[:, h // G]
                lse[t, h] = top + np.log(total)
                az = scale * (np.abs(ks[:, h // G]) @ np.abs(q[t, h]))
                dz = ((depth(D) + 4) * HALF_F32 * az + 8 * HALF_F32 * (1 + np.abs(z) + abs(top))).max()
                chain = depth(len(z)) * HALF_F32
                le[t, h] = dz + chain + 4 * HALF_F32 * abs(lse[t, h])
                ye[t, h] = (2 * dz + 2 * chain + p_round) * (w @ np.abs(vs[:, h // G]))
    return y, ye, lse, le


def plan(cached, fresh, table, free, n_free, T, P):
    """-> (q_start, kv_len, positions, slots, table, n_left, status), token by token."""
    table, width = table.copy(), table.shape[1]
    left = min(max(int(n_free), 0), len(free))
    q_start, kv_len, positions, slots = [0], [], [], []
    lacked = over = 0
    for b in range(len(cached)):
        have = max(int(cached[b]), 0)
        n = min(max(int(fresh[b]), 0), T - q_start[-1])
        for j in range(-(-have // P), -(-(have + n) // P)):
            if j >= width:
                over += 1
            elif left:
                left -= 1
                table[b, j] = free[left]
            else:
                lacked += 1
                table[b, j] = -1
        for p in range(have, have + n):
            page = table[b, p // P] if p // P < width else -1
            positions.append(p)
            slots.append(int(page) * P + p % P if page >= 0 else -1)
        q_start.append(q_start[-1] + n)
        kv_len.append(have + n)
    pad = T - len(slots)
    return (np.array(q_start), np.array(kv_len, np.int64), np.array(positions + [0] * pad), np.array(slots + [-1] * pad),
            table, left, np.array([lacked, over]))

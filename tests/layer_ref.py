"""64-bit references of the operators around the MoE block (test
infrastructure): plain loops and numpy from the definitions in e0moe.h."""
import numpy as np

# the non-negative finite e4m3 values by code
E4M3 = np.array([(m / 8) * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
                 for e in range(16) for m in range(8)][:127])


def decode(codes):
    """e4m3 codes (uint8) as numbers; the two NaN codes as +-480."""
    c = np.asarray(codes)
    v = np.append(E4M3, 480.0)[c & 127]
    return np.where(c & 128, -v, v)


def encode(x):
    """Nearest e4m3 code, ties to even, saturating."""
    x = np.asarray(x, np.float64)
    a = np.minimum(np.abs(x), 448.0)
    hi = np.minimum(np.searchsorted(E4M3, a), 126)
    lo = np.maximum(hi - 1, 0)
    below, above = a - E4M3[lo], E4M3[hi] - a
    c = np.where((above < below) | ((above == below) & (hi % 2 == 0)), hi, lo)
    return (c | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def border_distance(x):
    """Distance of |x| from the nearest rounding border of e4m3, relative to |x|."""
    a = np.minimum(np.abs(np.asarray(x, np.float64)), 448.0)
    mid = (E4M3[1:] + E4M3[:-1]) / 2
    i = np.clip(np.searchsorted(mid, a), 1, len(mid) - 1)
    d = np.minimum(np.abs(a - mid[i]), np.abs(a - mid[i - 1]))
    return d / np.maximum(a, 1e-300)


def pow2_scale(m):
    """Smallest power of two >= 2^-100 with m / 448 (rounded to fp32) <= it."""
    m = np.float32(m) / np.float32(448)
    e = -100
    while 2.0 ** e < m:
        e += 1
    return 2.0 ** e


class Cache:
    """The paged cache, held as codes and scales."""

    def __init__(self, n_blocks, Hkv, bs, D, rng=None):
        self.n, self.H, self.bs, self.D = n_blocks, Hkv, bs, D
        shape = (n_blocks, Hkv, bs, D)
        self.k = rng.integers(0, 256, shape).astype(np.uint8) if rng is not None else np.zeros(shape, np.uint8)
        self.v = rng.integers(0, 256, shape).astype(np.uint8) if rng is not None else np.zeros(shape, np.uint8)
        # what an unwritten block holds is anything, NaN among it
        fill = np.nan if rng is not None else 0
        self.ks = np.full((n_blocks, Hkv), fill, np.float32)
        self.vs = np.full((n_blocks, Hkv), fill, np.float32)

    def append(self, k, v, slots):
        """k, v float64 [T][Hkv][D]."""
        T = len(slots)
        t = 0
        while t < T:
            if slots[t] < 0 or slots[t] >= self.n * self.bs:
                t += 1
                continue
            blk, off = divmod(int(slots[t]), self.bs)
            n = 1
            while off + n < self.bs and t + n < T and slots[t + n] == slots[t] + n:
                n += 1
            for x, codes, scale in ((k, self.k, self.ks), (v, self.v, self.vs)):
                x = np.where(np.isfinite(x[t:t + n]), x[t:t + n], 0.0)
                for h in range(self.H):
                    s = pow2_scale(np.abs(x[:, h]).max())
                    if off:
                        old = float(scale[blk, h])
                        s = max(s, old)
                        if s > old:
                            codes[blk, h, :off] = encode(decode(codes[blk, h, :off]) * (old / s))
                    scale[blk, h] = s
                    codes[blk, h, off:off + n] = encode(x[:, h] / s)
            t += n

    def row(self, table_row, n):
        """The first n tokens' keys and values of one sequence, [n][Hkv][D] float64;
        positions whose block id is out of range come as NaN."""
        k = np.full((n, self.H, self.D), np.nan)
        v = np.full((n, self.H, self.D), np.nan)
        for j in range(-(-n // self.bs)):
            b = int(table_row[j])
            m = min(self.bs, n - j * self.bs)
            if 0 <= b < self.n:
                at = slice(j * self.bs, j * self.bs + m)
                k[at] = (decode(self.k[b, :, :m]) * self.ks[b][:, None, None]).transpose(1, 0, 2)
                v[at] = (decode(self.v[b, :, :m]) * self.vs[b][:, None, None]).transpose(1, 0, 2)
        return k, v


def attention(q, k, v, scale, ctx, window, weight_err=0.0):
    """q [n][Hq][D], the last n of ctx positions; k, v [ctx][Hkv][D] (NaN
    positions are not seen).  Returns out, lse and, for each output, a bound on what
    fp32 sums, 22-bit operands and weights that are weight_err (relative) off may
    be off by."""
    n, Hq, D = q.shape
    Hkv = k.shape[1] if k.ndim == 3 else 1
    G = Hq // Hkv
    out, lse = np.zeros(q.shape), np.full((n, Hq), -np.inf)
    tol, ltol = np.zeros(q.shape), np.zeros((n, Hq))
    eps = 2.0 ** -23
    ok = ~np.isnan(k[:, 0, 0]) if ctx else np.zeros(0, bool)
    for i in range(n):
        p = ctx - n + i
        j = np.arange(ctx)
        seen = ok & (j <= p) & ((j > p - window) if window else True)
        if not seen.any():
            continue
        for h in range(Hq):
            kk, vv = k[seen, h // G], v[seen, h // G]
            x = kk @ q[i, h] * scale
            mag = np.abs(kk) @ np.abs(q[i, h]) * abs(scale)
            m = x.max()
            e = np.exp(x - m)
            z = e.sum()
            out[i, h] = (e / z) @ vv
            lse[i, h] = m + np.log(z)
            # a score: D products of 22-bit operands summed in fp32, scaled by factors of 3 roundings;
            # exp2's argument and result; sums over the positions; the operands of the second product
            ds = (D + 16) * eps * mag.max() + 4 * eps * np.abs(x).max()
            rel = 2 * ds + (seen.sum() / 4 + 64) * eps
            tol[i, h] = (rel + weight_err) * ((e / z) @ np.abs(vv))
            ltol[i, h] = rel + 4 * eps * abs(lse[i, h])
    return out, lse, tol, ltol

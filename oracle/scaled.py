"""Oracle (test infrastructure only): e4m3 values, block scales, products on them, float64 NumPy."""
import numpy as np

BLOCK = 128


def e4m3_table():
    """Value of each of the 256 codes: sign, 4 exponent bits (bias 7), 3 mantissa bits; exponent 0
    is subnormal, all ones with mantissa 7 is NaN (there is no infinity)."""
    out = np.empty(256)
    for c in range(256):
        s, e, m = c >> 7, (c >> 3) & 15, c & 7
        v = m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        if e == 15 and m == 7:
            v = np.nan
        out[c] = -v if s else v
    return out


TABLE = e4m3_table()
_POS = TABLE[:127]  # ascending, 0 .. 448


def round_e4m3(v):
    """Codes of the nearest e4m3 values (ties to the even code), |v| <= 448; non-finite -> NaN."""
    v = np.asarray(v, np.float64)
    a = np.where(np.isfinite(v), np.abs(v), 0.0)
    hi = np.clip(np.searchsorted(_POS, a), 0, 126)
    lo = np.clip(hi - 1, 0, 126)
    dl, dh = a - _POS[lo], _POS[hi] - a
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    code = code + np.where(np.signbit(v), 128, 0)
    return np.where(np.isfinite(v), code, 127).astype(np.uint8)


def block_scale(m):
    """Smallest 2^e, e >= -126, with m <= 448 * 2^e; 1 for m = 0."""
    if m == 0:
        return 1.0
    e = -126
    while 448.0 * 2.0 ** e < m:
        e += 1
    return 2.0 ** e


def quantize(x, block_rows):
    """codes [rows][cols] uint8, scale [rows/block_rows up][cols/128 up]."""
    x = np.asarray(x, np.float64)
    R, C = x.shape
    nr, nc = -(-R // block_rows), -(-C // BLOCK)
    q, scale = np.zeros((R, C), np.uint8), np.ones((nr, nc))
    for i in range(nr):
        for j in range(nc):
            v = x[i * block_rows:(i + 1) * block_rows, j * BLOCK:(j + 1) * BLOCK]
            f = np.abs(v[np.isfinite(v)])
            scale[i, j] = block_scale(f.max() if f.size else 0.0)
            q[i * block_rows:(i + 1) * block_rows, j * BLOCK:(j + 1) * BLOCK] = round_e4m3(v / scale[i, j])
    return q, scale


def values(q, scale, block_rows):
    """What codes and scales stand for."""
    R, C = q.shape
    s = np.repeat(np.repeat(np.asarray(scale, np.float64), block_rows, 0)[:R], BLOCK, 1)[:, :C]
    return TABLE[q] * s


def gemm(x, w, offsets):
    """x [M][K], w [E][N][K] (values), rows offsets[e] .. of expert e; NaN rows elsewhere."""
    y = np.full((x.shape[0], w.shape[1]), np.nan)
    for e in range(w.shape[0]):
        a, b = offsets[e], offsets[e + 1]
        y[a:b] = x[a:b] @ w[e].T
    return y


def silu(z):
    return z / (1.0 + np.exp(-z))


def moe(x, idx, gate, w1, w2):
    """Expert FFN on values w1 [E][2I][H], w2 [E][H][I]; x and h quantised per row and 128 columns."""
    T, H = x.shape
    xq = values(*quantize(x, 1), 1)
    I = w2.shape[2]
    y = np.zeros((T, H))
    for t in range(T):
        for s in range(idx.shape[1]):
            e = idx[t, s]
            if e < 0:
                continue
            gu = w1[e] @ xq[t]
            h = (silu(gu[:I]) * gu[I:])[None]
            y[t] += float(gate[t, s]) * (w2[e] @ values(*quantize(h, 1), 1)[0])
    return y

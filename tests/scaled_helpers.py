"""Inputs and error bounds of the scaled-product tests.

Bounds (u = 2^-24).  A product of two e4m3 values is exact in fp32.  The tensor cores add the 128
products of a block in fp32 (their rounding is not documented: every addition is granted a whole unit,
2 u, of the sum of magnitudes): 256 u.  Folding a block costs the rounding of the two scales' product
and of the multiply-add; adding pieces of a split unit, one more per piece: with kb blocks and at most
kb pieces (2 kb + 2) u.  All relative to S = sum of |x w| over K."""
import numpy as np

from oracle import scaled as S

U = 2.0 ** -24


def sum_bound(kb):
    return (256 + 2 * kb + 2) * U


def weights(E, N, K, seed):
    """Codes [E][N][K] and general fp32 scales [E][N/128][K/128], as if quantised by amax / 448."""
    rng = np.random.default_rng([E, N, K, seed])
    q = S.round_e4m3(np.clip(rng.normal(size=(E, N, K)) * 120, -448, 448))
    s = np.exp(rng.normal(size=(E, -(-N // 128), -(-K // 128))) * 0.3 - 8).astype(np.float32)
    v = np.stack([S.values(q[e], np.repeat(s[e], 1, 0), 128) for e in range(E)])
    return q, s, v


def padded_codes(q):
    """Rows of K codes -> device uint8 rows of K rounded up to 16 (the rest e4m3 NaN: not read)."""
    import torch
    ld = -(-q.shape[-1] // 16) * 16
    t = torch.full((*q.shape[:-1], ld), 127, dtype=torch.uint8, device="cuda")
    t[..., :q.shape[-1]] = torch.from_numpy(q).cuda()
    return t, ld


def moe_bound(x, idx, gate, w1, w2):
    """Oracle output of the layer and an elementwise bound on the kernel's difference from it.

    h is quantised, so an fp32 error of h can move it to the neighbouring code where it lies within
    that error of a rounding border; those elements (and whole blocks whose maximum lies near a scale's
    border) are granted their step, all others only the sums' bounds."""
    T, H = x.shape
    E, I = w2.shape[0], w2.shape[2]
    xq = S.values(*S.quantize(x, 1), 1)
    y, tol = np.zeros((T, H)), np.zeros((T, H))
    b1, b2 = sum_bound(H // 128), sum_bound(I // 128)
    for t in range(T):
        for s in range(idx.shape[1]):
            e = idx[t, s]
            if e < 0:
                continue
            gu = w1[e] @ xq[t]
            err = b1 * (np.abs(w1[e]) @ np.abs(xq[t]))
            g, u, eg, eu = gu[:I], gu[I:], err[:I], err[I:]
            sg = S.silu(g)
            h = sg * u
            # |SiLU'| <= 1.1; the fast exponential is off by at most 2 + 1.173 |g| ulp, division 2 ulp,
            # the sum, the product and the quotient's operands one rounding each
            eh = 1.1 * eg * (np.abs(u) + eu) + np.abs(sg) * eu + np.abs(h) * (8 + 1.2 * np.abs(g)) * 2 * U
            q, sc = S.quantize(h[None], 1)
            hv = S.values(q, sc, 1)[0]
            scale = np.repeat(sc[0], 128)[:I]
            a = np.abs(h) / scale
            step = np.maximum(2.0 ** (np.floor(np.log2(np.maximum(a, 2.0 ** -6))) - 3), 2.0 ** -9)
            frac = a / step - np.floor(a / step)
            near = np.abs(frac - 0.5) * step <= eh / scale
            for b in range(I // 128):
                blk = slice(128 * b, 128 * b + 128)
                m, em = np.abs(h[blk]).max(), eh[blk].max()
                if S.block_scale(max(m - em, 0)) != S.block_scale(m + em):
                    near[blk] = True
                    step[blk] *= 2
            dh = np.where(near, step * scale * 1.001 + eh, 0)
            gt = float(gate[t, s])
            aw = np.abs(w2[e])
            o = w2[e] @ hv
            y[t] += gt * o
            tol[t] += abs(gt) * (aw @ dh + b2 * (aw @ (np.abs(hv) + dh))) + 4 * U * abs(gt) * np.abs(o)
    return y, tol

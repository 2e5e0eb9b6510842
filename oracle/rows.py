"""Oracle (test infrastructure only): token rows sorted by expert and back, float64 NumPy."""
import numpy as np


def sort(idx, E):
    """pos [T][k], src (rows in use only), offsets [E+1]: ascending slot within an expert."""
    T, k = idx.shape
    flat = idx.reshape(-1)
    src = np.concatenate([np.flatnonzero(flat == e) for e in range(E)]).astype(np.int64)
    offsets = np.concatenate([[0], np.cumsum([(flat == e).sum() for e in range(E)])])
    pos = np.full(T * k, -1, np.int64)
    pos[src] = np.arange(len(src))
    return pos.reshape(T, k), src, offsets


def dispatch(x, pos, rows):
    """xs [rows][H]: NaN where no slot put a row."""
    out = np.full((rows, x.shape[1]), np.nan)
    for t in range(pos.shape[0]):
        for r in pos[t]:
            if r >= 0:
                out[r] = x[t]
    return out


def combine(o, pos, gate):
    T, k = pos.shape
    y = np.zeros((T, o.shape[1]))
    for t in range(T):
        for s in range(k):
            if pos[t, s] >= 0:
                y[t] += float(gate[t, s]) * o[pos[t, s]].astype(np.float64)
    return y


def dispatch_grad(d_xs, pos):
    return combine(d_xs, pos, np.ones(pos.shape))


def combine_grad(d_y, o, pos, gate):
    """d_o [rows][H] (NaN where no slot), d_gate [T][k]."""
    T, k = pos.shape
    d_o = np.full(o.shape, np.nan)
    d_gate = np.zeros((T, k))
    for t in range(T):
        for s in range(k):
            r = pos[t, s]
            if r >= 0:
                d_o[r] = float(gate[t, s]) * d_y[t].astype(np.float64)
                d_gate[t, s] = np.dot(d_y[t].astype(np.float64), o[r].astype(np.float64))
    return d_o, d_gate

"""The oracles of the expert-row and scaled-product calls, pinned to hand cases, to torch's e4m3
cast and to differences."""
import numpy as np
import pytest
import torch

from oracle import rows as R
from oracle import scaled as S


def test_sort_hand_case():
    idx = np.array([[2, 0], [0, -1], [2, 2]])
    pos, src, offsets = R.sort(idx, 4)
    assert offsets.tolist() == [0, 2, 2, 5, 5]
    assert src.tolist() == [1, 2, 0, 4, 5]
    assert pos.tolist() == [[2, 0], [1, -1], [3, 4]]


def test_row_gradients_against_differences():
    rng = np.random.default_rng(1)
    idx = np.array([[1, 0, 2], [2, -1, 1], [-1, -1, -1], [0, 2, 1]])
    pos, src, _ = R.sort(idx, 3)
    n, H = len(src), 5
    o, gate, dy = rng.normal(size=(n, H)), rng.normal(size=idx.shape), rng.normal(size=(4, H))
    loss = lambda o_, g_: float((R.combine(o_, pos, g_) * dy).sum())  # noqa: E731
    d_o, d_gate = R.combine_grad(dy, o, pos, gate)
    h = 1e-6
    for r in range(n):
        for c in range(H):
            p, m = o.copy(), o.copy()
            p[r, c] += h
            m[r, c] -= h
            assert abs((loss(p, gate) - loss(m, gate)) / (2 * h) - d_o[r, c]) < 1e-8
    for t in range(4):
        for s in range(3):
            p, m = gate.copy(), gate.copy()
            p[t, s] += h
            m[t, s] -= h
            assert abs((loss(o, p) - loss(o, m)) / (2 * h) - d_gate[t, s]) < 1e-8
    # dispatch: loss = <dispatch(x), d_xs>, linear, so its gradient is exact in one step
    x, d_xs = rng.normal(size=(4, H)), rng.normal(size=(n, H))
    d_x = R.dispatch_grad(d_xs, pos)
    for t in range(4):
        e = np.zeros((4, H))
        e[t] = 1.0
        assert np.allclose((R.dispatch(e, pos, n) * d_xs).sum(0), d_x[t], atol=1e-12)
    assert x.shape == d_x.shape


def test_e4m3_values_and_rounding_match_torch():
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(np.isnan(codes), np.isnan(S.TABLE))
    ok = ~np.isnan(codes)
    assert np.array_equal(codes[ok], S.TABLE[ok])
    v = np.float32(np.random.default_rng(2).normal(size=20000) * 2.0 ** np.random.default_rng(3).integers(-12, 8, 20000))
    v = v[np.abs(v) <= 448]
    mid = (S._POS[:-1] + S._POS[1:]) / 2                       # every border: ties to even
    v = np.concatenate([v, np.float32(mid), -np.float32(mid)])
    want = torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(S.round_e4m3(v), want)


def test_block_scales():
    assert S.block_scale(448.0) == 1.0 and S.block_scale(448.0 * (1 + 2 ** -20)) == 2.0
    assert S.block_scale(0.0) == 1.0 and S.block_scale(1e-45) == 2.0 ** -126
    assert S.block_scale(3.4e38) == 2.0 ** 120
    x = np.zeros((3, 130))
    x[1, 5], x[2, 129], x[0, 0] = -900.0, 3.5, np.inf
    q, s = S.quantize(x, 1)
    assert s.tolist() == [[1.0, 1.0], [4.0, 1.0], [1.0, 2.0 ** -7]]
    v = S.values(q, s, 1)
    assert np.isnan(v[0, 0]) and v[1, 5] == -896.0 and v[2, 129] == 3.5


def test_moe_equals_dense_layer_of_its_values():
    rng = np.random.default_rng(4)
    E, H, I, T = 3, 128, 128, 4
    w1, w2 = rng.normal(size=(E, 2 * I, H)), rng.normal(size=(E, H, I))
    x = S.values(*S.quantize(rng.normal(size=(T, H)), 1), 1)   # already representable
    idx = np.array([[0, 2], [1, -1], [-1, -1], [2, 1]])
    gate = rng.random((T, 2))
    y = S.moe(x, idx, gate, w1, w2)
    assert np.all(y[2] == 0)
    gu = x[1] @ w1[1].T
    h = S.values(*S.quantize((gu[:I] / (1 + np.exp(-gu[:I])) * gu[I:])[None], 1), 1)[0]
    assert np.allclose(y[1], gate[1, 0] * (h @ w2[1].T), rtol=1e-12)


@pytest.mark.parametrize("E", [1, 4])
def test_gemm_rows_by_offset(E):
    rng = np.random.default_rng(5)
    off = [0, 3] if E == 1 else [0, 2, 2, 5, 6]
    x, w = rng.normal(size=(8, 4)), rng.normal(size=(E, 3, 4))
    y = S.gemm(x, w, off)
    assert np.isnan(y[off[-1]:]).all()
    for e in range(E):
        for r in range(off[e], off[e + 1]):
            assert np.allclose(y[r], w[e] @ x[r])

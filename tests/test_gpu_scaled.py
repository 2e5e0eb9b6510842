"""Quantisation to e4m3 and products on it, against the float64 oracle (bounds: scaled_helpers)."""
import numpy as np
import pytest

from any_precision_expert_pw_b200 import binding as B
from any_precision_expert_pw_b200.inputs import CONFIGS
from oracle import scaled as S
from scaled_helpers import U, moe_bound, padded_codes, sum_bound, weights
from test_gpu_rows import TYPES, Strided, _torch_type, gpu, half_step, routing

pytestmark = pytest.mark.gpu

QUANT = [(1, 1, 0, 0), (3, 128, 0, 0), (5, 100, 28, 0), (130, 257, 3, 1), (64, 384, 0, 0), (200, 1000, 8, 8)]


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("name", list(TYPES))
@pytest.mark.parametrize("rows,cols,extra,base", QUANT)
def test_quantize(libpw, rows, cols, extra, base, name, block_rows):
    import torch
    rng = np.random.default_rng([rows, cols, block_rows])
    v = rng.normal(size=(rows, cols)) * np.exp(rng.normal(size=(rows, 1)) * 3)
    v[0, 0] = 0.0
    v[rows // 2] = 0.0                                     # blocks of zeros
    if rows > 2:
        v[2, cols // 2] = np.inf
        v[2, 0] = np.nan
        v[1] *= 2.0 ** -20 if name == "f16" else 2.0 ** -130  # subnormal values
    x = Strided(rows, cols, name, extra, base, gpu(v))
    ld = -(-cols // 16) * 16 + 16
    q = torch.full((rows, ld), 0x5A, dtype=torch.uint8, device="cuda")
    scale = torch.full((-(-rows // block_rows), -(-cols // 128)), -7.0, device="cuda")
    B.check(B.pw_scaled_quantize(x.ptr, TYPES[name], rows, cols, x.ld, block_rows, q.data_ptr(), ld,
                                 scale.data_ptr()))
    want_q, want_s = S.quantize(x.np(), block_rows)
    assert np.array_equal(scale.double().cpu().numpy(), want_s)
    got = q.cpu().numpy()
    assert (got[:, cols:] == 0x5A).all()                   # behind the columns: left as they were
    a, b = S.TABLE[got[:, :cols]], S.TABLE[want_q]
    assert np.array_equal(np.isnan(a), np.isnan(b))
    assert np.array_equal(a[~np.isnan(a)], b[~np.isnan(b)])


@pytest.mark.parametrize("name", list(TYPES))
def test_quantize_borders(libpw, name):
    """Every e4m3 value and every border between two, both signs, and the scale's own borders."""
    import torch
    vals = np.concatenate([S._POS, (S._POS[:-1] + S._POS[1:]) / 2])
    vals = np.concatenate([vals, -vals])
    rows = []
    for e in (-8, 0, 5):
        for lead in (448.0, 449.0 if name != "bf16" else 450.0, 447.0 if name != "bf16" else 446.0):
            for i in range(0, len(vals), 127):
                r = np.zeros(128)
                c = vals[i:i + 127]
                r[:len(c)] = c
                r[127] = lead
                rows.append(r * 2.0 ** e)
    x = gpu(np.array(rows)).to(_torch_type(name))
    q = torch.empty(len(rows), 128, dtype=torch.uint8, device="cuda")
    s = torch.empty(len(rows), 1, device="cuda")
    B.check(B.pw_scaled_quantize(x.data_ptr(), TYPES[name], len(rows), 128, 128, 1, q.data_ptr(), 128,
                                 s.data_ptr()))
    want_q, want_s = S.quantize(x.double().cpu().numpy(), 1)
    assert np.array_equal(s.double().cpu().numpy(), want_s)
    assert np.array_equal(S.TABLE[q.cpu().numpy()], S.TABLE[want_q])


def product(x_np, q, s, off, N, y_name, extra=0, base=0, x_extra=0, w_extra=0, poison=0xFF):
    """Quantise x and multiply; returns (y Strided, quantised values of x)."""
    import torch
    M, K = x_np.shape
    E = q.shape[0]
    ld = -(-K // 16) * 16 + x_extra
    x = gpu(np.asarray(x_np, np.float32))
    xq = torch.full((M, ld), 127, dtype=torch.uint8, device="cuda")   # NaN behind the columns
    xs = torch.empty(M, -(-K // 128), device="cuda")
    B.check(B.pw_scaled_quantize(x.data_ptr(), B.PW_TYPE_F32, M, K, K, 1, xq.data_ptr(), ld, xs.data_ptr()))
    w, ldw = padded_codes(q)
    if w_extra:
        w2 = torch.full((E, N, ldw + w_extra), 127, dtype=torch.uint8, device="cuda")
        w2[..., :ldw] = w
        w, ldw = w2, ldw + w_extra
    ws = gpu(s)
    y = Strided(M, N, y_name, extra, base)
    n = B.pw_scaled_gemm_workspace_bytes(M, N, K, E)
    tmp = torch.full((n + 4096,), poison, dtype=torch.uint8, device="cuda")
    o = gpu(np.asarray(off, np.int32)) if off is not None else None
    B.check(B.pw_scaled_gemm(xq.data_ptr(), xs.data_ptr(), M, K, ld, w.data_ptr(), ws.data_ptr(), E, N,
                             ldw, o.data_ptr() if o is not None else 0, y.ptr, TYPES[y_name], y.ld,
                             tmp.data_ptr(), n))
    st = B.pw_get_status()
    assert st == B.PW_OK, B.pw_status_string(st)
    assert bool((tmp[n:] == poison).all())
    return y, S.values(*S.quantize(x.double().cpu().numpy(), 1), 1)


def check(y, y_name, xv, v, off, K):
    ref = S.gemm(xv, v, off)
    mag = S.gemm(np.abs(xv), np.abs(v), off)
    n = off[-1]
    tol = sum_bound(-(-K // 128)) * mag[:n]
    tol = tol + half_step(y_name) * (np.abs(ref[:n]) + tol) + (2.0 ** -25 if y_name == "f16" else 0)
    got = y.np()
    assert (np.abs(got[:n] - ref[:n]) <= tol).all(), float(np.max(np.abs(got[:n] - ref[:n]) / tol))
    assert (got[n:] == -77.0).all() and y.outside_untouched()


# both kernels (up to 32 rows an expert, and above), whole units and units cut into two and more pieces,
# more units than SMs, sizes that end inside a block, a row tile or a 16-row box
DENSE = [(1, 1, 1), (1, 128, 128), (4, 256, 128), (3, 300, 200), (17, 129, 136), (32, 300, 520),
         (33, 300, 520), (64, 512, 4096), (65, 255, 1111), (128, 256, 256), (129, 257, 640),
         (256, 512, 8192), (300, 700, 384), (1, 40000, 256), (2, 1000, 8192), (700, 9000, 128)]


@pytest.mark.parametrize("y_name", list(TYPES))
@pytest.mark.parametrize("M,N,K", DENSE)
def test_product_dense(libpw, M, N, K, y_name):
    rng = np.random.default_rng([M, N, K])
    q, s, v = weights(1, N, K, 1)
    y, xv = product(rng.normal(size=(M, K)), q, s, None, N, y_name)
    check(y, y_name, xv, v, [0, M], K)


GROUPED = [([0, 3], 256, 128), ([0, 0, 5, 5, 6], 300, 264), ([0, 1, 2, 3, 4, 5, 6, 7, 8], 384, 512),
           ([0, 130, 130, 131, 400], 520, 384), ([0, 0, 0], 256, 128), ([0, 200, 260], 8192, 256),
           ([0, 90, 91, 91, 95], 300, 384), ([0, 0, 64, 128, 129], 130, 3000)]


@pytest.mark.parametrize("off,N,K", GROUPED)
def test_product_grouped(libpw, off, N, K):
    E, M = len(off) - 1, off[-1] + 9                       # nine rows behind the last group
    rng = np.random.default_rng([E, N, K])
    q, s, v = weights(E, N, K, 2)
    y, xv = product(rng.normal(size=(M, K)), q, s, off, N, "bf16")
    check(y, "bf16", xv, v, off, K)


def test_product_many_experts(libpw):
    E, N, K = 1024, 130, 128
    rng = np.random.default_rng(7)
    rows = rng.integers(0, 3, E)
    off = np.concatenate([[0], np.cumsum(rows)])
    q, s, v = weights(E, N, K, 3)
    y, xv = product(rng.normal(size=(off[-1] + 1, K)), q, s, off, N, "f32")
    check(y, "f32", xv, v, off, K)


@pytest.mark.parametrize("extra,base,x_extra,w_extra", [(5, 0, 0, 0), (8, 0, 32, 16), (0, 1, 16, 0), (8, 8, 0, 48)])
@pytest.mark.parametrize("y_name", list(TYPES))
def test_product_strides(libpw, y_name, extra, base, x_extra, w_extra):
    rng = np.random.default_rng(8)
    q, s, v = weights(2, 392, 200, 4)
    off = [0, 70, 133]
    y, xv = product(rng.normal(size=(140, 200)), q, s, off, 392, y_name, extra, base, x_extra, w_extra)
    check(y, y_name, xv, v, off, 200)


def test_product_repeats_bit_for_bit(libpw):
    """Units cut along K are joined in piece order, whichever CTA joins."""
    rng = np.random.default_rng(9)
    q, s, v = weights(1, 1536, 8192, 5)
    x = rng.normal(size=(5, 8192))
    first = product(x, q, s, None, 1536, "f32")[0].np()
    for poison in (0, 0x7F, 0xFF):
        assert np.array_equal(product(x, q, s, None, 1536, "f32", poison=poison)[0].np(), first)


def test_product_non_finite_rows_stay_apart(libpw):
    rng = np.random.default_rng(10)
    q, s, v = weights(1, 256, 256, 6)
    x = rng.normal(size=(6, 256)).astype(np.float32)
    x[2, 3], x[4, 200] = np.nan, np.inf
    y, xv = product(x, q, s, None, 256, "f32")
    got = y.np()
    assert np.isnan(got[[2, 4]]).all() and np.isfinite(got[[0, 1, 3, 5]]).all()
    ref = S.gemm(xv[[0, 1, 3, 5]], v, [0, 4])
    assert (np.abs(got[[0, 1, 3, 5]] - ref) <= (sum_bound(2) + U) * S.gemm(np.abs(xv[[0, 1, 3, 5]]), np.abs(v), [0, 4])).all()


@pytest.mark.parametrize("off", [[0, 5, 3, 8], [0, 4, 20, 8], [-3, 2, 4, 8], [8, 0, 0, 0]])
def test_bad_offsets_are_recorded(libpw, off):
    """Rows outside [0, M] and groups that go backwards give no rows: nothing outside y is touched."""
    import torch
    M, N, K, E = 8, 256, 128, 3
    q, s, _ = weights(E, N, K, 7)
    w, ldw = padded_codes(q)
    xq = torch.zeros(M, 128, dtype=torch.uint8, device="cuda")
    xs, ws = torch.ones(M, 1, device="cuda"), gpu(s)
    y = Strided(M, N, "f32", 0, 64)
    n = B.pw_scaled_gemm_workspace_bytes(M, N, K, E)
    tmp = torch.empty(n, dtype=torch.uint8, device="cuda")
    o = gpu(np.asarray(off, np.int32))
    B.check(B.pw_scaled_gemm(xq.data_ptr(), xs.data_ptr(), M, K, 128, w.data_ptr(), ws.data_ptr(), E, N, ldw,
                             o.data_ptr(), y.ptr, B.PW_TYPE_F32, y.ld, tmp.data_ptr(), n))
    assert B.pw_get_status() == B.PW_ERR_BOUNDS
    assert y.outside_untouched()
    got = y.np()
    assert ((got == 0) | (got == -77.0)).all()


@pytest.mark.parametrize("M", [5, 70])                     # both kernels
def test_product_of_extreme_scales(libpw, M):
    """The product of two scales is rounded to fp32 first.  In the normal range that costs what
    sum_bound grants; below 2^-126 its absolute error is half of 2^-149, and |P| <= 128 * 448^2 < 2^25, so
    a block adds less than 2^-125."""
    import torch
    N, K = 140, 256
    rng = np.random.default_rng([28, M])
    q, _, _ = weights(1, N, K, 29)
    xq = S.round_e4m3(np.clip(rng.normal(size=(M, K)) * 120, -448, 448))
    e = np.array([[-126, -126], [120, -100], [-126, 100], [90, 119], [-60, 0]])
    xs = 2.0 ** e[np.arange(M) % 5]
    ws = (np.array([[[2.0 ** -20, 2.0 ** -12], [2.0 ** -13, 1.0]]]) * 1.1875).astype(np.float32)
    w, ldw = padded_codes(q)
    d = [gpu(xq), gpu(xs.astype(np.float32)), gpu(ws)]
    y, n = torch.empty(M, N, device="cuda"), B.pw_scaled_gemm_workspace_bytes(M, N, K, 1)
    tmp = torch.empty(n, dtype=torch.uint8, device="cuda")
    B.check(B.pw_scaled_gemm(d[0].data_ptr(), d[1].data_ptr(), M, K, K, w.data_ptr(), d[2].data_ptr(), 1, N, ldw, 0,
                             y.data_ptr(), B.PW_TYPE_F32, N, tmp.data_ptr(), n))
    assert B.pw_get_status() == B.PW_OK
    xv, v = S.values(xq, xs, 1), S.values(q[0], ws[0], 128)
    with np.errstate(over="ignore"):
        ref, mag = xv @ v.T, np.abs(xv) @ np.abs(v).T
    got = y.double().cpu().numpy()
    fits = np.broadcast_to(mag < 2.0 ** 127, got.shape)
    assert (np.abs(got - ref)[fits] <= (sum_bound(2) * mag + 2 * 2.0 ** -125)[fits]).all()
    assert fits[[0, 2, 4]].all() and fits[1].any() and np.isfinite(got[fits]).all()
    assert (np.abs(ref[0]) < 2.0 ** -100).any() and (got[0] != 0).all()


def groups_of(off, M):
    """The rows that offsets give: taken into [0, M], no group starts before an earlier offset."""
    o = np.clip(off, 0, M)
    return [(o[e], o[e + 1]) if o[e] >= max(o[:e + 1]) else (o[e], o[e]) for e in range(len(o) - 1)]


@pytest.mark.parametrize("scale", [1, 100])                # 100: the large-rows kernel
@pytest.mark.parametrize("off", [[0, 5, 3, 8], [0, 4, 20, 8], [-3, 2, 4, 8], [8, 0, 0, 0], [2, 6, 1, 8, 3, 8],
                                 [0, 8, 0, 8, 0, 8], [3, 1, 5, 6, 2, 7]])
def test_bad_offsets_keep_groups_apart(libpw, off, scale):
    """The valid groups are right, every other row is left as it was: no row has two writers."""
    off, M, N, K, E = np.array(off) * scale, 8 * scale, 300, 200, len(off) - 1
    check_groups(off, M, N, K, E)


def test_bad_offsets_of_many_experts(libpw):
    """A decrease in the middle of 200 experts, and one after it: looked at 32 experts at a time."""
    rows = np.random.default_rng(26).integers(0, 4, 200)
    off = np.concatenate([[0], np.cumsum(rows)])
    M = int(off[-1])
    off[77] -= 40
    off[130] = M
    check_groups(off, M, 130, 128, 200)


def check_groups(off, M, N, K, E):
    import torch
    rng = np.random.default_rng([M, E])
    q, s, v = weights(E, N, K, 27)
    w, ldw = padded_codes(q)
    x = gpu(rng.normal(size=(M, K)).astype(np.float32))
    ld = -(-K // 16) * 16
    xq, xs = torch.full((M, ld), 127, dtype=torch.uint8, device="cuda"), torch.empty(M, -(-K // 128), device="cuda")
    B.check(B.pw_scaled_quantize(x.data_ptr(), B.PW_TYPE_F32, M, K, K, 1, xq.data_ptr(), ld, xs.data_ptr()))
    y, ws, o = Strided(M, N, "f32", 4, 64), gpu(s), gpu(np.asarray(off, np.int32))
    n = B.pw_scaled_gemm_workspace_bytes(M, N, K, E)
    tmp = torch.empty(n, dtype=torch.uint8, device="cuda")
    B.check(B.pw_scaled_gemm(xq.data_ptr(), xs.data_ptr(), M, K, ld, w.data_ptr(), ws.data_ptr(), E, N, ldw,
                             o.data_ptr(), y.ptr, B.PW_TYPE_F32, y.ld, tmp.data_ptr(), n))
    assert B.pw_get_status() == B.PW_ERR_BOUNDS
    xv = S.values(*S.quantize(x.double().cpu().numpy(), 1), 1)
    got, left = y.np(), np.ones(M, bool)
    for e, (a, b) in enumerate(groups_of(off, M)):
        if a < b:
            assert left[a:b].all()
            left[a:b] = False
            ref, mag = xv[a:b] @ v[e].T, np.abs(xv[a:b]) @ np.abs(v[e]).T
            assert (np.abs(got[a:b] - ref) <= (sum_bound(-(-K // 128)) + U) * mag).all()
    assert (got[left] == -77.0).all() and y.outside_untouched()


def _layer(H, I, E, seed):
    q1, s1, v1 = weights(E, 2 * I, H, seed)
    q2, s2, v2 = weights(E, H, I, seed + 1)
    s1, s2 = s1 * 4, s2 * 4
    return (gpu(q1), gpu(s1), gpu(q2), gpu(s2)), v1 * 4, v2 * 4


LAYERS = [(1, 2, 8, 256, 512, "f32", "f32"), (4, 2, 8, 256, 512, "bf16", "f32"), (33, 4, 12, 128, 384, "bf16", "bf16"),
          (150, 1, 1, 4096, 128, "bf16", "f32"), (8, 1, 1, 4096, 256, "bf16", "f32"), (2, 1, 3, 128, 4096, "f16", "f32"),
          (1, 1, 1, 128, 128, "f16", "f16"), (70, 3, 5, 384, 128, "f32", "bf16"), (300, 2, 3, 256, 256, "bf16", "f32")]


@pytest.mark.parametrize("T,k,E,H,I,xt,yt", LAYERS)
def test_layer(libpw, T, k, E, H, I, xt, yt):
    import torch
    from any_precision_expert_pw_b200.scaled_layer import ScaledExperts
    rng = np.random.default_rng([T, k, E, H, I])
    tensors, v1, v2 = _layer(H, I, E, 11)
    ex = ScaledExperts(*tensors, max_tokens=T, k=k)
    ex.workspace.fill_(0xFF)
    idx = routing(T, E, k, 12, 0.1 if T > 4 else 0.0)
    if T > 10:
        idx[T - 3:] = -1
    gate = rng.random((T, k)).astype(np.float32)
    x = gpu(rng.normal(size=(T, H))).to(_torch_type(xt))
    y = torch.full((T, H), -7.0, dtype=_torch_type(yt), device="cuda")
    ex.forward(x, gpu(idx), gpu(gate), y)
    assert B.pw_get_status() == B.PW_OK
    ref, tol = moe_bound(x.double().cpu().numpy(), idx, gate, v1, v2)
    tol = tol + half_step(yt) * (np.abs(ref) + tol) + 2.0 ** -25
    got = y.double().cpu().numpy()
    assert (np.abs(got - ref) <= tol).all(), float(np.max(np.abs(got - ref) / tol))
    if T > 10:
        assert (got[T - 3:] == 0).all()
    # the bound itself is tight enough to see a wrong expert, gate or block
    assert float(np.median(tol)) < 0.05 * float(np.sqrt((ref ** 2).mean()))


class OnDemand:
    """The values of experts' weights on the device, one expert at a time."""

    def __init__(self, q, s):
        self.q, self.s, self.shape = q, s, tuple(q.shape)

    def __getitem__(self, e):
        return S.values(self.q[e].cpu().numpy(), self.s[e].cpu().numpy(), 128)


def device_weights(E, N, K, gen):
    import torch
    q = torch.empty(E, N, K, dtype=torch.uint8, device="cuda")
    for e in range(E):
        v = torch.randn(N, K, generator=gen, device="cuda").mul_(120).clamp_(-448, 448)
        q[e] = v.to(torch.float8_e4m3fn).view(torch.uint8)
    return q, torch.exp(torch.randn(E, N // 128, K // 128, generator=gen, device="cuda") * 0.3 - 7)


# the layers' own sizes: one token, a decode batch (both on the few-rows kernel), a prompt (large-rows)
@pytest.mark.parametrize("T,k,E,H,I,pick", [(1, 2, 8, 4096, 14336, [0]), (64, 8, 64, 3584, 2560, [0, 40]),
                                            (400, 8, 64, 3584, 2560, [3, 200, 396])])
def test_layer_at_its_real_sizes(libpw, T, k, E, H, I, pick):
    import torch
    from any_precision_expert_pw_b200.scaled_layer import ScaledExperts
    gen = torch.Generator(device="cuda")
    gen.manual_seed(T)
    q1, s1 = device_weights(E, 2 * I, H, gen)
    q2, s2 = device_weights(E, H, I, gen)
    ex = ScaledExperts(q1, s1, q2, s2, max_tokens=T, k=k)
    ex.workspace.fill_(0xFF)
    idx, gate = routing(T, E, k, 33), torch.rand(T, k, generator=gen, device="cuda")
    if T > 100:
        idx[T - 3:] = -1                                   # a padded batch
    x = torch.randn(T, H, generator=gen, device="cuda").bfloat16()
    y = ex.forward(x, gpu(idx), gate, torch.empty(T, H, device="cuda"))
    again = ex.forward(x, gpu(idx), gate, torch.empty(T, H, device="cuda"))
    assert B.pw_get_status() == B.PW_OK and bool((y == again).all())
    ref, tol = moe_bound(x[pick].double().cpu().numpy(), idx[pick], gate[pick].cpu().numpy(), OnDemand(q1, s1),
                         OnDemand(q2, s2))
    tol = tol + U * (np.abs(ref) + tol)
    got = y[pick].double().cpu().numpy()
    assert (np.abs(got - ref) <= tol).all(), float(np.max(np.abs(got - ref) / tol))
    # granting each of K terms its rounding moves many h to a border: the bound is 0.25 to 0.35 of the
    # outputs' rms here, and a wrong expert, gate or block moves thousands of outputs by more
    assert float(np.median(tol)) < 0.5 * float(np.sqrt((ref ** 2).mean()))
    if T > 100:
        assert bool((y[T - 3:] == 0).all())


@pytest.mark.parametrize("n", [2, 40])                     # tokens an expert: both kernels
def test_layer_of_very_negative_gates(libpw, n):
    """SiLU(g) u where e^-g passes 2^126 and 2^128 and u makes up for it.  x has one value, so g and u are
    known (one rounding, of g); h is off by (8 + 1.2 |g|) units (moe_bound), at most 2^-16 of its value,
    and where e^g is subnormal by half of 2^-149 in e^g >= 2^-133, another 2^-17: below 2^-15 in all.  It
    becomes its e4m3 value or, within that of a border, the next one."""
    import torch
    from any_precision_expert_pw_b200.scaled_layer import ScaledExperts
    gs = [-92.0, -89.5, -88.6, -88.0, -87.5, -86.0, -60.0, -20.0, -1.0, 0.0, 1.0, 30.0, 88.0]
    E, H, I, T = len(gs), 128, 128, len(gs) * n
    rng = np.random.default_rng(30)
    q1, q2 = np.zeros((E, 2 * I, H), np.uint8), S.round_e4m3(rng.normal(size=(E, H, I)) * 60)
    q1[:, :I, 0] = S.round_e4m3(448.0)
    q1[:, I:, 0] = S.round_e4m3(rng.uniform(64, 448, (E, I)) * rng.choice([-1, 1], (E, I)))
    s1, s2 = np.empty((E, 2, 1), np.float32), np.full((E, 1, 1), 2.0 ** -8, np.float32)
    s1[:, 0, 0] = np.array(gs) / 448
    s1[:, 1, 0] = 2.0 ** np.clip(np.round(-np.minimum(gs, 0) / np.log(2)) - 7, 0, 118)  # h up to about 100
    ex = ScaledExperts(gpu(q1), gpu(s1), gpu(q2), gpu(s2), max_tokens=T, k=1)
    x = torch.zeros(T, H, device="cuda")
    x[:, 0] = 1.0
    idx = (np.arange(T) % E).astype(np.int32)[:, None]
    y = ex.forward(x, gpu(idx), torch.ones(T, 1, device="cuda")).double().cpu().numpy()
    assert B.pw_get_status() == B.PW_OK
    for e in range(E):
        g, u = float(np.float32(448.0 * float(s1[e, 0, 0]))), S.values(q1[e, I:, :1], s1[e, 1:], 128)[:, 0]
        h = S.silu(g) * u
        q, sc = S.quantize(h[None], 1)
        hv, w2 = S.values(q, sc, 1)[0], S.values(q2[e], s2[e], 128)
        top, a = np.abs(h).max(), np.abs(h) / sc[0, 0]
        assert S.block_scale(top * (1 - 2.0 ** -15)) == S.block_scale(top * (1 + 2.0 ** -15))
        step = np.maximum(2.0 ** (np.floor(np.log2(np.maximum(a, 2.0 ** -6))) - 3), 2.0 ** -9)
        near = np.abs(a / step - np.floor(a / step) - 0.5) * step <= 2.0 ** -15 * a
        tol = np.abs(w2) @ np.where(near, step * sc[0, 0], 0) + sum_bound(1) * (np.abs(w2) @ (1.25 * np.abs(hv)))
        ref = w2 @ hv
        assert (np.abs(y[idx[:, 0] == e] - ref) <= tol).all(), gs[e]
        assert g == 0 or np.abs(y[idx[:, 0] == e]).max() > 0, gs[e]


def test_layer_bad_expert_is_recorded(libpw):
    import torch
    from any_precision_expert_pw_b200.scaled_layer import ScaledExperts
    tensors, _, _ = _layer(128, 128, 4, 13)
    ex = ScaledExperts(*tensors, max_tokens=4, k=2)
    x = torch.randn(4, 128, device="cuda")
    gate = torch.rand(4, 2, device="cuda")
    good = gpu(np.array([[0, 1], [2, 3], [1, -1], [3, 0]], np.int32))
    bad = good.clone()
    bad[2, 1] = 4
    a = ex.forward(x, good, gate)
    assert B.pw_get_status() == B.PW_OK
    b = ex.forward(x, bad, gate)
    assert B.pw_get_status() == B.PW_ERR_BAD_EXPERT
    assert bool((a == b).all())


def test_layer_after_the_router_in_a_graph(libpw):
    """Router, remap, expert layer: captured once on another stream, replayed on new activations;
    equal to the calls made one by one."""
    import torch
    from any_precision_expert_pw_b200.scaled_layer import ScaledExperts
    cfg = CONFIGS["qwen2_57b_a14b"].scaled(H=256, I=128, E=16)
    T, E, H, k = 24, cfg.E, cfg.H, cfg.k
    tensors, _, _ = _layer(H, cfg.I, E, 14)
    ex = ScaledExperts(*tensors, max_tokens=T, k=k)
    rc = B.pw_route_cfg(k=k, renorm=1, policy=0, threshold=0.15, critical_n=10)
    x = torch.randn(T, H, device="cuda").bfloat16()
    wr = torch.randn(E, H, device="cuda") * 0.1
    logits = torch.empty(T, E, device="cuda")
    idx = torch.empty(T, k, dtype=torch.int32, device="cuda")
    gate = torch.empty(T, k, device="cuda")
    y = torch.empty(T, H, device="cuda").bfloat16()

    def step(st):
        B.check(B.pw_route_topk(x.data_ptr(), wr.data_ptr(), 0, T, H, E, rc, logits.data_ptr(),
                                idx.data_ptr(), gate.data_ptr(), st))
        B.check(B.pw_remap(logits.data_ptr(), idx.data_ptr(), gate.data_ptr(), T, E, rc, 0, 0, st))
        ex.forward(x, idx, gate, y, stream=st)

    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    step(s.cuda_stream)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step(torch.cuda.current_stream().cuda_stream)
    for _ in range(3):
        x.normal_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = y.clone()
        step(torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()
        assert bool((y == got).all()) and bool(got.isfinite().all())
    assert B.pw_get_status() == B.PW_OK


def test_layer_two_streams_with_their_own_workspaces(libpw):
    import torch
    from any_precision_expert_pw_b200.scaled_layer import ScaledExperts
    H, I, E, T, k = 512, 512, 8, 40, 2
    tensors, _, _ = _layer(H, I, E, 15)
    xs = [torch.randn(T, H, device="cuda").bfloat16() for _ in range(2)]
    idx, gate = gpu(routing(T, E, k, 16)), torch.rand(T, k, device="cuda")
    ex = [ScaledExperts(*tensors, max_tokens=T, k=k) for _ in range(2)]
    want = [ex[0].forward(x, idx, gate).clone() for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    ys = [torch.empty_like(x) for x in xs]
    for _ in range(20):
        for i in range(2):
            ex[i].forward(xs[i], idx, gate, ys[i], stream=streams[i].cuda_stream)
    torch.cuda.synchronize()
    assert all(bool((a == b).all()) for a, b in zip(ys, want))
    assert B.pw_get_status() == B.PW_OK


def test_layer_on_another_stream_keeps_its_memory(libpw):
    """Experts and workspace may be dropped while a call on another stream waits there: their memory is
    not handed out again before that stream is done, and the call's own output belongs to both streams.
    (Given activations are the caller's to record.)"""
    import torch
    from any_precision_expert_pw_b200.scaled_layer import ScaledExperts
    H, I, E, T, k = 640, 384, 4, 50, 2
    tensors, _, _ = _layer(H, I, E, 31)
    x, idx, gate = torch.randn(T, H, device="cuda"), gpu(routing(T, E, k, 32)), torch.rand(T, k, device="cuda")
    want = ScaledExperts(*tensors, max_tokens=T, k=k).forward(x, idx, gate) + 0   # every kernel loaded
    torch.cuda.synchronize()

    def fresh():
        return [t.clone() for t in (*tensors, x, idx, gate)]

    s, done = torch.cuda.Stream(), torch.cuda.Event()
    mine = fresh()
    ex = ScaledExperts(*mine[:4], max_tokens=T, k=k)
    ex.workspace.zero_()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        torch.cuda._sleep(400_000_000)                     # about 0.2 s
    y = ex.forward(*mine[4:], stream=s.cuda_stream)
    for t in mine[4:]:
        t.record_stream(s)
    done.record(s)
    sizes = [t.numel() * t.element_size() for t in (*mine, ex.workspace)]
    held = [(t.data_ptr(), n) for t, n in zip((*mine, ex.workspace), sizes)]
    del mine, ex
    again = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes]
    assert not done.query()                                # the call has not run yet
    for t in again:
        assert all(t.data_ptr() + t.numel() <= p or p + n <= t.data_ptr() for p, n in held)
        t.fill_(0xFF)
    torch.cuda.current_stream().wait_event(done)
    assert bool((y == want).all())
    # the output: dropped while the current stream still reads it, it is not given to the other stream
    torch.cuda._sleep(400_000_000)
    z, at, n = y + 0, y.data_ptr(), y.numel() * 4
    done.record()
    del y
    with torch.cuda.stream(s):
        other = torch.empty(n, dtype=torch.uint8, device="cuda")
        assert not done.query()
        assert other.data_ptr() + n <= at or at + n <= other.data_ptr()
        other.fill_(0xFF)
    torch.cuda.synchronize()
    assert bool((z == want).all()) and B.pw_get_status() == B.PW_OK


def test_quantized_weights_object(libpw):
    """quantize_weights: 128 x 128 blocks of each matrix, odd sizes included, and a layer on them
    close to the unquantised one (both roundings are at most 2^-4 of a value)."""
    import torch
    from any_precision_expert_pw_b200.scaled_layer import ScaledExperts, quantize_weights
    w = torch.randn(3, 200, 150, device="cuda")
    q, s = quantize_weights(w)
    for e in range(3):
        wq, wsc = S.quantize(w[e].double().cpu().numpy(), 128)
        assert np.array_equal(q[e, :, :150].cpu().numpy(), wq)
        assert np.array_equal(s[e].double().cpu().numpy(), wsc)
    E, H, I, T, k = 4, 256, 128, 9, 2
    w1, w2 = torch.randn(E, 2 * I, H, device="cuda") * 0.05, torch.randn(E, H, I, device="cuda") * 0.05
    ex = ScaledExperts(*quantize_weights(w1.bfloat16()), *quantize_weights(w2.bfloat16()), max_tokens=T, k=k)
    idx, gate = routing(T, E, k, 17), np.random.default_rng(18).random((T, k)).astype(np.float32)
    x = torch.randn(T, H, device="cuda")
    y = ex.forward(x, gpu(idx), gpu(gate)).double().cpu().numpy()
    v = [[S.values(*S.quantize(m[e].bfloat16().double().cpu().numpy(), 128), 128) for e in range(E)] for m in (w1, w2)]
    ref, tol = moe_bound(x.double().cpu().numpy(), idx, gate, np.stack(v[0]), np.stack(v[1]))
    assert (np.abs(y - ref) <= tol + U * np.abs(ref)).all()
    assert B.pw_get_status() == B.PW_OK


def test_layer_without_any_assignment(libpw):
    import torch
    from any_precision_expert_pw_b200.scaled_layer import ScaledExperts
    tensors, _, _ = _layer(128, 128, 4, 19)
    ex = ScaledExperts(*tensors, max_tokens=70, k=2)
    ex.workspace.fill_(0xFF)
    for T in (1, 70):
        y = torch.full((T, 128), -7.0, device="cuda")
        ex.forward(torch.randn(T, 128, device="cuda"), torch.full((T, 2), -1, dtype=torch.int32, device="cuda"),
                   torch.full((T, 2), float("nan"), device="cuda"), y)
        assert B.pw_get_status() == B.PW_OK and bool((y == 0).all())


@pytest.mark.parametrize("T,E", [(3, 8), (200, 2)])
def test_layer_stays_inside_its_buffers(libpw, T, E):
    import torch
    H, I, k = 256, 384, 2
    (q1, s1, q2, s2), _, _ = _layer(H, I, E, 20)
    st = B.pw_scaled_experts(E=E, H=H, I=I, gate_up=q1.data_ptr(), gate_up_scale=s1.data_ptr(),
                             down=q2.data_ptr(), down_scale=s2.data_ptr())
    x = torch.randn(T, H, device="cuda")
    idx, gate = gpu(routing(T, E, k, 21)), torch.rand(T, k, device="cuda")
    y = torch.full((T + 64, H), -77.0, device="cuda")
    n = B.pw_moe_scaled_workspace_bytes(T, k, E, H, I)
    ws = torch.full((n + 65536,), 0xA5, dtype=torch.uint8, device="cuda")
    B.check(B.pw_moe_scaled_forward(st, x.data_ptr(), B.PW_TYPE_F32, T, k, idx.data_ptr(), gate.data_ptr(),
                                    y[32:].data_ptr(), B.PW_TYPE_F32, ws.data_ptr(), n))
    assert B.pw_get_status() == B.PW_OK
    assert bool((ws[n:] == 0xA5).all()) and bool((y[:32] == -77.0).all()) and bool((y[32 + T:] == -77.0).all())
    assert bool(y[32:32 + T].isfinite().all())


def test_gradient_on_transposed_blocks(libpw):
    """d_x = d_y W: square blocks transpose with their scales, so it is the product on W^T."""
    rng = np.random.default_rng(22)
    N, K, M = 300, 200, 40
    q, s, v = weights(1, N, K, 23)
    qt, st = np.ascontiguousarray(q.transpose(0, 2, 1)), np.ascontiguousarray(s.transpose(0, 2, 1))
    y, dyv = product(rng.normal(size=(M, N)), qt, st, None, K, "f32")
    ref = dyv @ v[0]
    mag = np.abs(dyv) @ np.abs(v[0])
    assert (np.abs(y.np() - ref) <= (sum_bound(-(-N // 128)) + U) * mag).all()


def test_products_beyond_32_bits(libpw):
    """Rows whose offsets pass 2^32 elements: the first, a middle one and the last against the oracle."""
    import torch
    M, N, K = 280000, 130, 16384
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB of device memory")
    x = torch.empty(M, K, dtype=torch.bfloat16, device="cuda").normal_()
    xq = torch.empty(M, K, dtype=torch.uint8, device="cuda")
    xs = torch.empty(M, K // 128, device="cuda")
    B.check(B.pw_scaled_quantize(x.data_ptr(), B.PW_TYPE_BF16, M, K, K, 1, xq.data_ptr(), K, xs.data_ptr()))
    q, s, v = weights(1, N, K, 24)
    w, ldw = padded_codes(q)
    ws = gpu(s)
    n = B.pw_scaled_gemm_workspace_bytes(M, N, K, 1)
    tmp = torch.empty(n, dtype=torch.uint8, device="cuda")
    y = torch.empty(M, 16400, device="cuda")                # rows 16400 apart: 2^32 elements too
    B.check(B.pw_scaled_gemm(xq.data_ptr(), xs.data_ptr(), M, K, K, w.data_ptr(), ws.data_ptr(), 1, N, ldw, 0,
                             y.data_ptr(), B.PW_TYPE_F32, 16400, tmp.data_ptr(), n))
    assert B.pw_get_status() == B.PW_OK
    pick = [0, 1, M // 2, M - 2, M - 1]
    xv = S.values(*S.quantize(x[pick].double().cpu().numpy(), 1), 1)
    ref, mag = xv @ v[0].T, np.abs(xv) @ np.abs(v[0]).T
    assert (np.abs(y[pick][:, :N].double().cpu().numpy() - ref) <= (sum_bound(K // 128) + U) * mag).all()


@pytest.mark.parametrize("M", [5, 300])                    # both kernels
def test_wait_that_never_completes_times_out(libpw, M):
    """The issuers wait for operands that never come: the call returns, the status reads PW_ERR_TIMEOUT
    once, the tiles are zeros, and the next call is right."""
    import torch
    N, K = 600, 4096
    q, s, v = weights(1, N, K, 25)
    w, ldw = padded_codes(q)
    ws = gpu(s)
    x = torch.randn(M, K, device="cuda")
    xq, xs = torch.empty(M, K, dtype=torch.uint8, device="cuda"), torch.empty(M, K // 128, device="cuda")
    B.check(B.pw_scaled_quantize(x.data_ptr(), B.PW_TYPE_F32, M, K, K, 1, xq.data_ptr(), K, xs.data_ptr()))
    n = B.pw_scaled_gemm_workspace_bytes(M, N, K, 1)
    tmp = torch.empty(n, dtype=torch.uint8, device="cuda")

    def run():
        y = torch.full((M, N), -7.0, device="cuda")
        B.check(B.pw_scaled_gemm(xq.data_ptr(), xs.data_ptr(), M, K, K, w.data_ptr(), ws.data_ptr(), 1, N, ldw, 0,
                                 y.data_ptr(), B.PW_TYPE_F32, N, tmp.data_ptr(), n))
        return y, B.pw_get_status()

    try:
        B.check(B.pw_set_wait_limit_ns(5_000_000))          # 5 ms
        B.check(B.pw_test_hold_down_items(1))
        y, st = run()
        assert st == B.PW_ERR_TIMEOUT and B.pw_get_status() == B.PW_OK
        assert bool((y == 0).all())
    finally:
        B.check(B.pw_test_hold_down_items(0))
        B.check(B.pw_set_wait_limit_ns(0))
    y, st = run()
    assert st == B.PW_OK
    xv = S.values(*S.quantize(x.double().cpu().numpy(), 1), 1)
    ref, mag = xv @ v[0].T, np.abs(xv) @ np.abs(v[0]).T
    assert (np.abs(y.double().cpu().numpy() - ref) <= (sum_bound(K // 128) + U) * mag).all()


@pytest.mark.parametrize("M,N,K,pick", [(1 << 24, 40, 48, [0, 1, 5_000_001, (1 << 24) - 1]), (3, 130, 1 << 18, [0, 2]),
                                        (70, 130, (1 << 18) - 3, [0, 69]), (2, 1 << 18, 136, [0, 1])])
def test_products_of_largest_sizes(libpw, M, N, K, pick):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(N)
    ld, kb = -(-K // 16) * 16, -(-K // 128)
    x = torch.randn(M, K, generator=g, device="cuda").bfloat16()
    xq, xs = torch.full((M, ld), 127, dtype=torch.uint8, device="cuda"), torch.empty(M, kb, device="cuda")
    B.check(B.pw_scaled_quantize(x.data_ptr(), B.PW_TYPE_BF16, M, K, K, 1, xq.data_ptr(), ld, xs.data_ptr()))
    q, s, v = weights(1, N, K, 34)
    w, ldw = padded_codes(q)
    ws, n = gpu(s), B.pw_scaled_gemm_workspace_bytes(M, N, K, 1)
    tmp, y = torch.empty(n, dtype=torch.uint8, device="cuda"), torch.full((M + 1, N), -7.0, device="cuda")
    B.check(B.pw_scaled_gemm(xq.data_ptr(), xs.data_ptr(), M, K, ld, w.data_ptr(), ws.data_ptr(), 1, N, ldw, 0,
                             y.data_ptr(), B.PW_TYPE_F32, N, tmp.data_ptr(), n))
    assert B.pw_get_status() == B.PW_OK and bool((y[M] == -7.0).all())
    xv = S.values(*S.quantize(x[pick].double().cpu().numpy(), 1), 1)
    ref, mag = xv @ v[0].T, np.abs(xv) @ np.abs(v[0]).T
    assert (np.abs(y[pick].double().cpu().numpy() - ref) <= (sum_bound(kb) + U) * mag).all()


def test_layer_of_the_largest_batch(libpw):
    """2^24 assignments: the rows of some tokens against the oracle, padding zero."""
    import torch
    from any_precision_expert_pw_b200.scaled_layer import ScaledExperts
    T, k, E, H, I = 1 << 21, 8, 16, 128, 128
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB of device memory")
    g = torch.Generator(device="cuda")
    g.manual_seed(35)
    tensors, v1, v2 = _layer(H, I, E, 36)
    ex = ScaledExperts(*tensors, max_tokens=T, k=k)
    x = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    idx = torch.rand(T, E, generator=g, device="cuda").topk(k, dim=1).indices.int()
    idx[T - 1000:] = -1
    gate = torch.rand(T, k, generator=g, device="cuda")
    y = ex.forward(x, idx, gate, torch.empty(T, H, device="cuda"))
    assert B.pw_get_status() == B.PW_OK and bool((y[T - 1000:] == 0).all()) and bool(y.isfinite().all())
    pick = [0, 1, 77_777, T // 2, T - 1001]
    ref, tol = moe_bound(x[pick].double().cpu().numpy(), idx[pick].cpu().numpy(), gate[pick].cpu().numpy(), v1, v2)
    assert (np.abs(y[pick].double().cpu().numpy() - ref) <= tol + U * (np.abs(ref) + tol)).all()

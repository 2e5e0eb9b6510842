"""Token rows sorted by expert and back, against the float64 oracle.

Tolerances: copies and whole numbers are equal.  A sum of n fp32 terms by fused multiply-adds is off
by at most n 2^-24 of the sum of its terms' magnitudes; a result rounded to a type adds half a step
(eps / 2 of the value: bf16 2^-8, fp16 2^-11, fp32 2^-24) and, in fp16, half a subnormal step."""
import numpy as np
import pytest

from any_precision_expert_pw_b200 import binding as B
from oracle import rows as R

pytestmark = pytest.mark.gpu

TYPES = {"f32": B.PW_TYPE_F32, "bf16": B.PW_TYPE_BF16, "f16": B.PW_TYPE_F16}
U = 2.0 ** -24


def _torch_type(name):
    import torch
    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[name]


def half_step(name):
    import torch
    return float(torch.finfo(_torch_type(name)).eps) / 2


def routing(T, E, k, seed, empty=0.0):
    rng = np.random.default_rng([T, E, k, seed])
    idx = np.stack([rng.permutation(E)[:k] if k <= E else rng.integers(0, E, k) for _ in range(T)])
    idx[rng.random(idx.shape) < empty] = -1
    return idx.astype(np.int32)


def gpu(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def run_sort(idx, E, stream=0):
    import torch
    T, k = idx.shape
    d = gpu(idx)
    pos = torch.full((T, k), -7, dtype=torch.int32, device="cuda")
    src = torch.full((T * k,), -7, dtype=torch.int32, device="cuda")
    off = torch.full((E + 1,), -7, dtype=torch.int32, device="cuda")
    n = B.pw_expert_sort_workspace_bytes(T, k, E)
    ws = torch.full((n,), 0xA5, dtype=torch.uint8, device="cuda")
    B.check(B.pw_expert_sort(d.data_ptr(), T, k, E, pos.data_ptr(), src.data_ptr(), off.data_ptr(),
                             ws.data_ptr(), n, stream))
    st = B.pw_get_status(stream)
    return pos, src, off, st


SORTS = [(1, 1, 1, 0.0), (1, 8, 16, 0.3), (7, 3, 2, 0.0), (16, 512, 10, 0.0), (33, 60, 4, 0.2),
         (257, 1024, 16, 0.1), (1024, 8, 8, 0.0), (1025, 8, 8, 0.5), (4099, 64, 8, 0.03),
         (20000, 5, 3, 1.0), (70001, 1000, 2, 0.0)]


@pytest.mark.parametrize("T,E,k,empty", SORTS)
def test_sort(libpw, T, E, k, empty):
    idx = routing(T, E, k, 1, empty) if T < 5000 else np.random.default_rng(T).integers(-1, E, (T, k)).astype(np.int32)
    if empty == 1.0:
        idx[:] = -1
    pos, src, off, st = run_sort(idx, E)
    assert st == B.PW_OK
    flat = idx.reshape(-1)
    order = np.argsort(np.where(flat < 0, E, flat), kind="stable")
    n = int((flat >= 0).sum())
    counts = np.bincount(flat[flat >= 0], minlength=E)
    assert np.array_equal(off.cpu().numpy(), np.concatenate([[0], np.cumsum(counts)]))
    assert np.array_equal(src.cpu().numpy()[:n], order[:n])
    assert (src.cpu().numpy()[n:] == -7).all()                       # left as they were
    want = np.full(T * k, -1)
    want[order[:n]] = np.arange(n)
    assert np.array_equal(pos.cpu().numpy().reshape(-1), want)
    if T <= 300:
        opos, osrc, ooff = R.sort(idx, E)
        assert np.array_equal(opos.reshape(-1), want) and np.array_equal(osrc, order[:n])


def test_sort_one_expert_and_repeated_ids(libpw):
    # every slot of every token on one expert: rows in slot order
    idx = np.full((50, 4), 3, np.int32)
    pos, src, off, st = run_sort(idx, 5)
    assert st == B.PW_OK
    assert np.array_equal(pos.cpu().numpy().reshape(-1), np.arange(200))
    assert off.cpu().numpy().tolist() == [0, 0, 0, 0, 200, 200]


@pytest.mark.parametrize("T,k,E,kind", [(1 << 24, 1, 1, "one"), (1 << 24, 1, 3, "dominant"),
                                        (1 << 20, 16, 1024, "blocks"), (650_001, 15, 2, "dominant")])
def test_sort_largest_batches(libpw, T, k, E, kind):
    """The largest batches, most of a run's slots on one expert: every row once, in slot order."""
    import torch
    n = T * k
    if kind == "one":
        flat = torch.zeros(n, dtype=torch.int32, device="cuda")
    elif kind == "dominant":                     # 3 of 100 slots elsewhere or empty
        g = torch.Generator(device="cuda")
        g.manual_seed(n)
        flat = torch.full((n,), E - 1, dtype=torch.int32, device="cuda")
        other = torch.rand(n, generator=g, device="cuda") < 0.03
        flat[other] = torch.randint(-1, E, (int(other.sum()),), generator=g, device="cuda", dtype=torch.int32)
    else:                                        # long runs of one id, each longer than a CTA's run
        flat = (torch.arange(n, device="cuda") // 200_000 * 37 % E).int()
    pos = torch.full((n,), -7, dtype=torch.int32, device="cuda")
    src = torch.full((n,), -7, dtype=torch.int32, device="cuda")
    off = torch.full((E + 1,), -7, dtype=torch.int32, device="cuda")
    size = B.pw_expert_sort_workspace_bytes(T, k, E)
    ws = torch.full((size + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    B.check(B.pw_expert_sort(flat.data_ptr(), T, k, E, pos.data_ptr(), src.data_ptr(), off.data_ptr(),
                             ws.data_ptr(), size))
    assert B.pw_get_status() == B.PW_OK and bool((ws[size:] == 0xA5).all())
    key = torch.where(flat < 0, E, flat)
    order = torch.sort(key, stable=True).indices
    live = int((flat >= 0).sum())
    assert bool((src[:live] == order[:live]).all()) and bool((src[live:] == -7).all())
    want = torch.full((n,), -1, dtype=torch.int32, device="cuda")
    want[order[:live]] = torch.arange(live, dtype=torch.int32, device="cuda")
    assert bool((pos == want).all())
    count = torch.bincount(key.long(), minlength=E + 1)[:E]
    assert off.tolist() == [0] + torch.cumsum(count, 0).tolist()


@pytest.mark.parametrize("T", [9, 3000])
def test_sort_records_bad_ids(libpw, T):
    idx = routing(T, 6, 3, 2)
    bad = idx.copy()
    bad[4, 1], bad[8, 0] = 6, -2
    clean = idx.copy()
    clean[4, 1] = clean[8, 0] = -1
    pos, src, off, st = run_sort(bad, 6)
    assert st == B.PW_ERR_BAD_EXPERT
    p2, s2, o2, st2 = run_sort(clean, 6)
    assert st2 == B.PW_OK and bool((pos == p2).all()) and bool((src == s2).all()) and bool((off == o2).all())


# T, E, k, H, stride added, element offset of the base, empty share
ROWS = [(1, 4, 1, 1, 0, 0, 0.0), (1, 8, 8, 2048, 0, 0, 0.0), (5, 3, 2, 7, 0, 0, 0.3),
        (16, 60, 4, 256, 0, 0, 0.0), (16, 60, 4, 264, 8, 0, 0.2), (33, 9, 3, 1001, 3, 1, 0.1),
        (64, 64, 8, 3584, 0, 0, 0.05), (9, 16, 16, 520, 0, 8, 0.1), (40, 16, 5, 130, 0, 0, 1.0)]


class Strided:
    """A [rows][H] tensor with a row stride and a base offset inside a sentinel-filled buffer."""

    def __init__(self, rows, H, name, extra, base, values=None):
        import torch
        self.ld = H + extra
        self.buf = torch.full((base + rows * self.ld + 64,), -77.0, dtype=_torch_type(name), device="cuda")
        self.t = self.buf[base:base + rows * self.ld].view(rows, self.ld)[:, :H] if rows else self.buf[:0]
        if values is not None:
            self.t.copy_(values)
        self.ptr = self.buf.data_ptr() + base * self.buf.element_size()
        self.base, self.rows, self.H = base, rows, H

    def outside_untouched(self):
        m = self.buf.clone()
        if self.rows:
            m[self.base:self.base + self.rows * self.ld].view(self.rows, self.ld)[:, :self.H] = -77.0
        return bool((m == -77.0).all())

    def np(self):
        return self.t.double().cpu().numpy()


@pytest.mark.parametrize("name", list(TYPES))
@pytest.mark.parametrize("T,E,k,H,extra,base,empty", ROWS)
def test_movement_and_gradients(libpw, name, T, E, k, H, extra, base, empty):
    import torch
    rng = np.random.default_rng([T, E, k, H])
    idx = routing(T, E, k, 3, empty)
    if empty == 1.0:
        idx[:] = -1
    pos, _, off, st = run_sort(idx, E)
    assert st == B.PW_OK
    p = pos.cpu().numpy()
    n, rows = int(off[-1]), T * k
    ty = TYPES[name]
    gate = rng.normal(size=(T, k)).astype(np.float32)
    d_gate_t = torch.full((T, k), -7.0, device="cuda")
    x = Strided(T, H, name, extra, base, gpu(rng.normal(size=(T, H))))
    xs = Strided(rows, H, name, extra, base)
    B.check(B.pw_expert_dispatch(x.ptr, ty, T, k, H, x.ld, pos.data_ptr(), xs.ptr, xs.ld))
    want = R.dispatch(x.np(), p, rows)
    assert np.array_equal(xs.np()[:n], want[:n])
    assert (xs.np()[n:] == -77.0).all() and xs.outside_untouched()

    o_v = rng.normal(size=(rows, H))
    o_v[n:] = np.nan                                        # rows behind the last are not read
    o = Strided(rows, H, name, extra, base, gpu(o_v))
    g = gpu(gate)
    hs = half_step(name)
    tiny = 2.0 ** -25 if name == "f16" else 0.0
    # combine, into each output type
    ref = R.combine(o.np(), p, gate)
    mag = R.combine(np.abs(o.np()), p, np.abs(gate))
    for out in TYPES:
        y = Strided(T, H, out, extra, base)
        B.check(B.pw_expert_combine(o.ptr, ty, T, k, H, o.ld, pos.data_ptr(), g.data_ptr(), y.ptr,
                                    TYPES[out], y.ld))
        tol = k * U * mag
        tol = tol + half_step(out) * (np.abs(ref) + tol) + (2.0 ** -25 if out == "f16" else 0)
        assert (np.abs(y.np() - ref) <= tol).all() and y.outside_untouched()
    # gradient of dispatch
    dx = Strided(T, H, name, extra, base)
    B.check(B.pw_expert_dispatch_grad(o.ptr, ty, T, k, H, o.ld, pos.data_ptr(), dx.ptr, dx.ld))
    ref = R.dispatch_grad(o.np(), p)
    tol = k * U * R.dispatch_grad(np.abs(o.np()), p)
    assert (np.abs(dx.np() - ref) <= tol + hs * (np.abs(ref) + tol) + tiny).all()
    assert dx.outside_untouched()
    # gradient of combine
    dy = Strided(T, H, name, extra, base, gpu(rng.normal(size=(T, H))))
    do = Strided(rows, H, name, extra, base)
    B.check(B.pw_expert_combine_grad(dy.ptr, o.ptr, ty, T, k, H, dy.ld, o.ld, pos.data_ptr(),
                                     g.data_ptr(), do.ptr, do.ld, d_gate_t.data_ptr()))
    ref_o, ref_g = R.combine_grad(dy.np(), o.np(), p, gate)
    _, mag_g = R.combine_grad(np.abs(dy.np()), np.abs(o.np()), p, gate)
    r = ref_o[:n]
    assert (np.abs(do.np()[:n] - r) <= (U + hs * (1 + U)) * np.abs(r) + tiny).all()
    assert (do.np()[n:] == -77.0).all() and do.outside_untouched()
    # a thread adds at most H / 256 + 8 products, then 5 shuffles and 8 warps
    depth = H / 256 + 8 + 5 + 8
    assert (np.abs(d_gate_t.double().cpu().numpy() - ref_g) <= depth * U * mag_g).all()
    # either gradient alone gives the same bits
    do2, dg2 = Strided(rows, H, name, extra, base), torch.full((T, k), -7.0, device="cuda")
    B.check(B.pw_expert_combine_grad(dy.ptr, 0, ty, T, k, H, dy.ld, 0, pos.data_ptr(), g.data_ptr(),
                                     do2.ptr, do2.ld, 0))
    B.check(B.pw_expert_combine_grad(dy.ptr, o.ptr, ty, T, k, H, dy.ld, o.ld, pos.data_ptr(),
                                     g.data_ptr(), 0, 0, dg2.data_ptr()))
    assert np.array_equal(do2.np(), do.np()) and bool((dg2 == d_gate_t).all())
    assert B.pw_get_status() == B.PW_OK


def test_bad_rows_are_skipped_and_recorded(libpw):
    import torch
    T, k, H = 4, 2, 64
    pos = gpu(np.array([[0, 1], [2, 8], [-5, 3], [4, 5]], np.int32))   # 8 and -5 are no rows of 8 slots
    x = torch.randn(T, H, device="cuda")
    xs = torch.full((T * k, H), -7.0, device="cuda")
    B.check(B.pw_expert_dispatch(x.data_ptr(), B.PW_TYPE_F32, T, k, H, H, pos.data_ptr(), xs.data_ptr(), H))
    assert B.pw_get_status() == B.PW_ERR_BOUNDS
    assert bool((xs[[0, 1]] == x[0]).all()) and bool((xs[2] == x[1]).all()) and bool((xs[3] == x[2]).all())
    assert bool((xs[6:] == -7.0).all())
    y = torch.empty(T, H, device="cuda")
    gate = torch.ones(T, k, device="cuda")
    B.check(B.pw_expert_combine(xs.data_ptr(), B.PW_TYPE_F32, T, k, H, H, pos.data_ptr(),
                                gate.data_ptr(), y.data_ptr(), B.PW_TYPE_F32, H))
    assert B.pw_get_status() == B.PW_ERR_BOUNDS
    assert bool((y[1] == xs[2]).all()) and bool((y[2] == xs[3]).all())
    assert B.pw_get_status() == B.PW_OK


def test_non_finite_rows_stay_with_their_tokens(libpw):
    import torch
    idx = np.array([[0, 1], [1, 0], [0, -1]], np.int32)
    pos, _, _, _ = run_sort(idx, 2)
    o = torch.ones(6, 32, device="cuda")
    o[int(pos[0, 1])] = float("nan")
    o[int(pos[2, 0])] = float("inf")
    y = torch.empty(3, 32, device="cuda")
    gate = torch.ones(3, 2, device="cuda")
    B.check(B.pw_expert_combine(o.data_ptr(), B.PW_TYPE_F32, 3, 2, 32, 32, pos.data_ptr(),
                                gate.data_ptr(), y.data_ptr(), B.PW_TYPE_F32, 32))
    assert bool(y[0].isnan().all()) and bool((y[1] == 2).all()) and bool(y[2].isinf().all())


def test_offsets_beyond_32_bits(libpw):
    """Rows whose byte offsets pass 2^32: the last tokens' rows of a 5 GB buffer."""
    import torch
    T, k, H = 40000, 2, 16384
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB of device memory")
    idx = np.random.default_rng(0).integers(0, 8, (T, k)).astype(np.int32)
    pos, src, off, st = run_sort(idx, 8)
    assert st == B.PW_OK
    x = torch.randint(-1000, 1000, (T, H), device="cuda", dtype=torch.int32).to(torch.float32)
    xs = torch.empty(T * k, H, device="cuda")
    B.check(B.pw_expert_dispatch(x.data_ptr(), B.PW_TYPE_F32, T, k, H, H, pos.data_ptr(), xs.data_ptr(), H))
    pick = torch.tensor([0, 1, T * k // 2, T * k - 2, T * k - 1], device="cuda")
    assert bool((xs[pick] == x[src[pick].long() // k]).all())
    y = torch.empty(T, H, device="cuda")
    gate = torch.full((T, k), 0.5, device="cuda")
    B.check(B.pw_expert_combine(xs.data_ptr(), B.PW_TYPE_F32, T, k, H, H, pos.data_ptr(),
                                gate.data_ptr(), y.data_ptr(), B.PW_TYPE_F32, H))
    assert bool((y == x).all())                               # 0.5 x + 0.5 x, exact
    assert B.pw_get_status() == B.PW_OK


def test_run_together_in_a_graph_on_another_stream(libpw):
    """sort, dispatch, combine and both gradients captured once and replayed on other data."""
    import torch
    T, E, k, H = 300, 11, 3, 192
    s = torch.cuda.Stream()
    idx = gpu(routing(T, E, k, 5, 0.1))
    x, dy = torch.randn(T, H, device="cuda"), torch.randn(T, H, device="cuda")
    gate = torch.rand(T, k, device="cuda")
    pos, src = (torch.empty(T * k, dtype=torch.int32, device="cuda") for _ in range(2))
    off = torch.empty(E + 1, dtype=torch.int32, device="cuda")
    n = B.pw_expert_sort_workspace_bytes(T, k, E)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    xs, d_o = (torch.zeros(T * k, H, device="cuda") for _ in range(2))
    y, dx = torch.empty(T, H, device="cuda"), torch.empty(T, H, device="cuda")
    dg = torch.empty(T, k, device="cuda")
    f = B.PW_TYPE_F32

    def step(st):
        B.check(B.pw_expert_sort(idx.data_ptr(), T, k, E, pos.data_ptr(), src.data_ptr(),
                                 off.data_ptr(), ws.data_ptr(), n, st))
        B.check(B.pw_expert_dispatch(x.data_ptr(), f, T, k, H, H, pos.data_ptr(), xs.data_ptr(), H, st))
        B.check(B.pw_expert_combine(xs.data_ptr(), f, T, k, H, H, pos.data_ptr(), gate.data_ptr(),
                                    y.data_ptr(), f, H, st))
        B.check(B.pw_expert_combine_grad(dy.data_ptr(), xs.data_ptr(), f, T, k, H, H, H, pos.data_ptr(),
                                         gate.data_ptr(), d_o.data_ptr(), H, dg.data_ptr(), st))
        B.check(B.pw_expert_dispatch_grad(d_o.data_ptr(), f, T, k, H, H, pos.data_ptr(), dx.data_ptr(),
                                          H, st))

    torch.cuda.synchronize()
    step(s.cuda_stream)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step(torch.cuda.current_stream().cuda_stream)
    for seed in (6, 7):
        idx.copy_(gpu(routing(T, E, k, seed, 0.2)))
        x.normal_()
        gate.uniform_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        p, _, _ = R.sort(idx.cpu().numpy(), E)
        X, G, D = x.double().cpu().numpy(), gate.double().cpu().numpy(), dy.double().cpu().numpy()
        live = p >= 0
        w = (G * live).sum(1, keepdims=True)
        # y = (sum of gates) x, dx = (sum of gates) dy, dgate = <dy, x>: k terms each
        assert (np.abs(y.cpu().numpy() - w * X) <= (k + 1) * U * np.abs(w * X) + 1e-30).all()
        assert (np.abs(dx.cpu().numpy() - w * D) <= (2 * k + 2) * U * np.abs(w * D) + 1e-30).all()
        dots = np.where(live, (X * D).sum(1, keepdims=True), 0)
        mag = (np.abs(X * D)).sum(1, keepdims=True)
        assert (np.abs(dg.cpu().numpy() - dots) <= (H / 256 + 21) * U * mag).all()
    assert B.pw_get_status() == B.PW_OK


@pytest.mark.parametrize("T,k,H,name", [(1 << 20, 16, 24, "bf16"), (1 << 24, 1, 3, "f16"), (2, 3, 1 << 18, "f32"),
                                        (3, 2, (1 << 18) - 1, "bf16")])
def test_movement_of_largest_sizes(libpw, T, k, H, name):
    """2^24 rows, and rows of 2^18 columns: small whole numbers, so that every sum is exact in fp32."""
    import torch
    E, ty, dt = 5, TYPES[name], _torch_type(name)
    g = torch.Generator(device="cuda")
    g.manual_seed(H)
    idx = torch.randint(-1, E, (T, k), generator=g, device="cuda", dtype=torch.int32)
    pos = torch.empty_like(idx)
    src, off = torch.full((T * k,), -7, dtype=torch.int32, device="cuda"), torch.empty(E + 1, dtype=torch.int32, device="cuda")
    n = B.pw_expert_sort_workspace_bytes(T, k, E)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    B.check(B.pw_expert_sort(idx.data_ptr(), T, k, E, pos.data_ptr(), src.data_ptr(), off.data_ptr(),
                             ws.data_ptr(), n))
    live = int(off[-1])
    x = torch.randint(-3, 4, (T, H), generator=g, device="cuda", dtype=torch.int8).to(dt)
    gate = torch.randint(1, 3, (T, k), generator=g, device="cuda").float()
    xs = torch.full((T * k, H), -77.0, dtype=dt, device="cuda")
    B.check(B.pw_expert_dispatch(x.data_ptr(), ty, T, k, H, H, pos.data_ptr(), xs.data_ptr(), H))
    token = src[:live].long() // k
    for a in range(0, live, 1 << 22):
        b = min(live, a + (1 << 22))
        assert bool((xs[a:b] == x[token[a:b]]).all())
    assert bool((xs[live:] == -77.0).all())
    there = (pos >= 0).float()
    y, d_x = torch.empty_like(x), torch.empty_like(x)
    B.check(B.pw_expert_combine(xs.data_ptr(), ty, T, k, H, H, pos.data_ptr(), gate.data_ptr(), y.data_ptr(), ty, H))
    B.check(B.pw_expert_dispatch_grad(xs.data_ptr(), ty, T, k, H, H, pos.data_ptr(), d_x.data_ptr(), H))
    # whole numbers up to 16 * 2 * 3 = 96 are exact in every type
    assert bool((y == ((gate * there).sum(1, keepdim=True) * x.float()).to(dt)).all())
    assert bool((d_x == (there.sum(1, keepdim=True) * x.float()).to(dt)).all())
    d_gate, d_o = torch.empty_like(gate), torch.full_like(xs, -77.0)
    B.check(B.pw_expert_combine_grad(x.data_ptr(), xs.data_ptr(), ty, T, k, H, H, H, pos.data_ptr(), gate.data_ptr(),
                                     d_o.data_ptr(), H, d_gate.data_ptr()))
    # at most 9 * 2^18 < 2^24: exact
    assert bool((d_gate == there * (x.float() ** 2).sum(1, keepdim=True)).all())
    weight = gate.reshape(-1)[src[:live].long()]
    for a in range(0, live, 1 << 22):
        b = min(live, a + (1 << 22))
        assert bool((d_o[a:b] == (weight[a:b, None] * xs[a:b].float()).to(dt)).all())
    assert bool((d_o[live:] == -77.0).all()) and B.pw_get_status() == B.PW_OK

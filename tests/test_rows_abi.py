"""Refusals of the expert-row and scaled-product calls: every bad argument returns before anything
touches a GPU (fake addresses, no device needed)."""
import pytest

from any_precision_expert_pw_b200 import binding as B

BAD, UNSUP = B.PW_ERR_INVALID_ARG, B.PW_ERR_UNSUPPORTED
F32, BF16 = B.PW_TYPE_F32, B.PW_TYPE_BF16
P = 4096  # a fake, well aligned address


def _bad(fn, good, changes):
    names = list(good)
    for ch in changes:
        a = dict(good, **ch)
        assert fn(*[a[n] for n in names]) == BAD, ch


def test_sort_refusals(libpw):
    ws = B.pw_expert_sort_workspace_bytes(8, 2, 4)
    assert ws > 0
    for T, k, E in ((0, 2, 4), (8, 0, 4), (8, 17, 4), (8, 2, 0), (8, 2, 1025), (1 << 24, 2, 4),
                    (-1, 2, 4)):
        assert B.pw_expert_sort_workspace_bytes(T, k, E) == 0
    good = dict(idx=P, T=8, k=2, E=4, pos=P, src=P, offsets=P, workspace=P, ws_bytes=ws)
    _bad(B.pw_expert_sort, good,
         [dict(idx=0), dict(pos=0), dict(src=0), dict(offsets=0), dict(workspace=0), dict(T=0),
          dict(k=17), dict(E=1025), dict(T=1 << 24), dict(ws_bytes=ws - 1), dict(workspace=P + 16),
          dict(idx=P + 2), dict(pos=P + 1)])


@pytest.mark.parametrize("T,k", [(1 << 24, 1), (1 << 20, 16), (600_000, 16), (9_800_000, 1), (70_001, 2)])
def test_sort_runs_fit_their_places(libpw, T, k):
    """Places within the run of a sort's CTA are 16 bits: the count table (one int32 per CTA and
    expert) has enough CTAs that no run is longer than 65535 slots, on any number of SMs."""
    E = 64                                       # 4 E = 256: the table's size has no padding
    ctas = B.pw_expert_sort_workspace_bytes(T, k, E) // (4 * E)
    assert -(-T * k // ctas) <= 65535


def test_row_movement_refusals(libpw):
    good = dict(x=P, type_=BF16, T=8, k=2, H=64, x_stride=64, pos=P, xs=P, xs_stride=64)
    _bad(B.pw_expert_dispatch, good,
         [dict(x=0), dict(xs=0), dict(pos=0), dict(type_=3), dict(type_=-1), dict(T=0), dict(k=0),
          dict(k=17), dict(H=0), dict(x_stride=63), dict(xs_stride=63), dict(x=P + 1),
          dict(xs=P + 1), dict(pos=P + 2), dict(H=1 << 19, x_stride=1 << 19, xs_stride=1 << 19)])
    # a grid beyond 2^31 blocks' worth of warps is outside what is implemented
    assert B.pw_expert_dispatch(P, BF16, 1 << 24, 1, 1 << 18, 1 << 18, P, P, 1 << 18) == UNSUP
    good = dict(d_xs=P, type_=BF16, T=8, k=2, H=64, d_xs_stride=64, pos=P, d_x=P, d_x_stride=64)
    _bad(B.pw_expert_dispatch_grad, good,
         [dict(d_xs=0), dict(d_x=0), dict(pos=0), dict(type_=9), dict(H=0), dict(d_x_stride=1)])
    good = dict(o=P, o_type=F32, T=8, k=2, H=64, o_stride=64, pos=P, gate=P, y=P, y_type=BF16,
                y_stride=64)
    _bad(B.pw_expert_combine, good,
         [dict(o=0), dict(gate=0), dict(y=0), dict(pos=0), dict(o_type=4), dict(y_type=4),
          dict(o=P + 2), dict(gate=P + 2), dict(y_stride=63), dict(o_stride=0)])
    good = dict(d_y=P, o=P, type_=F32, T=8, k=2, H=64, d_y_stride=64, o_stride=64, pos=P, gate=P,
                d_o=P, d_o_stride=64, d_gate=P)
    _bad(B.pw_expert_combine_grad, good,
         [dict(d_y=0), dict(o=0), dict(pos=0), dict(gate=0), dict(d_o=0, d_gate=0), dict(type_=5),
          dict(d_o_stride=63), dict(o_stride=63), dict(d_gate=P + 1)])


def test_quantize_refusals(libpw):
    good = dict(x=P, type_=F32, rows=4, cols=100, x_stride=100, block_rows=1, q=P, q_stride=112,
                scale=P)
    _bad(B.pw_scaled_quantize, good,
         [dict(x=0), dict(q=0), dict(scale=0), dict(type_=3), dict(rows=0), dict(cols=0),
          dict(rows=(1 << 24) + 1), dict(x_stride=99), dict(block_rows=2), dict(block_rows=0),
          dict(q_stride=100), dict(q_stride=96), dict(q=P + 8), dict(scale=P + 2)])


def test_product_refusals(libpw):
    ws = B.pw_scaled_gemm_workspace_bytes(4, 100, 200, 3)
    assert ws > 0
    for a in ((0, 1, 1, 1), (1, 0, 1, 1), (1, 1, 0, 1), (1, 1, 1, 0), (1, 1, 1, 1025),
              (1, (1 << 18) + 1, 1, 1), ((1 << 24) + 1, 1, 1, 1)):
        assert B.pw_scaled_gemm_workspace_bytes(*a) == 0
    good = dict(x_q=P, x_scale=P, M=4, K=200, x_stride=208, w_q=P, w_scale=P, E=3, N=100,
                w_stride=208, offsets=P, y=P, y_type=BF16, y_stride=100, workspace=P, ws_bytes=ws)
    _bad(B.pw_scaled_gemm, good,
         [dict(x_q=0), dict(x_scale=0), dict(w_q=0), dict(w_scale=0), dict(y=0), dict(workspace=0),
          dict(offsets=0), dict(M=0), dict(K=0), dict(N=0), dict(E=0), dict(E=1025),
          dict(x_stride=200), dict(x_stride=192), dict(w_stride=200), dict(w_stride=192),
          dict(x_q=P + 8), dict(w_q=P + 8), dict(y_stride=99), dict(y_type=3), dict(y=P + 1),
          dict(ws_bytes=ws - 1), dict(workspace=P + 128), dict(offsets=P + 2)])


def test_layer_refusals(libpw):
    ws = B.pw_moe_scaled_workspace_bytes(4, 2, 8, 256, 512)
    assert ws > 0 and ws % 256 == 0
    for a in ((0, 2, 8, 256, 512), (4, 2, 8, 200, 512), (4, 2, 8, 256, 500), (4, 17, 8, 256, 512),
              (4, 2, 1025, 256, 512), (4, 2, 0, 256, 512), (1 << 24, 2, 8, 256, 512)):
        assert B.pw_moe_scaled_workspace_bytes(*a) == 0
    ex = B.pw_scaled_experts(E=8, H=256, I=512, gate_up=P, gate_up_scale=P, down=P, down_scale=P)
    good = dict(ex=ex, x=P, x_type=BF16, T=4, k=2, idx=P, gate=P, y=P, y_type=F32, workspace=P,
                ws_bytes=ws)
    changes = [dict(x=0), dict(idx=0), dict(gate=0), dict(y=0), dict(workspace=0), dict(x_type=3),
               dict(y_type=3), dict(T=0), dict(k=0), dict(ws_bytes=ws - 1), dict(workspace=P + 64),
               dict(ex=None)]
    for field, value in (("gate_up", 0), ("down", 0), ("gate_up_scale", 0), ("down_scale", 0),
                         ("H", 200), ("I", 100), ("E", 0), ("gate_up", P + 8), ("down", P + 8)):
        e = B.pw_scaled_experts.from_buffer_copy(ex)
        setattr(e, field, value)
        changes.append(dict(ex=e))
    _bad(B.pw_moe_scaled_forward, good, changes)


@pytest.mark.parametrize("T,k,E,H,I", [(1, 2, 8, 4096, 14336), (64, 8, 64, 3584, 2560), (4096, 8, 64, 3584, 2560)])
def test_layer_workspace_holds_what_is_used(libpw, T, k, E, H, I):
    """Positions, quantised rows and hidden rows with their scales, fp32 expert outputs, one set of
    partials (up to 160 CTAs x 256 columns x 128 rows), counters and the sort's table: nothing twice."""
    n = T * k
    partials = 4 * 160 * 256 * min(128, -(-n // 32) * 32)
    rows = n * (H + H // 32 + I + I // 32 + 4 * H)
    small = 4 * n + 4 * (E + 1) + 8 * 160 + B.pw_expert_sort_workspace_bytes(T, k, E)
    assert B.pw_moe_scaled_workspace_bytes(T, k, E, H, I) <= rows + partials + small + 12 * 256


def test_experts_object_refuses_other_tensors():
    torch = pytest.importorskip("torch")
    from any_precision_expert_pw_b200.scaled_layer import ScaledExperts, type_of
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)  # noqa: E731
    f = lambda *s: torch.zeros(*s)                       # noqa: E731
    with pytest.raises(ValueError):                      # down does not match gate_up
        ScaledExperts(u8(2, 512, 128), f(2, 4, 1), u8(2, 128, 128), f(2, 1, 1), 4, 2)
    with pytest.raises(ValueError):                      # scales of another shape
        ScaledExperts(u8(2, 512, 128), f(2, 4, 2), u8(2, 128, 256), f(2, 1, 2), 4, 2)
    with pytest.raises(ValueError):                      # not on a GPU
        ScaledExperts(u8(2, 512, 128), f(2, 4, 1), u8(2, 128, 256), f(2, 1, 2), 4, 2)
    with pytest.raises(TypeError):
        type_of(torch.zeros(1, dtype=torch.float64))

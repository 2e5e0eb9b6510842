"""Cases of the expert-row and scaled-product operators, and their plain forms.

Five kinds of case, each one pass through operators as a program calls them:

* ``sort``     the routed assignments of a batch sorted by expert and the tokens' rows copied into
               that order (what stands between the router and the experts' products);
* ``combine``  the experts' rows brought back to their tokens, weighted by the gates and summed;
* ``grad``     the gradients of both row movements: of the combine with respect to the rows and
               the gates, and of the sorted copy with respect to the tokens;
* ``product``  y = x W^T with both operands in 8-bit floating point (e4m3): x quantised within the
               call, one scale per row and 128 columns, the weights held with one scale per
               128 x 128 block; one matrix, or one per expert over sorted rows;
* ``layer``    the whole expert feed-forward on such weights: sort, quantise, gate_up product with
               SiLU(gate) * up, quantise, down product, weighted combine.

With ``own`` false, ``run`` computes the plain form in 32 bits with elementary torch operations;
with ``own`` true it calls libpw.
"""
import math

import torch

own = False

BLOCK = 128
E4M3_MAX = 448.0
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
DEV = "cuda"


# ------------------------------------------------------------------------------------- cases
def listed():
    return [
        # a decode step of a layer with many small experts
        dict(name="sort_decode", kind="sort", T=16, H=2048, E=512, k=10, pad=0, type="bf16"),
        # a prompt; the last tokens of the batch are padding and have no expert
        dict(name="sort_prompt", kind="sort", T=16384, H=3584, E=64, k=8, pad=389, type="bf16"),
        # a decode step on the way back, and a prompt whose rows are kept in 32 bits
        dict(name="combine_decode", kind="combine", T=8, H=3584, E=64, k=8, pad=0, type="bf16"),
        dict(name="combine_prompt", kind="combine", T=8192, H=2048, E=60, k=4, pad=101, type="f32"),
        # training: a micro-batch, and a short one with odd sizes
        dict(name="grad_batch", kind="grad", T=4096, H=3584, E=64, k=8, pad=64, type="bf16"),
        dict(name="grad_odd", kind="grad", T=509, H=1001, E=7, k=3, pad=5, type="f32"),
        # one projection of a decode step of four tokens: bound by the weights' bytes
        dict(name="product_decode", kind="product", T=4, N=28672, K=4096, E=1, type="bf16", out="bf16"),
        # one projection of a prompt: bound by the tensor cores
        dict(name="product_prompt", kind="product", T=4096, N=5120, K=3584, E=1, type="bf16", out="f32"),
        # ragged groups, several experts with few rows or none, sizes that end inside a block
        dict(name="product_ragged", kind="product", T=3001, N=2808, K=2040, E=60, type="f16", out="bf16"),
        # the whole expert layer: one token, a decode batch, a prompt
        dict(name="layer_one", kind="layer", T=1, H=4096, I=14336, E=8, k=2, pad=0, type="bf16", out="bf16"),
        dict(name="layer_decode", kind="layer", T=64, H=3584, I=2560, E=64, k=8, pad=0, type="bf16", out="bf16"),
        dict(name="layer_prompt", kind="layer", T=4096, H=3584, I=2560, E=64, k=8, pad=100, type="bf16", out="bf16"),
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["sort", "combine", "grad", "product", "layer"])
    like = [work(c) for c in listed() if c["kind"] == kind]
    most = {n: max(w[n] for w in like) for n in ("bytes", "flops")}
    while True:
        T = _logint(rng, 1, 16384)
        E = _logint(rng, 1, 512)
        if kind == "product":
            c = dict(kind=kind, T=T, N=_logint(rng, 1, 28672), K=_logint(rng, 1, 8192),
                     E=1 if rng.random() < 0.5 else E, type=rng.choice(list(TYPES)),
                     out=rng.choice(list(TYPES)))
            large = c["E"] * c["N"] * c["K"]
        elif kind == "layer":
            k = rng.randint(1, min(10, E))
            c = dict(kind=kind, T=T, H=BLOCK * rng.randint(1, 32), I=BLOCK * _logint(rng, 1, 112),
                     E=E, k=k, pad=rng.choice([0, T // 7]), type="bf16", out="bf16")
            large = max(3 * E * c["H"] * c["I"], E * T * max(2 * c["I"], c["H"]) // 2)
        else:
            k = rng.randint(1, min(16, E))
            c = dict(kind=kind, T=T, H=_logint(rng, 1, 8192), E=E, k=k,
                     pad=rng.choice([0, T // 5]), type=rng.choice(list(TYPES)))
            large = 0
        w = work(c)
        if large <= 1_800_000_000 and all(w[n] <= most[n] for n in most):
            return c


def work(case):
    """Bytes each input and output moves once, and the products' operations.  Weights count for
    the experts that can have a row (at most one per assignment)."""
    T, E = case["T"], case["E"]
    size = 4 if case["type"] == "f32" else 2
    if case["kind"] == "product":
        N, K = case["N"], case["K"]
        out = 4 if case["out"] == "f32" else 2
        used = min(E, T)
        blocks = math.ceil(N / BLOCK) * math.ceil(K / BLOCK)
        return {"bytes": T * K * size + used * (N * K + 4 * blocks) + T * N * out,
                "flops": 2.0 * T * N * K}
    H, k = case["H"], case["k"]
    real = T - case["pad"]
    rows = real * k
    if case["kind"] == "sort":
        return {"bytes": 4 * T * k * 3 + 4 * E + real * H * size + rows * H * size, "flops": 0.0}
    if case["kind"] == "combine":
        return {"bytes": 8 * T * k + rows * H * size + T * H * size, "flops": 2.0 * rows * H}
    if case["kind"] == "grad":
        # dy, rows and their gradient, the gradient of the sorted copy in, dx and dgate out
        return {"bytes": 12 * T * k + (2 * T + 3 * rows) * H * size, "flops": 4.0 * rows * H}
    I = case["I"]
    used = min(E, rows)
    return {"bytes": T * H * (size + (4 if case["out"] == "f32" else 2)) + 8 * T * k +
            used * 3 * I * H * (1 + 4 / BLOCK ** 2), "flops": 6.0 * rows * H * I}


# ------------------------------------------------------------------------------------ inputs
def _routing(T, E, k, pad, gen):
    """Assignments with a skewed load, as a trained router gives them; the last `pad` tokens have
    none (-1).  Gates are the renormalised softmax of the selected logits."""
    skew = -0.3 * torch.log(1.0 + torch.randperm(E, generator=gen, device=DEV))
    logits = torch.randn(T, E, generator=gen, device=DEV) + skew
    top, idx = torch.topk(logits, k, dim=1)
    gate = torch.softmax(top, dim=1)
    idx = idx.to(torch.int32)
    if pad:
        idx[T - pad:] = -1
    return idx.contiguous(), gate.contiguous()


def _activations(rows, cols, type_, gen):
    """Normal values, tokens of differing size and a few channels far larger than the others."""
    x = torch.randn(rows, cols, generator=gen, device=DEV)
    x *= torch.exp(0.5 * torch.randn(rows, 1, generator=gen, device=DEV))
    x *= 1.0 + 15.0 * (torch.rand(1, cols, generator=gen, device=DEV) < 0.003)
    return x.to(TYPES[type_])


def _blocks(n):
    return -(-n // BLOCK)


def _weights(E, N, K, gen):
    """e4m3 weights [E][N][ld] (ld = K rounded up to 16) and their fp32 scales
    [E][N/128][K/128]: normal weights divided by each block's own scale, so that the block's
    largest magnitude is the format's."""
    ld = -(-K // 16) * 16
    q = torch.zeros(E, N, ld, dtype=torch.uint8, device=DEV)
    scale = torch.empty(E, _blocks(N), _blocks(K), dtype=torch.float32, device=DEV)
    step = max(1, min(E, 268_435_456 // (N * K)))
    for e in range(0, E, step):
        n = min(step, E - e)
        w = torch.randn(n, _blocks(N) * BLOCK, _blocks(K) * BLOCK, generator=gen, device=DEV) * 0.02
        w[:, N:] = 0
        w[:, :, K:] = 0
        b = w.view(n, _blocks(N), BLOCK, _blocks(K), BLOCK)
        s = b.abs().amax(dim=(2, 4)) / E4M3_MAX
        scale[e:e + n] = s
        b /= s[:, :, None, :, None]
        q[e:e + n, :, :K] = w[:, :N, :K].to(torch.float8_e4m3fn).view(torch.uint8)
        del w, b
    return q, scale


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    kind, T, E = case["kind"], case["T"], case["E"]
    st = dict(case=case, stream=torch.cuda.current_stream().cuda_stream)
    if kind == "product":
        N, K = case["N"], case["K"]
        st["x"] = _activations(T, K, case["type"], gen)
        st["w"], st["ws"] = _weights(E, N, K, gen)
        load = torch.rand(E, generator=gen, device=DEV) ** 2
        if E > 3:
            load[1] = 0.0  # an expert without rows
        edge = torch.cumsum(load, 0) / load.sum().clamp(min=1e-6)
        cut = torch.round(edge * T).to(torch.int32)
        cut[-1] = T
        st["offsets"] = torch.cat([torch.zeros(1, dtype=torch.int32, device=DEV), cut])
        st["most"] = int((st["offsets"][1:] - st["offsets"][:-1]).max())
        st["y"] = torch.zeros(T, N, dtype=TYPES[case["out"]], device=DEV)
        ld = st["w"].shape[2]
        st["xq"] = torch.zeros(T, ld, dtype=torch.uint8, device=DEV)
        st["xs"] = torch.zeros(T, _blocks(K), dtype=torch.float32, device=DEV)
        if own:
            from any_precision_expert_pw_b200 import binding as B
            st["tmp"] = torch.empty(B.pw_scaled_gemm_workspace_bytes(T, N, K, E),
                                    dtype=torch.uint8, device=DEV)
        return st
    H, k, type_ = case["H"], case["k"], TYPES[case["type"]]
    st["idx"], st["gate"] = _routing(T, E, k, case["pad"], gen)
    if kind == "layer":
        I = case["I"]
        st["x"] = _activations(T, H, case["type"], gen)
        st["w1"], st["s1"] = _weights(E, 2 * I, H, gen)
        st["w2"], st["s2"] = _weights(E, H, I, gen)
        count = torch.bincount(st["idx"].reshape(-1).long() + 1, minlength=E + 1)[1:]
        st["most"] = max(1, int(count.max()))
        st["y"] = torch.zeros(T, H, dtype=TYPES[case["out"]], device=DEV)
        if own:
            from any_precision_expert_pw_b200.scaled_layer import ScaledExperts
            st["experts"] = ScaledExperts(st["w1"], st["s1"], st["w2"], st["s2"], max_tokens=T, k=k)
        return st
    rows = T * k
    pos, src, offsets, _ = _sorted(st["idx"], E)
    if kind == "sort":
        st["x"] = _activations(T, H, case["type"], gen)
        st["out"] = dict(pos=torch.full((T, k), -1, dtype=torch.int32, device=DEV),
                         src=torch.full((rows,), -1, dtype=torch.int32, device=DEV),
                         offsets=torch.zeros(E + 1, dtype=torch.int32, device=DEV),
                         rows=torch.zeros(rows, H, dtype=type_, device=DEV))
        if own:
            from any_precision_expert_pw_b200 import binding as B
            st["tmp"] = torch.empty(B.pw_expert_sort_workspace_bytes(T, k, E), dtype=torch.uint8, device=DEV)
        return st
    st["pos"] = pos
    st["o"] = torch.randn(rows, H, generator=gen, device=DEV).to(type_)
    if kind == "combine":
        st["y"] = torch.zeros(T, H, dtype=type_, device=DEV)
        return st
    st["dy"] = torch.randn(T, H, generator=gen, device=DEV).to(type_)
    st["drows"] = torch.randn(rows, H, generator=gen, device=DEV).to(type_)
    st["out"] = dict(d_o=torch.zeros(rows, H, dtype=type_, device=DEV),
                     d_gate=torch.zeros(T, k, dtype=torch.float32, device=DEV),
                     d_x=torch.zeros(T, H, dtype=type_, device=DEV))
    return st


# ------------------------------------------------------------------------------- plain forms
def _sorted(idx, E):
    """pos [T][k] (row of each slot, -1 for an empty one), src (slot behind each row, -1 behind
    the last), offsets [E+1], and the rows that hold something."""
    T, k = idx.shape
    key = torch.where(idx >= 0, idx, E).reshape(-1).long()
    count = (torch.zeros(E + 1, dtype=torch.int64, device=idx.device)
             .scatter_add_(0, key, torch.ones_like(key)))[:E]
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=idx.device)
    offsets[1:] = torch.cumsum(count, 0)
    order = torch.sort(key, stable=True).indices
    row = torch.arange(T * k, device=idx.device)
    live = row < offsets[E]
    src = torch.where(live, order, -1).to(torch.int32)
    pos = torch.empty_like(row)
    pos[order] = torch.where(live, row, -1)
    return pos.to(torch.int32).view(T, k), src, offsets, live


def _quantised(x):
    """The values that x stands for after quantising: e4m3 with one power-of-two scale for each
    row and 128 columns, the smallest whose 448 covers the block."""
    rows, cols = x.shape
    v = torch.zeros(rows, _blocks(cols) * BLOCK, dtype=torch.float32, device=x.device)
    v[:, :cols] = x
    v = v.view(rows, _blocks(cols), BLOCK)
    m, e = torch.frexp(v.abs().amax(dim=2, keepdim=True))
    s = torch.ldexp(torch.ones_like(m), torch.clamp(torch.where(m <= 0.875, e - 9, e - 8), min=-126))
    s = torch.where(m == 0, torch.ones_like(s), s)
    return ((v / s).to(torch.float8_e4m3fn).float() * s).view(rows, -1)[:, :cols]


def _values(q, scale, K, type_=torch.float32):
    """The weights that [..][N][ld] e4m3 bytes and their block scales stand for."""
    N = q.shape[-2]
    s = scale.to(type_).repeat_interleave(BLOCK, dim=-1).repeat_interleave(BLOCK, dim=-2)
    return q[..., :K].view(torch.float8_e4m3fn).to(type_) * s[..., :N, :K]


def _by_expert(x, offsets, most):
    """Sorted rows as one padded block per expert, and where each row went."""
    E = offsets.shape[0] - 1
    row = torch.arange(x.shape[0], device=x.device)
    e = torch.searchsorted(offsets[1:].contiguous().long(), row, right=True).clamp(max=E - 1)
    at = e * most + (row - offsets[e].long()).clamp(max=most - 1)
    return e, at


def _grouped(x, w, offsets, most):
    E = offsets.shape[0] - 1
    if E == 1:
        return x @ w[0].t()
    _, at = _by_expert(x, offsets, most)
    live = torch.arange(x.shape[0], device=x.device) < offsets[-1]
    padded = torch.zeros(E * most, x.shape[1], dtype=x.dtype, device=x.device)
    padded[at[live]] = x[live]
    y = torch.bmm(padded.view(E, most, -1), w.transpose(1, 2)).view(E * most, -1)
    return torch.where(live[:, None], y[at], torch.zeros((), dtype=y.dtype, device=y.device))


def _silu(z):
    return z / (1.0 + torch.exp(-z))


def _plain(st):
    case = st["case"]
    kind = case["kind"]
    if kind == "sort":
        pos, src, offsets, live = _sorted(st["idx"], case["E"])
        rows = st["x"][(src.long().clamp(min=0)) // case["k"]]
        return dict(pos=pos, src=src, offsets=offsets,
                    rows=torch.where(live[:, None], rows, torch.zeros_like(rows[:1])))
    if kind in ("combine", "grad"):
        pos = st["pos"].long()
        there = (pos >= 0)[:, :, None]
        zero = torch.zeros((), device=pos.device)
        o = torch.where(there, st["o"][pos.clamp(min=0)].float(), zero)
        if kind == "combine":
            return (o * st["gate"][:, :, None]).sum(1).to(st["y"].dtype)
        dy = st["dy"].float()
        d_o = torch.zeros(st["o"].shape, dtype=torch.float32, device=pos.device)
        live = pos.reshape(-1) >= 0
        d_o[pos.reshape(-1)[live]] = (st["gate"][:, :, None] * dy[:, None, :]).reshape(-1, dy.shape[1])[live]
        d_x = torch.where(there, st["drows"][pos.clamp(min=0)].float(), zero).sum(1)
        return dict(d_o=d_o.to(st["o"].dtype), d_gate=(o * dy[:, None, :]).sum(2), d_x=d_x.to(st["dy"].dtype))
    if kind == "product":
        x = _quantised(st["x"].float())
        return _grouped(x, _values(st["w"], st["ws"], case["K"]), st["offsets"], st["most"]).to(st["y"].dtype)
    x, idx, E = st["x"].float(), st["idx"], case["E"]
    T, k = idx.shape
    H, I = case["H"], case["I"]
    x = _quantised(x)
    if T * k <= E:  # few assignments: the weights of each one's expert
        e = idx.reshape(-1).long()
        rows = x[torch.arange(T * k, device=x.device) // k]
        live = e >= 0
        e = e.clamp(min=0)
        gu = torch.bmm(_values(st["w1"][e], st["s1"][e], H), rows[:, :, None])[:, :, 0]
        h = _quantised(_silu(gu[:, :I]) * gu[:, I:])
        o = torch.bmm(_values(st["w2"][e], st["s2"][e], I), h[:, :, None])[:, :, 0]
        o = torch.where(live[:, None], o, torch.zeros((), device=x.device)).view(T, k, H)
        return (o * st["gate"][:, :, None]).sum(1).to(st["y"].dtype)
    pos, src, offsets, live = _sorted(idx, E)
    rows = x[src.long().clamp(min=0) // k]
    gu = _grouped(rows, _values(st["w1"], st["s1"], H), offsets, st["most"])
    h = _quantised(_silu(gu[:, :I]) * gu[:, I:])
    o = _grouped(h, _values(st["w2"], st["s2"], I), offsets, st["most"])
    there = (pos >= 0)[:, :, None]
    o = torch.where(there, o[pos.long().clamp(min=0)], torch.zeros((), device=x.device))
    return (o * st["gate"][:, :, None]).sum(1).to(st["y"].dtype)


# ------------------------------------------------------------------------ the framework's calls
def _calls(st):
    from any_precision_expert_pw_b200 import binding as B
    case = st["case"]
    kind, T, E, s = case["kind"], case["T"], case["E"], st["stream"]
    kinds = {"f32": B.PW_TYPE_F32, "bf16": B.PW_TYPE_BF16, "f16": B.PW_TYPE_F16}
    t = kinds[case["type"]]
    if kind == "layer":
        st["experts"].forward(st["x"], st["idx"], st["gate"], st["y"], stream=s)
        return st["y"]
    if kind == "product":
        N, K, ld = case["N"], case["K"], st["w"].shape[2]
        B.check(B.pw_scaled_quantize(st["x"].data_ptr(), t, T, K, K, 1, st["xq"].data_ptr(), ld,
                                     st["xs"].data_ptr(), s))
        B.check(B.pw_scaled_gemm(st["xq"].data_ptr(), st["xs"].data_ptr(), T, K, ld,
                                 st["w"].data_ptr(), st["ws"].data_ptr(), E, N, ld,
                                 st["offsets"].data_ptr(), st["y"].data_ptr(), kinds[case["out"]], N,
                                 st["tmp"].data_ptr(), st["tmp"].numel(), s))
        return st["y"]
    H, k = case["H"], case["k"]
    if kind == "sort":
        out = st["out"]
        B.check(B.pw_expert_sort(st["idx"].data_ptr(), T, k, E, out["pos"].data_ptr(),
                                 out["src"].data_ptr(), out["offsets"].data_ptr(),
                                 st["tmp"].data_ptr(), st["tmp"].numel(), s))
        B.check(B.pw_expert_dispatch(st["x"].data_ptr(), t, T, k, H, H, out["pos"].data_ptr(),
                                     out["rows"].data_ptr(), H, s))
        return out
    if kind == "combine":
        B.check(B.pw_expert_combine(st["o"].data_ptr(), t, T, k, H, H, st["pos"].data_ptr(),
                                    st["gate"].data_ptr(), st["y"].data_ptr(), t, H, s))
        return st["y"]
    out = st["out"]
    B.check(B.pw_expert_combine_grad(st["dy"].data_ptr(), st["o"].data_ptr(), t, T, k, H, H, H,
                                     st["pos"].data_ptr(), st["gate"].data_ptr(),
                                     out["d_o"].data_ptr(), H, out["d_gate"].data_ptr(), s))
    B.check(B.pw_expert_dispatch_grad(st["drows"].data_ptr(), t, T, k, H, H, st["pos"].data_ptr(),
                                      out["d_x"].data_ptr(), H, s))
    return out


def run(st):
    return _calls(st) if own else _plain(st)


# ---------------------------------------------------------------- the definition, in 64 bits
def _round_e4m3(v):
    """The nearest e4m3 value (ties to even) of |v| <= 448, in 64 bits: steps of 2^-9 below 2^-6,
    of an eighth of the power of two above."""
    _, e = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), torch.clamp(e - 4, min=-9))
    return torch.round(v / step) * step


def _exact_quantised(x):
    out = torch.empty_like(x)
    for c in range(0, x.shape[1], BLOCK):
        v = x[:, c:c + BLOCK]
        top = v.abs().amax(dim=1, keepdim=True)
        e = torch.ceil(torch.log2(top / E4M3_MAX))
        e = torch.where(top / E4M3_MAX > torch.exp2(e), e + 1, e)      # where log2 was rounded
        e = torch.where(top / E4M3_MAX <= torch.exp2(e - 1), e - 1, e)
        s = torch.where(top > 0, torch.exp2(torch.clamp(e, min=-126.0)), torch.ones_like(top))
        out[:, c:c + BLOCK] = _round_e4m3(v / s) * s
    return out


def exact(case, seed):
    st = prepare(case, seed)
    kind, T, E = case["kind"], case["T"], case["E"]
    if kind == "product":
        x, y = _exact_quantised(st["x"].double()), torch.zeros(T, case["N"], dtype=torch.float64, device=DEV)
        edge = st["offsets"].tolist()
        for e in range(E):
            a, b = edge[e], edge[e + 1]
            if a < b:
                y[a:b] = x[a:b] @ _values(st["w"][e], st["ws"][e], case["K"], torch.float64).t()
        return y
    H, k, idx, gate = case["H"], case["k"], st["idx"].long(), st["gate"].double()
    if kind == "sort":
        flat = idx.reshape(-1)
        rows = torch.zeros(T * k, H, dtype=torch.float64, device=DEV)
        at = 0
        for e in range(E):
            slots = torch.nonzero(flat == e)[:, 0]
            rows[at:at + len(slots)] = st["x"][slots // k].double()
            at += len(slots)
        return dict(pos=None, src=None, offsets=None, rows=rows)
    if kind == "layer":
        I = case["I"]
        x, y = _exact_quantised(st["x"].double()), torch.zeros(T, H, dtype=torch.float64, device=DEV)
        for e in range(E):
            hit = torch.nonzero(idx == e)
            if not len(hit):
                continue
            t = hit[:, 0]
            gu = x[t] @ _values(st["w1"][e], st["s1"][e], H, torch.float64).t()
            g, u = gu[:, :I], gu[:, I:]
            h = _exact_quantised(g * torch.sigmoid(g) * u)
            o = h @ _values(st["w2"][e], st["s2"][e], I, torch.float64).t()
            y.index_add_(0, t, gate[t, hit[:, 1]][:, None] * o)
        return y
    pos = st["pos"].long()
    if kind == "combine":
        y = torch.zeros(T, H, dtype=torch.float64, device=DEV)
        for j in range(k):
            t = torch.nonzero(pos[:, j] >= 0)[:, 0]
            y[t] += gate[t, j, None] * st["o"][pos[t, j]].double()
        return y
    dy = st["dy"].double()
    d_o = torch.zeros(T * k, H, dtype=torch.float64, device=DEV)
    d_gate = torch.zeros(T, k, dtype=torch.float64, device=DEV)
    d_x = torch.zeros(T, H, dtype=torch.float64, device=DEV)
    for j in range(k):
        t = torch.nonzero(pos[:, j] >= 0)[:, 0]
        r = pos[t, j]
        d_o[r] = gate[t, j, None] * dy[t]
        d_gate[t, j] = (st["o"][r].double() * dy[t]).sum(1)
        d_x[t] += st["drows"][r].double()
    return dict(d_o=d_o, d_gate=d_gate, d_x=d_x)

"""Expert FFN on e4m3 weights (libpw's pw_moe_scaled_forward) with torch tensors as the buffers.

Beside ``device_layer.DeviceLayer`` (any-precision experts): the same layer on experts held in 8-bit
floating point with one scale per 128 x 128 block, for batches of up to 2^24 assignments.  PyTorch allocates
device memory and names the stream; quantisation, sorting, both products and the combine run in
libpw's kernels.  Routing comes from ``pw_route_topk`` and the rewrites (``DeviceLayer.route``).
"""
from __future__ import annotations

from . import binding as B


def _torch():
    import torch
    return torch


def type_of(t) -> int:
    """PW_TYPE_* of a tensor."""
    torch = _torch()
    kinds = {torch.float32: B.PW_TYPE_F32, torch.bfloat16: B.PW_TYPE_BF16,
             torch.float16: B.PW_TYPE_F16}
    if t.dtype not in kinds:
        raise TypeError(f"float32, bfloat16 or float16 expected, got {t.dtype}")
    return kinds[t.dtype]


def quantize_weights(w):
    """[E][N][K] (or [N][K]) float weights -> e4m3 bytes [E][N][K up to 16] and their scales
    [E][N/128 up][K/128 up] (pw_scaled_quantize, blocks of 128 x 128), on the current stream."""
    torch = _torch()
    lead = w.shape[:-2]
    w3 = w.reshape(-1, *w.shape[-2:]).contiguous()
    E, N, K = w3.shape
    ld = -(-K // 16) * 16
    with torch.cuda.device(w.device):
        s = torch.cuda.current_stream().cuda_stream
        q = torch.zeros(E, N, ld, dtype=torch.uint8, device=w.device)
        scale = torch.empty(E, -(-N // 128), -(-K // 128), dtype=torch.float32, device=w.device)
        for e in range(E):
            B.check(B.pw_scaled_quantize(w3[e].data_ptr(), type_of(w3), N, K, K, 128,
                                         q[e].data_ptr(), ld, scale[e].data_ptr(), s),
                    "pw_scaled_quantize")
    return q.view(*lead, N, ld), scale.view(*lead, *scale.shape[1:])


class ScaledExperts:
    """The experts of one layer and the workspace of their forward.

    gate_up uint8 [E][2I][H] and down uint8 [E][H][I] e4m3 bytes, their fp32 scales
    [E][2I/128][H/128] and [E][H/128][I/128] (quantize_weights gives both), kept by reference.
    max_tokens x k assignments at most in one call.  Calls on different streams that may overlap
    need an object each (they would share the workspace); a stream other than the one current at
    construction has to be ordered behind it.  Streams given to forward have to exist as long as
    this object, and the object as long as a graph that captured its calls."""

    def __init__(self, gate_up, gate_up_scale, down, down_scale, max_tokens: int, k: int):
        torch = _torch()
        E, I2, H = gate_up.shape
        I = I2 // 2
        if tuple(down.shape) != (E, H, I) or I2 % 2:
            raise ValueError(f"gate_up {tuple(gate_up.shape)} and down {tuple(down.shape)}: "
                             "[E][2I][H] and [E][H][I] expected")
        for t, shape in ((gate_up_scale, (E, I2 // 128, H // 128)),
                         (down_scale, (E, H // 128, I // 128))):
            if tuple(t.shape) != shape or t.dtype != torch.float32:
                raise ValueError(f"scales {tuple(t.shape)} {t.dtype}: float32 {shape} expected")
        for t in (gate_up, down, gate_up_scale, down_scale):
            if not t.is_cuda or t.device != gate_up.device or not t.is_contiguous():
                raise ValueError("contiguous tensors on one CUDA device expected")
        if gate_up.dtype != torch.uint8 or down.dtype != torch.uint8:
            raise TypeError("e4m3 bytes (uint8) expected")
        self.device = gate_up.device
        self.E, self.H, self.I, self.k, self.max_tokens = E, H, I, k, max_tokens
        self._keep = (gate_up, gate_up_scale, down, down_scale)
        self.ws_bytes = B.pw_moe_scaled_workspace_bytes(max_tokens, k, E, H, I)
        if not self.ws_bytes:
            raise B.PwError(B.PW_ERR_INVALID_ARG, "pw_moe_scaled_workspace_bytes")
        self.workspace = torch.empty(self.ws_bytes, dtype=torch.uint8, device=self.device)
        self._streams = set()  # streams that the workspace and the weights are recorded on
        self._ws_ptr = self.workspace.data_ptr()
        self.experts = B.pw_scaled_experts(E=E, H=H, I=I, gate_up=gate_up.data_ptr(),
                                           gate_up_scale=gate_up_scale.data_ptr(),
                                           down=down.data_ptr(), down_scale=down_scale.data_ptr())

    def forward(self, x, idx, gate, y=None, stream=None):
        """y[t] = sum over s of gate[t][s] * FFN(expert idx[t][s], x[t]); idx -1 = empty slot.
        x, y [T][H] float32, bfloat16 or float16, idx int32 [T][k], gate float32 [T][k], T >= 1.
        stream: handle of the stream to run on (the current one if None).  It has to be ordered behind
        what made the tensors.  The experts and the workspace may be dropped while it still runs, and a
        y that is made here is safe on both streams; given tensors stay with the caller, who keeps them
        or records the stream on them (Tensor.record_stream) if they are another stream's."""
        torch = _torch()
        if torch.cuda.current_device() != self.device.index:
            with torch.cuda.device(self.device):
                return self.forward(x, idx, gate, y, stream)
        if stream is None:
            stream = torch.cuda.current_stream().cuda_stream
            if y is None:
                y = torch.empty_like(x)
        elif y is None:  # of the stream that writes it, known to the one that will read it
            with torch.cuda.stream(torch.cuda.ExternalStream(stream, self.device)):
                y = torch.empty_like(x)
            y.record_stream(torch.cuda.current_stream())
        T = x.shape[0]
        if x.shape != (T, self.H) or y.shape != (T, self.H):
            raise ValueError(f"x {tuple(x.shape)}, y {tuple(y.shape)}: [T][{self.H}] expected")
        if idx.shape != (T, self.k) or gate.shape != (T, self.k) or T > self.max_tokens:
            raise ValueError(f"idx {tuple(idx.shape)}, gate {tuple(gate.shape)}: [T][{self.k}] with "
                             f"T <= {self.max_tokens} expected")
        if idx.dtype != torch.int32 or gate.dtype != torch.float32:
            raise TypeError("idx int32 and gate float32 expected")
        for t in (x, idx, gate, y):
            if t.device != self.device or not t.is_contiguous():
                raise ValueError("contiguous tensors on the experts' device expected")
        if stream not in self._streams:  # the allocator keeps this memory until that stream is done with it
            on = torch.cuda.ExternalStream(stream, self.device)
            for t in (self.workspace, *self._keep):
                t.record_stream(on)
            self._streams.add(stream)
        B.check(B.pw_moe_scaled_forward(self.experts, x.data_ptr(), type_of(x), T, self.k,
                                        idx.data_ptr(), gate.data_ptr(), y.data_ptr(), type_of(y),
                                        self._ws_ptr, self.ws_bytes, stream), "pw_moe_scaled_forward")
        return y

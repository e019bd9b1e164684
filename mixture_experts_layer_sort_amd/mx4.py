"""The layer's forward with experts in microscaled 4-bit floating point.

  MoEMx4Tensor        a tensor in 4 bits: weights [count, K, cols] or rows [N, K],
                      in blocks of 32 along K (moe_mx4_quantize, moe_mx4_dequantize)
  MoEMx4DecodeRunner  the layer for the few tokens of a decoding step
                      (moe_mx4_decode): only the weights are in 4 bits
  MoEMx4Runner        the layer for many tokens (a prompt): the rows of both
                      products are quantised too, which lets them run on the 4-bit
                      matrix instruction (moe_mx4_gate_up, moe_mx4_down)

A trained layer's weights are quantised once and serve both:

    w = [MoEMx4Tensor.weights(t) for t in (w_gate, w_up, w_down)]
    y = MoEMx4Runner(N, H, F, E, K, dtype).forward(x, w_r, *w)   # shared=: a shared expert's, in both
    y = MoEMx4DecodeRunner(16, H, F, E, K, dtype).forward(x, w_r, *w)
"""
from __future__ import annotations

from typing import Optional

import torch

from . import _lib as L
from .layer import _Made, _cuda_device, _expect, _on, _stream_of


class MoEMx4Tensor:
    """Codes and scales of a tensor in 4 bits, in device memory of its own.
    ``shape`` is that of the values it stands for; ``order`` a moe_mx4_order.
    As with any tensor, a call on another stream than the one that filled it comes
    behind that one in the caller's order, and record_stream() keeps its memory
    from new tensors until such a call has ended."""

    def __init__(self, order: int, shape, device="cuda"):
        """Room for weights of shape [count, K, cols] or rows [N, K]; fill it
        with quantize()."""
        shape = tuple(int(n) for n in shape)
        if len(shape) != (3 if order == L.MOE_MX4_WEIGHTS else 2):
            raise ValueError("weights have the shape [count, K, cols], rows [N, K]")
        self.order, self.shape = order, shape
        self._sizes = (shape[0], shape[1], shape[2] if len(shape) == 3 else 1)
        need = L.moe_mx4_code_bytes(order, *self._sizes), L.moe_mx4_scale_bytes(order, *self._sizes)
        if 2 ** 64 - 1 in need:
            raise ValueError(f"no 4-bit form for {shape}: K and cols have to be multiples of 128, at most 2^20")
        self.device = dev = _cuda_device(device)
        self.codes = torch.empty((max(16, need[0]),), dtype=torch.uint8, device=dev)
        self.scales = torch.empty((max(16, need[1]),), dtype=torch.uint8, device=dev)
        self.mx4 = L.mx4(self.codes, self.scales)
        self._made = _Made(dev)

    @classmethod
    def weights(cls, w, stream=None) -> "MoEMx4Tensor":
        """Quantised weights w [count, K, cols] or [K, cols] (one matrix), float32
        or bfloat16."""
        w = w[None] if w.dim() == 2 else w
        with _stream_of(w.device, stream):
            q = cls(L.MOE_MX4_WEIGHTS, w.shape, w.device)
        return q.quantize(w, stream)

    @classmethod
    def rows(cls, x, stream=None) -> "MoEMx4Tensor":
        """Quantised token rows x [N, K]."""
        with _stream_of(x.device, stream):
            q = cls(L.MOE_MX4_ROWS, x.shape, x.device)
        return q.quantize(x, stream)

    def record_stream(self, stream):
        """As torch.Tensor.record_stream."""
        self.codes.record_stream(stream)
        self.scales.record_stream(stream)

    def quantize(self, v, stream=None) -> "MoEMx4Tensor":
        """Take over the values of v; returns self."""
        _expect("v", v, self.shape, v.dtype, self.device)
        code = L.dtype_code(v.dtype)
        if self.shape[0]:
            with _on(self.device):
                L.moe_mx4_quantize(self.order, *self._sizes, code, v, self.mx4, self._made.before(self.device, stream))
        return self

    def dequantize(self, dtype: Optional[torch.dtype] = None, out=None, stream=None):
        """The values, as a new tensor (bfloat16 by default) or in ``out``."""
        if out is None:
            with _stream_of(self.device, stream):
                out = torch.empty(self.shape, dtype=torch.bfloat16 if dtype is None else dtype, device=self.device)
        _expect("out", out, self.shape, out.dtype if dtype is None else dtype, self.device)
        code = L.dtype_code(out.dtype)
        if self.shape[0]:
            with _on(self.device):
                L.moe_mx4_dequantize(self.order, *self._sizes, code, self.mx4, out, stream)
        return out


def _expect_mx4(name: str, q, order: int, shape, dev):
    if not isinstance(q, MoEMx4Tensor) or q.order != order or q.shape != shape or q.device != dev:
        what = "weights" if order == L.MOE_MX4_WEIGHTS else "rows"
        raise ValueError(f"{name}: expected a MoEMx4Tensor of {what} {tuple(shape)} on {dev}")
    return q.mx4


def _shared_weights(shared, H: int, Fs: int, dev):
    return [_expect_mx4(name, q, L.MOE_MX4_WEIGHTS, shape, dev)
            for name, q, shape in zip(("shared w_gate", "shared w_up", "shared w_down"), shared,
                                      ((1, H, Fs), (1, H, Fs), (1, Fs, H)))]


class MoEMx4DecodeRunner:
    """The layer's forward for the few tokens of a decoding step with experts in
    4 bits: MoEDecodeRunner with MoEMx4Tensor weights.  Outputs are the runner's
    own buffers and live until the next call, so one runner serves one call at a
    time."""

    def __init__(self, max_tokens: int, H: int, F: int, E: int, K: int, dtype: torch.dtype, device="cuda",
                 shared_ffn: Optional[int] = None):
        self.max_tokens, self.H, self.F, self.E, self.K = max_tokens, H, F, E, K
        self.dtype, self.shared_ffn = dtype, shared_ffn
        code = L.dtype_code(dtype)
        self._dims = [(L.dims(n, H, F, E, K, code), None if shared_ffn is None else L.dims(n, H, shared_ffn, 1, 1, code))
                      for n in range(max_tokens + 1)]
        need = [L.moe_mx4_decode_workspace_bytes(*p) for p in self._dims]
        if not need or max(need) == 2 ** 64 - 1:
            raise L.MoEError("moe_mx4_decode_workspace_bytes",
                             L.MOE_EUNSUPPORTED if max_tokens > L.MOE_DECODE_MAX_TOKENS else L.MOE_EINVAL)
        self.device = dev = _cuda_device(device)
        self._ws_bytes = max(16, *need)
        self.ws = torch.empty((self._ws_bytes,), dtype=torch.uint8, device=dev)
        self._topk = torch.empty((max_tokens, K), dtype=torch.int32, device=dev)
        self._gates = torch.empty((max_tokens, K), dtype=torch.float32, device=dev)
        self._y = torch.empty((max_tokens, H), dtype=dtype, device=dev)
        self.topk, self.gates, self.y = self._topk, self._gates, self._y
        # of any first n rows too
        self._at = self._topk.data_ptr(), self._gates.data_ptr(), self._y.data_ptr(), self.ws.data_ptr()
        self._made = _Made(dev)

    def forward(self, x, w_r, w_gate, w_up, w_down, bias=None, stream=None, shared=None):
        """Returns y [n, H] of x [n, H], n <= max_tokens; topk and gates [n, K]
        are attributes.  ``shared`` = (W_gate_s [1,H,Fs], W_up_s, W_down_s
        [1,Fs,H]), MoEMx4Tensor weights too, exactly when the runner has a shared
        expert."""
        H, F, E, dt, dev = self.H, self.F, self.E, self.dtype, self.device
        n = x.shape[0]
        if n > self.max_tokens:
            raise ValueError(f"{n} tokens, the runner holds {self.max_tokens}")
        if (shared is None) != (self.shared_ffn is None):
            raise ValueError("shared weights must be given exactly when the runner has a shared expert")
        _expect("x", x, (n, H), dt, dev)
        _expect("w_r", w_r, (H, E), dt, dev)
        if bias is not None:
            _expect("bias", bias, (E,), torch.float32, dev)
        w = (_expect_mx4("w_gate", w_gate, L.MOE_MX4_WEIGHTS, (E, H, F), dev),
             _expect_mx4("w_up", w_up, L.MOE_MX4_WEIGHTS, (E, H, F), dev),
             _expect_mx4("w_down", w_down, L.MOE_MX4_WEIGHTS, (E, F, H), dev))
        s = (None, None, None)
        if shared is not None:
            s = _shared_weights(shared, H, self.shared_ffn, dev)
        d, ds = self._dims[n]
        if n:
            with _on(dev):
                L.moe_mx4_decode(d, x, w_r, bias, *w, ds, *s, *self._at, self._made.before(dev, stream), self._ws_bytes)
        if n != self.y.shape[0]:  # not before the call: a refused one changes nothing
            self.topk, self.gates, self.y = self._topk[:n], self._gates[:n], self._y[:n]
        return self.y


class MoEMx4Runner:
    """The layer's forward for N tokens with experts in 4 bits.  The token rows and
    the activations are quantised to 4 bits in front of their products; the router,
    the activations before that and the sum over a token's experts are those of
    MoELayerRunner.  Outputs are the runner's own buffers; one call at a time."""

    def __init__(self, N: int, H: int, F: int, E: int, K: int, dtype: torch.dtype, device="cuda",
                 capacity: Optional[int] = None, shared_ffn: Optional[int] = None):
        """capacity: rows per expert, the overflow dropped; None is the dropless layer.
        shared_ffn: intermediate size of a shared expert that every token passes through
        (weights passed to forward as ``shared``); None: no shared expert."""
        self.N, self.H, self.F, self.E, self.K, self.dtype, self.capacity = N, H, F, E, K, dtype, capacity
        if capacity is not None and capacity < 0:
            raise ValueError("capacity must not be negative")
        self.d = L.dims(N, H, F, E, K, L.dtype_code(dtype))
        mt = L.moe_max_tiles(self.d)
        if mt < 0:
            raise L.MoEError("moe_max_tiles", L.MOE_EINVAL)
        self.device = dev = _cuda_device(device)
        i32, NK = torch.int32, N * K
        self.topk = torch.empty((N, K), dtype=i32, device=dev)
        self.gates = torch.empty((N, K), dtype=torch.float32, device=dev)
        self.sorted_flat = torch.empty((NK,), dtype=i32, device=dev)
        self.inv = torch.empty((NK,), dtype=i32, device=dev)
        self.counts = torch.empty((E,), dtype=i32, device=dev)
        self.offsets = torch.empty((E + 1,), dtype=i32, device=dev)
        self.tiles = torch.empty((max(1, mt) * 3,), dtype=i32, device=dev)
        # no tiles until meta() or forward() has run, so that products behind a captured one do nothing
        self.num_tiles = torch.zeros((1,), dtype=i32, device=dev)
        self._grouped = False
        need = [L.moe_workspace_bytes(self.d, e) for e in (L.MOE_ENTRY_ROUTE_META, L.MOE_ENTRY_PERMUTE_META)]
        self.ws = torch.empty((max(16, *need),), dtype=torch.uint8, device=dev)
        self.xq = MoEMx4Tensor(L.MOE_MX4_ROWS, (N, H), dev)
        self.aq = MoEMx4Tensor(L.MOE_MX4_ROWS, (NK, F), dev)
        # rows that a capacity drops are never written, but quantised with the others
        make = torch.empty if capacity is None else torch.zeros
        self.act = make((NK, F), dtype=dtype, device=dev)
        self.ys = make((NK, H), dtype=dtype, device=dev)
        self.y = torch.empty((N, H), dtype=dtype, device=dev)
        self.shared_ffn = shared_ffn
        if shared_ffn is not None:
            # one expert that every token has chosen: all rows, in their order
            self.ds = L.dims(N, H, shared_ffn, 1, 1, L.dtype_code(dtype))
            if L.moe_max_tiles(self.ds) < 0:
                raise L.MoEError("moe_max_tiles", L.MOE_EINVAL)
            self.rows_s = torch.arange(max(1, N), dtype=i32, device=dev)
            first = self.rows_s[::L.MOE_TILE_M]
            self.tiles_s = torch.stack([torch.zeros_like(first), first, (N - first).clamp(max=L.MOE_TILE_M)], 1)
            self.num_tiles_s = torch.full((1,), first.numel(), dtype=i32, device=dev)
            self.aq_s = MoEMx4Tensor(L.MOE_MX4_ROWS, (N, shared_ffn), dev)
            self.act_s = torch.empty((N, shared_ffn), dtype=dtype, device=dev)
            self.ys_s = torch.empty((N, H), dtype=dtype, device=dev)
        self._made = _Made(dev)

    def meta(self, topk, stream=None):
        """Group the rows by a given choice topk [N, K] int32, values in [0, E)."""
        _expect("topk", topk, (self.N, self.K), torch.int32, self.device)
        cap = 2 ** 31 - 1 if self.capacity is None else self.capacity
        if self.N:
            with _on(self.device):
                L.moe_permute_meta_capacity(self.d, topk, cap, self.sorted_flat, self.inv, self.counts, self.offsets,
                                            self.tiles, self.num_tiles, self.ws, self._made.before(self.device, stream))
        self._grouped = True

    def _expect_groups(self, name: str):
        if not self._grouped:
            raise RuntimeError(f"{name} before meta or forward")

    def gate_up(self, xq, w_gate, w_up, stream=None):
        """silu(G) * U [N*K, F] of quantised token rows xq [N, H], in the grouped order of
        the last meta() or forward()."""
        E, H, F, dev = self.E, self.H, self.F, self.device
        q = (_expect_mx4("xq", xq, L.MOE_MX4_ROWS, (self.N, H), dev),
             _expect_mx4("w_gate", w_gate, L.MOE_MX4_WEIGHTS, (E, H, F), dev),
             _expect_mx4("w_up", w_up, L.MOE_MX4_WEIGHTS, (E, H, F), dev))
        if self.N:
            self._expect_groups("gate_up")
            with _on(dev):
                L.moe_mx4_gate_up(self.d, q[0], self.sorted_flat, q[1], q[2], self.tiles, self.num_tiles, self.act,
                                  self._made.before(dev, stream))
        return self.act

    def down(self, aq, w_down, stream=None):
        """The down product ys [N*K, H] of quantised activations aq [N*K, F] in the same order."""
        dev = self.device
        a = _expect_mx4("aq", aq, L.MOE_MX4_ROWS, (self.N * self.K, self.F), dev)
        w = _expect_mx4("w_down", w_down, L.MOE_MX4_WEIGHTS, (self.E, self.F, self.H), dev)
        if self.N:
            self._expect_groups("down")
            with _on(dev):
                L.moe_mx4_down(self.d, a, w, self.tiles, self.num_tiles, self.ys, self._made.before(dev, stream))
        return self.ys

    def forward(self, x, w_r, w_gate, w_up, w_down, bias=None, stream=None, shared=None):
        """Returns y [N, H] of x [N, H]; topk and gates are attributes.  w_gate, w_up
        [E,H,F] and w_down [E,F,H]: MoEMx4Tensor weights.  ``shared`` as in
        MoEMx4DecodeRunner.forward."""
        E, H, F, dev = self.E, self.H, self.F, self.device
        if (shared is None) != (self.shared_ffn is None):
            raise ValueError("shared weights must be given exactly when the runner has a shared expert")
        _expect("x", x, (self.N, H), self.dtype, dev)
        _expect("w_r", w_r, (H, E), self.dtype, dev)
        if bias is not None:
            _expect("bias", bias, (E,), torch.float32, dev)
        for name, q, shape in (("w_gate", w_gate, (E, H, F)), ("w_up", w_up, (E, H, F)), ("w_down", w_down, (E, F, H))):
            _expect_mx4(name, q, L.MOE_MX4_WEIGHTS, shape, dev)
        if shared is not None:
            s = _shared_weights(shared, H, self.shared_ffn, dev)
        if self.N == 0:
            return self.y
        cap = 2 ** 31 - 1 if self.capacity is None else self.capacity
        with _on(dev):
            L.moe_route_meta(self.d, x, w_r, bias, cap, self.topk, self.gates, self.sorted_flat, self.inv,
                             self.counts, self.offsets, self.tiles, self.num_tiles, self.ws,
                             self._made.before(dev, stream))
        self._grouped = True
        act = self.gate_up(self.xq.quantize(x, stream), w_gate, w_up, stream)
        self.down(self.aq.quantize(act, stream), w_down, stream)
        with _on(dev):
            if shared is None:
                L.moe_combine(self.d, self.ys, self.gates, self.inv, self.y, stream)
                return self.y
            L.moe_mx4_gate_up(self.ds, self.xq.mx4, self.rows_s, s[0], s[1], self.tiles_s, self.num_tiles_s, self.act_s,
                              stream)
            self.aq_s.quantize(self.act_s, stream)
            L.moe_mx4_down(self.ds, self.aq_s.mx4, s[2], self.tiles_s, self.num_tiles_s, self.ys_s, stream)
            L.moe_combine_shared(self.d, self.ys, self.gates, self.inv, self.ys_s, self.y, stream)
        return self.y

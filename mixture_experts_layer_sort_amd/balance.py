"""Balance and z loss of router logits, with the counts of every expert and the
gradient of the logits (moe_balance_loss, moe_balance_loss_bwd).

MoELayerRunner's aux_alpha is the Switch loss of the layer's own logits over the
whole batch.  Here the logits are given, sequences are balanced one by one, padding is
left out, scores may be sigmoids, and the z loss keeps the logits small:

    y, topk = moe_layer(x, w_r, w_gate, w_up, w_down, K, return_topk=True)
    logits = x.float() @ w_r.float()
    loss, counts = moe_balance_loss(logits, K, topk=topk, seq_len=T, mask=mask, alpha=0.01, z_coef=1e-3)
    (task_loss + loss).backward()

topk is the layer's own choice: it is made on wider logits than a bfloat16 x @ w_r holds,
whose equals are frequent, so a choice made again on those would count other experts.
"""
from __future__ import annotations

from typing import Optional

import torch
from torch.autograd.function import once_differentiable

from . import _lib as L
from .layer import _Made, _cuda_device, _dense, _expect, _on, _stream_of

_SCORES = {"softmax": L.MOE_SCORE_SOFTMAX, "sigmoid": L.MOE_SCORE_SIGMOID}


def _problem(N, E, K, dtype, seq_len, alpha, z_coef, score):
    if score not in _SCORES:
        raise ValueError(f"score: one of {sorted(_SCORES)}")
    return L.moe_balance(N, E, K, max(1, N) if seq_len is None else seq_len, L.dtype_code(dtype), _SCORES[score], alpha,
                         z_coef)


def _bytes(b):
    need = L.moe_balance_state_bytes(b), L.moe_balance_workspace_bytes(b)
    if 2 ** 64 - 1 in need:
        raise L.MoEError("moe_balance_workspace_bytes", L.MOE_EINVAL)
    return [max(16, n) for n in need]


def _mask(mask, N, dev):
    """A token's byte, from bool or uint8 of any shape with N elements."""
    if mask is None:
        return None
    if mask.dtype not in (torch.bool, torch.uint8) or mask.numel() != N or mask.device != dev:
        raise ValueError(f"mask: expected bool or uint8 with {N} elements on {dev}")
    return _dense(mask)


class MoEBalanceRunner:
    """The loss of N tokens' logits, in buffers of its own: loss [1], counts [E]
    int32 and dlogits.  One call at a time."""

    def __init__(self, N: int, E: int, K: int, dtype: torch.dtype, device="cuda", seq_len: Optional[int] = None,
                 alpha: float = 0.01, z_coef: float = 0.0, score: str = "softmax"):
        """seq_len: tokens of a sequence, N a multiple of it; None: all tokens are one."""
        self.N, self.E, self.K, self.dtype = N, E, K, dtype
        self.b = _problem(N, E, K, dtype, seq_len, alpha, z_coef, score)
        state, ws = _bytes(self.b)
        self.device = dev = _cuda_device(device)
        self.state = torch.empty((state,), dtype=torch.uint8, device=dev)
        self.ws = torch.empty((ws,), dtype=torch.uint8, device=dev)
        self.loss = torch.zeros((1,), dtype=torch.float32, device=dev)
        self.counts = torch.zeros((E,), dtype=torch.int32, device=dev)
        self.dlogits = torch.empty((N, E), dtype=dtype, device=dev)
        self._at = self.loss.data_ptr(), self.counts.data_ptr(), self.state.data_ptr(), self.ws.data_ptr()
        self._sizes, self._d_at = (state, ws), self.dlogits.data_ptr()
        self._made = _Made(dev)
        self.inputs = None

    def forward(self, logits, topk=None, mask=None, bias=None, stream=None):
        """Returns the loss of logits [N, E]; counts is an attribute.  topk [N, K] int32: the
        experts that the tokens chose; None: those of largest logit (+ bias [E] float32)."""
        dev = self.device
        _expect("logits", logits, (self.N, self.E), self.dtype, dev)
        if topk is not None:
            _expect("topk", topk, (self.N, self.K), torch.int32, dev)
        if bias is not None:
            _expect("bias", bias, (self.E,), torch.float32, dev)
            if topk is not None:
                raise ValueError("a bias moves the choice of experts: it goes without topk")
        if mask is not None:
            with _stream_of(dev, stream):
                mask = _mask(mask, self.N, dev)
        with _on(dev):
            stream = self._made.before(dev, stream)
            if self.N:
                L.moe_balance_loss(self.b, logits, topk, bias, mask, *self._at, stream, self._sizes)
        self.inputs = logits, mask
        return self.loss

    def backward(self, dloss=None, stream=None):
        """dlogits [N, E] of the last forward; dloss [1] float32 on the device, None for 1."""
        if self.inputs is None:
            raise RuntimeError("backward before forward")
        if dloss is not None:
            _expect("dloss", dloss, (1,), torch.float32, self.device)
        logits, mask = self.inputs
        if self.N:
            with _on(self.device):
                L.moe_balance_loss_bwd(self.b, logits, mask, self._at[2], dloss, self._d_at, stream)
        return self.dlogits


class MoEBalanceFunction(torch.autograd.Function):
    """(loss, counts) of logits, the loss with a gradient for the logits."""

    @staticmethod
    def forward(ctx, logits, K, topk, mask, bias, seq_len, alpha, z_coef, score):
        E, dev = logits.shape[-1], logits.device
        N = logits.numel() // E if E else 0
        b = _problem(N, E, K, logits.dtype, seq_len, alpha, z_coef, score)
        need, ws = _bytes(b)
        logits = _dense(logits)
        if topk is not None:
            if topk.dtype != torch.int32 or topk.numel() != N * K or topk.device != dev:
                raise ValueError(f"topk: expected int32 with {N} x {K} elements on {dev}")
            if bias is not None:
                raise ValueError("a bias moves the choice of experts: it goes without topk")
            topk = _dense(topk)
        if bias is not None:
            _expect("bias", bias, (E,), torch.float32, dev)
            bias = _dense(bias)
        mask = _mask(mask, N, dev)
        state = torch.empty((need,), dtype=torch.uint8, device=dev)
        if N:
            loss = torch.empty((1,), dtype=torch.float32, device=dev)
            counts = torch.empty((E,), dtype=torch.int32, device=dev)
            with _on(dev):
                L.moe_balance_loss(b, logits, topk, bias, mask, loss, counts, state,
                                   torch.empty((ws,), dtype=torch.uint8, device=dev))
        else:
            loss = torch.zeros((1,), dtype=torch.float32, device=dev)
            counts = torch.zeros((E,), dtype=torch.int32, device=dev)
        ctx.save_for_backward(logits, mask, state)
        ctx.b = b
        ctx.mark_non_differentiable(counts)
        return loss, counts

    @staticmethod
    @once_differentiable
    def backward(ctx, dloss, _dcounts):
        logits, mask, state = ctx.saved_tensors
        d = torch.empty_like(logits)
        if ctx.b.N:
            with _on(logits.device):
                L.moe_balance_loss_bwd(ctx.b, logits, mask, state, _dense(dloss), d)
        return (d,) + (None,) * 8


def moe_balance_loss(logits, K: int, topk=None, mask=None, bias=None, seq_len: Optional[int] = None,
                     alpha: float = 0.01, z_coef: float = 0.0, score: str = "softmax"):
    """Balance and z loss of router logits [..., E] with autograd support: (loss [1] float32,
    counts [E] int32).

    The last axis but one and those before it are tokens, seq_len of them (None: all) a
    sequence.  topk: the K experts that each token chose, int32 [..., K] (moe_layer's, with
    return_topk); None: those of largest logit (+ bias [E] float32, which moves the choice
    alone).  mask: bool or uint8 [...], false for padding.  score: "softmax" or "sigmoid"
    (normalised over the experts).
    loss = alpha / sequences * sum_s sum_e f_s,e P_s,e + z_coef * mean(logsumexp^2), f_s,e the
    share of a sequence's choices that expert e has, times E, and P_s,e its mean probability.
    A backward pass is captured into a graph only while no eager graph of the same leaves lives
    (torch then waits on that graph's stream, which ends the process); MoEBalanceRunner can be
    captured at any time.
    """
    return MoEBalanceFunction.apply(logits, K, topk, mask, bias, seq_len, alpha, z_coef, score)

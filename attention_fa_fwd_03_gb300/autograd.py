"""Differentiable attention: a node of PyTorch's graph over the C ABI.

Follows page "mlx-bun 0.0.4: package/src/model/flash-attention.ts", section
"Differentiable op: flash forward + manual backward via CustomVjp": the
forward returns O and keeps the per-row log-sum-exp L beside q, k, v and O;
the backward is the hand-written VJP (D-vector, dK/dV, dQ kernels), which
recomputes the probabilities from L instead of storing them. The cotangent of
L is discarded (L is marked non-differentiable here), as on that page.

Differences from the page: fp16 and bf16 both run natively (no cast to fp16
and back), and sliding windows run in the same kernels instead of falling
back to another attention op. Only argument marshalling happens here: output
and workspace tensors are allocated by PyTorch, every step of the computation
runs in the library's kernels, and there is no CPU path (a CPU tensor raises).

``flash_attention`` is the compiled node (csrc/autograd_binding.h), whose
backward does not wait for the interpreter's lock. ``FlashAttention.apply`` is
the same node under the name and arguments of a ``torch.autograd.Function``.
There is no second derivative: differentiating the gradients raises.

    from attention_fa_fwd_03_gb300.autograd import flash_attention
    o = flash_attention(q, k, v, causal=True)          # q [B,Hq,Tq,D], k/v [B,Hkv,Tkv,D]
    o.backward(do)                                      # fills q.grad, k.grad, v.grad
"""
from __future__ import annotations

import math

import torch

from . import _paged_calls

__all__ = ["FlashAttention", "flash_attention"]


class FlashAttention(torch.autograd.Function):
    """``apply(q, k, v, scale, causal, window[, sinks])`` -> (O, LSE); gradients for q, k, v only."""

    @staticmethod
    def apply(q, k, v, scale: float, causal: bool, window: int, sinks: int = 0):
        return _paged_calls().attention(q, k, v, scale, causal, window, sinks)


def flash_attention(q, k, v, scale: float | None = None, causal: bool = False, window: int = 0,
                    return_lse: bool = False, sinks: int = 0):
    """Exact attention O = softmax(s Q K^T + mask) V with a backward pass.

    q [B,Hq,Tq,D], k and v [B,Hkv,Tkv,D] on one CUDA device, fp16 or bf16,
    Hq a multiple of Hkv (query head h reads KV head h // (Hq // Hkv)).
    ``scale`` defaults to 1/sqrt(D). ``causal`` masks keys after the query
    (top-left aligned); ``window`` W > 0 masks past keys with q - k >= W, but for
    the first ``sinks`` keys, which stay visible.
    Non-contiguous inputs are copied to contiguous ones first. With
    ``return_lse`` the natural-log LSE [B,Hq,Tq] (fp32, no gradient) is
    returned beside O. Gradients made with ``create_graph`` raise where they
    are differentiated again.
    """
    if scale is None:
        scale = 1.0 / math.sqrt(q.shape[-1])
    o, lse = _paged_calls().attention(q.contiguous(), k.contiguous(), v.contiguous(), float(scale), bool(causal),
                                      int(window), int(sinks))
    return (o, lse) if return_lse else o

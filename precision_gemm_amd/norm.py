"""Norms of the hidden states in front of a projection (include/lora_lowp.h): layer norm and RMS
norm, with the residual's addition, and their gradients.

Every call enqueues on the current stream of its tensors' device and synchronises nothing.  They are
no operations of autograd: outputs have no graph, and buffers are written without version counters.
"""

from __future__ import annotations

import torch

from ._binding import call
from ._lib import lib


def layer_norm(x: torch.Tensor, weight=None, bias=None, *, residual=None, eps: float = 1e-6, rms: bool = False, out=None,
               sum_out=None):
    """Norm of each row of ``x`` (lora_layer_norm), bf16 [T, K], rows of any stride; ``rms`` without
    the mean.  ``weight`` and ``bias`` float32 [K] or None.  With ``residual`` (as ``x``) the norm is of
    h = bf16(x + residual).  Returns ``(y, h)``, bf16 [T, K], h being ``x`` itself without a residual;
    in ``out`` and ``sum_out`` if given, which may be ``x`` or ``residual``.  Without a residual, ``out=x``
    leaves no h for :func:`layer_norm_backward`: None is returned in its place."""
    return call("layer_norm", x, x, weight, bias, residual, eps, rms, out, sum_out)


def layer_norm_backward_workspace_bytes(T: int, K: int) -> int:
    """Bytes of the workspace lora_layer_norm_backward needs for the weights' gradients."""
    return int(lib().lora_layer_norm_backward_workspace_bytes(T, K))


def layer_norm_backward(dy: torch.Tensor, h: torch.Tensor, weight=None, *, dsum=None, eps: float = 1e-6, rms: bool = False,
                        weight_grad: bool = True, bias_grad: bool = True, dx=None, dweight=None, dbias=None,
                        workspace=None):
    """Gradients of :func:`layer_norm` (lora_layer_norm_backward): ``dy`` bf16 [T, K] and ``h`` as the
    forward returned it -> ``(dx, dweight, dbias)``: bf16 [T, K], the gradient of ``x`` and of
    ``residual`` alike, and float32 [K], None where ``weight_grad`` or ``bias_grad`` is False
    (frozen weights, an RMS norm without a bias: each of the two takes time of its own).  ``dsum`` is the
    gradient that reaches h along the residual stream, added to ``dx`` (which may be its buffer, or ``dy``'s).  Output buffers and the workspace (calls that overlap in time need their own) may be
    passed in; then the call allocates nothing."""
    return call("layer_norm_backward", dy, dy, h, weight, dsum, eps, rms, weight_grad, bias_grad, dx, dweight, dbias, workspace)

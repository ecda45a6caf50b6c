"""What stands around the layer in a step, in fp64: norms of the hidden states, their gradients, and
an AdamW step.  Written from the definitions; shares no code with the HIP path."""

from __future__ import annotations

import numpy as np

__all__ = ["layer_norm", "layer_norm_backward", "adamw", "clip_factor", "held", "BLOCK"]

BLOCK = 64  # values that share a scale of the 8-bit states


def _center(h, eps, rms):
    h = np.asarray(h, np.float64)
    mean = np.zeros_like(h[:, :1]) if rms else h.mean(1, keepdims=True)
    return h - mean, np.sqrt(((h - mean) ** 2).mean(1, keepdims=True) + eps)


def layer_norm(h, weight, bias, eps, rms=False):
    d, dev = _center(h, eps, rms)
    y = d / dev
    if weight is not None:
        y = y * np.asarray(weight, np.float64)
    return y if bias is None else y + np.asarray(bias, np.float64)


def layer_norm_backward(dy, h, weight, eps, rms=False, dsum=None):
    """(dx, dweight, dbias)."""
    d, dev = _center(h, eps, rms)
    dy = np.asarray(dy, np.float64)
    xh = d / dev
    g = dy if weight is None else dy * np.asarray(weight, np.float64)
    dx = g - xh * (g * xh).mean(1, keepdims=True)
    if not rms:
        dx = dx - g.mean(1, keepdims=True)
    dx = dx / dev
    if dsum is not None:
        dx = dx + np.asarray(dsum, np.float64)
    return dx, (dy * xh).sum(0), dy.sum(0)


def clip_factor(norm, largest):
    return min(1.0, largest / (norm + 1e-6)) if largest > 0 else 1.0


def adamw(p, g, m, v, step, rate, beta1, beta2, eps, decay):
    """(p, m, v) after step number ``step`` (the first is 1)."""
    p, g, m, v = (np.asarray(a, np.float64) for a in (p, g, m, v))
    m = beta1 * m + (1 - beta1) * g
    v = beta2 * v + (1 - beta2) * g * g
    mh, vh = m / (1 - beta1 ** step), v / (1 - beta2 ** step)
    return p - rate * decay * p - rate * mh / (np.sqrt(vh) + eps), m, v


def held(x):
    """Scale of each block of 64 values of ``x`` in 8 bits: its largest magnitude / 448."""
    x = np.abs(np.asarray(x, np.float64).ravel())
    x = np.concatenate([x, np.zeros(-len(x) % BLOCK)]).reshape(-1, BLOCK)
    return x.max(1) / 448.0

"""fp64 oracle of the attention's backward pass — TEST INFRASTRUCTURE ONLY.

The gradients of softmax attention under the explicit frame-window-plus-
reference mask ("HeyGen x Google Cloud: Avatar IV on TPU", section "Deleting
the Mask"; the page has no training), one query row at a time:
P = exp(s q.k - lse), dS = P (dout.v - dout.out), dq = s dS k, dk = s dS^T q,
dv = P^T dout.
"""
from __future__ import annotations

import numpy as np

from .reference import bf16_bits_to_f64, token_mask

__all__ = ["attention_backward"]


def attention_backward(q, k, v, out, lse, dout, frame_tokens, ref_frames: int, window_radius: int) -> dict:
    """dq, dk, dv (fp64, [H, N, d]) from bf16 bits q, k, v, out, dout
    [H, N, d] and lse [H, N]; frame_tokens: one span or per-frame spans."""
    q, k, v, out, dout = (bf16_bits_to_f64(t) for t in (q, k, v, out, dout))
    H, N, d = q.shape
    s = 1.0 / np.sqrt(d)
    mask = token_mask(np.arange(N), N, frame_tokens, ref_frames, window_radius)
    grads = {name: np.zeros((H, N, d)) for name in ("dq", "dk", "dv")}
    for h in range(H):
        for i in range(N):
            j = np.flatnonzero(mask[i])
            p = np.exp(s * (k[h, j] @ q[h, i]) - lse[h, i])
            ds = p * (v[h, j] @ dout[h, i] - dout[h, i] @ out[h, i])
            grads["dq"][h, i] = s * ds @ k[h, j]
            grads["dk"][h, j] += s * ds[:, None] * q[h, i]
            grads["dv"][h, j] += p[:, None] * dout[h, i]
    return grads

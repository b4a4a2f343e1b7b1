"""fp64 CPU oracle of linear attention with a decay for each head and of layer norm.

TEST INFRASTRUCTURE, like ``oracle.rnn``; it shares no code with the HIP
library.  Definitions (t a token, h a head; head h of q, o and the decay uses
head h // (H // Hkv) of k and v):

    S[t] = exp(log_decay[h]) S[t-1] + k[t] v[t]^T,   o[t] = scale S[t]^T q[t]
    y = (x - mean) rstd weight + bias,   rstd = 1 / sqrt(var + eps)

computed token by token and row by row.  The gradients are the adjoint
recurrence (R[t] the gradient of S[t]):

    R[t] = exp(log_decay) R[t+1] + scale q[t] do[t]^T
    dq[t] = scale S[t] do[t],   dk[t] = R[t] v[t],   dv[t] = R[t]^T k[t]

``tests/test_sequence_oracle.py`` pins them against the sums over pairs of
tokens, closed forms and differences.
"""
from __future__ import annotations

import numpy as np


def _f64(a):
    return np.asarray(a, dtype=np.float64)


def _heads(x, H):
    """[T, B, Hkv, D] -> [T, B, H, D]."""
    return np.repeat(_f64(x), H // x.shape[2], axis=2)


def _lengths(lengths, T, B):
    return np.full(B, T) if lengths is None else np.clip(np.asarray(lengths), 0, T)


def linear_attention(q, k, v, log_decay, scale=None, S0=None, lengths=None):
    """o [T, B, H, Dv] and the final states [B, H, Dk, Dv]; rows past a
    sequence's length are zeros."""
    q = _f64(q)
    T, B, H, Dk = q.shape
    k, v = _heads(k, H), _heads(v, H)
    scale = Dk ** -0.5 if scale is None else scale
    decay = np.exp(_f64(log_decay))[:, None, None]
    S = np.zeros((B, H, Dk, v.shape[3])) if S0 is None else _f64(S0).copy()
    o = np.zeros((T, B, H, v.shape[3]))
    n = _lengths(lengths, T, B)
    for t in range(T):
        for b in range(B):
            if t < n[b]:
                S[b] = decay * S[b] + k[t, b, :, :, None] * v[t, b, :, None, :]
                o[t, b] = scale * np.sum(q[t, b, :, :, None] * S[b], axis=1)
    return o, S


def linear_attention_backward(q, k, v, log_decay, do, scale=None, S0=None, dS1=None, lengths=None):
    """dq, dk, dv and the gradient of the initial states."""
    q, do = _f64(q), _f64(do)
    T, B, H, Dk = q.shape
    Hkv = k.shape[2]
    kh, vh = _heads(k, H), _heads(v, H)
    Dv = vh.shape[3]
    scale = Dk ** -0.5 if scale is None else scale
    decay = np.exp(_f64(log_decay))[:, None, None]
    S = np.zeros((B, H, Dk, Dv)) if S0 is None else _f64(S0).copy()
    R = np.zeros((B, H, Dk, Dv)) if dS1 is None else _f64(dS1).copy()
    dq, dk, dv = np.zeros_like(q), np.zeros_like(kh), np.zeros_like(vh)
    n = _lengths(lengths, T, B)
    for b in range(B):
        for t in range(n[b]):
            S[b] = decay * S[b] + kh[t, b, :, :, None] * vh[t, b, :, None, :]
            dq[t, b] = scale * np.sum(S[b] * do[t, b, :, None, :], axis=2)
        for t in reversed(range(n[b])):
            R[b] = R[b] + scale * q[t, b, :, :, None] * do[t, b, :, None, :]
            dk[t, b] = np.sum(R[b] * vh[t, b, :, None, :], axis=2)
            dv[t, b] = np.sum(R[b] * kh[t, b, :, :, None], axis=1)
            R[b] = decay * R[b]

    def shared(x):
        return x.reshape(T, B, Hkv, H // Hkv, x.shape[3]).sum(axis=3)

    return dq, shared(dk), shared(dv), R


def layer_norm(x, weight=None, bias=None, eps=1e-5):
    """y, mean and rstd over the last axis."""
    x = _f64(x)
    mean = x.mean(axis=-1)
    rstd = 1.0 / np.sqrt(np.square(x - mean[..., None]).mean(axis=-1) + eps)
    y = (x - mean[..., None]) * rstd[..., None]
    if weight is not None:
        y = y * _f64(weight)
    if bias is not None:
        y = y + _f64(bias)
    return y, mean, rstd


def layer_norm_backward(dy, x, weight=None, eps=1e-5):
    """dx, dweight and dbias."""
    dy, x = _f64(dy), _f64(x)
    _, mean, rstd = layer_norm(x, eps=eps)
    n = (x - mean[..., None]) * rstd[..., None]
    g = dy if weight is None else dy * _f64(weight)
    dx = rstd[..., None] * (g - g.mean(axis=-1, keepdims=True) - n * (g * n).mean(axis=-1, keepdims=True))
    rows = tuple(range(x.ndim - 1))
    return dx, (dy * n).sum(axis=rows), dy.sum(axis=rows)

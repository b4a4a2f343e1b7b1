"""fp64 CPU oracle of the gated delta rule and of rms norm.

TEST INFRASTRUCTURE, like ``oracle.rnn``; it shares no code with the HIP
library.  Definitions (t a token, h a head; head h of v, o, the decay, beta and
the state uses head h // (H // Hk) of q and k):

    Sd = exp(log_decay[t]) S[t-1],   m = v[t] - Sd^T k[t]
    S[t] = Sd + beta[t] k[t] m^T,    o[t] = scale S[t]^T q[t]
    s = x + residual,   y = s rstd weight,   rstd = 1 / sqrt(mean(s^2) + eps)

computed token by token and row by row; the gradients are the adjoint
recurrence.  ``tests/test_delta_oracle.py`` pins them against closed forms, the
product of the tokens' transition matrices and differences.
"""
from __future__ import annotations

import numpy as np


def _f64(a):
    return np.asarray(a, dtype=np.float64)


def _lengths(lengths, T, B):
    return np.full(B, T) if lengths is None else np.clip(np.asarray(lengths), 0, T)


def _token(S, k, v, g, beta):
    Sd = np.exp(g)[:, None, None] * S
    m = v - np.einsum("hij,hi->hj", Sd, k)
    return Sd, m, Sd + k[:, :, None] * (beta[:, None] * m)[:, None, :]


def _inputs(q, k, v, log_decay, beta):
    v, beta = _f64(v), _f64(beta)
    H = v.shape[2]
    q, k = (np.repeat(_f64(x), H // x.shape[2], axis=2) for x in (q, k))
    g = np.zeros_like(beta) if log_decay is None else _f64(log_decay)
    return q, k, v, g, beta


def gated_delta_rule(q, k, v, log_decay, beta, scale=None, S0=None, lengths=None):
    """o [T, B, H, Dv], the final states [B, H, Dk, Dv], and the largest 2-norm of
    every column of the states and of the values, [B, H, Dv]; rows past a
    sequence's length are zeros."""
    Hk = np.shape(q)[2]
    q, k, v, g, beta = _inputs(q, k, v, log_decay, beta)
    T, B, H, Dv = v.shape
    Dk = q.shape[3]
    assert H % Hk == 0
    scale = Dk ** -0.5 if scale is None else scale
    S = np.zeros((B, H, Dk, Dv)) if S0 is None else _f64(S0).copy()
    o = np.zeros((T, B, H, Dv))
    size = np.sqrt(np.square(S).sum(axis=2))
    n = _lengths(lengths, T, B)
    for b in range(B):
        for t in range(n[b]):
            S[b] = _token(S[b], k[t, b], v[t, b], g[t, b], beta[t, b])[2]
            o[t, b] = scale * np.einsum("hij,hi->hj", S[b], q[t, b])
            size[b] = np.maximum(size[b], np.maximum(np.sqrt(np.square(S[b]).sum(axis=1)), np.abs(v[t, b])))
    return o, S, size


def gated_delta_rule_backward(q, k, v, log_decay, beta, do, scale=None, S0=None, dS1=None, lengths=None):
    """(dq, dk, dv, dlog_decay, dbeta, dS0), and bounds of what their rounding is
    relative to: the same six from products of 2-norms (largest Frobenius norm of
    the states and of their gradients along the sequence)."""
    Hk = np.shape(q)[2]
    q, k, v, g, beta = _inputs(q, k, v, log_decay, beta)
    do = _f64(do)
    T, B, H, Dv = v.shape
    Dk = q.shape[3]
    scale = Dk ** -0.5 if scale is None else scale
    S0 = np.zeros((B, H, Dk, Dv)) if S0 is None else _f64(S0)
    R = np.zeros((B, H, Dk, Dv)) if dS1 is None else _f64(dS1).copy()
    dq, dk, dv, dg, db = (np.zeros_like(x) for x in (q, k, v, g, beta))
    bq, bk, bv, bg, bb = (np.zeros_like(x) for x in (q, k, v, g, beta))
    bR = np.zeros((B, H, 1, 1))
    n = _lengths(lengths, T, B)
    norm = lambda x, axes: np.sqrt(np.square(x).sum(axis=axes))
    for b in range(B):
        S, kept = S0[b], []
        for t in range(n[b]):
            Sd, m, S1 = _token(S, k[t, b], v[t, b], g[t, b], beta[t, b])
            kept.append((S, Sd, m, S1))
            S = S1
        sizeS = np.max([norm(x[i], (1, 2)) for x in kept for i in (0, 3)] + [norm(S0[b], (1, 2))], axis=0)
        sizeM = np.max([norm(x[2], 1) for x in kept] + [np.zeros(H)], axis=0)
        sizeR = norm(R[b], (1, 2))
        sizeW = np.zeros(H)
        for t in reversed(range(n[b])):
            S, Sd, m, S1 = kept[t]
            kt, bt = k[t, b], beta[t, b][:, None]
            dq[t, b] = scale * np.einsum("hij,hj->hi", S1, do[t, b])
            R[b] = R[b] + scale * q[t, b][:, :, None] * do[t, b][:, None, :]
            sizeR = np.maximum(sizeR, norm(R[b], (1, 2)))
            du = np.einsum("hij,hi->hj", R[b], kt)
            db[t, b] = (du * m).sum(axis=1)
            dv[t, b] = bt * du
            dk[t, b] = np.einsum("hij,hj->hi", R[b], bt * m) - np.einsum("hij,hj->hi", Sd, dv[t, b])
            sizeW = np.maximum(sizeW, norm(dv[t, b], 1))
            R[b] = R[b] - kt[:, :, None] * dv[t, b][:, None, :]
            dg[t, b] = (R[b] * Sd).sum(axis=(1, 2))
            R[b] = np.exp(g[t, b])[:, None, None] * R[b]
            sizeR = np.maximum(sizeR, norm(R[b], (1, 2)))
        for t in range(n[b]):
            nk, bt = norm(k[t, b], 1), np.abs(beta[t, b])
            bq[t, b] = (abs(scale) * sizeS * norm(do[t, b], 1))[:, None]
            bk[t, b] = (sizeR * bt * sizeM + sizeS * sizeW)[:, None]
            bv[t, b] = (sizeR * bt * nk)[:, None]
            bb[t, b] = sizeR * nk * sizeM
            bg[t, b] = sizeR * sizeS
        bR[b, :, 0, 0] = sizeR

    def shared(x):
        return x.reshape(T, B, Hk, H // Hk, Dk).sum(axis=3)

    return (shared(dq), shared(dk), dv, dg, db, R), (shared(bq), shared(bk), bv, bg, bb, np.broadcast_to(bR, R.shape))


def rms_norm(x, weight=None, eps=1e-6, residual=None):
    """y, rstd and the sum over the last axis."""
    s = _f64(x) if residual is None else _f64(x) + _f64(residual)
    rstd = 1.0 / np.sqrt(np.square(s).mean(axis=-1) + eps)
    y = s * rstd[..., None]
    return y if weight is None else y * _f64(weight), rstd, s


def rms_norm_backward(dy, x, rstd, weight=None, dsum=None):
    """dx and dweight, from the statistics given."""
    dy, x, rstd = _f64(dy), _f64(x), _f64(rstd)[..., None]
    n = x * rstd
    g = dy if weight is None else dy * _f64(weight)
    dx = rstd * (g - n * (g * n).mean(axis=-1, keepdims=True))
    if dsum is not None:
        dx = dx + _f64(dsum)
    return dx, (dy * n).sum(axis=tuple(range(x.ndim - 1)))


def e4m3_values():
    """The finite values of OCP e4m3 that are not negative, by their code."""
    code = np.arange(127)
    e, m = code >> 3, code & 7
    return np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))

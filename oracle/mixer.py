"""The mixer block's serving operators, oracle side (fp64, plain loops).  Test infrastructure.

RMS norm with the residual's addition, rows in 8 bits with a scale, the product
of 8-bit rows and weights, and the gated delta rule token by token.
"""
from __future__ import annotations

import numpy as np


def rmsnorm(x, w, eps, residual=None):
    """(y, s): s = x + residual, y = s w / sqrt(mean(s^2) + eps), float64."""
    s = np.asarray(x, dtype=np.float64)
    if residual is not None:
        s = s + np.asarray(residual, dtype=np.float64)
    return s * np.asarray(w, np.float64) / np.sqrt(np.mean(s * s, axis=1, keepdims=True) + eps), s


def quant_rows_q8(t):
    """8-bit rows of t and their step a / 127, decided in fp32 as the kernel
    decides: q = rne(t * (127 * (1 / a))) with each operation rounded to fp32.
    The step of a row that holds a NaN or an infinity is not finite (and q unspecified)."""
    t = np.asarray(t, dtype=np.float32)
    a = np.max(np.abs(t), axis=1)
    small = a < np.float32(1e-30)  # a NaN is not
    inv = np.where(small, np.float32(0.0), np.float32(127.0) * (np.float32(1.0) / np.maximum(a, np.float32(1e-30))))
    q = np.rint(t * inv.astype(np.float32)[:, None])
    return (np.clip(np.where(np.isnan(q), 0.0, q), -127, 127).astype(np.int8),
            np.where(small, 0.0, a).astype(np.float64) / 127.0)


def rmsnorm_q8(x, w, eps, residual=None):
    """(q, scale, s): the fp32 rows s w in 8 bits (q does not see the norm's divisor)."""
    s = np.asarray(x, dtype=np.float32)
    if residual is not None:
        s = s + np.asarray(residual, dtype=np.float32)
    q, step = quant_rows_q8(s * np.asarray(w, dtype=np.float32))
    _, s64 = rmsnorm(x, w, eps, residual)
    return q, step / np.sqrt(np.mean(s64 * s64, axis=1) + eps), s64


def linear_i8(xq, x_scale, wq, w_scale, bias=None):
    """Integer sums, then the scales and the bias, float64."""
    acc = np.asarray(xq, dtype=np.int64) @ np.asarray(wq, dtype=np.int64).T
    y = acc.astype(np.float64) * np.asarray(x_scale, np.float64)[:, None] * np.asarray(w_scale, np.float64)
    return y if bias is None else y + np.asarray(bias, np.float64)


def gated_delta(q, k, v, g, beta, offsets, *, scale, unit_qk, state=None):
    """(o [total, hv, dv], state [nseq, hv, dk, dv]): the rule token by token."""
    q, k, v = (np.asarray(a, dtype=np.float64) for a in (q, k, v))
    g, beta = np.asarray(g, np.float64), np.asarray(beta, np.float64)
    nseq, (total, hv, dv), hk, dk = len(offsets) - 1, v.shape, q.shape[1], q.shape[2]
    S = np.zeros((nseq, hv, dk, dv)) if state is None else np.array(state, dtype=np.float64)
    o = np.zeros((total, hv, dv))
    for s in range(nseq):
        for t in range(int(offsets[s]), int(offsets[s + 1])):
            for h in range(hv):
                qt, kt = q[t, h * hk // hv], k[t, h * hk // hv]
                if unit_qk:
                    qt = qt / np.sqrt(qt @ qt + 1e-6)
                    kt = kt / np.sqrt(kt @ kt + 1e-6)
                M = np.exp(g[t, h]) * S[s, h]
                u = beta[t, h] * (v[t, h] - kt @ M)
                S[s, h] = M + np.outer(kt, u)
                o[t, h] = scale * (qt @ S[s, h])
    return o, S

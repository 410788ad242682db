"""Attention in serving, oracle side (fp64, plain loops).  Test infrastructure.

Rows into the pages of a cache and back, attention of packed prompts, and
attention of one new token of each stream over its pages.
"""
from __future__ import annotations

import numpy as np

from .mixer import quant_rows_q8


def _place(table, s, p, npages, page):
    """(page, row in it) of position p of stream s, or None where it has no page."""
    if p < 0 or p // page >= table.shape[1] or not 0 <= table[s, p // page] < npages:
        return None
    return int(table[s, p // page]), p % page


def kv_write(rows, offsets, table, pages, *, start=None, scale=None):
    """rows [total, heads, d] into a copy of pages [npages, heads, page, d] (and of scale
    [npages, heads, page] with 8-bit pages): returns (pages, scale)."""
    pages, scale = pages.copy(), None if scale is None else scale.copy()
    npages, _, page, _ = pages.shape
    for s in range(len(offsets) - 1):
        for i in range(int(offsets[s + 1] - offsets[s])):
            at = _place(table, s, (0 if start is None else int(start[s])) + i, npages, page)
            if at is None:
                continue
            row = rows[int(offsets[s]) + i]
            if scale is None:
                pages[at[0], :, at[1]] = row
            else:
                pages[at[0], :, at[1]], scale[at[0], :, at[1]] = quant_rows_q8(row)
    return pages, scale


def kv_read(pages, offsets, table, *, start=None, scale=None):
    """The positions start[s] .. of every sequence as packed rows [offsets[-1], heads, d], float64."""
    npages, heads, page, d = pages.shape
    out = np.zeros((int(offsets[-1]), heads, d))
    for s in range(len(offsets) - 1):
        for i in range(int(offsets[s + 1] - offsets[s])):
            at = _place(table, s, (0 if start is None else int(start[s])) + i, npages, page)
            if at is not None:
                row = pages[at[0], :, at[1]].astype(np.float64)
                out[int(offsets[s]) + i] = row if scale is None else row * scale[at[0], :, at[1]].astype(np.float64)[:, None]
    return out


def _attend(q, k, v, t, seen, scale, cap, slope, key):
    """Queries [n, d] at positions t over the keys `key` that they see: (o, sum of weights times |v|,
    largest sum of |q k| times scale over a query's keys)."""
    x = scale * (q @ k.T)
    if cap:
        x = cap * np.tanh(x / cap)
    x = x - slope * np.abs(t[:, None] - key[None, :])
    x = np.where(seen, x, -np.inf)
    top = np.max(x, axis=1, initial=-np.inf)
    p = np.where(seen, np.exp(x - np.where(np.isfinite(top), top, 0.0)[:, None]), 0.0)
    total = p.sum(1, keepdims=True)
    w = p / np.where(total > 0, total, 1.0)
    return w @ v, w @ np.abs(v), np.max(np.where(seen, abs(scale) * (np.abs(q) @ np.abs(k).T), 0.0), axis=1, initial=0.0)


def attention(q, k, v, offsets, *, k_offsets=None, scale=None, causal=True, window=None, cap=None, slopes=None, prefix=None,
              there=None, sizes=False):
    """o [total, hq, d] of the packed batch, float64; with sizes also the sums that bound its error.
    ``there`` [total_k] marks the keys that exist (all without it)."""
    q, k, v = (np.asarray(a, np.float64) for a in (q, k, v))
    k_offsets = offsets if k_offsets is None else k_offsets
    (total, hq, d), hkv = q.shape, k.shape[1]
    o, size, reach = np.zeros(q.shape), np.zeros(q.shape), np.zeros((total, hq))
    for s in range(len(offsets) - 1):
        a, b, ka, kb = (int(x) for x in (offsets[s], offsets[s + 1], k_offsets[s], k_offsets[s + 1]))
        t, key = np.arange(b - a) + (kb - ka) - (b - a), np.arange(kb - ka)
        seen = np.ones((b - a, kb - ka), bool)
        if causal:
            seen &= key[None, :] <= t[:, None]
        if window:
            seen &= np.abs(t[:, None] - key[None, :]) < window
        if prefix is not None:
            seen |= (key < prefix[s])[None, :]
        if there is not None:
            seen &= there[ka:kb][None, :]
        for h in range(hq):
            g = h * hkv // hq
            o[a:b, h], size[a:b, h], reach[a:b, h] = _attend(
                q[a:b, h], k[ka:kb, g], v[ka:kb, g], t, seen, d ** -0.5 if scale is None else scale, cap,
                0.0 if slopes is None else float(slopes[h]), key)
    return (o, size, reach) if sizes else o


def attention_step(q, k_pages, v_pages, table, lengths, *, k_scale=None, v_scale=None, sizes=False, **more):
    """One query of each stream over the first lengths[s] positions of its pages."""
    npages, _, page, _ = k_pages.shape
    n = np.clip(lengths, 0, table.shape[1] * page)
    k_offsets = np.concatenate([[0], np.cumsum(n)])
    k, v = kv_read(k_pages, k_offsets, table, scale=k_scale), kv_read(v_pages, k_offsets, table, scale=v_scale)
    there = np.array([_place(table, s, p, npages, page) is not None for s in range(len(n)) for p in range(n[s])], bool)
    return attention(q, k, v, np.arange(len(n) + 1), k_offsets=k_offsets, there=there, sizes=sizes, **more)

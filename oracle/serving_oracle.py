"""Plain fp64 reference of the windowed layer and of the paged serving calls.

TEST INFRASTRUCTURE ONLY, like saf_oracle.py: dense matrices, one exp per element.

* Window: query i of an ordinary head sees the keys j <= i with i - j < window or
  j < sinks (window 0: every j <= i). Frozen heads (Eq. 3) are not cut.
* Rotation: pair c of a row turned by pos * inv_freq[c]; pairs are (c, c + n) of the first
  2n elements, or (2c, 2c + 1) when interleaved.
* Paged attention: the same rows of weights over keys gathered from pages.

A row that sees no key has weights 0, output 0 and log-sum-exp -inf.
"""
from __future__ import annotations

import numpy as np


def visible(i, j, window, sinks):
    """Boolean [len(i), len(j)]: whether an ordinary head's query at i sees the key at j."""
    gap = np.asarray(i)[:, None] - np.asarray(j)[None, :]
    seen = gap >= 0
    if window:
        seen &= (gap < window) | (np.asarray(j)[None, :] < sinks)
    return seen


def row_weights(q, k, i, a, r, frozen, window=0, sinks=0):
    """Weights [n, m] and log-sum-exp [n] of the queries q [n, d] at positions i [n]
    (negative: no query there) over the keys k [m, d] at positions 0 .. m - 1."""
    i = np.asarray(i)
    m = k.shape[0]
    j = np.arange(m)
    if frozen:
        logits = a[None, :m] + r[np.clip(i[:, None] - j[None, :], 0, None)]
        seen = visible(i, j, 0, 0)
    else:
        logits = q @ k.T / np.sqrt(k.shape[1])
        seen = visible(i, j, window, sinks)
    logits = np.where(seen, logits, -np.inf)
    top = logits.max(axis=1, initial=-np.inf)
    e = np.exp(logits - np.where(np.isfinite(top), top, 0.0)[:, None])
    z = e.sum(axis=1)
    with np.errstate(divide="ignore", invalid="ignore"):
        return e / np.where(z > 0, z, 1.0)[:, None], np.where(z > 0, top + np.log(z), -np.inf)


def window_fwd(q, k, v, a, r, frozen, window, sinks):
    """q [B, H, T, d], k, v [B, Hkv, T, d] fp64; returns o [B, H, T, d], lse [B, H, T]."""
    B, H, T, _ = q.shape
    G = H // k.shape[1]
    o, lse = np.zeros(q.shape), np.zeros((B, H, T))
    for b in range(B):
        for h in range(H):
            W, lse[b, h] = row_weights(q[b, h], k[b, h // G], np.arange(T), a[h], r[h], frozen[h], window, sinks)
            o[b, h] = W @ v[b, h // G]
    return o, lse


def window_bwd(q, k, v, do, a, r, frozen, window, sinks):
    """dq [B, H, T, d] (zeros for frozen heads), dk, dv [B, Hkv, T, d]."""
    B, H, T, d = q.shape
    G = H // k.shape[1]
    dq, dk, dv = np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape)
    for b in range(B):
        for h in range(H):
            kk, vv = k[b, h // G], v[b, h // G]
            W, _ = row_weights(q[b, h], kk, np.arange(T), a[h], r[h], frozen[h], window, sinks)
            dv[b, h // G] += W.T @ do[b, h]
            if frozen[h]:
                continue
            dW = do[b, h] @ vv.T
            dS = W * (dW - (W * dW).sum(axis=1, keepdims=True)) / np.sqrt(d)
            dq[b, h] = dS @ kk
            dk[b, h // G] += dS.T @ q[b, h]
    return dq, dk, dv


def rotate(x, pos, inv_freq, interleaved):
    """x [..., n, d] at positions pos [n], turned by the angles pos * inv_freq."""
    n = len(inv_freq)
    ang = np.asarray(pos, dtype=np.float64)[:, None] * np.asarray(inv_freq, dtype=np.float64)
    c, s = np.cos(ang), np.sin(ang)
    y = np.array(x, dtype=np.float64)
    first, second = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
    x0, x1 = y[..., first].copy(), y[..., second].copy()
    y[..., first] = x0 * c - x1 * s
    y[..., second] = x0 * s + x1 * c
    return y


def gather(cache, pages, n):
    """The first n slots [n, Hkv, d] of the pages of a cache [num_pages, Hkv, page, d]."""
    page = cache.shape[2]
    at = np.arange(n)
    return cache[np.asarray(pages, dtype=np.int64)[at // page], :, at % page]


def paged_fwd(q, k_cache, v_cache, table, ctx, n_new, a, r, frozen, window=0, sinks=0, prefix=(), prefix_len=0):
    """q [B, H, T, d]; caches, tables and counts as the library takes them; fp64 results."""
    B, H, T, _ = q.shape
    G = H // v_cache.shape[1]
    o, lse = np.zeros(q.shape), np.full((B, H, T), -np.inf)
    kp, vp = gather(k_cache, prefix, prefix_len), gather(v_cache, prefix, prefix_len)
    for b in range(B):
        n, L = int(n_new[b]), int(ctx[b] + n_new[b])
        if n == 0:
            continue
        k = np.concatenate([kp, gather(k_cache, table[b], L)])
        v = np.concatenate([vp, gather(v_cache, table[b], L)])
        i = prefix_len + int(ctx[b]) + np.arange(n)
        for h in range(H):
            W, lse[b, h, :n] = row_weights(q[b, h, :n], k[:, h // G], i, None if a is None else a[h],
                                           None if r is None else r[h], frozen[h], window, sinks)
            o[b, h, :n] = W @ v[:, h // G]
    return o, lse

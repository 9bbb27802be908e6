"""Cache append, paged attention and prompt attention by their definitions, in float64.

Inputs and caches are bf16 bit patterns (uint16), as the library takes them; outputs are
float64, with nothing rounded.  Besides each output row the attention functions return
what an error bound needs: the row's sum of p |v| and its largest scale * sum |q| |k|.
"""
from __future__ import annotations

import numpy as np

from .context_kv import bf16_decode

__all__ = ["append", "paged", "prompt"]


def append(x_bits, norm_w_bits, positions, eps, theta):
    """[M, heads, hd]: RMSNorm over hd (norm_w_bits None: none), then the pair (x_i,
    x_{i + hd/2}) rotated by positions[m] * theta^(-2i/hd)."""
    x = bf16_decode(x_bits)
    hd = x.shape[-1]
    half = hd // 2
    if norm_w_bits is not None:
        x = x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps) * bf16_decode(norm_w_bits)
    ang = np.asarray(positions, np.float64)[:, None] * theta ** (-2.0 * np.arange(half) / hd)
    c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
    a, b = x[..., :half], x[..., half:]
    return np.concatenate([a * c - b * s, b * c + a * s], axis=-1)


def _row(q, k, v, scale):
    """One query over the keys it sees -> (out, lse, sum p |v|, max scale sum |q| |k|)."""
    if k.shape[0] == 0:
        z = np.zeros(v.shape[-1])
        return z, -np.inf, z, 0.0
    x = (k @ q) * scale
    m = x.max()
    e = np.exp(x - m)
    p = e / e.sum()
    return p @ v, m + np.log(e.sum()), p @ np.abs(v), scale * (np.abs(k) @ np.abs(q)).max()


def _empty(T, nh, hd):
    return dict(out=np.full((T, nh, hd), np.nan), lse=np.full((T, nh), np.nan), mag=np.zeros((T, nh, hd)),
                dot=np.zeros((T, nh)), keys=np.zeros(T, np.int64), written=np.zeros(T, bool))


def _fill(r, t, h, *row):
    r["out"][t, h], r["lse"][t, h], r["mag"][t, h], r["dot"][t, h] = row


def paged(q_bits, k_cache, v_cache, page_table, kv_len, cu_q, page_size, causal, scale):
    """Rows of request b: the tokens cu_q[b] .. cu_q[b+1] - 1, the last of kv_len[b] cached
    ones; a page outside the cache hides its keys."""
    q = bf16_decode(q_bits)
    T, nh, hd = q.shape
    S, nkv, _ = k_cache.shape
    width = page_table.shape[1]
    r = _empty(T, nh, hd)
    for b in range(len(kv_len)):
        n = int(cu_q[b + 1]) - int(cu_q[b])
        kv = min(max(int(kv_len[b]), 0), width * page_size)
        pages = page_table[b][np.arange(kv) // page_size].astype(np.int64)
        there = (pages >= 0) & (pages < S // page_size)
        slots = np.where(there, pages * page_size + np.arange(kv) % page_size, 0)
        k, v = bf16_decode(k_cache[slots]), bf16_decode(v_cache[slots])
        for j in range(n):
            t = int(cu_q[b]) + j
            seen = there & (np.arange(kv) <= kv - n + j) if causal else there
            r["keys"][t], r["written"][t] = seen.sum(), True
            for h in range(nh):
                g = h // (nh // nkv)
                _fill(r, t, h, *_row(q[t, h], k[seen, g], v[seen, g], scale))
    return r


def prompt(q_bits, k_bits, v_bits, cu_seqlens, causal, scale):
    q, k, v = bf16_decode(q_bits), bf16_decode(k_bits), bf16_decode(v_bits)
    T, nh, hd = q.shape
    nkv = k.shape[1]
    r = _empty(T, nh, hd)
    for b in range(len(cu_seqlens) - 1):
        lo, hi = int(cu_seqlens[b]), int(cu_seqlens[b + 1])
        for t in range(lo, hi):
            end = t + 1 if causal else hi
            r["keys"][t], r["written"][t] = end - lo, True
            for h in range(nh):
                g = h // (nh // nkv)
                _fill(r, t, h, *_row(q[t, h], k[lo:end, g], v[lo:end, g], scale))
    return r

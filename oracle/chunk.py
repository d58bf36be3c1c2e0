"""Oracle for chunk attention and the append of a chunk's K/V (float64, loops).

A sequence with L tokens in its paged cache brings n new ones.  Their K/V go
to slots L .. L + n - 1; token i (position L + i) attends the positions
j <= L + i, with a window w > 0 only those with j > L + i - w or j < sink.

Readings: softmax scale 1/sqrt(D) unless given; query head h uses KV head
floor(h / G); Q and K arrive with positions already applied.

Test infrastructure only.
"""

from __future__ import annotations

import math
from typing import Optional

import numpy as np


def chunk_visible(ctx_len: int, new: int, window: int = 0, sink: int = 0) -> np.ndarray:
    """mask[i, j] is True iff new token i attends position j, [n, L + n]."""
    mask = np.zeros((new, ctx_len + new), dtype=bool)
    for i in range(new):
        me = ctx_len + i
        for j in range(me + 1):
            mask[i, j] = window == 0 or me - j < window or j < sink
    return mask


def chunk_attention(q, k_cache, v_cache, block_table, ctx_lens, cu_tokens, *, window: int = 0, sink: int = 0,
                    sm_scale: Optional[float] = None, page_size: int = 16):
    """All arrays hold values (any float type): q [T, Hq, D], caches [pages,
    Hkv, P, D].  Returns (out, lse) in float64; rows no sequence owns are NaN."""
    T, Hq, D = q.shape
    Hkv = k_cache.shape[1]
    G = Hq // Hkv
    scale = 1.0 / math.sqrt(D) if sm_scale is None else float(sm_scale)
    out = np.full((T, Hq, D), np.nan)
    lse = np.full((T, Hq), np.nan)
    for b, L in enumerate(int(x) for x in ctx_lens):
        n0, n1 = int(cu_tokens[b]), int(cu_tokens[b + 1])
        if n1 == n0:
            continue
        end = L + n1 - n0
        pos = np.arange(end)
        phys, row = np.asarray(block_table[b])[pos // page_size], pos % page_size
        mask = chunk_visible(L, n1 - n0, window, sink)
        for kh in range(Hkv):
            K = k_cache[phys, kh, row].astype(np.float64)
            V = v_cache[phys, kh, row].astype(np.float64)
            for h in range(kh * G, (kh + 1) * G):
                s = np.where(mask, q[n0:n1, h].astype(np.float64) @ K.T * scale, -np.inf)
                m = s.max(axis=1, keepdims=True)
                p = np.exp(s - m)
                l = p.sum(axis=1, keepdims=True)
                out[n0:n1, h] = p @ V / l
                lse[n0:n1, h] = (m + np.log(l))[:, 0]
    return out, lse


def kv_append(k, v, k_cache, v_cache, block_table, ctx_lens, cu_tokens, page_size: int = 16):
    """k/v [layers, T, Hkv, D] into caches [layers, pages, Hkv, P, D], bit for
    bit.  Returns (k_new, v_new, new_ctx_lens); inputs are not modified."""
    k_new, v_new = np.array(k_cache, copy=True), np.array(v_cache, copy=True)
    lens = []
    for b, L in enumerate(int(x) for x in ctx_lens):
        n0, n1 = int(cu_tokens[b]), int(cu_tokens[b + 1])
        for i in range(n1 - n0):
            page, row = int(block_table[b][(L + i) // page_size]), (L + i) % page_size
            k_new[:, page, :, row] = k[:, n0 + i]
            v_new[:, page, :, row] = v[:, n0 + i]
        lens.append(L + n1 - n0)
    return k_new, v_new, np.asarray(lens, dtype=np.int32)

"""Oracle for the append with the position rotation and for token sampling
(float64, loops).  Attention over a shared prefix is chunk attention
(oracle/chunk.py): what is shared does not show in the result.

Rotation: pair j of a head, the elements (j, j + r/2) or (2 j, 2 j + 1), turns by
position * inv_freq[j]; elements from r on stay.

Sampling: w = exp((l - max l) / T); in descending order (equal logits: lower index
first) the kept entries are the longest prefix within the first top_k, within the
fewest that sum to top_p of the top_k ones' weight, and of weight >= min_p; at
least one.  The token is the smallest index whose kept weights up to and including
it sum to more than u times all of them; T = 0 takes the first of the order.

Test infrastructure only.
"""

from __future__ import annotations

import numpy as np


def rotate(x, positions, inv_freq, interleaved: bool = False, amplitude: float = 1.0):
    """x [T, H, D] turned to positions [T]; inv_freq holds float32 values."""
    out = np.array(x, dtype=np.float64, copy=True)
    half = len(inv_freq)
    for t, pos in enumerate(positions):
        for j, f in enumerate(inv_freq):
            angle = int(pos) * float(f)  # exact up to position 2^29: 24 bits times 29
            c, s = amplitude * np.cos(angle), amplitude * np.sin(angle)
            a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
            xa, xb = out[t, :, a].copy(), out[t, :, b].copy()
            out[t, :, a] = xa * c - xb * s
            out[t, :, b] = xa * s + xb * c
    return out


def rope_append(q, k, v, k_cache, v_cache, block_table, ctx_lens, cu_tokens, inv_freq, *, interleaved: bool = False,
                amplitude: float = 1.0, positions=None, page_size: int = 16):
    """q [T, Hq, D], k/v [T, Hkv, D], caches [pages, Hkv, P, D].  Returns (q_out,
    k_cache, v_cache, new lengths) in float64; q rows no sequence owns are NaN."""
    kc, vc = np.array(k_cache, dtype=np.float64), np.array(v_cache, dtype=np.float64)
    q_out = np.full(q.shape, np.nan)
    lens = []
    for b, L in enumerate(int(x) for x in ctx_lens):
        n0, n1 = int(cu_tokens[b]), int(cu_tokens[b + 1])
        lens.append(L + n1 - n0)
        pos = np.arange(L, L + n1 - n0) if positions is None else np.asarray(positions)[n0:n1]
        q_out[n0:n1] = rotate(q[n0:n1], pos, inv_freq, interleaved, amplitude)
        turned = rotate(k[n0:n1], pos, inv_freq, interleaved, amplitude)
        for i in range(n1 - n0):
            page, row = int(block_table[b][(L + i) // page_size]), (L + i) % page_size
            kc[page, :, row] = turned[i]
            vc[page, :, row] = v[n0 + i]
    return q_out, kc, vc, np.asarray(lens, dtype=np.int32)


def kept(logits, temperature: float = 1.0, top_k: int = 0, top_p: float = 1.0, min_p: float = 0.0):
    """(indices of the kept entries in descending order, their weights)."""
    x = np.asarray(logits, dtype=np.float64)
    order = sorted((i for i in range(len(x)) if x[i] > -np.inf), key=lambda i: (-x[i], i))
    if temperature == 0:
        return order[:1], [1.0]
    w = [float(np.exp((x[i] - x[order[0]]) / temperature)) for i in order]
    n = len(order) if top_k <= 0 else min(top_k, len(order))
    limit = np.sum(np.array(w[:n], dtype=np.longdouble)) * np.longdouble(top_p)
    stay, running = 0, np.longdouble(0)
    for i in range(n):
        if stay > 0 and (w[i] < min_p or (top_p < 1 and running >= limit)):
            break
        running += w[i]
        stay += 1
    return order[:stay], w[:stay]


def sample_token(logits, u: float, temperature: float = 1.0, top_k: int = 0, top_p: float = 1.0, min_p: float = 0.0):
    """(token, natural logarithm of its share, all shares, distance of u from the nearest border that would change it)."""
    order, w = kept(logits, temperature, top_k, top_p, min_p)
    probs = np.zeros(len(logits))
    total = np.sum(np.array(w, dtype=np.longdouble))
    running, token, gap = np.longdouble(0), -1, np.inf
    for i, x in sorted(zip(order, w)):
        probs[i] = float(x / total)
        before, running = running, running + x
        if token < 0 and running > np.longdouble(u) * total:
            token = i
            gap = float(min(abs(running / total - u), abs(u - before / total) if before > 0 else np.inf))
    return token, float(np.log(probs[token])), probs, gap

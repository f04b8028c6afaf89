"""Float64 oracle of the prompt operators: the rotary position, the packed append and causal
attention of packed query rows over the paged cache (test infrastructure only).

Packed rows: sequence ``b``'s new tokens are rows ``cu[b] .. cu[b+1]-1`` and take its last
``n_b`` positions, ``seq_lens[b] - n_b + i``.
"""

from __future__ import annotations

import numpy as np


def rope(x, pos, inv_freq, interleaved=False):
    """Rows ``x`` [T][H][D] with the first ``2 * len(inv_freq)`` columns turned pair by pair by
    ``pos * inv_freq`` (pairs ``(j, j + r/2)``, or ``(2j, 2j + 1)`` when interleaved), and the
    magnitude ``|a| + |b|`` of each column's pair, which rounding errors scale with."""
    x = np.asarray(x, dtype=np.float64)
    out, mag = x.copy(), np.abs(x)
    half = len(inv_freq)
    for j in range(half):
        lo, hi = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
        angle = np.asarray(pos, dtype=np.float64) * float(inv_freq[j])
        c, s = np.cos(angle)[:, None], np.sin(angle)[:, None]
        a, b = x[..., lo], x[..., hi]
        out[..., lo], out[..., hi] = a * c - b * s, a * s + b * c
        mag[..., lo] = mag[..., hi] = np.abs(a) + np.abs(b)
    return out, mag


def row_places(cu, seq_lens):
    """(sequence, position) of every packed row."""
    seq, pos = [], []
    for b in range(len(seq_lens)):
        n = int(cu[b + 1]) - int(cu[b])
        for i in range(n):
            seq.append(b)
            pos.append(int(seq_lens[b]) - n + i)
    return np.array(seq, dtype=np.int64), np.array(pos, dtype=np.int64)


def cached_rows(pool, page_table, b, length, page_size):
    """The ``length`` cached rows of sequence ``b``: [length][Hkv][D] float64."""
    t = np.arange(length)
    phys = np.asarray(page_table)[b][t // page_size]
    return np.asarray(pool)[phys, :, t % page_size].astype(np.float64)


def prefill(q, k_pool, v_pool, page_table, seq_lens, cu, page_size, sm_scale):
    """Causal attention of packed rows: ``out`` [T][Hq][D], ``lse`` [T][Hq], and what the error
    bounds need, ``mass`` = sum_t p_t |v_t| like out and ``logit`` = sm_scale * the largest
    sum_d |q_d k_d| like lse. Rows that belong to no sequence stay NaN."""
    T, Hq, D = q.shape
    Hkv = k_pool.shape[1]
    G = Hq // Hkv
    out, mass = np.full((T, Hq, D), np.nan), np.full((T, Hq, D), np.nan)
    lse, logit = np.full((T, Hq), np.nan), np.full((T, Hq), np.nan)
    for b in range(len(seq_lens)):
        n, L = int(cu[b + 1]) - int(cu[b]), int(seq_lens[b])
        if n == 0:
            continue
        K = cached_rows(k_pool, page_table, b, L, page_size)
        V = cached_rows(v_pool, page_table, b, L, page_size)
        rows = slice(int(cu[b]), int(cu[b + 1]))
        hidden = np.arange(L)[None, :] > np.arange(L - n, L)[:, None]
        for h in range(Hq):
            x = np.asarray(q[rows, h], dtype=np.float64)
            k, v = K[:, h // G], V[:, h // G]
            z = sm_scale * (x @ k.T)
            z[hidden] = -np.inf
            m = z.max(axis=1, keepdims=True)
            p = np.exp(z - m)
            l = p.sum(axis=1, keepdims=True)
            out[rows, h] = p @ v / l
            mass[rows, h] = p @ np.abs(v) / l
            lse[rows, h] = (m + np.log(l))[:, 0]
            size = sm_scale * (np.abs(x) @ np.abs(k).T)
            size[hidden] = 0.0
            logit[rows, h] = size.max(axis=1)
    return out, lse, mass, logit

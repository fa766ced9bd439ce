"""CPU oracle of sparse decode attention: block bounds, the choice of blocks and attention
over the chosen rows (test infrastructure only, like the rest of ``oracle/``; numpy only).

Bounds of a block and KV head: the elementwise smallest and largest stored key, rounded
outward to bf16 (down and up). Score of block j for query rows r of the KV head:

    score_j = max_r sum_d max(q_rd lo_jd, q_rd hi_jd)

summed exactly (products of bf16 values are exact in float64; ``math.fsum`` rounds the sum
once). The choice keeps all blocks when there are at most ``top_k``, else the ``first``
first, the ``last`` last and the best-scored between, ties to the lower block.
"""

from __future__ import annotations

import math

import numpy as np

from .paged_decode import kv_head, softmax_weights


def bf16_outward(x, up: bool) -> np.ndarray:
    """float64 values to bf16 values (as float64), never past them: the largest bf16 <= x, or smallest >= x."""
    x = np.asarray(x, dtype=np.float64)
    _, e = np.frexp(x)
    step = np.ldexp(1.0, np.maximum(e - 8, -133))  # 8 significant bits; subnormals below 2^-126
    return (np.ceil(x / step) if up else np.floor(x / step)) * step


def update_bounds(bounds, values, block_tables, seq_lens, n_new: int, whole_blocks: bool = False) -> np.ndarray:
    """``bounds`` [NB, HK, 2, D] after the last ``n_new`` rows of every sequence were appended.
    ``values``: the stored keys [NB, HK, BS, D], float64. ``whole_blocks``: touched blocks are
    read whole (e4m3 pages) instead of widened."""
    out = np.array(bounds, dtype=np.float64)
    bs = values.shape[2]
    for b, length in enumerate(seq_lens):
        begin = max(0, length - n_new)
        if length <= 0 or n_new == 0:
            continue
        for j in range(begin // bs, (length - 1) // bs + 1):
            blk = int(block_tables[b][j])
            old = j * bs < begin and not whole_blocks
            lo, hi = (begin - j * bs if old else 0), min(length - j * bs, bs)
            rows = values[blk, :, lo:hi]
            low, high = bf16_outward(rows.min(1), False), bf16_outward(rows.max(1), True)
            out[blk, :, 0] = np.minimum(low, out[blk, :, 0]) if old else low
            out[blk, :, 1] = np.maximum(high, out[blk, :, 1]) if old else high
    return out


def block_scores(q_rows, lo, hi) -> list:
    """Exact scores of blocks (``lo``, ``hi`` [n, D]) for query rows [R, D]."""
    out = []
    for j in range(len(lo)):
        out.append(max(math.fsum(np.maximum(q * lo[j], q * hi[j])) for q in q_rows))
    return out


def choose(scores, top_k: int, first: int, last: int) -> list:
    n = len(scores)
    if n <= top_k:
        return list(range(n))
    mid = sorted(range(first, n - last), key=lambda j: (-scores[j], j))[:top_k - first - last]
    return sorted(list(range(first)) + mid + list(range(n - last, n)))


def choose_blocks(q, bounds, block_tables, seq_lens, block_size: int, top_k: int, first: int, last: int):
    """Chosen block places per (sequence, KV head): a list of lists of lists."""
    q = np.asarray(q, dtype=np.float64)
    hk = bounds.shape[1]
    rep = q.shape[1] // hk
    out = []
    for b, length in enumerate(seq_lens):
        t = [int(x) for x in block_tables[b][:-(-length // block_size)]]
        out.append([])
        for h in range(hk):
            rows = q[b, h * rep:(h + 1) * rep].reshape(-1, q.shape[-1])
            scores = block_scores(rows, bounds[t, h, 0], bounds[t, h, 1]) if len(t) > top_k else [0] * len(t)
            out[-1].append(choose(scores, top_k, first, last))
    return out


def sparse_attention(q, k_values, v_values, block_tables, seq_lens, scale: float, chosen) -> np.ndarray:
    """Attention over the chosen blocks' rows, float64 [B, HQ, N, Dv]; pools as float64 values."""
    q = np.asarray(q, dtype=np.float64)
    B, HQ, N, _ = q.shape
    hk, bs = k_values.shape[1], k_values.shape[2]
    out = np.zeros((B, HQ, N, v_values.shape[-1]))
    for b in range(B):
        length = int(seq_lens[b])
        for h in range(HQ):
            kv = kv_head(h, HQ, hk)
            pos = np.concatenate([np.arange(j * bs, (j + 1) * bs) for j in chosen[b][kv]])
            for i in range(N):
                at = pos[pos <= length - N + i]
                blk = np.asarray(block_tables[b], dtype=np.int64)[at // bs]
                K, V = k_values[blk, kv, at % bs], v_values[blk, kv, at % bs]
                out[b, h, i] = softmax_weights(scale * (K @ q[b, h, i])) @ V
    return out

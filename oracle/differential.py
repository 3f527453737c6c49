"""fp64 reference definition of differential attention over a paged KV cache (test
infrastructure): the difference of two softmax maps over one value row, and the heads'
root-mean-square norm.

Query head 2h + j is map j of head h; KV heads 2g + j hold map j's keys of KV group g, and KV
heads 2g and 2g + 1 the two halves of its value row.  Everything is written out map by map.
"""

from __future__ import annotations

import numpy as np

from .paged_attention import decode_bits, gather_kv, query_positions


def diff_map(q64, K64, V64, positions, scale: float, causal: bool = True, window: int = 0, key_offset: int = 0,
             readable=None):
    """One map of one head: (out [n][2d], sum of weight x |value| [n][2d], largest sum scale |q| |k| [n]).

    q64 [n][d], K64 [T][d], V64 [T][2d]; row 0 of K64 and V64 is position ``key_offset``; keys that are not
    ``readable`` are left out, and a row that attends none is 0."""
    n = len(positions)
    key = key_offset + np.arange(K64.shape[0])
    keep = np.ones((n, K64.shape[0]), dtype=bool)
    if causal:
        keep &= key[None, :] <= np.asarray(positions)[:, None]
    if window:
        keep &= key[None, :] > np.asarray(positions)[:, None] - window
    if readable is not None:
        keep &= np.asarray(readable)[None, :]
    score = np.where(keep, scale * (q64 @ K64.T), -np.inf)
    some = keep.any(axis=1)
    top = np.where(some, score.max(axis=1, initial=-np.inf), 0.0)
    weight = np.exp(score - top[:, None])
    weight /= np.where(some, weight.sum(axis=1), 1.0)[:, None]
    V = np.where((weight > 0).any(axis=0)[:, None], V64, 0.0)  # what nobody attends may hold anything
    reach = np.where(keep, scale * (np.abs(q64) @ np.abs(K64).T), 0.0).max(axis=1, initial=0.0)
    return weight @ V, weight @ np.abs(V), reach


def diff_norm(o64, norm_weight, norm_eps: float):
    """o / sqrt(mean(o^2) + eps) * weight over the last axis; no norm where the weight is None."""
    if norm_weight is None:
        return o64
    return o64 / np.sqrt((o64 ** 2).mean(axis=-1, keepdims=True) + norm_eps) * np.asarray(norm_weight, np.float64)


def diff_varlen(q_bits, q_dtype: str, k_cache, v_cache, kv_dtype: str, block_tables, query_start_loc, seq_lens,
                block_size: int, scale: float, lam, norm_weight=None, norm_eps: float = 1e-5, causal: bool = True,
                k_scale=1.0, v_scale=1.0, window: int = 0, rows=None, num_blocks: int | None = None):
    """(out, difference, spread, reach, keys) of a flattened batch: out [T][H][2d] with its norm; the difference before
    it; A_1 + |lambda| A_2 with A_j the weighted sums of |value|; the largest sum of scale |q| |k| [T][H]; keys
    attended at most [T].  ``lam`` [T][H].  Rows of requests that are not in ``rows`` (flattened rows) are NaN."""
    q64 = decode_bits(q_bits, q_dtype)
    total, hq, d = q64.shape
    hkv = k_cache.shape[1]
    heads, per = hq // 2, hq // hkv
    lam = np.broadcast_to(np.asarray(lam, np.float64), (total, heads))
    diff, spread = np.full((total, heads, 2 * d), np.nan), np.full((total, heads, 2 * d), np.nan)
    reach, keys = np.full((total, heads), np.nan), np.zeros(total)
    for r in range(len(seq_lens)):
        lo, hi, n = int(query_start_loc[r]), int(query_start_loc[r + 1]), int(seq_lens[r])
        sel = [t for t in range(lo, hi) if rows is None or t in rows]
        if not sel:
            continue
        pos = query_positions(n, hi - lo)[np.array(sel) - lo]
        first = max(0, n - (hi - lo) - window + 1) if window else 0
        table = np.array(block_tables[r], dtype=np.int64)
        readable = None
        if num_blocks is not None:
            good = (table >= 0) & (table < num_blocks)
            readable = good[np.arange(first, n) // block_size]
            table = np.where(good, table, 0)
        K = gather_kv(k_cache, table, n, block_size, kv_dtype, k_scale, first)
        V = gather_kv(v_cache, table, n, block_size, kv_dtype, v_scale, first)
        for h in range(heads):
            g = h // per
            value = np.concatenate([V[:, 2 * g], V[:, 2 * g + 1]], axis=1)
            parts = [diff_map(q64[sel, 2 * h + j], K[:, 2 * g + j], value, pos, scale, causal, window, first, readable)
                     for j in (0, 1)]
            w = lam[sel, h][:, None]
            diff[sel, h] = parts[0][0] - w * parts[1][0]
            spread[sel, h] = parts[0][1] + np.abs(w) * parts[1][1]
            reach[sel, h] = np.maximum(parts[0][2], parts[1][2])
        keys[sel] = n
    return diff_norm(diff, norm_weight, norm_eps), diff, spread, reach, keys

"""fp64 reference definitions of the operators around attention in a decoding step
(test infrastructure): rotary positions on one axis or several, positions and slots of
sequences with media, beam selection, and the pages of sequences that branch, grow and end.

Rotary positions and beam search are textbook definitions; the pages' state (one pool,
reference counts, copy-on-write) is [AGENTIC] "統一分頁 + 共用池" and [LINEAGE] "Prefix
reuse".  Every function works row by row, in the order the definition names.
"""

from __future__ import annotations

import math

import numpy as np


# --------------------------------------------------------------------------
# Rotary positions
# --------------------------------------------------------------------------

def rotary_frequencies(rotary_dim: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                       original_max_position: float = 0.0, low_turns: float = 1.0, high_turns: float = 32.0):
    """(float64 inverse frequencies [rotary_dim / 2], factor on the rotated values)."""
    out = []
    for i in range(rotary_dim // 2):
        if scaling == "ntk":
            f = (base * factor ** (rotary_dim / (rotary_dim - 2))) ** (-2.0 * i / rotary_dim)
        else:
            f = base ** (-2.0 * i / rotary_dim)
        if scaling == "linear":
            f /= factor
        elif scaling == "by_parts":
            turns = original_max_position * f / (2 * math.pi)
            if turns <= low_turns:
                f /= factor
            elif turns < high_turns:
                keep = (turns - low_turns) / (high_turns - low_turns)
                f = keep * f + (1 - keep) * f / factor
        out.append(f)
    return np.array(out), (0.1 * math.log(factor) + 1.0 if scaling == "by_parts" else 1.0)


def rotate(x64, positions, inv_freq, interleaved: bool = False, attn_factor: float = 1.0) -> np.ndarray:
    """Rows ``x64`` [tokens][heads][head] with the first 2 * len(inv_freq) elements of each
    head rotated pair by pair by position x inv_freq; inv_freq's fp32 values are exact."""
    y = np.array(x64, dtype=np.float64)
    freq = np.asarray(inv_freq, dtype=np.float32).astype(np.float64)
    half = len(freq)
    theta = np.asarray(positions, dtype=np.float64)[:, None] * freq                # [tokens][half]
    c = (np.cos(theta) * attn_factor)[:, None, :]
    s = (np.sin(theta) * attn_factor)[:, None, :]
    a, b = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half))
    first, second = y[..., a].copy(), y[..., b].copy()
    y[..., a] = first * c - second * s
    y[..., b] = second * c + first * s
    return y


def rotate_axes(x64, positions, inv_freq, pair_axis, interleaved: bool = False,
                attn_factor: float = 1.0) -> np.ndarray:
    """``rotate`` with positions [axes][tokens]: pair i turns by the position on axis pair_axis[i]."""
    y = np.array(x64, dtype=np.float64)
    freq = np.asarray(inv_freq, dtype=np.float32).astype(np.float64)
    for i, axis in enumerate(pair_axis):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + len(freq))
        theta = np.asarray(positions[axis], dtype=np.float64) * freq[i]
        c, s = (np.cos(theta) * attn_factor)[:, None], (np.sin(theta) * attn_factor)[:, None]
        y[..., a], y[..., b] = x64[..., a] * c - x64[..., b] * s, x64[..., b] * c + x64[..., a] * s
    return y


# --------------------------------------------------------------------------
# Positions and slots
# --------------------------------------------------------------------------

def sequence_positions(num_tokens: int, media) -> np.ndarray:
    """Positions [3][num_tokens] of a sequence's tokens, one after the other; ``media`` are
    (first token, frames, rows, columns, step), ascending."""
    out = np.zeros((3, num_tokens), dtype=np.int64)
    starts = {int(m[0]): [int(v) for v in m] for m in media}
    at = place = 0
    while at < num_tokens:
        if at not in starts:
            out[:, at] = place
            at += 1
            place += 1
            continue
        _, frames, rows, cols, step = starts[at]
        highest = place
        for f in range(frames):
            for r in range(rows):
                for c in range(cols):
                    if at < num_tokens:
                        out[:, at] = place + f * step, place + r, place + c
                    highest = max(highest, place + f * step, place + r, place + c)
                    at += 1
        place = highest + 1
    return out


def positions_and_slots(query_start_loc, seq_lens, block_tables, block_size: int, media):
    """(positions [3][tokens], slots [tokens]) of a step's new tokens; ``media`` holds a list for every sequence."""
    positions, slots = [], []
    for i, n in enumerate(seq_lens):
        n, new = int(n), int(query_start_loc[i + 1]) - int(query_start_loc[i])
        positions.append(sequence_positions(n, media[i])[:, n - new:])
        slots += [int(block_tables[i][t // block_size]) * block_size + t % block_size for t in range(n - new, n)]
    return np.concatenate(positions, 1).astype(np.int32), np.array(slots, dtype=np.int64)


# --------------------------------------------------------------------------
# Beam selection
# --------------------------------------------------------------------------

def beam_select(logits64, beam_scores, num_candidates: int, largest: float = np.finfo(np.float32).max):
    """Best candidates of one step: (scores float64, tokens, parents), each [seqs][num_candidates].

    ``logits64`` [seqs * beams][vocab], ``beam_scores`` [seqs][beams].  A NaN logit is -inf, +inf is ``largest``; a
    beam with a score of -inf or NaN gives nothing; equal scores go to the lower beam, within it to the larger logit
    (two that the sum with a far larger maximum rounds together), then to the lower token; what is missing is score
    -inf, token -1, parent -1."""
    x = np.where(np.isnan(logits64), -np.inf, np.minimum(logits64, largest))
    beam_scores = np.asarray(beam_scores, dtype=np.float64)
    seqs, beams = beam_scores.shape
    scores = np.full((seqs, num_candidates), -np.inf)
    tokens = np.full((seqs, num_candidates), -1, dtype=np.int32)
    parents = np.full((seqs, num_candidates), -1, dtype=np.int32)
    for b in range(seqs):
        found = []
        for w in range(beams):
            row = x[b * beams + w]
            live = np.flatnonzero(row > -np.inf)
            if live.size == 0 or not beam_scores[b, w] > -np.inf:
                continue
            top = row[live].max()
            log_sum = math.log(math.fsum(np.exp(row[live] - top)))
            for v in live:
                found.append((-(beam_scores[b, w] + ((row[v] - top) - log_sum)), w, -row[v], int(v)))
        for k, (neg, w, _, v) in enumerate(sorted(found)[:num_candidates]):
            scores[b, k], tokens[b, k], parents[b, k] = -neg, v, b * beams + w
    return scores, tokens, parents


# --------------------------------------------------------------------------
# Pages of sequences
# --------------------------------------------------------------------------

def fork_blocks(tables_out, lens_out, tables, lens, parents, ref_counts, block_size: int) -> None:
    """Row i of ``tables_out`` / ``lens_out`` becomes row parents[i]; its blocks count one holder more."""
    for i, p in enumerate(parents):
        if p < 0 or p >= len(lens) or not 0 <= lens[p] <= tables.shape[1] * block_size:
            lens_out[i] = 0
            continue
        lens_out[i] = lens[p]
        for j in range(-(-int(lens[p]) // block_size)):
            tables_out[i, j] = tables[p, j]
            if 0 <= tables[p, j] < len(ref_counts):
                ref_counts[tables[p, j]] += 1


def append_blocks(tables, lens, query_start_loc, ref_counts, block_size: int):
    """Serve the rows in order; returns (slots, pairs), or None where the call is refused (nothing is changed)."""
    t, n, r = tables.copy(), lens.copy(), ref_counts.copy()
    free = [b for b in range(len(r)) if r[b] == 0]
    slots, pairs = [], []
    qsl = [int(v) for v in query_start_loc]
    if qsl[0] != 0:
        return None
    for i in range(len(n)):
        add = qsl[i + 1] - qsl[i]
        if add < 0 or not 0 <= n[i] <= t.shape[1] * block_size or n[i] + add > t.shape[1] * block_size:
            return None
        pair = (0, 0)
        for pos in range(int(n[i]), int(n[i]) + add):
            j = pos // block_size
            if pos % block_size == 0:
                if not free:
                    return None
                t[i, j] = free.pop(0)
                r[t[i, j]] = 1
            elif pos == n[i]:
                b = int(t[i, j])
                if not 0 <= b < len(r) or r[b] < 1:
                    return None
                if r[b] > 1:
                    if not free:
                        return None
                    pair = (b, free.pop(0))
                    r[b] -= 1
                    t[i, j] = pair[1]
                    r[pair[1]] = 1
            slots.append(int(t[i, j]) * block_size + pos % block_size)
        n[i] += add
        pairs.append(pair)
    tables[:], lens[:], ref_counts[:] = t, n, r
    return np.array(slots, dtype=np.int64), np.array(pairs, dtype=np.int64).reshape(-1, 2)


def release_blocks(tables, lens, ref_counts, block_size: int, keep_lens=None) -> None:
    """Row i keeps its first keep_lens[i] tokens; the blocks behind them lose a holder."""
    for i in range(len(lens)):
        keep = 0 if keep_lens is None else int(keep_lens[i])
        if keep < 0 or keep >= lens[i] or lens[i] > tables.shape[1] * block_size:
            continue
        for j in range(-(-keep // block_size), -(-int(lens[i]) // block_size)):
            b = tables[i, j]
            if 0 <= b < len(ref_counts) and ref_counts[b] > 0:
                ref_counts[b] -= 1
        lens[i] = keep

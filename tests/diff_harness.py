"""Helpers of the differential-attention tests: a workload on the device, the calls, and how far an
output may be from the oracle's.

Tolerances count roundings.  u is half a step of the type that the maps' weights are rounded to for
their product with V (2^-8 bf16, 2^-11 f16; 0 where they stay fp32; single-token rows keep more).  For a row with n keys,
A = A_1 + |lambda| A_2 (A_j: map j's weighted sum of |value|) and R the largest sum of scale |q_i k_i|:
a score of d fp32 products and sums is off by (d + 4) 2^-24 R, its exponential by as much and 2^-21
relative (argument and exponential), each sum over keys by n 2^-24 at most; numerator and denominator
each, so the difference is off by

    E = 2 A (u + (d + 4) 2^-24 R + 2^-21 + n 2^-24) + n 2^-25 max|value| where weights are f16

(f16 weights below 2^-14 round to multiples of 2^-24; the largest is at least 1).  FP8 and NVFP4
values are exact in f16.  A norm o r w with r = 1 / sqrt(mean(o^2) + eps) passes E on as
|w| r (E + |o| r sqrt(mean(E^2))) to first order: a tenth is added for the second.  Storing rounds
once more: half a step of the output's type.
"""

from __future__ import annotations

import numpy as np
import torch

import oracle
import workloads
from tests.harness import DeviceBatch

HALF_STEP = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f32": 2.0 ** -150, "f16": 2.0 ** -25, "bf16": 2.0 ** -134}


class Diff:
    """A batch for both calls: lambda by head or by row and head, a norm or none."""

    def __init__(self, seq_lens, q_lens, hq, hkv, d, bs, kv, q_dtype=None, window=0, norm=True, per_token=False,
                 seed=0, causal=True, dev="cuda:0", cache_scale=None):
        kw = {} if cache_scale is None else {"fp8_scale": cache_scale, "nvfp4_scale": cache_scale}
        self.b = b = workloads.build("diff", seed, seq_lens, q_lens, hq, hkv, d, bs, kv, q_dtype=q_dtype, causal=causal,
                                     **kw)
        rng = np.random.default_rng(seed + 99)
        self.heads, self.window, self.dev = hq // 2, window, dev
        self.lam = rng.uniform(0.2, 0.8, (b.total_q, self.heads) if per_token else (self.heads,)).astype(np.float32)
        self.norm = rng.uniform(0.1, 0.5, 2 * d).astype(np.float32) if norm else None
        self.tables = b.block_tables.copy()
        if window:  # blocks before every window are released: entries that nobody reads
            for r, (n, q) in enumerate(zip(seq_lens, q_lens)):
                self.tables[r, :max(0, int(n) - int(q) - window + 1) // bs] = -5

    def to_device(self):
        self.db = DeviceBatch(self.b, self.dev)
        self.db.tables = torch.from_numpy(self.tables).to(self.dev)
        self.d_lam = torch.from_numpy(self.lam).to(self.dev)
        self.d_norm = None if self.norm is None else torch.from_numpy(self.norm).to(self.dev)
        self.out = torch.full((self.b.total_q, self.heads, 2 * self.b.head_size), 9.0, dtype=self.db.q.dtype,
                              device=self.dev)

    def workspace(self, pa, varlen, part=0):
        b = self.b
        if varlen:
            n = pa.pa_diff_varlen_workspace_size(b.num_seqs, b.total_q, b.max_query_len, b.num_q_heads, b.num_kv_heads,
                                                 b.head_size, b.max_seq_len, b.block_size, part)
        else:
            n = pa.pa_diff_decode_workspace_size(b.num_seqs, b.num_q_heads, b.num_kv_heads, b.head_size, b.max_seq_len,
                                                 b.block_size, part)
        return pa.workspace_tensor(n, self.dev)

    def call(self, pa, varlen, part=0, ws=None, stream=None):
        b, db = self.b, self.db
        ws = self.workspace(pa, varlen, part) if ws is None else ws
        if varlen:
            pa.pa_diff_varlen_attn(self.out, db.q, db.kc, db.vc, db.tables, db.qsl, db.lens, b.max_query_len,
                                   b.max_seq_len, b.scale, self.d_lam, ws, self.d_norm, 1e-5, b.causal, db.k_scale,
                                   db.v_scale, part, stream, self.window)
        else:
            pa.pa_diff_decode(self.out, db.q, db.kc, db.vc, db.tables, db.lens, b.max_seq_len, b.scale, self.d_lam, ws,
                              self.d_norm, 1e-5, db.k_scale, db.v_scale, part, stream, self.window)
        return self.out

    def oracle(self, rows=None):
        b = self.b
        return oracle.diff_varlen(b.q, b.q_dtype, b.k_cache, b.v_cache, b.kv_dtype, self.tables, b.query_start_loc,
                                  b.seq_lens, b.block_size, b.scale, self.lam, self.norm, 1e-5, b.causal, b.k_scale,
                                  b.v_scale, self.window, rows, num_blocks=b.num_blocks)

    def tolerance(self, want, diff, spread, reach, keys):
        b = self.b
        weights = "f32" if b.q_dtype == "f32" else "f16" if b.kv_dtype in workloads.SCALED else b.q_dtype
        u = 0.0 if weights == "f32" else HALF_STEP[weights]
        d = b.head_size
        n = keys[:, None, None]
        e = 2 * spread * (u + (d + 4) * 2.0 ** -24 * reach[..., None] + 2.0 ** -21 + n * 2.0 ** -24)
        if weights == "f16":
            e = e + n * 2.0 ** -25 * self.largest_value()
        if self.norm is not None:
            r = 1.0 / np.sqrt((diff ** 2).mean(-1, keepdims=True) + 1e-5)
            e = 1.1 * np.abs(self.norm) * r * (e + np.abs(diff) * r * np.sqrt((e ** 2).mean(-1, keepdims=True)))
        return np.maximum(HALF_STEP[b.q_dtype] * (np.abs(want) + e), TINY[b.q_dtype]) + e

    def largest_value(self):
        b = self.b
        return float(np.abs(b.v_scale).max()) * {"f16": 6.0, "bf16": 6.0, "fp8_e4m3": 448.0, "fp8_e5m2": 57344.0,
                                                 "nvfp4": 6.0 * 448.0}[b.kv_dtype]

    def check(self, got=None, rows=None):
        want, diff, spread, reach, keys = self.oracle(rows)
        tol = self.tolerance(want, diff, spread, reach, keys)
        got = (self.out if got is None else got).double().cpu().numpy()
        live = ~np.isnan(want[:, 0, 0])
        off = np.abs(got - want)[live]
        assert np.all(np.isfinite(got[live]))
        worst = float((off / tol[live]).max()) if off.size else 0.0
        assert worst <= 1.0, worst
        return worst

"""How far an output of differential attention may be from the oracle's when every rounding is counted
once and at its own size, so that a lost product or a coarser type shows.

For a row of n keys, with A = A_1 + |lambda| A_2 (A_j: map j's weighted sum of |value|) and R the largest
sum of scale |q_i k_i|:

* a weight's rounding for its product with V, in the numerator alone (the sums are of unrounded
  weights): u A.  Chunks on the tensor cores: half a step of 16 bits (2^-8 bf16, 2^-11 f16).  Single-token
  rows there: a weight is two 16-bit numbers, the second the rounded remainder of the first, so half a
  step of half a step (2^-16, 2^-22); but of a bf16 output on an FP8 cache one f16, and the sums are of
  it, so twice 2^-11.  Without the tensor cores: none.  f16 numbers below 2^-14 are multiples of
  2^-24: n 2^-25 max |value| / 1, as a row's largest weight is at least 1;
* scores: products are exact, a matrix instruction cuts its 16 products and its sum at 24 bits below the
  largest of them, so at most 20 x 2^-24 of the sum of magnitudes for each 16 elements, as do the scale,
  the maximum's subtraction and their product, 32 in all: (1.25 d + 32) 2^-24 R, the same relative to the
  exponential; its own error and that of joining partitions: 2^-20;
* sums over keys, likewise for each 16 keys, two products for each where weights are two numbers:
  (2.5 n + 64) 2^-24;
* the last three in numerator and denominator.

A norm passes that on as in diff_harness.  The result is rounded once: half a step at its own binade."""

import numpy as np

import oracle
import workloads
from tests.diff_harness import Diff

BITS = {"f32": 24, "f16": 11, "bf16": 8}
SMALLEST = {"f32": -149, "f16": -24, "bf16": -133}


def half_step(x, dtype):
    """Half of the distance between the type's neighbours at |x|."""
    e = np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -140)))
    return 2.0 ** (np.maximum(e - BITS[dtype] + 1, SMALLEST[dtype]) - 1)


class CountedDiff(Diff):
    """Diff, whose check counts every rounding at its own size."""

    def weight_rounding(self):
        """(u [rows], whether weights are f16 [rows])."""
        b = self.b
        new = np.diff(b.query_start_loc)
        single = np.repeat(new == 1, new)
        fp8 = b.kv_dtype in workloads.FP8
        cores = b.q_dtype != "f32" and b.block_size % 16 == 0 and \
            (b.head_size in (64, 128) if b.kv_dtype == b.q_dtype else fp8 and b.head_size == 128)
        tiles = cores and b.block_size in (16, 32, 64)
        weights = "f16" if fp8 else b.q_dtype
        step = 2.0 ** -BITS[weights]
        one = 0.0 if not cores else 2 * step if fp8 and b.q_dtype == "bf16" else step ** 2
        return np.where(single, one, step if tiles else 0.0), np.where(single, cores, tiles) & (weights == "f16")

    def largest_values(self):
        """The largest |value| of each row's keys."""
        b = self.b
        top = []
        for r, n in enumerate(b.seq_lens):
            v = oracle.gather_kv(b.v_cache, np.maximum(b.block_tables[r], 0), int(n), b.block_size, b.kv_dtype, b.v_scale)
            top.append(np.abs(v).max())
        return np.repeat(top, np.diff(b.query_start_loc))

    def error(self, diff, spread, reach, keys):
        u, f16 = (x[:, None, None] for x in self.weight_rounding())
        n = keys[:, None, None]
        both = (1.25 * self.b.head_size + 32) * 2.0 ** -24 * reach[..., None] + 2.0 ** -20 + (2.5 * n + 64) * 2.0 ** -24
        return spread * (u + 2 * both) + np.where(f16, n * 2.0 ** -25 * self.largest_values()[:, None, None], 0.0)

    def tolerance(self, want, diff, spread, reach, keys):
        e = self.error(diff, spread, reach, keys)
        if self.norm is not None:
            r = 1.0 / np.sqrt((diff ** 2).mean(-1, keepdims=True) + 1e-5)
            e = 1.1 * np.abs(self.norm) * r * (e + np.abs(diff) * r * np.sqrt((e ** 2).mean(-1, keepdims=True)))
            e = e + np.abs(want) * (2 * self.b.head_size + 16) * 2.0 ** -24  # the mean of 2 d squares, 1 / sqrt, products
        return e + half_step(np.abs(want) + e, self.b.q_dtype)


def short_contexts(kv, q_dtype=None, hq=64, hkv=4, seed=71):
    """Single tokens on few keys of nearly equal scores: the output's rounding and the weights' are all that
    is left, scores and sums being off by 2^-15 at most."""
    lens = [2, 3, 5, 7, 8, 11, 13, 16, 17, 23, 30]
    c = CountedDiff(lens, [1] * len(lens), hq, hkv, 128, 16, kv, q_dtype, norm=False, per_token=True, seed=seed,
                    dev="cpu", cache_scale=0.25 if kv in workloads.FP8 else None)
    c.b.scale *= 0.1
    return c

"""pa_beam_select on rows that a mask empties by whole tiles (a grammar allows a few tokens of a large
vocabulary), against the fp64 oracle.  A block goes through its segment of a row in tiles of 16 KB; what
its first tiles, or only some segments of a row, leave out must not change what the later ones give.

A returned score is off by the rounding of the output (2^-24 of it) and by the relative error of the sum of
exponentials.  With d <= D the distance of a logit from its reference: the difference and its product with
log2 e are rounded (together d 2^-23, as a relative error of the exponential) and the exponential is good to
2^-22; a term is rescaled once a tile at most, each time off by as much again; a thread adds at most 8 terms of
a tile, two joins of these and one sum a tile one after the other, and 8 more joins follow, 2^-24 each; whole
numbers of 2^-32 join the segments, and the logarithm is good to 2^-23 of its value, 16 at most.  Distances above
104 give exponentials below fp32's range, so D stops there.
"""

import numpy as np
import pytest
import torch

import oracle
import workloads

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
KEEP = 16
LARGEST = {"f32": float(np.finfo(np.float32).max), "f16": 65504.0, "bf16": float(torch.finfo(torch.bfloat16).max)}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}


@pytest.fixture(scope="module")
def pa():
    import paged_kv_cache_pagedattention_gb300 as lib
    lib.pa_get_error_flags(clear=True)
    return lib


def select(pa, logits, cum):
    b, w = cum.shape
    out = (torch.full((b, KEEP), 9.0, device=DEV), torch.full((b, KEEP), 99, dtype=torch.int32, device=DEV),
           torch.full((b, KEEP), 99, dtype=torch.int32, device=DEV))
    ws = torch.full((pa.pa_beam_select_workspace_size(b, w, logits.shape[1], KEEP),), 0xff, dtype=torch.uint8, device=DEV)
    pa.pa_beam_select(*out, logits, torch.from_numpy(cum).to(DEV), ws)
    torch.cuda.synchronize()
    return [t.cpu().numpy() for t in out]


def score_error(x, tiles):
    live = np.where(np.isfinite(x), x, np.nan)
    span = 0.0 if np.all(np.isnan(live)) else min(104.0, float(np.nanmax(live) - np.nanmin(live)))
    return (tiles + 1) * (span * 2.0 ** -23 + 2.0 ** -22) + (8 + 2 + tiles + 8) * 2.0 ** -24 + 16 * 2.0 ** -23


def patterns(tile, first, vocab):
    """Rows of True where a token is allowed; `first` holds the segments' first elements."""
    rng = np.random.default_rng(41)
    heads = np.zeros(vocab, bool)                # the first tile of every segment
    for f in first:
        heads[f:f + tile] = True
    none = np.zeros(vocab, bool)

    def only(*tokens):
        row = none.copy()
        row[list(tokens)] = True
        return row

    late = np.flatnonzero(~heads)
    rows = [~heads, only(tile + 11), only(vocab - 1), only(late[0], late[-1])]
    row = ~none
    for f in first[::2]:
        row[f:f + tile] = False                  # every other segment begins empty
    rows.append(row)
    row = ~none
    row[:first[1] if len(first) > 1 else 2 * tile] = False
    rows.append(row)                             # a whole segment, or all but one's end
    row = ~none
    row[first[-1] + tile:first[-1] + 2 * tile] = False
    rows.append(row)                             # a tile in the middle
    row = none.copy()
    row[-5:] = True
    rows.append(row)
    rows.append(only(*rng.choice(late, 40, replace=False)))
    rows.append(rng.random(vocab) < 0.02)
    rows.append(none)
    return np.array(rows)


@pytest.mark.parametrize("mask", ["-inf", "nan", "both", "lowest"])
@pytest.mark.parametrize("segments", [1, 4])
@pytest.mark.parametrize("aligned", [True, False], ids=["aligned", "shifted"])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_masked_tiles(pa, dtype, aligned, segments, mask):
    tile, piece = 16384 // SIZE[dtype], 16 // SIZE[dtype]
    vocab = 3 * segments * tile - (0 if aligned else 2 * piece - 3)
    pieces = vocab // piece
    first = [pieces * s // segments * piece for s in range(segments)]
    allowed = patterns(tile, first, vocab)
    if mask == "lowest":                         # every token is a candidate: a few rows of the dense kind
        allowed = allowed[[0, 1, 4, 8]]
    rng = np.random.default_rng(42)
    x = rng.standard_normal(allowed.shape) * 2.0
    x[0, 2 * tile:] += 60.0                      # references rise far after they began late
    off = {"-inf": -np.inf, "nan": np.nan, "lowest": -LARGEST[dtype]}
    x[~allowed] = np.where(np.arange(vocab) % 3 == 1, np.nan, -np.inf)[None].repeat(len(x), 0)[~allowed] \
        if mask == "both" else off[mask]
    dev = torch.from_numpy(x).float().to(workloads.torch_dtype(dtype)).to(DEV)
    x = dev.double().cpu().numpy()
    repeats = -(-{1: 320, 4: 140}[segments] // len(x))
    rows = repeats * len(x)                      # 608 / rows blocks a row
    assert 608 // rows == segments and (rows == 1 or vocab * SIZE[dtype] % 16 == 0) == aligned
    cum = -np.arange(rows, dtype=np.float32).reshape(-1, 1) % 7
    scores, tokens, parents = select(pa, dev.repeat(repeats, 1), cum)
    tiles = -(-(-(-vocab // segments)) // tile) + 1
    want_scores, want_tokens, _ = oracle.beam_select(x, np.zeros((len(x), 1)), KEEP, LARGEST[dtype])
    for r in range(rows):
        i = r % len(x)
        live = want_tokens[i] >= 0
        assert np.array_equal(tokens[r], want_tokens[i]), (r, i)
        assert np.array_equal(parents[r], np.where(live, r, -1))
        assert np.all(np.isneginf(scores[r, ~live]))
        want = want_scores[i, live] + cum[r, 0]
        tol = np.abs(want) * 2.0 ** -24 + score_error(x[i], tiles)
        assert np.all(np.abs(scores[r, live] - want) <= tol), (r, i, float(np.abs(scores[r, live] - want).max()))
    assert pa.pa_get_error_flags(clear=True) == 0


@pytest.mark.parametrize("dtype,beams", [("f32", 4), ("bf16", 8)])
def test_masked_beams_beside_full_ones(pa, dtype, beams):
    """Beams of one sequence under different masks are weighed by their whole sums."""
    tile, piece = 16384 // SIZE[dtype], 16 // SIZE[dtype]
    vocab, seqs, segments = 8 * tile, 128 // beams, 4
    first = [vocab // piece * s // segments * piece for s in range(segments)]
    rng = np.random.default_rng(43)
    rows = patterns(tile, first, vocab)
    allowed = np.concatenate([rows, ~np.zeros((3, vocab), bool)])[rng.integers(0, len(rows) + 3, 128)]
    x = np.where(allowed, rng.standard_normal(allowed.shape, dtype=np.float32) * 2, -np.inf)
    dev = torch.from_numpy(x).float().to(workloads.torch_dtype(dtype)).to(DEV)
    x = dev.double().cpu().numpy()
    cum = -np.cumsum(rng.random((seqs, beams)).astype(np.float32), 1)
    scores, tokens, parents = select(pa, dev, cum)
    error = max(score_error(row, 3) for row in x)
    for s in range(seqs):
        mine = x[s * beams:(s + 1) * beams]
        top = mine.max(1, keepdims=True)
        top = np.where(np.isfinite(top), top, 0.0)
        total = np.exp(mine - top).sum(1, keepdims=True)
        every = (cum[s][:, None] + ((mine - top) - np.log(np.where(total > 0, total, 1.0)))).ravel()
        best = -np.sort(-every)[:KEEP]
        live = np.isfinite(best)
        assert np.array_equal(tokens[s] >= 0, live) and np.array_equal(parents[s] >= 0, live)
        own = every[(parents[s][live] - s * beams).astype(np.int64) * vocab + tokens[s][live]]
        tol = np.abs(own) * 2.0 ** -24 + error
        assert np.all(np.abs(scores[s][live] - own) <= tol) and np.all(own >= best[live] - 2 * error)
        assert len(set(zip(parents[s][live].tolist(), tokens[s][live].tolist()))) == int(live.sum())
    assert pa.pa_get_error_flags(clear=True) == 0

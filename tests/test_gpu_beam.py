"""GPU parity of pa_beam_select against the fp64 oracle.

A returned score may be off from the fp64 score by the fp32 rounding of the output (2^-24 of
it) and by the error of log-sum-exp: every exponential and rescale is good to 2^-21, and a
thread adds in fp32, one after the other, at most 32 terms (four of a tile of 4096 elements,
two joins of these, and the tiles of its segment, few in these tests) before sums are joined
in a tree of depth 8 (TOL).  Candidates closer than that across beams may swap, so general inputs are checked by
the oracle's score of what came back; where scores are equal by construction, or one beam
is alone, tokens and parents have to be the oracle's.
"""

import numpy as np
import pytest
import torch

import oracle
import workloads

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TOL = 2.0 ** -21 + (32 + 8) * 2.0 ** -24
LARGEST = {"f32": float(np.finfo(np.float32).max), "f16": 65504.0, "bf16": float(torch.finfo(torch.bfloat16).max)}


@pytest.fixture(scope="module")
def pa():
    import paged_kv_cache_pagedattention_gb300 as lib
    lib.pa_get_error_flags(clear=True)
    return lib


def run(pa, logits, cum, k, stream=None, ws=None):
    b, w = cum.shape
    out = (torch.full((b, k), 9.0, device=DEV), torch.full((b, k), 99, dtype=torch.int32, device=DEV),
           torch.full((b, k), 99, dtype=torch.int32, device=DEV))
    if ws is None:
        ws = torch.full((pa.pa_beam_select_workspace_size(b, w, logits.shape[1], k),), 0xff, dtype=torch.uint8,
                        device=DEV)
    pa.pa_beam_select(*out, logits, cum, ws, stream)
    torch.cuda.synchronize()
    return [t.cpu().numpy() for t in out]


def dense_scores(x, cum, dtype):
    """fp64 score of every (beam, token): [seqs][beams][vocab], -inf where it gives nothing."""
    x = np.where(np.isnan(x), -np.inf, np.minimum(x, LARGEST[dtype]))
    b, w = cum.shape
    top = x.max(1, keepdims=True)
    top = np.where(np.isfinite(top), top, 0.0)
    total = np.exp(x - top).sum(1, keepdims=True)
    cum = np.where(np.isnan(cum), -np.inf, cum).astype(np.float64)
    return cum[..., None] + ((x - top) - np.log(np.where(total > 0, total, 1.0))).reshape(b, w, -1)


def check(x, cum, got, k, dtype, exact):
    scores, tokens, parents = got
    b, w = cum.shape
    every = dense_scores(x, cum, dtype)
    vocab = every.shape[2]
    flat = every.reshape(b, -1)
    best = -np.sort(-flat, axis=1)[:, :k]
    for i in range(b):
        live = int(min(k, np.isfinite(best[i]).sum()))
        assert np.all(tokens[i, live:] == -1) and np.all(parents[i, live:] == -1)
        assert np.all(np.isneginf(scores[i, live:]))
        at = (parents[i, :live] - i * w).astype(np.int64) * vocab + tokens[i, :live]
        assert len(set(at.tolist())) == live and np.all(at >= 0) and np.all(at < w * vocab)
        own = flat[i, at]
        tol = np.abs(own) * 2.0 ** -24 + TOL
        assert np.all(np.abs(scores[i, :live] - own) <= tol), float(np.abs(scores[i, :live] - own).max())
        assert np.all(own >= best[i, :live] - 2 * TOL)
        assert np.all(np.diff(scores[i, :live]) <= 0)
        for r in range(w):  # within a beam: by logit, then by token
            mine = np.flatnonzero(parents[i, :live] == i * w + r)
            row = np.where(np.isnan(x[i * w + r]), -np.inf, np.minimum(x[i * w + r], LARGEST[dtype]))
            order = np.lexsort((np.arange(vocab), -row))[:mine.size]
            assert np.array_equal(tokens[i, mine], order)
    if exact:
        s, t, p = oracle.beam_select(x, cum, k, LARGEST[dtype])
        assert np.array_equal(tokens, t) and np.array_equal(parents, p)


def make(rng, rows, vocab, dtype, stride=None, shift=0, spread=2.0):
    """(device logits, their fp64 values): rows `stride` apart, the rest of a row NaN."""
    stride = stride or vocab
    x = (rng.standard_normal((rows, stride)) * spread).astype(np.float32)
    x[:, vocab:] = np.nan
    flat = torch.from_numpy(np.concatenate([np.full(shift, np.nan, np.float32), x.ravel()]))
    flat = flat.to(workloads.torch_dtype(dtype)).to(DEV)[shift:]
    dev = flat.view(rows, stride)[:, :vocab]
    return dev, dev.double().cpu().numpy()


CASES = [  # sequences, beams, vocabulary, candidates, type, row stride, shift
    (1, 1, 1, 1, "f32", 0, 0), (1, 1, 5, 32, "f32", 0, 0), (2, 3, 7, 32, "f16", 0, 0), (1, 4, 32000, 8, "f32", 0, 0),
    (3, 4, 1000, 8, "bf16", 0, 0), (2, 5, 4099, 10, "f32", 0, 0), (2, 5, 65537, 10, "bf16", 0, 0),
    (4, 2, 2049, 4, "f16", 2056, 0), (4, 2, 2048, 4, "f32", 2051, 1), (2, 16, 9001, 32, "bf16", 9007, 3),
    (1, 1024, 33, 32, "f32", 0, 0), (40, 16, 300, 16, "f16", 0, 0), (1, 1, 262144, 1, "f32", 0, 0),
    (7, 8, 131072, 16, "bf16", 0, 0), (160, 4, 8195, 4, "bf16", 0, 0), (2000, 2, 40, 3, "f32", 0, 0),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_parity(pa, case):
    b, w, v, k, dtype, stride, shift = case
    rng = np.random.default_rng(21)
    logits, x = make(rng, b * w, v, dtype, stride, shift)
    cum = -np.cumsum(rng.random((b, w)).astype(np.float32), 1)
    got = run(pa, logits, torch.from_numpy(cum).to(DEV), k)
    check(x, cum, got, k, dtype, exact=w == 1)
    assert pa.pa_get_error_flags(clear=True) == 0


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("v,k", [(50, 8), (5000, 32), (70001, 16)])
def test_equal_scores_go_to_the_lower_beam_and_token(pa, dtype, v, k):
    """Rows of few distinct values, the same in every beam: all ties are exact."""
    rng = np.random.default_rng(22)
    row = rng.integers(-2, 3, v).astype(np.float32)
    x = np.tile(row, (6, 1))
    logits = torch.from_numpy(x).to(workloads.torch_dtype(dtype)).to(DEV)
    cum = np.zeros((2, 3), np.float32)
    cum[1, 0] = -20.0
    check(x.astype(np.float64), cum, run(pa, logits, torch.from_numpy(cum).to(DEV), k), k, dtype, exact=True)


@pytest.mark.parametrize("v", [100, 9000])
@pytest.mark.parametrize("fill", [0.0, -5.5, float("-inf")])
def test_constant_rows(pa, v, fill):
    x = np.full((4, v), fill)
    cum = np.zeros((2, 2), np.float32)
    check(x, cum, run(pa, torch.from_numpy(x).float().to(DEV), torch.from_numpy(cum).to(DEV), 12), 12, "f32", True)


@pytest.mark.parametrize("w,v", [(10, 64), (40, 3000), (700, 40)])
def test_many_equal_beams(pa, w, v):
    """More candidates with the best score than are ranked at once."""
    x = np.zeros((2 * w, v))
    cum = np.full((2, w), -1.5, np.float32)
    check(x, cum, run(pa, torch.zeros(2 * w, v, device=DEV), torch.from_numpy(cum).to(DEV), 32), 32, "f32", exact=True)


@pytest.mark.parametrize("k", [1, 7, 32])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rising_and_falling_references(pa, dtype, k):
    """Rows whose later parts lie far above, or below, the first part that sets the reference
    of the sums, a few segments long; flat rows; one that overflows fp32 exponentials of the
    first reference."""
    rng = np.random.default_rng(26)
    v = 40000
    x = rng.standard_normal((6, v))
    x[0] += np.linspace(0, 200, v)
    x[1] -= np.linspace(0, 200, v)
    x[2] *= 1e-3
    x[3, v // 2:] += 300
    x[4, :5000] -= 1e4
    x[5, ::4096] = 150.0
    dev = torch.from_numpy(x).float().to(workloads.torch_dtype(dtype)).to(DEV)
    x = dev.double().cpu().numpy()
    cum = np.zeros((6, 1), np.float32)
    check(x, cum, run(pa, dev, torch.from_numpy(cum).to(DEV), k), k, dtype, exact=True)
    many = dev.repeat(120, 1)                    # one segment a row
    got = run(pa, many, torch.zeros(720, 1, device=DEV), k)
    for r in range(0, 720, 6):
        assert np.array_equal(got[1][r:r + 6], got[1][:6]) and np.array_equal(got[0][r:r + 6], got[0][:6])
    check(x, cum, [g[:6] for g in got], k, dtype, exact=False)


@pytest.mark.parametrize("order", [1, -1])
@pytest.mark.parametrize("v", [3000, 120000])
def test_sorted_rows(pa, v, order):
    x = (np.arange(v)[::order] * 2.0 ** -10)[None].repeat(3, 0).astype(np.float32)
    cum = np.array([[0.0, 0.0, 0.0]], np.float32)
    check(x.astype(np.float64), cum, run(pa, torch.from_numpy(x.copy()).to(DEV), torch.from_numpy(cum).to(DEV), 32), 32,
          "f32", exact=True)


def test_signed_zeros_are_equal(pa):
    x = np.full((1, 600), -1.0, np.float32)
    x[0, [100, 200, 300]] = [-0.0, 0.0, -0.0]
    got = run(pa, torch.from_numpy(x).to(DEV), torch.zeros(1, 1, device=DEV), 3)
    assert got[1].tolist() == [[100, 200, 300]]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_masked_and_non_finite_logits(pa, dtype):
    rng = np.random.default_rng(23)
    logits, x = make(rng, 12, 2500, dtype)
    x = x.copy()
    x[rng.random(x.shape) < 0.5] = -np.inf
    x[1] = -np.inf                               # a row with nothing left
    x[2] = np.nan
    x[3, 700:] = -np.inf
    x[4, :] = -np.inf
    x[4, 2499] = 1.0                             # one token left
    x[5, 17] = np.inf
    x[6, ::50] = np.nan
    x[7, [3, 9]] = np.inf
    x[8] = -LARGEST[dtype]                       # masked by the type's lowest value: still candidates
    x[9, 5] = LARGEST[dtype]
    logits = torch.from_numpy(x).to(logits.dtype).to(DEV)
    cum = -np.cumsum(rng.random((4, 3)).astype(np.float32), 1)
    check(x, cum, run(pa, logits, torch.from_numpy(cum).to(DEV), 10), 10, dtype, exact=False)
    alone = cum.reshape(12, 1)
    check(x, alone, run(pa, logits, torch.from_numpy(alone).to(DEV), 10), 10, dtype, exact=True)


def test_first_step_and_ended_beams(pa):
    rng = np.random.default_rng(24)
    logits, x = make(rng, 12, 900, "f32")
    cum = np.full((3, 4), -np.inf, np.float32)
    cum[0, 0] = 0.0                              # the first step: one beam lives
    cum[1, 2] = -3.0
    cum[1, 3] = np.nan                           # sequence 2 has ended
    check(x, cum, run(pa, logits, torch.from_numpy(cum).to(DEV), 8), 8, "f32", exact=True)


def test_large_magnitudes(pa):
    x = np.array([[1e30, -1e30, 9.9e29, 0.0], [-3e38, -3.1e38, -3e38, -2.9e38]])
    cum = np.array([[-1.0, -1e10]], np.float32)
    logits = torch.from_numpy(x).float().to(DEV)
    check(logits.double().cpu().numpy(), cum, run(pa, logits, torch.from_numpy(cum).to(DEV), 4), 4, "f32", exact=True)


def test_another_stream_two_workspaces_and_graphs(pa):
    rng = np.random.default_rng(25)
    first, x1 = make(rng, 8, 50000, "bf16")
    second, x2 = make(rng, 8, 50000, "bf16")
    cum = -np.cumsum(rng.random((2, 4)).astype(np.float32), 1)
    dev_cum = torch.from_numpy(cum).to(DEV)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    outs = []
    for s, logits in zip(streams, (first, second)):  # at once, each with its own workspace
        ws = pa.workspace_tensor(pa.pa_beam_select_workspace_size(2, 4, 50000, 8))
        out = (torch.empty(2, 8, device=DEV), torch.empty(2, 8, dtype=torch.int32, device=DEV),
               torch.empty(2, 8, dtype=torch.int32, device=DEV))
        torch.cuda.synchronize()
        outs.append((out, ws))
    for _ in range(20):
        for s, logits, (out, ws) in zip(streams, (first, second), outs):
            pa.pa_beam_select(*out, logits, dev_cum, ws, s)
    torch.cuda.synchronize()
    for x, (out, ws) in zip((x1, x2), outs):
        check(x, cum, [t.cpu().numpy() for t in out], 8, "bf16", exact=False)
    # two graphs that share a workspace, replayed in turn on one stream
    ws = outs[0][1]
    graphs = []
    for logits, (out, _) in zip((first, second), outs):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            pa.pa_beam_select(*out, logits, dev_cum, ws)
        graphs.append(graph)
    eager = [[t.clone() for t in out] for out, _ in outs]
    for _ in range(3):
        for graph, (out, _), want in zip(graphs, outs, eager):
            for t in out:
                t.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, want))  # the same bits every time


@pytest.mark.parametrize("dtype,gap", [("bf16", 8), ("f32", 7)])
def test_rows_behind_2_to_31_elements(pa, dtype, gap):
    """Rows far apart: the last one starts behind 2^31 elements."""
    rng = np.random.default_rng(26)
    v, rows, stride = 5003, 4, 2 ** 30 + gap
    flat = torch.empty((rows - 1) * stride + v, dtype=workloads.torch_dtype(dtype), device=DEV)
    far = flat.as_strided((rows, v), (stride, 1))
    near, x = make(rng, rows, v, dtype)
    far.copy_(near)
    cum = -np.cumsum(rng.random((2, 2)).astype(np.float32), 1)
    got = run(pa, far, torch.from_numpy(cum).to(DEV), 8)
    check(x, cum, got, 8, dtype, exact=False)
    for a, b in zip(got, run(pa, near, torch.from_numpy(cum).to(DEV), 8)):
        assert np.array_equal(a, b)


def test_outputs_over_inputs_are_refused(pa):
    logits, cum = torch.zeros(4, 50, device=DEV), torch.zeros(2, 2, device=DEV)
    out = (torch.empty(2, 2, device=DEV), torch.empty(2, 2, dtype=torch.int32, device=DEV),
           torch.empty(2, 2, dtype=torch.int32, device=DEV))
    ws = pa.workspace_tensor(pa.pa_beam_select_workspace_size(2, 2, 50, 2))
    for bad in ((cum, out[1], out[2]), (out[0], cum.view(torch.int32), out[2]),
                (out[0], out[1], ws[:16].view(torch.int32).view(2, 2))):
        with pytest.raises(pa.PAError):
            pa.pa_beam_select(*bad, logits, cum, ws)

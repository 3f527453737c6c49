"""A whole beam search on the device with the library's calls together: append blocks, copy
shared tails, rotate and write, attend, select, fork and release, as eager calls and as
one captured graph replayed for the whole generation, against a dense fp64 beam search
that knows no pages.  The model is one attention layer with random weights; the reference
checks that no choice was closer than 1e-3, far above fp32's error, so tokens are equal."""

import math

import numpy as np
import pytest
import torch

import oracle

DEV = "cuda:0"
VOCAB, E, HQ, HKV, D, ROT, BS = 97, 32, 4, 2, 64, 48, 16
BEAMS, STEPS = 3, 20
PROMPTS = [1, 2, 16, 17, 33, 48]
LONGEST = max(PROMPTS) + STEPS


def weights(seed=10):
    rng = np.random.default_rng(seed)
    f = lambda *s: rng.standard_normal(s).astype(np.float32)  # noqa: E731
    return {"embed": f(VOCAB, E), "qkv": f(E, (HQ + 2 * HKV) * D) / 4, "out": f(HQ * D, VOCAB) / 3,
            "skip": f(E, VOCAB) / 5, "freq": oracle.rotary_frequencies(ROT)[0].astype(np.float32),
            "prompts": [rng.integers(0, VOCAB, n) for n in PROMPTS]}


def dense_beam_search(w):
    """Tokens [seq][beam][STEPS] and scores of the hypotheses, each attended from scratch."""
    w64 = {k: v.astype(np.float64) for k, v in w.items() if k not in ("prompts", "freq")}
    all_tokens, all_scores, gap = [], [], math.inf
    for prompt in w["prompts"]:
        beams = [(0.0, [int(t) for t in prompt])]
        for _ in range(STEPS):
            cands = []
            for cum, toks in beams:
                x = w64["embed"][toks]
                q, k, v = np.split(x @ w64["qkv"], [HQ * D, (HQ + HKV) * D], axis=1)
                pos = np.arange(len(toks))
                q = oracle.rotate(q.reshape(-1, HQ, D), pos, w["freq"])[-1]
                k = oracle.rotate(k.reshape(-1, HKV, D), pos, w["freq"])
                v = v.reshape(-1, HKV, D)
                heads = []
                for h in range(HQ):
                    s = k[:, h // (HQ // HKV)] @ q[h] / math.sqrt(D)
                    p = np.exp(s - s.max())
                    heads.append((p / p.sum()) @ v[:, h // (HQ // HKV)])
                logits = np.concatenate(heads) @ w64["out"] + x[-1] @ w64["skip"]
                logp = logits - logits.max()
                logp -= math.log(np.exp(logp).sum())
                cands += [(cum + lp, toks + [t]) for t, lp in enumerate(logp)]
            cands.sort(key=lambda c: -c[0])
            scores = [c[0] for c in cands[:BEAMS + 1]]
            gap = min(gap, -max(np.diff(scores)))
            beams = cands[:BEAMS]
        all_tokens.append([b[1][len(prompt):] for b in beams])
        all_scores.append([b[0] for b in beams])
    return np.array(all_tokens), np.array(all_scores), gap


@pytest.fixture(scope="module")
def reference():
    w = weights()
    tokens, scores, gap = dense_beam_search(w)
    assert gap > 1e-3
    return w, tokens, scores


def test_reference_has_clear_choices(reference):
    """On the CPU: the dense search's choices are far apart, and beams cross."""
    w, tokens, scores = reference
    assert tokens.shape == (len(PROMPTS), BEAMS, STEPS) and np.all(np.diff(scores, axis=1) < 0)


@pytest.mark.gpu
@pytest.mark.parametrize("graph", [False, True], ids=["eager", "graph"])
def test_beam_search(reference, graph):
    import paged_kv_cache_pagedattention_gb300 as pa

    pa.pa_get_error_flags(clear=True)
    w, want_tokens, want_scores = reference
    seqs, rows = len(PROMPTS), len(PROMPTS) * BEAMS
    width = -(-LONGEST // BS)
    blocks = sum(-(-n // BS) for n in PROMPTS) + rows * 4
    d = {k: torch.from_numpy(v).to(DEV) for k, v in w.items() if k != "prompts"}
    kc = torch.full((blocks, HKV, BS, D), 100.0, device=DEV)   # stale contents that nothing may read
    vc = torch.full_like(kc, 100.0)
    refs = torch.zeros(blocks, dtype=torch.int32, device=DEV)
    state = [(torch.full((rows, width), -1, dtype=torch.int32, device=DEV),
              torch.zeros(rows, dtype=torch.int32, device=DEV)) for _ in range(2)]

    def write(tokens, table, lens, qsl, slots, pairs, positions, ws):
        """Room for the tokens, their k and v in the cache; their rotated q."""
        pa.pa_append_blocks(table, lens, qsl, slots, pairs, refs, BS, ws)
        pa.pa_copy_blocks(kc, vc, pairs)
        x = d["embed"][tokens]
        q, k, v = (t.unflatten(1, (-1, D)) for t in (x @ d["qkv"]).split([HQ * D, HKV * D, HKV * D], 1))
        q_out = torch.empty(len(x), HQ, D, device=DEV)
        pa.pa_rotary_and_cache(q_out, q, k, v, kc, vc, positions, slots, d["freq"])
        return x, q_out

    # prompts but for their last token, in the first row of each sequence
    lens = np.zeros(rows, np.int32)
    lens[::BEAMS] = np.array(PROMPTS) - 1
    qsl = torch.from_numpy(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)).to(DEV)
    total = int(lens.sum())
    body = torch.from_numpy(np.concatenate([p[:-1] for p in w["prompts"]])).to(DEV)
    at = torch.from_numpy(np.concatenate([np.arange(n - 1) for n in PROMPTS]).astype(np.int32)).to(DEV)
    slots = torch.empty(total, dtype=torch.int64, device=DEV)
    pairs = torch.empty(rows, 2, dtype=torch.int64, device=DEV)
    write(body, *state[0], qsl, slots, pairs, at, pa.workspace_tensor(pa.pa_append_workspace_size(rows, total, BS)))
    pa.pa_fork_blocks(*state[1], *state[0], torch.arange(rows, dtype=torch.int32, device=DEV) // BEAMS * BEAMS, refs, BS)
    pa.pa_release_blocks(*state[0], refs, BS)
    state.reverse()

    cum = torch.full((seqs, BEAMS), -math.inf, device=DEV)
    cum[:, 0] = 0.0
    tokens = torch.tensor([int(p[-1]) for p in w["prompts"] for _ in range(BEAMS)], dtype=torch.int32, device=DEV)
    one = torch.arange(rows + 1, dtype=torch.int32, device=DEV)
    slots = torch.empty(rows, dtype=torch.int64, device=DEV)
    picked = [torch.empty(seqs, BEAMS, dtype=torch.int32, device=DEV) for _ in range(4)]
    ws_append = pa.workspace_tensor(pa.pa_append_workspace_size(rows, rows, BS))
    ws_beam = pa.workspace_tensor(pa.pa_beam_select_workspace_size(seqs, BEAMS, VOCAB, BEAMS))
    ws_decode = pa.workspace_tensor(pa.pa_decode_workspace_size(rows, HQ, HKV, D, LONGEST, BS))

    def step(now, then, out_tokens, out_parents):
        table, lens = now
        x, q = write(tokens, table, lens, one, slots, pairs, lens.clone(), ws_append)
        attn = torch.empty_like(q)
        pa.pa_decode(attn, q, kc, vc, table, lens, LONGEST, 1 / math.sqrt(D), ws_decode)
        logits = attn.flatten(1) @ d["out"] + x @ d["skip"]
        scores = torch.empty_like(cum)
        pa.pa_beam_select(scores, out_tokens, out_parents, logits, cum, ws_beam)
        cum.copy_(scores)
        tokens.copy_(out_tokens.flatten())
        pa.pa_fork_blocks(*then, table, lens, out_parents.flatten(), refs, BS)
        pa.pa_release_blocks(table, lens, refs, BS)

    def two_steps():
        step(state[0], state[1], picked[0], picked[1])
        step(state[1], state[0], picked[2], picked[3])

    replay = two_steps
    if graph:
        saved = [t.clone() for t in (kc, vc, refs, cum, tokens, *state[0], *state[1])]
        two_steps()                             # warm-up outside the capture, then back to the start
        for t, s in zip((kc, vc, refs, cum, tokens, *state[0], *state[1]), saved):
            t.copy_(s)
        torch.cuda.synchronize()
        captured = torch.cuda.CUDAGraph()
        with torch.cuda.graph(captured):
            two_steps()
        replay = captured.replay
    got = np.zeros((seqs, BEAMS, 0), np.int64)
    for _ in range(STEPS // 2):
        replay()
        for tok, par in ((picked[0], picked[1]), (picked[2], picked[3])):
            par = par.cpu().numpy() - np.arange(seqs)[:, None] * BEAMS
            got = np.concatenate([got[np.arange(seqs)[:, None], par], tok.cpu().numpy()[..., None]], -1)
    assert pa.pa_get_error_flags(clear=True) == 0
    assert np.array_equal(got, want_tokens)
    assert np.abs(cum.cpu().numpy() - want_scores).max() < 1e-3
    assert state[0][1].tolist() == [n + STEPS - 1 for n in PROMPTS for _ in range(BEAMS)]
    pa.pa_release_blocks(*state[0], refs, BS)
    assert not bool(refs.any()) and pa.pa_get_error_flags(clear=True) == 0


def state(seed):
    import paged_kv_cache_pagedattention_gb300 as pa
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g).to(DEV)  # noqa: E731
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device=DEV)  # noqa: E731
    n, blocks = 6, 64
    s = {"tables": i32(n, 8), "lens": i32(n), "refs": i32(blocks), "t2": i32(n, 8), "l2": i32(n),
         "qsl": (torch.arange(n + 1) * 9).int().to(DEV), "slots": torch.zeros(9 * n, dtype=torch.int64, device=DEV),
         "pairs": torch.zeros(n, 2, dtype=torch.int64, device=DEV),
         "ws": pa.workspace_tensor(pa.pa_append_workspace_size(n, 9 * n, BS)),
         "q": rnd(9 * n, HQ, D), "k": rnd(9 * n, HKV, D), "v": rnd(9 * n, HKV, D), "q_out": rnd(9 * n, HQ, D),
         "kc": torch.zeros(blocks, HKV, BS, D, device=DEV), "vc": torch.zeros(blocks, HKV, BS, D, device=DEV),
         "pos": (torch.arange(9 * n) % 9).int().to(DEV), "freq": pa.pa_rotary_frequencies(ROT)[0],
         "logits": rnd(n, VOCAB), "cum": rnd(2, 3), "scores": rnd(2, 3), "tokens": i32(2, 3), "parents": i32(2, 3),
         "bws": pa.workspace_tensor(pa.pa_beam_select_workspace_size(2, 3, VOCAB, 3))}
    return s


def step(s, between=lambda: None):
    import paged_kv_cache_pagedattention_gb300 as pa
    between()
    pa.pa_append_blocks(s["tables"], s["lens"], s["qsl"], s["slots"], s["pairs"], s["refs"], BS, s["ws"])
    between()
    pa.pa_copy_blocks(s["kc"], s["vc"], s["pairs"])
    between()
    pa.pa_rotary_and_cache(s["q_out"], s["q"], s["k"], s["v"], s["kc"], s["vc"], s["pos"], s["slots"], s["freq"])
    between()
    pa.pa_beam_select(s["scores"], s["tokens"], s["parents"], s["logits"], s["cum"], s["bws"])
    between()
    pa.pa_fork_blocks(s["t2"], s["l2"], s["tables"], s["lens"], s["parents"].view(-1), s["refs"], BS)
    between()
    pa.pa_release_blocks(s["tables"], s["lens"], s["refs"], BS)
    for a, b in (("tables", "t2"), ("lens", "l2")):
        s[a], s[b] = s[b], s[a]


@pytest.mark.gpu
def test_traced_calls_and_two_streams_at_once():
    """Every call is traced under its own kind; with tracing off again, two streams run steps side by
    side on pools and buffers of their own and get what one after the other gives."""
    import paged_kv_cache_pagedattention_gb300 as pa

    kinds = ("rotary_and_cache", "beam_select", "fork_blocks", "append_blocks", "release_blocks")
    want = [state(1), state(2)]
    pa.pa_trace_enable(True)
    try:
        pa.pa_trace_read(0, reset=True)
        for s in want:
            for _ in range(4):
                step(s)
        torch.cuda.synchronize()
        for kind, name in enumerate(pa.TRACE_KINDS):
            count, ms = pa.pa_trace_read(kind)
            assert count == (8 if name in kinds or name == "copy_blocks" else 0), name
            assert ms > 0 or count == 0
    finally:
        pa.pa_trace_enable(False)
        pa.pa_trace_read(0, reset=True)
    got, streams = [state(1), state(2)], [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(4):
        for s, stream in zip(got, streams):
            with torch.cuda.stream(stream):
                step(s)
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(a[k], b[k]) for k in ("lens", "refs", "slots", "pairs", "kc", "vc", "q_out", "scores",
                                                     "tokens", "parents"))
        held = -(-a["lens"] // BS)
        for row, n in enumerate(held.tolist()):
            assert torch.equal(a["tables"][row, :n], b["tables"][row, :n])
    assert pa.pa_get_error_flags(clear=True) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("before", ["nothing", "memset", "copy", "join", "kernel"])
def test_calls_behind_other_work(before):
    """The calls may begin while the work before them ends: a fill, a copy, another stream's kernel
    or a long kernel that writes what they read is waited for, eagerly and as a graph."""
    import paged_kv_cache_pagedattention_gb300 as pa

    side = torch.cuda.Stream()
    filler, big = torch.zeros(1 << 24, device=DEV), torch.ones(1 << 24, device=DEV)

    def between():
        if before == "memset":
            filler.zero_()
        elif before == "copy":
            filler.copy_(big)
        elif before == "kernel":
            torch.add(big, 1.0, out=filler)
        elif before == "join":
            main = torch.cuda.current_stream()
            side.wait_stream(main)
            with torch.cuda.stream(side):
                torch.add(big, 1.0, out=filler)
            main.wait_stream(side)

    def late_inputs(s, g):
        """Every input of the calls is written by the kernel right before them."""
        def between_writes():
            between()
            for name in ("q", "k", "v", "logits", "cum"):
                s[name].copy_(g[name])
            torch.mul(g["pos"], 1, out=s["pos"])
        return between_writes

    want, good = state(5), state(5)
    for _ in range(3):
        step(want)
    torch.cuda.synchronize()
    got = state(5)
    for name in ("q", "k", "v", "logits", "cum", "pos"):
        got[name].zero_()
    for _ in range(3):
        step(got, late_inputs(got, good))
    torch.cuda.synchronize()
    same = ("lens", "refs", "slots", "pairs", "kc", "vc", "q_out", "scores", "tokens", "parents")
    assert all(torch.equal(want[k], got[k]) for k in same)
    # captured: two steps a graph, so that tables and lengths end in the arrays they began in
    ref, cap = state(6), state(6)
    for _ in range(6):
        step(ref)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step(cap, between)
        step(cap, between)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(ref[k], cap[k]) for k in same)
    assert pa.pa_get_error_flags(clear=True) == 0


@pytest.mark.gpu
def test_default_stream_waits_for_blocking_streams():
    """The default stream waits by itself for streams that are not created as non-blocking: inputs that
    such a stream writes behind long kernels are there when the calls read them, without an event."""
    import ctypes

    import paged_kv_cache_pagedattention_gb300 as pa

    handle = ctypes.c_size_t(0)
    assert int(torch.cuda.cudart().cudaStreamCreate(ctypes.addressof(handle))) == 0
    other = torch.cuda.ExternalStream(handle.value)
    big, filler = torch.ones(1 << 26, device=DEV), torch.zeros(1 << 26, device=DEV)
    want, got, good = state(8), state(8), state(8)
    for name in ("q", "k", "v", "logits", "cum"):
        got[name].zero_()
    assert torch.cuda.current_stream().cuda_stream == 0

    def between():
        with torch.cuda.stream(other):
            torch.add(big, 1.0, out=filler)
            for name in ("q", "k", "v", "logits", "cum"):
                got[name].copy_(good[name])
            torch.mul(good["pos"], 1, out=got["pos"])

    for _ in range(3):
        step(want)
    torch.cuda.synchronize()
    for _ in range(3):
        step(got, between)
    torch.cuda.synchronize()
    assert all(torch.equal(want[k], got[k]) for k in ("lens", "refs", "slots", "pairs", "kc", "vc", "q_out", "scores",
                                                      "tokens", "parents"))
    assert int(torch.cuda.cudart().cudaStreamDestroy(handle.value)) == 0
    assert pa.pa_get_error_flags(clear=True) == 0

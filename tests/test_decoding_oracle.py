"""Pins of the oracle of rotary positions, beam selection and the pages of sequences, and
the host checks of their entry points (no GPU)."""

import ctypes
import itertools
import math

import numpy as np
import pytest
import torch

import oracle
from test_abi import pa  # noqa: F401  (builds and loads the library)


# ---------------------------------------------------------------- rotary positions

@pytest.mark.parametrize("interleaved", [False, True])
def test_rotate_is_a_complex_product(interleaved):
    rng = np.random.default_rng(1)
    x = rng.standard_normal((5, 3, 16))
    freq = np.array([1.0, 0.3, 0.01], np.float32)
    pos = np.array([0, 1, -7, 1000, 262143])
    y = oracle.rotate(x, pos, freq, interleaved, 1.5)
    for t, h, i in itertools.product(range(5), range(3), range(3)):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + 3)
        z = complex(x[t, h, a], x[t, h, b]) * 1.5 * np.exp(1j * float(freq[i]) * float(pos[t]))
        assert abs(complex(y[t, h, a], y[t, h, b]) - z) < 1e-11
    assert np.array_equal(y[..., 6:], x[..., 6:])


def test_rotated_products_depend_on_distance_alone():
    rng = np.random.default_rng(2)
    q, k = rng.standard_normal((2, 1, 1, 64))
    freq, _ = oracle.rotary_frequencies(64)
    dots = [float((oracle.rotate(q, [p + 11], freq) * oracle.rotate(k, [p], freq)).sum()) for p in (0, 3, 500, 40000)]
    assert np.ptp(dots) < 1e-9


def test_frequency_scalings():
    f, m = oracle.rotary_frequencies(8)
    assert np.allclose(f, [1, 0.1, 0.01, 0.001]) and m == 1.0
    assert np.allclose(oracle.rotary_frequencies(8, scaling="linear", factor=4)[0], f / 4)
    ntk = oracle.rotary_frequencies(8, scaling="ntk", factor=4)[0]
    assert ntk[0] == 1.0 and math.isclose(ntk[-1], f[-1] / 4)      # the last pair is stretched by the factor
    by, m = oracle.rotary_frequencies(8, scaling="by_parts", factor=4, original_max_position=2000)
    # turns over the trained range: 318, 31.8, 3.18, 0.318
    keep = (2000 * f / (2 * math.pi) - 1) / 31
    assert by[0] == f[0] and math.isclose(by[3], f[3] / 4)
    assert math.isclose(by[2], f[2] * keep[2] + f[2] / 4 * (1 - keep[2]))
    assert math.isclose(m, 1 + 0.1 * math.log(4))


@pytest.mark.parametrize("kw", [{}, {"base": 500000.0}, {"scaling": "linear", "factor": 8.0},
                                {"scaling": "ntk", "factor": 3.5},
                                {"scaling": "by_parts", "factor": 16.0, "original_max_position": 8192.0},
                                {"scaling": "by_parts", "factor": 8.0, "original_max_position": 8192.0,
                                 "low_turns": 1.0, "high_turns": 4.0, "base": 500000.0}])
@pytest.mark.parametrize("rot", [4, 64, 128])
def test_library_frequencies(pa, rot, kw):  # noqa: F811
    got, m = pa.pa_rotary_frequencies(rot, device="cpu", **kw)
    want, wm = oracle.rotary_frequencies(rot, **kw)
    # fp64 arithmetic of a few operations, then one rounding to fp32 (half a step)
    assert np.all(np.abs(got.double().numpy() - want) <= want * (2.0 ** -24 + 2.0 ** -45))
    assert math.isclose(m, wm, rel_tol=2.0 ** -23)


def test_library_frequency_refusals(pa):  # noqa: F811
    bad = [{"rotary_dim": 0}, {"rotary_dim": 7}, {"rotary_dim": 8, "base": 0.0}, {"rotary_dim": 8, "base": math.inf},
           {"rotary_dim": 8, "scaling": "linear", "factor": 0.5}, {"rotary_dim": 2, "scaling": "ntk", "factor": 2.0},
           {"rotary_dim": 8, "scaling": "by_parts", "factor": 2.0},
           {"rotary_dim": 8, "scaling": "by_parts", "factor": 2.0, "original_max_position": 4096.0, "low_turns": 3.0,
            "high_turns": 3.0}, {"rotary_dim": 8, "scaling": "linear", "factor": math.nan}]
    for kw in bad:
        with pytest.raises(pa.PAError) as e:
            pa.pa_rotary_frequencies(device="cpu", **kw)
        assert e.value.status == pa.PA_ERR_INVALID_ARG, kw
    with pytest.raises(ValueError):
        pa.pa_rotary_frequencies(8, scaling="cubic", device="cpu")


# ---------------------------------------------------------------- beam selection

def test_beam_select_against_a_full_sort():
    g = torch.Generator().manual_seed(3)
    x = torch.randn(6, 50, generator=g, dtype=torch.float64)
    cum = -torch.rand(2, 3, generator=g, dtype=torch.float64)
    scores, tokens, parents = oracle.beam_select(x.numpy(), cum.numpy(), 7)
    full = (cum.view(6, 1) + torch.log_softmax(x, -1)).view(2, 150)
    val, at = full.sort(dim=1, descending=True, stable=True)
    assert np.allclose(scores, val[:, :7].numpy(), atol=1e-12)
    assert np.array_equal(tokens, (at[:, :7] % 50).numpy())
    assert np.array_equal(parents, (at[:, :7] // 50 + torch.tensor([[0], [3]])).numpy())


def test_beam_select_ties_masks_and_missing():
    x = np.full((2, 5), -np.inf)
    x[0, [1, 3]] = 2.0                      # equal: the lower token first
    x[1, 4] = np.nan                        # a row with nothing to give
    s, t, p = oracle.beam_select(x, [[0.0, 0.0]], 4)
    assert t.tolist() == [[1, 3, -1, -1]] and p.tolist() == [[0, 0, -1, -1]]
    assert np.allclose(s[0, :2], -math.log(2)) and np.all(np.isneginf(s[0, 2:]))
    x = np.zeros((2, 3))
    s, t, p = oracle.beam_select(x, [[-np.inf, -1.0]], 2)  # an ended beam gives nothing
    assert t.tolist() == [[0, 1]] and p.tolist() == [[1, 1]]
    x[0, 2] = np.inf                        # as the largest finite value: all of the probability
    s, t, p = oracle.beam_select(x, [[-3.0, -1.0]], 1)
    assert t.tolist() == [[0]] and p.tolist() == [[1]]
    s, t, p = oracle.beam_select(x[:1], [[-3.0]], 1)
    assert s[0, 0] == -3.0 and t[0, 0] == 2
    lowest = float(np.finfo(np.float32).min)  # masked by the lowest value alone: still a distribution
    s, t, p = oracle.beam_select(np.full((1, 4), lowest), [[0.0]], 2)
    assert np.allclose(s, -math.log(4)) and t.tolist() == [[0, 1]]


# ---------------------------------------------------------------- pages

def test_pages_keep_their_books():
    """Random forks, appends and releases against dense histories: every row reads back the
    tokens it was given, counts equal the holders, and a free block has none."""
    rng = np.random.default_rng(5)
    bs, width, rows, pool = 4, 6, 5, 40
    refs = np.zeros(pool, np.int32)
    mem = np.full(pool * bs, -1)
    tables = np.full((rows, width), -1, np.int32)
    lens = np.zeros(rows, np.int32)
    dense = [[] for _ in range(rows)]
    token = 0
    for _ in range(300):
        op = rng.integers(3)
        if op == 0:
            add = np.minimum(rng.integers(0, 6, rows), width * bs - lens)
            qsl = np.concatenate([[0], np.cumsum(add)])
            got = oracle.append_blocks(tables, lens, qsl, refs, bs)
            if got is None:
                continue
            slots, pairs = got
            for src, dst in pairs:
                mem[dst * bs:(dst + 1) * bs] = mem[src * bs:(src + 1) * bs]
            at = 0
            for i in range(rows):
                for _ in range(add[i]):
                    mem[slots[at]] = token
                    dense[i].append(token)
                    token, at = token + 1, at + 1
        elif op == 1:
            parents = rng.integers(-1, rows, rows)
            t2, l2 = np.full_like(tables, -1), np.zeros_like(lens)
            oracle.fork_blocks(t2, l2, tables, lens, parents, refs, bs)
            oracle.release_blocks(tables, lens, refs, bs)
            tables, lens = t2, l2
            dense = [list(dense[p]) if p >= 0 else [] for p in parents]
        else:
            keep = rng.integers(0, width * bs, rows)
            oracle.release_blocks(tables, lens, refs, bs, keep)
            dense = [d[:k] for d, k in zip(dense, keep)]
        held = np.zeros(pool, np.int64)
        for i in range(rows):
            assert lens[i] == len(dense[i])
            n = -(-len(dense[i]) // bs)
            held[tables[i, :n]] += 1
            assert [mem[tables[i, p // bs] * bs + p % bs] for p in range(lens[i])] == dense[i]
        assert np.array_equal(held, refs)
    assert token > 500


# ---------------------------------------------------------------- host checks

def _fn(pa, name):  # noqa: F811
    fn = getattr(ctypes.CDLL(pa.LIB_PATH), name)
    fn.restype, fn.argtypes = pa.SIGNATURES[name]
    return fn


def _edited(args, edits):
    args = list(args)
    for i, v in edits.items():
        args[i] = v
    return args


FAKE = 1 << 20  # aligned, never dereferenced: the checks return first


def test_rotary_host_validation_without_a_gpu(pa):  # noqa: F811
    fn = _fn(pa, "pa_rotary_and_cache")
    # q_out q key value kc vc pos slots freq | T nb hq hkv d rot bs inter attn | strides | dtypes scales stream
    good = [FAKE] * 9 + [3, 10, 8, 2, 128, 64, 16, 0, 1.0, 1024, 1024, 256, 256, pa.PA_BF16, pa.PA_BF16, None, None,
                         None]
    bad, unsup = pa.PA_ERR_INVALID_ARG, pa.PA_ERR_UNSUPPORTED
    assert fn(*_edited(good, {9: 0})) == pa.PA_OK                              # nothing to do
    for edits, want in [({9: -1}, bad), ({10: 0}, bad), ({11: -1}, bad), ({12: 0}, bad), ({15: 0}, bad),
                        ({14: 0}, bad), ({14: 63}, bad), ({14: 130}, bad), ({17: 0.0}, bad),
                        ({17: math.inf}, bad), ({17: math.nan}, bad), ({17: -1.0}, bad), ({18: 1023}, bad),
                        ({19: 8}, bad), ({20: 0}, bad), ({21: -256}, bad), ({2: FAKE + 1}, bad), ({4: FAKE + 8}, bad),
                        ({0: FAKE + 1}, bad), ({22: pa.PA_FP8_E4M3}, unsup), ({23: pa.PA_F16}, unsup), ({23: 99}, unsup),
                        ({23: pa.PA_FP8_E4M3}, bad), ({23: pa.PA_NVFP4_PER_HEAD}, bad),
                        ({13: 68, 20: 1 << 20, 21: 1 << 20, 18: 1 << 20, 19: 1 << 20}, unsup),
                        ({13: 24, 14: 24, 23: pa.PA_FP8_E5M2, 24: FAKE, 25: FAKE}, unsup),
                        ({0: FAKE, 1: FAKE, 18: 2048}, bad)]:                  # in place with two strides
        assert fn(*_edited(good, edits)) == want, edits
    for i in range(9):
        assert fn(*_edited(good, {i: None})) == bad, i


def test_beam_host_validation_without_a_gpu(pa):  # noqa: F811
    fn = _fn(pa, "pa_beam_select")
    need = pa.pa_beam_select_workspace_size(2, 4, 1000, 8)
    assert need >= 256 and pa.pa_beam_select_workspace_size(0, 4, 1000, 8) == 256
    # scores tokens parents logits stride cum | B W V K dtype ws bytes stream
    good = [FAKE, FAKE, FAKE, FAKE, 1000, FAKE, 2, 4, 1000, 8, pa.PA_BF16, FAKE, need, None]
    bad, unsup = pa.PA_ERR_INVALID_ARG, pa.PA_ERR_UNSUPPORTED
    assert fn(*_edited(good, {6: 0})) == pa.PA_OK
    for edits, want in [({6: -1}, bad), ({7: 0}, bad), ({8: 0}, bad), ({9: 0}, bad), ({4: 999}, bad),
                        ({3: FAKE + 1}, bad), ({9: 33}, unsup), ({10: pa.PA_FP8_E4M3}, unsup),
                        ({6: 66, 7: 1024, 12: 1 << 40}, unsup), ({6: 1, 7: 1025, 12: 1 << 40}, unsup),
                        ({11: FAKE + 16}, pa.PA_ERR_WORKSPACE), ({12: need - 1}, pa.PA_ERR_WORKSPACE)]:
        assert fn(*_edited(good, edits)) == want, edits
    for i in (0, 1, 2, 3, 5, 11):
        assert fn(*_edited(good, {i: None})) == bad, i


def test_pages_host_validation_without_a_gpu(pa):  # noqa: F811
    bad = pa.PA_ERR_INVALID_ARG
    fork = _fn(pa, "pa_fork_blocks")
    far = FAKE + (1 << 16)
    # out_tables out_lens tables lens parents refs | children parents width blocks bs stream
    good = [FAKE, FAKE + 4096, far, far + 4096, far + 8192, FAKE, 4, 3, 8, 100, 16, None]
    assert fork(*_edited(good, {6: 0})) == pa.PA_OK
    for edits in ({6: -1}, {7: -1}, {8: 0}, {9: 0}, {10: 0}, {0: None}, {1: None}, {2: None}, {3: None}, {4: None},
                  {5: None}, {2: FAKE}, {2: FAKE + 4 * 8 * 4 - 4}, {3: FAKE + 4096}, {4: FAKE + 4096}, {4: FAKE + 8}):
        assert fork(*_edited(good, edits)) == bad, edits
    append = _fn(pa, "pa_append_blocks")
    need = pa.pa_append_workspace_size(4, 40, 16)
    assert need >= 256 and pa.pa_append_workspace_size(0, 0, 16) == 256
    # tables lens qsl slots pairs refs | rows total width blocks bs ws bytes stream
    good = [FAKE] * 6 + [4, 40, 8, 100, 16, FAKE, need, None]
    assert append(*_edited(good, {6: 0, 7: 0})) == pa.PA_OK
    for edits in ({6: -1}, {7: -1}, {8: 0}, {9: 0}, {10: 0}, {6: 0}, {0: None}, {1: None}, {2: None}, {3: None},
                  {4: None}, {5: None}, {11: None}):
        assert append(*_edited(good, edits)) == bad, edits
    assert append(*_edited(good, {6: 8193, 12: 1 << 30})) == pa.PA_ERR_UNSUPPORTED
    assert append(*_edited(good, {11: FAKE + 8})) == pa.PA_ERR_WORKSPACE
    assert append(*_edited(good, {12: need - 1})) == pa.PA_ERR_WORKSPACE
    release = _fn(pa, "pa_release_blocks")
    good = [FAKE, FAKE, None, FAKE, 4, 8, 100, 16, None]
    assert release(*_edited(good, {4: 0})) == pa.PA_OK
    for edits in ({4: -1}, {5: 0}, {6: 0}, {7: 0}, {0: None}, {1: None}, {3: None}):
        assert release(*_edited(good, edits)) == bad, edits


def test_outputs_over_inputs_are_refused(pa):  # noqa: F811
    bad, far = pa.PA_ERR_INVALID_ARG, [FAKE + (i << 24) for i in range(12)]
    rotary = _fn(pa, "pa_rotary_and_cache")
    # three tokens of 8 and 2 heads of 128 bf16, rows of 1536 elements
    row = 1536
    good = [far[0], far[1], far[2], far[3], far[4], far[5], far[6], far[7], far[8], 3, 10, 8, 2, 128, 64, 16, 0, 1.0,
            row, row, row, row, pa.PA_BF16, pa.PA_BF16, None, None, None]
    packed = {1: far[0], 2: far[0] + 2048, 3: far[0] + 2048 + 512}
    for edits in ({1: far[0] + 16}, {1: far[0] - 16}, {1: far[0] + 2 * row}, {2: far[0] + 2048 - 16},
                  {3: far[0] + 2 * row - 16}, {3: far[0] - 512 + 2}, {**packed, 0: far[0] + 1024},
                  {**packed, 0: far[0] + 2048},
                  {9: 1, 1: far[0] + 2046}, {9: 1, 2: far[0] - 510}):
        assert rotary(*_edited(good, edits)) == bad, edits
    beam = _fn(pa, "pa_beam_select")
    need = pa.pa_beam_select_workspace_size(2, 4, 1000, 8)
    good = [far[0], far[1], far[2], far[3], 1000, far[4], 2, 4, 1000, 8, pa.PA_BF16, far[5], need, None]
    for i in range(3):
        for at in (far[3], far[3] + 2 * 7999, far[4], far[4] + 28, far[5] + need - 4, far[3] - 63, far[4] - 60):
            assert beam(*_edited(good, {i: at})) == bad, (i, at)


def test_counts_past_32_bit_steps_are_refused(pa):  # noqa: F811
    unsup, most = pa.PA_ERR_UNSUPPORTED, 1 << 30
    far = [FAKE + (i << 50) for i in range(8)]
    assert _fn(pa, "pa_fork_blocks")(*far[:6], 4, 3, most + 1, 100, 16, None) == unsup
    append = _fn(pa, "pa_append_blocks")
    assert append(*far[:6], 4, most + 1, 8, 100, 16, far[6], 1 << 40, None) == unsup
    assert append(*far[:6], 4, 40, 8, most + 1, 16, far[6], 1 << 40, None) == unsup
    assert _fn(pa, "pa_release_blocks")(far[0], far[1], None, far[2], 4, most + 1, 100, 16, None) == unsup
    assert pa.pa_beam_select_workspace_size(1, 1, pa.PA_MAX_VOCAB + 1, 1) == 256
    assert _fn(pa, "pa_beam_select")(*far[:4], most + 1, far[4], 1, 1, pa.PA_MAX_VOCAB + 1, 8, pa.PA_BF16, far[5],
                                     1 << 40, None) == unsup
    freq = (ctypes.c_float * 2)()
    assert _fn(pa, "pa_rotary_frequencies")(freq, None, 4, 1e300, pa.ROTARY_SCALINGS["ntk"], 1e10, 0.0, 0.0,
                                            0.0) == pa.PA_ERR_INVALID_ARG


def test_bindings_refuse_wrong_tensors_on_the_cpu(pa):  # noqa: F811
    z = torch.zeros
    i32, i64 = torch.int32, torch.int64
    key = z(3, 2, 64)
    cache = z(4, 2, 16, 64)
    pos, slots, freq = z(3, dtype=i32), z(3, dtype=i64), z(32)
    with pytest.raises(ValueError, match="CUDA"):
        pa.pa_rotary_and_cache(z(3, 8, 64), z(3, 8, 64), key, key, cache, cache, pos, slots, freq)
    for args, kw in [((z(3, 8, 64), None, key, key, cache, cache, pos, slots, freq), {}),
                     ((z(3, 8, 64), z(3, 8, 32), key, key, cache, cache, pos, slots, freq), {}),
                     ((None, None, key.transpose(0, 1), key, cache, cache, pos, slots, freq), {}),
                     ((None, None, key, z(3, 2, 32), cache, cache, pos, slots, freq), {}),
                     ((None, None, key, key, cache, cache, slots, slots, freq), {}),
                     ((None, None, key, key, cache, cache, pos, pos, freq), {}),
                     ((None, None, key, key, cache, cache, pos, slots, freq.double()), {}),
                     ((None, None, key, key, cache, cache, z(2, dtype=i32), slots, freq), {})]:
        with pytest.raises(ValueError):
            pa.pa_rotary_and_cache(*args, **kw)
    out = (z(2, 4), z(2, 4, dtype=i32), z(2, 4, dtype=i32))
    ws = z(256, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):
        pa.pa_beam_select(*out, z(6, 50), z(2, 3), ws)
    for bad_logits in (z(5, 50), z(6, 50, 1), z(50, 6).t()):
        with pytest.raises(ValueError):
            pa.pa_beam_select(*out, bad_logits, z(2, 3), ws)
    with pytest.raises(ValueError):
        pa.pa_beam_select(out[0], out[0], out[2], z(6, 50), z(2, 3), ws)
    with pytest.raises(ValueError):
        pa.pa_beam_select(*out, z(6, 50), z(2, 3, dtype=torch.float64), ws)
    tables, lens, refs = z(2, 5, dtype=i32), z(2, dtype=i32), z(9, dtype=i32)
    with pytest.raises(ValueError, match="CUDA"):
        pa.pa_release_blocks(tables, lens, refs, 16)
    for call in (lambda: pa.pa_release_blocks(tables.long(), lens, refs, 16),
                 lambda: pa.pa_release_blocks(tables, lens, refs, 16, keep_lens=z(3, dtype=i32)),
                 lambda: pa.pa_fork_blocks(z(4, 6, dtype=i32), z(4, dtype=i32), tables, lens, z(4, dtype=i32), refs, 16),
                 lambda: pa.pa_fork_blocks(z(4, 5, dtype=i32), z(4, dtype=i32), tables, lens, z(4, dtype=i64), refs, 16),
                 lambda: pa.pa_append_blocks(tables, lens, z(2, dtype=i32), z(1, dtype=i64), z(2, 2, dtype=i64), refs,
                                             16, ws),
                 lambda: pa.pa_append_blocks(tables, lens, z(3, dtype=i32), z(1, dtype=i32), z(2, 2, dtype=i64), refs,
                                             16, ws)):
        with pytest.raises(ValueError):
            call()

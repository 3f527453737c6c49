"""CPU: positions of media against hand-written ones, rotation on several axes against the one-axis
oracle, and what pa_rotary_pair_axes, pa_rotary_axes_and_cache and pa_positions_and_slots refuse."""

import ctypes

import numpy as np
import pytest

import oracle


@pytest.fixture(scope="module")
def pa():
    import __graft_entry__ as g
    g.build()
    import paged_kv_cache_pagedattention_gb300 as lib
    return lib


def test_positions_by_hand():
    # two words, an image of 2 x 3, a word, a clip of 2 frames of 1 x 2 three positions apart, a word
    want = np.array([[0, 1, 2, 2, 2, 2, 2, 2, 5, 6, 6, 9, 9, 10],
                     [0, 1, 2, 2, 2, 3, 3, 3, 5, 6, 6, 6, 6, 10],
                     [0, 1, 2, 3, 4, 2, 3, 4, 5, 6, 7, 6, 7, 10]])
    media = [(2, 1, 2, 3, 1), (9, 2, 1, 2, 3)]
    assert np.array_equal(oracle.sequence_positions(14, media), want)
    for n in range(14):  # a prefix's positions do not depend on what follows
        assert np.array_equal(oracle.sequence_positions(n, media), want[:, :n])
    pos, slots = oracle.positions_and_slots([0, 3, 4], [14, 2], [[7, 3, 9, 1], [4, 0, 0, 0]], 4, [media, []])
    assert np.array_equal(pos, np.concatenate([want[:, 11:], [[1]] * 3], 1))
    assert slots.tolist() == [9 * 4 + 3, 1 * 4, 1 * 4 + 1, 4 * 4 + 1]


@pytest.mark.parametrize("interleaved", [False, True])
def test_equal_axes_are_one_axis(interleaved):
    rng = np.random.default_rng(3)
    x, pos = rng.normal(size=(5, 2, 16)), rng.integers(0, 999, 5)
    freq = oracle.rotary_frequencies(12)[0]
    axes = rng.integers(0, 3, 6)
    got = oracle.rotate_axes(x, np.tile(pos, (3, 1)), freq, axes, interleaved, 1.5)
    assert np.allclose(got, oracle.rotate(x, pos, freq, interleaved, 1.5), rtol=0, atol=1e-14)


def test_pair_axes(pa):
    assert list(pa.pa_rotary_pair_axes([2, 3, 1])) == [0, 0, 1, 1, 1, 2]
    assert list(pa.pa_rotary_pair_axes([0, 2])) == [1, 1]
    assert list(pa.pa_rotary_pair_axes([4])) == [0] * 4
    assert list(pa.pa_rotary_pair_axes([4, 2, 2], cycled=True)) == [0, 1, 2, 0, 1, 2, 0, 0]
    assert list(pa.pa_rotary_pair_axes([24, 20, 20], cycled=True)) == [i % 3 if i < 60 else 0 for i in range(64)]
    assert len(pa.pa_rotary_pair_axes([256])) == 256
    for sections in ([], [0], [257], [3, -1]):
        with pytest.raises((ValueError, pa.PAError)):
            pa.pa_rotary_pair_axes(sections)
    with pytest.raises(pa.PAError):
        pa.pa_rotary_pair_axes([1, 5, 2], cycled=True)     # dealt round, axis 1 cannot have five of eight
    with pytest.raises(pa.PAError):
        pa.pa_rotary_pair_axes([1] * 5)                    # five axes
    two = (ctypes.c_int32 * 2)(2, 1)
    out = (ctypes.c_uint8 * 4)()
    lib = pa._lib
    assert lib.pa_rotary_pair_axes(out, 8, two, 2, 0) == pa.PA_ERR_INVALID_ARG    # three of four pairs
    assert lib.pa_rotary_pair_axes(out, 7, two, 2, 0) == pa.PA_ERR_INVALID_ARG
    assert lib.pa_rotary_pair_axes(None, 6, two, 2, 0) == pa.PA_ERR_INVALID_ARG
    assert lib.pa_rotary_pair_axes(out, 514, two, 2, 0) == pa.PA_ERR_UNSUPPORTED
    assert list(out) == [0] * 4                            # a refused call writes nothing


def test_rotary_axes_refusals(pa):
    fn, f = pa._lib.pa_rotary_axes_and_cache, 1 << 20  # an aligned address that no refused call touches

    def call(axes=bytes(64), num_axes=3, tokens=4, rot=128, q_out=1 << 26):
        return fn(q_out, f, f + (1 << 16), f + (1 << 17), f, f, f, f, f, axes, num_axes, tokens, 9, 8, 2, 128, rot, 16,
                  0, 1.0, 1024, 1024, 256, 256, pa.PA_BF16, pa.PA_BF16, None, None, None)

    assert call(tokens=0) == pa.PA_OK
    assert call(axes=None) == pa.PA_ERR_INVALID_ARG
    assert call(axes=bytes(63) + b"\x03") == pa.PA_ERR_INVALID_ARG     # an axis that is not there
    assert call(num_axes=0) == pa.PA_ERR_INVALID_ARG
    assert call(num_axes=5) == pa.PA_ERR_UNSUPPORTED
    assert call(rot=514) == pa.PA_ERR_UNSUPPORTED
    assert call(rot=130) == pa.PA_ERR_INVALID_ARG                      # what the one-axis call refuses: wider than the head
    assert call(rot=127) == pa.PA_ERR_INVALID_ARG
    assert call(tokens=-1) == pa.PA_ERR_INVALID_ARG


def test_positions_refusals(pa):
    fn, f = pa._lib.pa_positions_and_slots, 1 << 20

    def call(pos=f, slots=f + (1 << 12), qsl=f + (2 << 12), lens=f + (3 << 12), tables=f + (4 << 12), ms=f + (5 << 12),
             media=f + (6 << 12), n=4, total=9, axes=3, records=2, width=8, blocks=9, bs=16):
        return fn(pos, slots, qsl, lens, tables, ms, media, n, total, axes, records, width, blocks, bs, None)

    bad, no = pa.PA_ERR_INVALID_ARG, pa.PA_ERR_UNSUPPORTED
    assert call(n=0, total=0) == call(total=0) == pa.PA_OK
    assert call(n=0) == call(n=-1) == call(total=-1) == call(records=-1) == bad
    assert call(axes=2) == call(axes=0) == call(total=(1 << 30) + 1) == call(n=(1 << 30) + 1) == no
    assert call(axes=1) == call(axes=1, records=0) == bad              # media have three axes
    assert call(pos=None, slots=None) == call(qsl=None) == call(lens=None) == call(tables=None) == bad
    assert call(width=0) == call(blocks=0) == call(bs=0) == bad
    assert call(ms=None) == call(media=None) == bad
    for read in ("qsl", "lens", "tables", "ms", "media"):              # results over what is still read
        assert call(**{read: f + 8}) == bad and call(**{read: f + (1 << 12) + 16}) == bad, read
    assert call(slots=f + 64) == bad


def test_binding_refusals(pa):
    import torch
    i32 = dict(dtype=torch.int32)
    lens, qsl, pos = torch.zeros(2, **i32), torch.zeros(3, **i32), torch.zeros(3, 4, **i32)
    slots, tables = torch.zeros(4, dtype=torch.int64), torch.zeros(2, 5, **i32)
    ms, media = torch.zeros(3, **i32), torch.zeros(2, 5, **i32)
    good = [pos, slots, qsl, lens, tables, 9, 16, ms, media]
    for i, wrong in ((0, pos.long()), (0, pos[:, ::2]), (0, torch.zeros(3, 5, **i32)), (0, torch.zeros(1, 1, 4, **i32)),
                     (1, slots.int()), (1, slots[::2]), (2, qsl[:2]), (3, lens.long()), (4, tables[:1]), (4, None),
                     (7, None), (7, ms[:2]), (8, None), (8, media[:, :4]), (8, media.long())):
        args = list(good)
        args[i] = wrong
        with pytest.raises(ValueError):
            pa.pa_positions_and_slots(*args)
    with pytest.raises(ValueError):
        pa.pa_positions_and_slots(*good)                               # not on a CUDA device
    row = torch.zeros(4, 2, 64)
    cache = torch.zeros(3, 2, 16, 64)
    freq = torch.ones(32)
    for axes, where in ((None, pos), ([0] * 32, pos), (bytes(31), pos), (bytes(32), pos[0]), (bytes(32), pos[:, :3])):
        with pytest.raises(ValueError):
            pa.pa_rotary_axes_and_cache(row, row.clone(), row, row, cache, cache.clone(), where, slots, freq, axes)

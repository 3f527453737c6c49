"""GPU: positions and slots of sequences with media (whole numbers: equal to the oracle's), and the
rotary write on several axes: bit for bit the one-axis write's element of the pair's axis, and near
the fp64 rotation by roundings alone.
"""

import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
I32 = dict(dtype=torch.int32, device=DEV)


@pytest.fixture(scope="module")
def pa():
    import paged_kv_cache_pagedattention_gb300 as lib
    lib.pa_get_error_flags(clear=True)
    return lib


# ---------------------------------------------------------------- positions and slots


def grids(rng, length, most, side=6):
    """Up to ``most`` media in ascending order; the last ones may lie behind the sequence's end."""
    media, at = [], int(rng.integers(0, 4))
    for _ in range(most):
        m = (at, int(rng.integers(1, 4)), int(rng.integers(1, side)), int(rng.integers(1, side)),
             int(rng.integers(0, 4)))
        media.append(m)
        at += m[1] * m[2] * m[3] + int(rng.choice([0, 0, 1, 5]))
        if at > length + 30:
            break
    return media


class Step:
    def __init__(self, lens, new, most, bs=16, seed=0, side=6):
        rng = np.random.default_rng(seed)
        self.lens, self.bs = np.array(lens, np.int32), bs
        self.qsl = np.concatenate(([0], np.cumsum(new))).astype(np.int32)
        self.width = -(-max(list(lens) + [1]) // bs) + 1
        self.nb = len(lens) * self.width + 2
        self.tables = rng.permutation(self.nb)[:len(lens) * self.width].reshape(len(lens), -1).astype(np.int32)
        self.media = [grids(rng, n, int(rng.integers(0, most + 1)), side) for n in lens]

    def call(self, pa, axes=3, slots=True, positions=True, stream=None):
        t = int(self.qsl[-1])
        flat = [m for one in self.media for m in one]
        dev = lambda x: torch.tensor(np.asarray(x), **I32)  # noqa: E731
        self.pos = torch.full((3, t) if axes == 3 else (t,), -7, **I32) if positions else None
        self.slots = torch.full((t,), -7, dtype=torch.int64, device=DEV) if slots else None
        starts = dev(np.concatenate(([0], np.cumsum([len(m) for m in self.media]))).astype(np.int32))
        media = dev(np.array(flat, np.int32).reshape(-1, 5))
        self.args = [self.pos, self.slots, dev(self.qsl), dev(self.lens), dev(self.tables) if slots else None, self.nb,
                     self.bs, starts if axes == 3 else None, media if axes == 3 else None]
        pa.pa_positions_and_slots(*self.args, stream=stream)
        torch.cuda.synchronize()

    def check(self):
        pos, slots = oracle.positions_and_slots(self.qsl, self.lens, self.tables, self.bs, self.media)
        if self.pos is not None:
            assert np.array_equal(self.pos.cpu().numpy(), pos if self.pos.dim() == 2 else pos[0])
        if self.slots is not None:
            assert np.array_equal(self.slots.cpu().numpy(), slots)


@pytest.mark.parametrize("bs", [1, 16, 48])
@pytest.mark.parametrize("most", [0, 1, 3, 31, 32, 33, 64, 200])
def test_positions_parity(pa, most, bs):
    lens = [1, 2, 700, 129, 128, 127, 33, 1500, 400, 1]
    new = [1, 0, 700, 129, 1, 127, 32, 300, 257, 1]   # whole prompts, chunks, decodes, and one that rests
    s = Step(lens, new, most, bs, seed=most + bs)
    s.call(pa)
    assert pa.pa_get_error_flags(clear=True) == 0
    s.check()


@pytest.mark.parametrize("n", [1, 5, 300, 5000])
def test_positions_of_decodes(pa, n):
    rng = np.random.default_rng(n)
    s = Step(rng.integers(1, 260, n), [1] * n, 9, seed=n)
    s.call(pa)
    s.check()


def test_positions_of_long_media(pa):
    s = Step([5000, 4000], [5000, 1], 0, seed=5)
    s.media = [[(0, 1, 1, 1, 0), (1, 40, 10, 10, 2), (4003, 1, 9, 9, 1)], [(10, 1, 60, 60, 1), (3999, 1, 1, 1, 9)]]
    s.call(pa)
    s.check()


def test_text_alone_and_parts_of_the_call(pa):
    s = Step([300, 20, 64], [130, 20, 1], 0, seed=6)
    s.call(pa, axes=1)
    s.check()
    s = Step([300, 20, 64], [130, 20, 1], 7, seed=6)
    s.call(pa, slots=False)
    s.check()
    s.call(pa, positions=False)
    s.check()
    assert pa.pa_get_error_flags(clear=True) == 0


def test_positions_up_to_31_bits(pa):
    """Far text behind media, without slots; a position that would pass 2^31 - 1 is refused."""
    top = 2 ** 31 - 1
    s = Step([20, 20], [2, 2], 0, seed=7)
    s.lens[:] = [top, 100]
    s.media = [[(5, 10, 100, 100, 1)], [(3, 2, 1, 1, top - 10)]]
    s.call(pa, slots=False)
    far = 5 + 100 + (top - 5 - 100000)                # the image's 100,000 tokens take 100 positions
    got = s.pos.cpu().numpy()
    assert np.array_equal(got[:, :2], np.tile([far - 2, far - 1], (3, 1))) and not got[:, 2:].any()
    assert pa.pa_get_error_flags(clear=True) == pa.PA_ERRFLAG_MEDIA


@pytest.mark.parametrize("wrong", [(5, 0, 2, 2, 1), (5, 1, -1, 2, 1), (5, 1, 2, 2, -1), (-1, 1, 2, 2, 1),
                                   (1, 1, 1, 1, 1), (5, 2 ** 20, 2 ** 20, 1, 0), (5, 1, 2 ** 31 - 1, 2 ** 31 - 1, 1),
                                   (5, 2 ** 31 - 1, 1, 1, 2 ** 31 - 1), (2 ** 31 - 1, 1, 1, 1, 1)])
def test_a_malformed_medium(pa, wrong):
    """Every token of its sequence gets slot -1 and position 0; the others are placed."""
    s = Step([200, 200, 40], [200, 1, 40], 3, seed=8)
    s.media[0] = [(0, 1, 2, 2, 1)] + s.media[0][:0] + [wrong]
    s.call(pa)
    assert pa.pa_get_error_flags(clear=True) == pa.PA_ERRFLAG_MEDIA
    assert bool((s.slots[:200] == -1).all()) and not bool(s.pos[:, :200].any())
    bad, s.media[0] = s.media[0], []
    pos, slots = oracle.positions_and_slots(s.qsl, s.lens, s.tables, s.bs, s.media)
    assert np.array_equal(s.pos.cpu().numpy()[:, 200:], pos[:, 200:])
    assert np.array_equal(s.slots.cpu().numpy()[200:], slots[200:])


def test_malformed_requests(pa):
    s = Step([50, 60, 70, 80], [50, 10, 1, 5], 2, seed=9)
    s.lens[1] = 9                                     # ten new tokens of nine
    s.lens[2] = s.width * s.bs + 1                    # longer than its table
    s.tables[3, 4] = s.nb                             # tokens 64 .. 79 lie there
    s.call(pa)
    assert pa.pa_get_error_flags(clear=True) == pa.PA_ERRFLAG_QUERY | pa.PA_ERRFLAG_SEQ_LEN | \
        pa.PA_ERRFLAG_BLOCK_TABLE
    assert bool((s.slots[50:66] == -1).all()) and not bool(s.pos[:, 50:61].any())
    want = oracle.sequence_positions(80, s.media[3])[:, 75:]
    assert np.array_equal(s.pos[:, 61:].cpu().numpy(), want)
    for start, end in ((1, 66), (0, 65)):             # does not run from 0 to the tokens' number
        s.args[2].copy_(torch.tensor([start, 50, 60, 61, end], **I32))
        s.args[1].fill_(5), s.args[0].fill_(5)
        pa.pa_positions_and_slots(*s.args)
        assert pa.pa_get_error_flags(clear=True) == pa.PA_ERRFLAG_QUERY
        assert bool((s.slots == -1).all()) and not bool(s.pos.any())
    s.args[2].copy_(torch.tensor([0, 50, 40, 61, 66], **I32))
    pa.pa_positions_and_slots(*s.args)
    assert pa.pa_get_error_flags(clear=True) == pa.PA_ERRFLAG_QUERY and bool((s.slots == -1).all())
    s.args[7][1] = 10 ** 6                            # a sequence's media end outside the records
    s.args[2].copy_(torch.tensor([0, 50, 60, 61, 66], **I32))
    pa.pa_positions_and_slots(*s.args)
    assert pa.pa_get_error_flags(clear=True) & pa.PA_ERRFLAG_MEDIA and bool((s.slots[:50] == -1).all())


def test_slots_are_those_append_gave(pa):
    """Append hands out blocks and writes slots; from its tables and lengths the same slots follow."""
    lens, new, bs = [0, 5, 16, 31], [20, 3, 1, 40], 16
    tables = torch.zeros(4, 6, **I32)
    refs = torch.zeros(40, **I32)
    for i, n in enumerate(lens):
        for j in range(-(-n // bs)):
            tables[i, j] = 4 * i + j
            refs[4 * i + j] = 1
    seq_lens, qsl = torch.tensor(lens, **I32), torch.tensor(np.concatenate(([0], np.cumsum(new))), **I32)
    slots = torch.zeros(sum(new), dtype=torch.int64, device=DEV)
    pairs = torch.zeros(4, 2, dtype=torch.int64, device=DEV)
    ws = pa.workspace_tensor(pa.pa_append_workspace_size(4, sum(new), bs))
    pa.pa_append_blocks(tables, seq_lens, qsl, slots, pairs, refs, bs, ws)
    again, pos = torch.zeros_like(slots), torch.zeros(sum(new), **I32)
    pa.pa_positions_and_slots(pos, again, qsl, seq_lens, tables, 40, bs)
    assert torch.equal(slots, again)
    assert pos.tolist() == [n + j for n, m in zip(lens, new) for j in range(m)]


# ---------------------------------------------------------------- the rotary write on several axes

HALF_STEP = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}


class Write:
    def __init__(self, t, hq, hkv, d, rot, src, cache, bs=16, axes=3, seed=0, far=5000, gap=0):
        gen = torch.Generator(device=DEV).manual_seed(seed)
        rows = torch.randn(t, (hq + 2 * hkv) * d + gap, device=DEV, generator=gen).to(src)
        self.q, self.key, self.value = (rows[:, a * d:b * d].unflatten(1, (b - a, d)) for a, b in
                                        ((0, hq), (hq, hq + hkv), (hq + hkv, hq + 2 * hkv)))
        nb = 2 * t // bs + 3
        if cache == "nvfp4":
            self.kc = torch.zeros(nb, hkv, 9 * bs * d // 16, dtype=torch.uint8, device=DEV)
        else:
            self.kc = torch.zeros(nb, hkv, bs, d, device=DEV).to(cache)
        self.vc = self.kc.clone()
        scaled = self.kc.element_size() == 1
        self.scale = torch.full((1,), 2.0 ** -6, device=DEV) if scaled else None
        self.pos = torch.randint(-far, far, (axes, t), generator=gen, **I32)
        self.slots = torch.randperm(nb * bs, device=DEV, generator=gen)[:t]
        self.slots[::5] = -1
        self.freq = torch.from_numpy(oracle.rotary_frequencies(rot)[0].astype(np.float32)).to(DEV)
        self.rot, self.bs = rot, bs

    def run(self, pa, interleaved, pair_axis=None, axis=None, stream=None):
        """(q_out, k_cache, v_cache) of the several-axes call, or of the one-axis call on one axis."""
        out = torch.full(self.q.shape, 3.0, dtype=self.q.dtype, device=DEV)
        kc, vc = self.kc.clone(), self.vc.clone()
        if pair_axis is not None:
            pa.pa_rotary_axes_and_cache(out, self.q, self.key, self.value, kc, vc, self.pos, self.slots, self.freq,
                                        pair_axis, interleaved, 1.25, self.scale, self.scale, stream)
        else:
            pa.pa_rotary_and_cache(out, self.q, self.key, self.value, kc, vc, self.pos[axis].contiguous(), self.slots,
                                   self.freq, interleaved, 1.25, self.scale, self.scale, stream)
        torch.cuda.synchronize()
        return out, kc, vc


B, H, F, E4, E5 = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn, torch.float8_e5m2
WRITES = [  # tokens, q heads, kv heads, head, rotated, source, cache, block, axes, gap
    (1, 28, 4, 128, 128, B, B, 16, 3, 0),
    (37, 32, 8, 128, 128, B, B, 16, 3, 0),
    (300, 16, 2, 128, 64, H, H, 32, 4, 0),
    (21, 8, 2, 64, 32, F, F, 16, 2, 0),
    (19, 8, 2, 96, 24, H, H, 16, 3, 1),       # no whole pieces: the kernel for any rows
    (65, 8, 4, 128, 128, B, E4, 32, 3, 0),
    (12, 8, 2, 160, 40, H, E5, 16, 3, 0),
    (9, 4, 2, 256, 256, F, F, 16, 1, 0),
    (5, 2, 1, 512, 512, B, B, 16, 4, 0),      # the most pairs
]


@pytest.mark.parametrize("interleaved", [False, True], ids=["half", "interleaved"])
@pytest.mark.parametrize("shape", WRITES, ids=lambda s: "-".join(str(x).split(".")[-1] for x in s))
def test_every_pair_turns_on_its_axis(pa, shape, interleaved):
    t, hq, hkv, d, rot, src, cache, bs, axes, gap = shape
    w = Write(t, hq, hkv, d, rot, src, cache, bs, axes, seed=t, gap=gap)
    rng = np.random.default_rng(t)
    pair_axis = bytes(rng.integers(0, axes, rot // 2).tolist())
    out, kc, vc = w.run(pa, interleaved, pair_axis)
    assert pa.pa_get_error_flags(clear=True) == 0
    # element j belongs to pair i: the one-axis call's value on that pair's axis, bit for bit
    element = torch.full((d,), 0, device=DEV)
    for i, a in enumerate(pair_axis):
        for j in (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2):
            element[j] = a
    parts = [w.run(pa, interleaved, axis=a) for a in range(axes)]
    for a, (o, k, v) in enumerate(parts):
        mine = element == a
        assert torch.equal(out[..., mine], o[..., mine])
        assert torch.equal(kc.view(torch.uint8 if kc.element_size() == 1 else kc.dtype)[..., mine],
                           k.view(torch.uint8 if kc.element_size() == 1 else kc.dtype)[..., mine])
    assert torch.equal(vc.view(torch.uint8), parts[0][2].view(torch.uint8))
    assert bool((out[w.slots < 0] == 3.0).all())
    # and the fp64 rotation: cos and sin off by 2^-21 together at most (see the one-axis tests), |theta| 2^-52 far
    # below it here, then half a step of the type
    x = w.q.double().cpu().numpy()
    want = oracle.rotate_axes(x, w.pos.cpu().numpy(), w.freq.cpu().numpy(), pair_axis, interleaved, 1.25)
    live = (w.slots >= 0).cpu().numpy()
    e = 2 * np.abs(x).max() * 1.25 * 2.0 ** -21
    off = np.abs(out.double().cpu().numpy() - want)[live]
    assert np.all(off <= HALF_STEP[src] * (np.abs(want[live]) + e) + 2.0 ** -25 + e)


@pytest.mark.parametrize("src,cache,rot", [(B, "nvfp4", 128), (F, "nvfp4", 32), (H, E4, 128), (B, B, 24)])
def test_equal_axes_are_the_one_axis_call(pa, src, cache, rot):
    w = Write(70, 8, 2, 128, rot, src, cache, seed=4)
    w.pos[1:] = w.pos[0]
    for interleaved in (False, True):
        got = w.run(pa, interleaved, pa.pa_rotary_pair_axes([rot // 2 - 2 * (rot // 8), rot // 8, rot // 8]))
        for a, b in zip(got, w.run(pa, interleaved, axis=0)):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_a_step_of_text_and_images(pa):
    """Positions and slots, then the rotary write that reads them, in a graph replayed as the lengths
    grow: what the eager calls give, and the oracle's rows at the oracle's slots."""
    s = Step([40, 90, 33], [40, 1, 9], 5, seed=12)
    s.call(pa)
    t = int(s.qsl[-1])
    w = Write(t, 8, 2, 128, 128, B, B, seed=12)
    kc = torch.zeros(s.nb, 2, 16, 128, dtype=B, device=DEV)
    vc, out = torch.zeros_like(kc), torch.zeros_like(w.q)
    axes = pa.pa_rotary_pair_axes([16, 24, 24])

    def step():
        pa.pa_positions_and_slots(*s.args)
        pa.pa_rotary_axes_and_cache(out, w.q, w.key, w.value, kc, vc, s.args[0], s.args[1], w.freq, axes)

    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        step()
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for grow in (0, 1):
        s.lens += grow
        s.args[3].add_(grow)                          # a decode further on: the replay reads the lengths of its time
        kc.zero_(), vc.zero_(), out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        s.check()
        slots = s.slots
        key = oracle.rotate_axes(w.key.double().cpu().numpy(), s.pos.cpu().numpy(), w.freq.cpu().numpy(), axes)
        got = kc[slots // 16, :, slots % 16].double().cpu().numpy()
        e = 2 * np.abs(key).max() * 2.0 ** -20
        assert np.all(np.abs(got - key) <= 2.0 ** -8 * (np.abs(key) + e) + e)
        assert torch.equal(vc[slots // 16, :, slots % 16], w.value)
    assert pa.pa_get_error_flags(clear=True) == 0


def test_several_axes_behind_slots_out_of_range(pa):
    w = Write(20, 8, 2, 128, 128, B, B, seed=13)
    w.slots[3] = 10 ** 9
    out, kc, _ = w.run(pa, False, pa.pa_rotary_pair_axes([16, 24, 24]))
    assert pa.pa_get_error_flags(clear=True) == pa.PA_ERRFLAG_SLOT
    assert bool((out[3] == 3.0).all())

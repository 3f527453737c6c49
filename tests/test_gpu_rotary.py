"""GPU parity of pa_rotary_and_cache against the fp64 oracle: element types, cache formats,
both pair layouts, partial heads, odd sizes and alignments, far positions, padding, bad
slots, in-place q, another stream, graph capture.

Tolerances count roundings.  With x, y the pair's values, m the factor and theta the angle:
cos and sin are each off by at most 2^-22 (the angle's turn is held to 2^-32 and rounded to
fp32 within an eighth of a turn: 2^-24; sincospi: 2 units of 2^-24; product with m: half a
unit) plus |theta| 2^-52 (the frequency's turn is rounded once to fp64), so a rotated value is
off by E = (|x| + |y|) m (2^-21 + |theta| 2^-52) before it is stored, three fp32 operations
included; storing adds half a step of the element type.
"""

import numpy as np
import pytest
import torch

import oracle
import workloads

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
HALF_STEP = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8, "fp8_e4m3": 2.0 ** -4, "fp8_e5m2": 2.0 ** -3}
# half of the smallest subnormal's step
TINY = {"f32": 2.0 ** -150, "f16": 2.0 ** -25, "bf16": 2.0 ** -134, "fp8_e4m3": 2.0 ** -10, "fp8_e5m2": 2.0 ** -17}


@pytest.fixture(scope="module")
def pa():
    import paged_kv_cache_pagedattention_gb300 as lib
    lib.pa_get_error_flags(clear=True)
    return lib


class Case:
    def __init__(self, t, hq, hkv, d, rot, src, kv, bs=16, seed=0, far=4096, per_head=False, gap=0, shift=0,
                 negative=False):
        rng = np.random.default_rng(seed)
        self.t, self.hq, self.hkv, self.d, self.rot, self.src, self.kv, self.bs = t, hq, hkv, d, rot, src, kv, bs
        width = (hq + 2 * hkv) * d + gap
        # one projection; `shift` elements of offset and an odd row length break 16-byte alignment
        bits = workloads.normal_bits(rng, (t * width + shift,), src)
        flat = workloads.bits_to_torch(bits, src, DEV)[shift:]
        rows = flat.view(t, width)
        self.q = rows[:, :hq * d].unflatten(1, (hq, d)) if hq else None
        self.key = rows[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d))
        self.value = rows[:, (hq + hkv) * d:(hq + 2 * hkv) * d].unflatten(1, (hkv, d))
        x = oracle.decode_bits(bits[shift:], src).reshape(t, width)
        self.q64 = x[:, :hq * d].reshape(t, hq, d)
        self.k64 = x[:, hq * d:(hq + hkv) * d].reshape(t, hkv, d)
        self.v64 = x[:, (hq + hkv) * d:(hq + 2 * hkv) * d].reshape(t, hkv, d)
        nb = 2 * t // bs + 3
        self.nb = nb
        self.scaled = kv in workloads.SCALED
        self.k_scale = np.float32(2.0 ** -5) if self.scaled else None
        self.v_scale = np.float32(0.03) if self.scaled else None
        if self.scaled and per_head:
            self.k_scale = (0.02 + 0.01 * np.arange(hkv)).astype(np.float32)
            self.v_scale = self.k_scale[::-1].copy()
        if kv == "nvfp4":
            self.kb = workloads.nvfp4_random_cache(rng, nb, hkv, bs, d)
            self.vb = workloads.nvfp4_random_cache(rng, nb, hkv, bs, d)
        else:
            self.kb = workloads.normal_bits(rng, (nb, hkv, bs, d), kv)
            self.vb = workloads.normal_bits(rng, (nb, hkv, bs, d), kv)
        self.slots = rng.permutation(nb * bs)[:t].astype(np.int64)
        self.pos = rng.integers(-far if negative else 0, far, t).astype(np.int32)
        self.freq = oracle.rotary_frequencies(rot)[0].astype(np.float32)

    def to_device(self):
        self.kc = workloads.bits_to_torch(self.kb, self.kv, DEV)
        self.vc = workloads.bits_to_torch(self.vb, self.kv, DEV)
        self.q_out = torch.full((self.t, self.hq, self.d), 7.0, dtype=self.key.dtype, device=DEV) if self.hq else None
        sc = lambda s: None if s is None else torch.tensor(np.atleast_1d(s), device=DEV)  # noqa: E731
        self.ks, self.vs = sc(self.k_scale), sc(self.v_scale)
        self.dev_pos = torch.from_numpy(self.pos).to(DEV)
        self.dev_slots = torch.from_numpy(self.slots).to(DEV)
        self.dev_freq = torch.from_numpy(self.freq).to(DEV)

    def call(self, pa, interleaved, attn=1.0, stream=None, in_place=False):
        self.to_device()
        pa.pa_rotary_and_cache(self.q if in_place else self.q_out, self.q, self.key, self.value, self.kc, self.vc,
                               self.dev_pos, self.dev_slots, self.dev_freq, interleaved, attn, self.ks, self.vs,
                               stream)
        torch.cuda.synchronize()

    def check(self, interleaved, attn=1.0, q=None):
        live = (self.slots >= 0) & (self.slots < self.nb * self.bs)
        theta = np.abs(np.outer(self.pos.astype(np.float64), self.freq.astype(np.float64)))[:, None, :]
        half = self.rot // 2
        a, b = (slice(0, self.rot, 2), slice(1, self.rot, 2)) if interleaved else (slice(0, half),
                                                                                   slice(half, self.rot))

        def error(x):
            e = np.zeros_like(x)
            e[..., a] = e[..., b] = (np.abs(x[..., a]) + np.abs(x[..., b])) * attn * (2.0 ** -21 + theta * 2.0 ** -52)
            return e

        def near(got, x, where):
            want, e = oracle.rotate(x, self.pos, self.freq, interleaved, attn), error(x)
            tol = np.maximum(HALF_STEP[self.src] * (np.abs(want) + e), TINY[self.src]) + e
            off = np.abs(got - want)[live]
            assert np.all(off <= tol[live]), (where, float((off / tol[live]).max()))

        if self.hq:
            q = self.q_out if q is None else q
            got = oracle.decode_bits(workloads.torch_to_bits(q, self.src), self.src)
            near(got, self.q64, "q")
            assert np.array_equal(got[live][..., self.rot:], self.q64[live][..., self.rot:])
        kb, vb = workloads.torch_to_bits(self.kc, self.kv), workloads.torch_to_bits(self.vc, self.kv)
        phys, off = self.slots[live] // self.bs, self.slots[live] % self.bs
        # v as pa_reshape_and_cache writes it, byte for byte; k's untouched slots too
        k_ref, v_ref = self.kb.copy(), self.vb.copy()
        one = np.float32(1.0)
        ks, vs = (self.k_scale, self.v_scale) if self.scaled else (one, one)
        src_bits = lambda t: workloads.torch_to_bits(t, self.src)  # noqa: E731
        oracle.reshape_and_cache(src_bits(self.key)[live], src_bits(self.value)[live], k_ref, v_ref, self.slots[live],
                                 self.bs, self.src, self.kv, ks, vs)
        assert np.array_equal(vb, v_ref)
        if self.kv == "nvfp4":
            got = oracle.nvfp4_rows(kb, phys, off, self.bs, ks)
            want = oracle.rotate(self.k64, self.pos, self.freq, interleaved, attn)[live]
            e = error(self.k64)[live]
            # Of a group's largest magnitude A: the block scale b is A / (6 s) to half a step of e4m3 (2^-4), so codes
            # end at 6 b s >= A (1 - 2^-4), and half of the widest step between codes (4 to 6) is b s <= A (1 + 2^-4) / 6.
            groups = (np.abs(want) + e).reshape(*want.shape[:2], -1, 16).max(-1).repeat(16, -1)
            assert np.all(np.abs(got - want) <= groups * (1 + 2.0 ** -4) / 6 + e)
            return
        rest = np.ones(kb.shape[:1] + kb.shape[2:3], bool)
        rest[phys, off] = False
        assert np.array_equal(kb.transpose(0, 2, 1, 3)[rest], self.kb.transpose(0, 2, 1, 3)[rest])
        got = oracle.decode_bits(kb[phys, :, off], self.kv, ks)
        want = oracle.rotate(self.k64, self.pos, self.freq, interleaved, attn)[live]
        e = error(self.k64)[live]
        step = HALF_STEP[self.kv] * (np.abs(want) + e) * (1 + 2.0 ** -23)  # x / scale is rounded to fp32 first
        unit = np.reshape(ks, (-1, 1)) if np.ndim(ks) else ks
        assert np.all(np.abs(got - want) <= np.maximum(step, TINY[self.kv] * unit) + e)
        assert np.array_equal(kb[phys, :, off][..., self.rot:], k_ref[phys, :, off][..., self.rot:])


SHAPES = [  # tokens, q heads, kv heads, head, rotated, source, cache, block
    (37, 32, 8, 128, 128, "bf16", "bf16", 16),
    (1, 32, 8, 128, 128, "bf16", "bf16", 16),
    (5, 8, 2, 64, 32, "f32", "f32", 16),
    (33, 8, 8, 64, 64, "f16", "f16", 32),
    (19, 28, 4, 96, 48, "bf16", "bf16", 16),
    (19, 28, 4, 96, 24, "f16", "f16", 16),      # halves of 12: not whole 16-byte pieces
    (7, 5, 1, 80, 2, "bf16", "bf16", 48),       # one pair
    (7, 3, 3, 8, 6, "bf16", "bf16", 16),        # the smallest head
    (9, 4, 2, 256, 256, "f32", "f32", 16),
    (300, 16, 2, 128, 128, "bf16", "fp8_e4m3", 32),
    (21, 8, 2, 128, 64, "f32", "fp8_e4m3", 16),
    (21, 8, 2, 160, 40, "f16", "fp8_e5m2", 64),  # halves of 20
    (65, 8, 4, 128, 128, "bf16", "fp8_e5m2", 16),
    (12, 8, 2, 128, 128, "bf16", "nvfp4", 32),
    (12, 8, 2, 64, 32, "f32", "nvfp4", 16),
    (11, 8, 2, 96, 72, "f16", "nvfp4", 16),      # halves of 36
    (2049, 12, 2, 64, 64, "bf16", "bf16", 16),
]


@pytest.mark.parametrize("interleaved", [False, True], ids=["half", "interleaved"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s)))
def test_parity(pa, shape, interleaved):
    c = Case(*shape, seed=11, per_head=shape[0] % 2 == 1)
    c.slots[::7] = np.where(np.arange(c.slots[::7].size) % 3 == 1, -1, c.slots[::7])
    c.call(pa, interleaved, 1.25)
    assert pa.pa_get_error_flags(clear=True) == 0
    c.check(interleaved, 1.25)
    pad = torch.from_numpy(np.flatnonzero(c.slots < 0)).to(DEV)
    assert bool((c.q_out[pad] == 7.0).all())    # padding rows are left as they were


@pytest.mark.parametrize("interleaved", [False, True], ids=["half", "interleaved"])
@pytest.mark.parametrize("kv,gap,shift", [("bf16", 0, 1), ("bf16", 1, 0), ("bf16", 8, 0), ("fp8_e4m3", 3, 5),
                                          ("nvfp4", 1, 1), ("bf16", 4, 4)])
def test_rows_at_any_element_alignment(pa, kv, gap, shift, interleaved):
    c = Case(23, 8, 2, 128, 64, "bf16", kv, gap=gap, shift=shift, seed=12)
    c.call(pa, interleaved)
    assert pa.pa_get_error_flags(clear=True) == 0
    c.check(interleaved)


@pytest.mark.parametrize("interleaved", [False, True], ids=["half", "interleaved"])
@pytest.mark.parametrize("rot,shift", [(128, 0), (32, 0), (24, 0), (128, 1)])
def test_q_in_place(pa, rot, shift, interleaved):
    c = Case(130, 8, 2, 128, rot, "f16", "f16", seed=13, shift=shift)
    key, value = c.key.clone(), c.value.clone()
    c.call(pa, interleaved, in_place=True)
    c.check(interleaved, q=c.q)
    assert torch.equal(key, c.key) and torch.equal(value, c.value)


@pytest.mark.parametrize("interleaved", [False, True], ids=["half", "interleaved"])
@pytest.mark.parametrize("far", [262144, 2 ** 24 + 3, 2 ** 31 - 1])
def test_far_and_negative_positions(pa, far, interleaved):
    c = Case(64, 4, 2, 64, 64, "f32", "f32", seed=14, far=far, negative=True)
    c.pos[:4] = [far, -far, 2 ** 31 - 1, -2 ** 31]
    c.call(pa, interleaved)
    c.check(interleaved)


@pytest.mark.parametrize("src,kv", [("bf16", "bf16"), ("f32", "f32"), ("f16", "f16"), ("bf16", "fp8_e4m3"),
                                    ("f32", "fp8_e5m2"), ("f16", "nvfp4"), ("bf16", "nvfp4")])
@pytest.mark.parametrize("rot", [128, 24])
def test_position_zero_is_the_plain_write(pa, src, kv, rot):
    """No angle: q unchanged, k and v byte for byte as pa_reshape_and_cache stores them."""
    c = Case(41, 8, 2, 128, rot, src, kv, seed=15, per_head=True)
    c.pos[:] = 0
    for interleaved in (False, True):
        c.call(pa, interleaved)
        kc, vc = workloads.bits_to_torch(c.kb, kv, DEV), workloads.bits_to_torch(c.vb, kv, DEV)
        pa.pa_reshape_and_cache(c.key.contiguous(), c.value.contiguous(), kc, vc, c.dev_slots, c.ks, c.vs)
        assert torch.equal(c.kc.view(torch.uint8), kc.view(torch.uint8))
        assert torch.equal(c.vc.view(torch.uint8), vc.view(torch.uint8))
        assert torch.equal(c.q_out, c.q)


def test_keys_alone(pa):
    c = Case(18, 0, 2, 128, 128, "bf16", "bf16", seed=16)
    c.call(pa, False)
    c.check(False)


@pytest.mark.parametrize("rot", [128, 24])
def test_slots_out_of_range_are_skipped_and_flagged(pa, rot):
    c = Case(20, 8, 2, 128, rot, "bf16", "bf16", seed=17)
    c.slots[3] = c.nb * c.bs
    c.slots[9] = 2 ** 62
    c.slots[12] = -2 ** 62
    c.call(pa, False)
    assert pa.pa_get_error_flags(clear=True) == pa.PA_ERRFLAG_SLOT
    c.check(False)
    assert bool((c.q_out[[3, 9, 12]] == 7.0).all())


def test_first_and_last_slot_and_no_tokens(pa):
    c = Case(2, 8, 2, 64, 64, "bf16", "fp8_e4m3", seed=18)
    c.slots[:] = [0, c.nb * c.bs - 1]
    c.call(pa, True)
    c.check(True)
    before = c.kc.clone()
    pa.pa_rotary_and_cache(c.q_out[:0], c.q[:0], c.key[:0], c.value[:0], c.kc, c.vc, c.dev_pos[:0], c.dev_slots[:0],
                           c.dev_freq, k_scale=c.ks, v_scale=c.vs)
    assert torch.equal(before, c.kc) and pa.pa_get_error_flags(clear=True) == 0


def test_another_stream_and_a_graph(pa):
    c = Case(50, 8, 2, 128, 128, "bf16", "bf16", seed=19)
    s = torch.cuda.Stream()
    c.call(pa, False, stream=s)
    c.check(False)
    eager = c.q_out.clone()
    k_eager = c.kc.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.pa_rotary_and_cache(c.q_out, c.q, c.key, c.value, c.kc, c.vc, c.dev_pos, c.dev_slots, c.dev_freq)
    for shift in (0, 5):
        c.dev_pos.add_(shift)                    # a replay reads the positions of its time
        c.pos += shift
        c.q_out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        c.check(False)
        assert torch.equal(c.q_out, eager) == (shift == 0) and torch.equal(c.kc, k_eager) == (shift == 0)


@pytest.mark.parametrize("rot,kv", [(128, "bf16"), (24, "bf16"), (128, "fp8_e4m3"), (24, "nvfp4")])
def test_slots_behind_2_to_32_elements(pa, rot, kv):
    """A block's rows are the same wherever it lies: in a cache of more than 2^32 elements too."""
    nb, far = 4 * 10 ** 5, 399990               # blocks of 8 heads x 16 x 128 elements (6.5 GB of bf16)
    c = Case(23, 8, 8, 128, rot, "bf16", kv, seed=20)
    c.call(pa, False)
    k_far, v_far = (torch.zeros((nb,) + tuple(t.shape[1:]), dtype=t.dtype, device=DEV) for t in (c.kc, c.vc))
    k_far[far:far + c.nb], v_far[far:far + c.nb] = (workloads.bits_to_torch(b, kv, DEV) for b in (c.kb, c.vb))
    q_out = torch.zeros_like(c.q_out)
    pa.pa_rotary_and_cache(q_out, c.q, c.key, c.value, k_far, v_far, c.dev_pos, c.dev_slots + far * c.bs, c.dev_freq,
                           k_scale=c.ks, v_scale=c.vs)
    assert torch.equal(q_out, c.q_out) and pa.pa_get_error_flags(clear=True) == 0
    raw = lambda t: t.view(torch.uint8)  # noqa: E731
    assert torch.equal(raw(k_far[far:far + c.nb]), raw(c.kc)) and torch.equal(raw(v_far[far:far + c.nb]), raw(c.vc))
    assert not bool(raw(k_far[:c.nb]).any()) and not bool(raw(v_far[:c.nb]).any())


def test_q_out_between_the_rows_it_comes_from(pa):
    """Slices of one array that lie side by side: written ones and read ones do not touch."""
    c = Case(40, 8, 2, 128, 128, "bf16", "bf16", seed=22)
    c.call(pa, False)
    want = c.q_out.clone()
    rows = torch.zeros(40, 2 * 8 * 128 + 4 * 128, dtype=torch.bfloat16, device=DEV)
    rows[:, :12 * 128] = torch.cat([c.q.flatten(1), c.key.flatten(1), c.value.flatten(1)], 1)
    q, key, value = (rows[:, a * 128:b * 128].unflatten(1, (-1, 128)) for a, b in ((0, 8), (8, 10), (10, 12)))
    q_out = rows[:, 12 * 128:].unflatten(1, (8, 128))
    pa.pa_rotary_and_cache(q_out, q, key, value, c.kc, c.vc, c.dev_pos, c.dev_slots, c.dev_freq)
    assert torch.equal(q_out, want)
    for over in (rows[:, 128:9 * 128], rows[:, 9 * 128:17 * 128], rows[:, 11 * 128:19 * 128]):
        with pytest.raises(pa.PAError):
            pa.pa_rotary_and_cache(over.unflatten(1, (8, 128)), q, key, value, c.kc, c.vc, c.dev_pos, c.dev_slots,
                                   c.dev_freq)

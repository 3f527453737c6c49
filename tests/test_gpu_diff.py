"""GPU: differential attention against the fp64 oracle, element by element within its roundings (see
diff_harness): both calls, every cache format, head layouts, odd sizes, windows, partitions, norms,
strides of lambda; caches that hold NaN wherever no token lies; bad tables and lengths; streams,
graphs and workspaces."""

import numpy as np
import pytest
import torch

import oracle
import workloads
from tests.diff_harness import Diff

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def pa():
    import paged_kv_cache_pagedattention_gb300 as lib
    lib.pa_get_error_flags(clear=True)
    return lib


def poison(c):
    """NaN in every slot of the caches that holds no token of any sequence."""
    b = c.b
    used = np.zeros((b.num_blocks, b.block_size), bool)
    for r, n in enumerate(b.seq_lens):
        pos = np.arange(int(n))
        used[b.block_tables[r, pos // b.block_size], pos % b.block_size] = True
    nan = {"f32": 0x7fc00000, "f16": 0x7e00, "bf16": 0x7fc0, "fp8_e4m3": 0x7f, "fp8_e5m2": 0x7f}
    if b.kv_dtype in nan:
        at = np.broadcast_to(~used[:, None, :, None], b.k_cache.shape)
        for x in (b.k_cache, b.v_cache):
            x.view({1: np.uint8, 2: np.uint16, 4: np.uint32}[x.dtype.itemsize])[at] = nan[b.kv_dtype]


LENS = [1, 17, 16, 200, 333, 64]
SHAPES = [  # q heads, kv heads, head, block, cache, q
    (8, 4, 64, 16, "f32", None),
    (8, 4, 128, 16, "bf16", None),
    (16, 4, 128, 16, "f16", None),
    (32, 8, 128, 32, "bf16", None),
    (64, 8, 128, 16, "bf16", None),      # eight heads to a group
    (24, 4, 128, 16, "f16", None),       # six
    (44, 4, 64, 16, "bf16", None),       # eleven
    (16, 16, 64, 32, "f16", None),       # one
    (16, 4, 64, 64, "bf16", None),
    (12, 4, 128, 64, "f16", None),
    (8, 4, 128, 48, "bf16", None),
    (8, 2, 128, 16, "fp8_e4m3", "bf16"),
    (32, 8, 128, 32, "fp8_e4m3", "f16"),
    (64, 4, 128, 64, "fp8_e5m2", "bf16"),
    (20, 4, 128, 16, "fp8_e5m2", "f16"),
    (8, 4, 64, 32, "fp8_e4m3", "bf16"),
    (8, 4, 128, 16, "fp8_e4m3", "f32"),
    (8, 4, 128, 16, "nvfp4", "bf16"),
    (4, 2, 64, 32, "nvfp4", "f32"),
    (6, 2, 80, 16, "bf16", None),        # no tensor-core shapes
    (4, 4, 7, 5, "f32", None),
    (4, 2, 256, 16, "f32", None),
    (2, 2, 192, 24, "f16", None),
    (2, 2, 1, 1, "f32", None),
]
ID = lambda s: "-".join(str(x) for x in s)  # noqa: E731


@pytest.mark.parametrize("shape", SHAPES, ids=ID)
@pytest.mark.parametrize("window,part", [(0, 0), (0, 64), (50, 0), (50, 32), (1, 0)])
def test_decode_parity(pa, shape, window, part):
    hq, hkv, d, bs, kv, qd = shape
    part = -(-part // bs) * bs
    c = Diff(LENS, [1] * len(LENS), hq, hkv, d, bs, kv, qd, window, norm=part == 0, per_token=window == 0,
             seed=hq + d + window)
    poison(c)
    c.to_device()
    c.call(pa, False, part)
    assert pa.pa_get_error_flags(clear=True) == 0
    c.check()


@pytest.mark.parametrize("shape", SHAPES, ids=ID)
@pytest.mark.parametrize("window,part", [(0, 0), (0, 64), (50, 0), (70, 64)])
def test_varlen_parity(pa, shape, window, part):
    """Whole prompts, chunks on prefixes, single tokens and a request that rests."""
    hq, hkv, d, bs, kv, qd = shape
    part = -(-part // bs) * bs
    lens, new = [1, 2, 37, 300, 129, 260, 70], [1, 2, 37, 1, 100, 260, 0]
    c = Diff(lens, new, hq, hkv, d, bs, kv, qd, window, norm=part != 0, per_token=window != 0, seed=hq + d + part)
    poison(c)
    c.to_device()
    c.call(pa, True, part)
    assert pa.pa_get_error_flags(clear=True) == 0
    c.check()


@pytest.mark.parametrize("kv,qd,d,bs", [("bf16", None, 128, 16), ("f16", None, 64, 32), ("fp8_e4m3", "bf16", 128, 32),
                                        ("f32", None, 64, 16)])
def test_not_causal(pa, kv, qd, d, bs):
    c = Diff([77, 140, 9], [20, 140, 1], 16, 4, d, bs, kv, qd, causal=False, seed=3)
    poison(c)
    c.to_device()
    c.call(pa, True)
    assert pa.pa_get_error_flags(clear=True) == 0
    c.check()


@pytest.mark.parametrize("kv", ["bf16", "f16", "fp8_e4m3"])
@pytest.mark.parametrize("hq,part", [(16, 0), (16, 512), (48, 0)])
def test_long_contexts(pa, kv, hq, part):
    """Many partitions of a row; sampled rows of long contexts."""
    c = Diff([9000, 16384, 4097, 1], [1, 1, 1, 1], hq, 4, 128, 16, kv, "bf16" if kv[0] == "f" and kv != "f16" else None,
             seed=5)
    c.to_device()
    c.call(pa, False, part)
    first = c.out.clone()
    c.check()
    c.call(pa, False, part)
    assert torch.equal(first, c.out)
    c.call(pa, True, part)
    c.check()
    assert pa.pa_get_error_flags(clear=True) == 0


@pytest.mark.parametrize("kv,qd,d", [("bf16", None, 128), ("bf16", None, 64), ("fp8_e4m3", "bf16", 128)])
def test_long_chunks(pa, kv, qd, d):
    """Chunks of hundreds of tokens on long prefixes, with decodes beside them: sampled rows."""
    lens, new = [3000, 700, 20000, 2500, 1], [600, 700, 300, 1, 1]
    c = Diff(lens, new, 16, 4, d, 16, kv, qd, per_token=True, seed=6)
    c.to_device()
    for part in (0, 4096):
        c.call(pa, True, part)
        rows = {0, 1, 127, 128, 255, 300, 599, 600, 601, 1100, 1299, 1300, 1500, 1599, 1600, 1601}
        c.check(rows=rows)
    first = c.out.clone()
    c.call(pa, True, 4096)
    assert torch.equal(first, c.out)
    assert pa.pa_get_error_flags(clear=True) == 0


@pytest.mark.parametrize("kv,bs", [("fp8_e4m3", 16), ("fp8_e5m2", 32), ("nvfp4", 16)])
def test_scales_for_every_head(pa, kv, bs):
    """One scale a KV head: the two maps' keys and the two value halves each have their own."""
    scales = [0.25, 0.5, 0.375, 1.0] if kv == "nvfp4" else [2.0 ** -6, 2.0 ** -5, 0.01, 0.02]
    for varlen in (False, True):
        c = Diff([150, 33, 90], [1, 33, 40] if varlen else [1, 1, 1], 8, 4, 128, bs, kv, "bf16", seed=7,
                 cache_scale=scales)
        poison(c)
        c.to_device()
        c.call(pa, varlen)
        c.check()
    assert pa.pa_get_error_flags(clear=True) == 0


def test_strides_of_lambda(pa):
    """A number, a row of heads, a column, a transposed matrix: what an expanded matrix gives."""
    c = Diff([70, 5, 300], [30, 5, 1], 16, 4, 128, 16, "bf16", per_token=True, seed=8)
    c.to_device()
    for lam in (torch.tensor(0.37, device=DEV), torch.rand(8, device=DEV), torch.rand(36, 1, device=DEV),
                torch.rand(1, 8, device=DEV), torch.rand(8, 36, device=DEV).t(), torch.rand(72, 24, device=DEV)[::2, ::3],
                torch.rand(1, device=DEV)):
        c.d_lam = lam.expand(36, 8).contiguous()
        want = c.call(pa, True).clone()
        c.d_lam = lam
        assert torch.equal(want, c.call(pa, True))
        c.lam = lam.expand(36, 8).cpu().numpy()
    c.check()


@pytest.mark.parametrize("lam", [0.0, -0.5, 1.0])
def test_values_of_lambda(pa, lam):
    c = Diff([70, 5], [1, 1], 8, 4, 128, 16, "f16", norm=False, seed=9)
    c.lam[:] = lam
    c.to_device()
    c.call(pa, False)
    c.check()


@pytest.mark.parametrize("kv,d", [("bf16", 128), ("f16", 64), ("f32", 64)])
def test_equal_maps_cancel(pa, kv, d):
    """Both maps alike and lambda 1: nothing is left but roundings, and exactly nothing in one kernel's sums."""
    c = Diff([100, 37], [1, 1], 8, 4, d, 16, kv, norm=False, seed=10)
    c.lam[:] = 1.0
    b = c.b
    b.q[:, 1::2] = b.q[:, 0::2]
    b.k_cache[:, 1::2] = b.k_cache[:, 0::2]
    c.to_device()
    c.call(pa, False)
    c.check()


@pytest.mark.parametrize("kv,qd,bs", [("bf16", None, 16), ("fp8_e4m3", "bf16", 32), ("f32", None, 16)])
def test_bad_tables_and_lengths(pa, kv, qd, bs):
    c = Diff([100, 60, 40, 80], [1, 1, 1, 1], 8, 4, 128, bs, kv, qd, seed=11)
    c.tables[0, 1] = c.b.num_blocks
    c.tables[2, :] = -1                            # nothing can be read: 0
    c.to_device()
    c.call(pa, False)
    assert pa.pa_get_error_flags(clear=True) == pa.PA_ERRFLAG_BLOCK_TABLE
    c.check()
    assert not bool(c.out[2].any())
    lens = c.db.lens.clone()
    for wrong in (0, -3, 81, 2 ** 31 - 1):
        c.db.lens[1] = wrong
        c.b.seq_lens[1] = 60
        c.out.fill_(9.0)
        if wrong == 81:
            c.db.lens[1] = c.b.max_seq_len + 1
        c.call(pa, False)
        assert pa.pa_get_error_flags(clear=True) & pa.PA_ERRFLAG_SEQ_LEN
        assert not bool(c.out[1].any())
        c.db.lens.copy_(lens)
    # in a flattened batch
    c = Diff([100, 60, 40, 80], [40, 1, 40, 3], 8, 4, 128, bs, kv, qd, seed=12)
    c.tables[0, 1] = -7
    c.tables[2, :] = c.b.num_blocks + 5
    c.to_device()
    c.call(pa, True)
    assert pa.pa_get_error_flags(clear=True) == pa.PA_ERRFLAG_BLOCK_TABLE
    c.check()
    assert not bool(c.out[41:81].any())
    c.db.qsl[2] = 39                               # starts that decrease: nothing is written
    c.out.fill_(9.0)
    c.call(pa, True)
    assert pa.pa_get_error_flags(clear=True) & pa.PA_ERRFLAG_QUERY
    assert bool((c.out == 9.0).all())


def growing(c):
    """Keys whose magnitude grows along every sequence, from a fifth to ten times: the maxima rise chunk
    after chunk by far more than the slack within which sums are not rescaled."""
    b = c.b
    factor = np.ones((b.num_blocks, b.block_size))
    for r, n in enumerate(b.seq_lens):
        pos = np.arange(int(n))
        factor[b.block_tables[r, pos // b.block_size], pos % b.block_size] = 0.2 + 10 * pos / int(n)
    k = oracle.decode_bits(b.k_cache, b.kv_dtype, b.k_scale) * factor[:, None, :, None]
    b.k_cache = workloads._cast_bits(torch.from_numpy(k.astype(np.float32)), b.kv_dtype, b.k_scale)


@pytest.mark.parametrize("kv,qd,hq,d,bs", [
    ("bf16", None, 16, 128, 16), ("f16", None, 16, 128, 32), ("bf16", None, 40, 128, 64), ("f16", None, 16, 64, 16),
    ("bf16", None, 8, 64, 64), ("fp8_e4m3", "bf16", 16, 128, 16), ("fp8_e5m2", "f16", 64, 128, 32), ("f32", None, 8, 64, 16)])
@pytest.mark.parametrize("part", [0, 128])
def test_maxima_that_rise(pa, kv, qd, hq, d, bs, part):
    for new in ([1, 1, 1], [300, 1, 90], [129, 40, 600]):
        c = Diff([900, 333, 600], new, hq, 4, d, bs, kv, qd, seed=31, cache_scale=0.25 if kv[:3] == "fp8" else None)
        growing(c)
        c.to_device()
        for varlen in (True, False) if max(new) == 1 else (True,):
            c.out.fill_(9.0)
            c.call(pa, varlen, part)
            c.check()
    assert pa.pa_get_error_flags(clear=True) == 0


@pytest.mark.parametrize("kv,d", [("f32", 64), ("bf16", 128), ("bf16", 96)])
def test_a_request_longer_than_told(pa, kv, d):
    """More new tokens than max_query_len: flagged, and the other requests' rows are what they are without it."""
    c = Diff([90, 500, 300, 7], [40, 20, 1, 1], 8, 4, d, 16, kv, seed=21)
    c.to_device()
    c.b.__class__.max_query_len, keep = property(lambda b: 30), c.b.__class__.max_query_len
    try:
        c.call(pa, True, 64)
    finally:
        c.b.__class__.max_query_len = keep
    assert pa.pa_get_error_flags(clear=True) == pa.PA_ERRFLAG_QUERY
    rows = set(range(40, 62))
    c.check(rows=rows)
    assert bool((c.out[:40] == 9.0).all()) or not bool(c.out[:40].any())     # left, or zero


@pytest.mark.parametrize("n,new", [(2, 2), (37, 37), (1000, 37), (700, 300), (513, 513), (4000, 129)])
@pytest.mark.parametrize("kv,qd,d", [("bf16", None, 128), ("f16", None, 64), ("fp8_e4m3", "bf16", 128)])
@pytest.mark.parametrize("window,part,causal", [(0, 0, True), (0, 64, True), (100, 64, True), (0, 128, False)])
def test_one_request_alone(pa, n, new, kv, qd, d, window, part, causal):
    c = Diff([n], [new], 24, 4, d, 16, kv, qd, window, norm=part != 64, seed=n + window, causal=causal)
    poison(c)
    c.to_device()
    c.call(pa, True, part)
    assert pa.pa_get_error_flags(clear=True) == 0
    c.check()


def test_one_request_out_of_range(pa):
    """Starts that do not run to the rows' number, a length out of range: nothing is written."""
    c = Diff([300], [100], 8, 4, 128, 16, "bf16", seed=23)
    c.to_device()
    ws = torch.full_like(c.workspace(pa, True, 64), 0xff)
    for starts, length, flag in (([0, 99], 300, pa.PA_ERRFLAG_QUERY), ([1, 101], 300, pa.PA_ERRFLAG_QUERY),
                                 ([0, 100], 99, pa.PA_ERRFLAG_QUERY), ([0, 100], 0, pa.PA_ERRFLAG_QUERY),
                                 ([0, 100], 301, pa.PA_ERRFLAG_SEQ_LEN), ([0, -5], 300, pa.PA_ERRFLAG_QUERY)):
        c.db.qsl.copy_(torch.tensor(starts, dtype=torch.int32))
        c.db.lens.fill_(length)
        c.out.fill_(9.0)
        c.call(pa, True, 64, ws)
        assert pa.pa_get_error_flags(clear=True) == flag
        assert bool((c.out == 9.0).all())
    c.db.qsl.copy_(torch.tensor([0, 100], dtype=torch.int32))
    c.db.lens.fill_(300)
    c.call(pa, True, 64, ws)
    c.check()


@pytest.mark.parametrize("d,heads", [(128, 16), (64, 8)])
@pytest.mark.parametrize("lens,new", [
    ([900, 333], [130, 333]),                                   # two requests, two warps of the plan each
    ([1500, 700, 640], [1300, 33, 2]),                          # more than 32 tiles beside a few
    ([400, 64, 2100, 77, 1200], [399, 64, 40, 2, 1100]),        # more requests than warps
])
def test_tiles_of_split_requests(pa, lens, new, d, heads):
    """Every tile over every partition is listed once, for few tiles and for many."""
    c = Diff(lens, new, heads, 4, d, 16, "bf16", seed=sum(new))
    poison(c)
    c.to_device()
    c.call(pa, True, 64)
    assert pa.pa_get_error_flags(clear=True) == 0
    c.check()


def test_two_streams_at_once(pa):
    """Mixed batches on two streams, each call with a workspace of its own and the side stream between
    them, give what they give one after the other."""
    cs = [Diff([700, 90, 33, 400], [200, 1, 33, 1], 16, 4, 128, 16, kv, per_token=True, seed=22 + i)
          for i, kv in enumerate(("bf16", "f16", "bf16"))]
    for c in cs:
        c.to_device()
        c.ws = c.workspace(pa, True)
    want = [c.call(pa, True, ws=c.ws).clone() for c in cs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    for c in cs:
        c.out.fill_(9.0)
    torch.cuda.synchronize()
    for _ in range(5):
        for c, s in zip(cs, streams):
            c.call(pa, True, ws=c.ws, stream=s)
    torch.cuda.synchronize()
    for c, w in zip(cs, want):
        assert torch.equal(c.out, w)
    assert pa.pa_get_error_flags(clear=True) == 0


@pytest.mark.parametrize("seed", range(12))
def test_batches_of_any_shape(pa, seed):
    """Shapes, lengths, windows and options drawn at random, both calls."""
    rng = np.random.default_rng(1000 + seed)
    d = int(rng.choice([64, 128]))
    kv = str(rng.choice(["bf16", "f16", "fp8_e4m3", "fp8_e5m2"] if d == 128 else ["bf16", "f16"]))
    qd = str(rng.choice(["bf16", "f16"])) if kv[:3] == "fp8" else None
    hkv = 2 * int(rng.integers(1, 5))
    hq = hkv * int(rng.integers(1, 10))
    n = int(rng.integers(1, 9))
    new = [int(rng.choice([0, 1, 1, 2, 17, 63, 64, 65, 128, 200])) for _ in range(n)]
    if not sum(new):
        new[0] = 1
    lens = [max(1, q + int(rng.choice([0, 0, 1, 15, 16, 100, 700]))) for q in new]
    c = Diff(lens, new, hq, hkv, d, int(rng.choice([16, 32, 64])), kv, qd, int(rng.choice([0, 0, 0, 1, 16, 77])),
             bool(rng.integers(2)), bool(rng.integers(2)), seed)
    poison(c)
    c.to_device()
    c.call(pa, True, int(rng.choice([0, 0, 64, 128])))
    assert pa.pa_get_error_flags(clear=True) == 0
    c.check()


@pytest.mark.parametrize("varlen", [False, True])
def test_streams_graphs_and_workspaces(pa, varlen):
    """Another stream; a workspace full of NaN; two graphs that share it, replayed in turn, each on
    the lengths of its time."""
    new = [1, 30, 1, 200] if varlen else [1, 1, 1, 1]
    cs = [Diff([500, 90, 3, 400], new, 16, 4, 128, 16, kv, per_token=True, seed=13) for kv in ("bf16", "f16")]
    for c in cs:
        c.to_device()
    ws = torch.full_like(cs[0].workspace(pa, varlen, 64), 0xff)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    want = []
    for c in cs:
        c.call(pa, varlen, 64, ws, stream=side)
        side.synchronize()
        c.check()
        want.append(c.out.clone())
    graphs = []
    for c in cs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.call(pa, varlen, 64, ws)
        graphs.append(g)
    for _ in range(2):
        for c, g, w in zip(cs, graphs, want):
            c.out.fill_(9.0)
            g.replay()
            assert torch.equal(c.out, w)
    cs[0].db.lens[0] -= 7
    cs[0].b.seq_lens[0] -= 7
    graphs[0].replay()
    torch.cuda.synchronize()
    cs[0].check()
    assert pa.pa_get_error_flags(clear=True) == 0


def test_cache_behind_2_to_32_elements(pa):
    """Blocks that lie behind 2^32 elements of the cache."""
    for kv, varlen in (("bf16", False), ("bf16", True), ("fp8_e4m3", False)):
        c = Diff([90, 300], [40, 1] if varlen else [1, 1], 32, 16, 128, 16, kv, "bf16", seed=14)
        c.to_device()
        want = c.call(pa, varlen).clone()
        c.check()
        per = 16 * 16 * 128
        far = 2 ** 32 // per + 5
        big = []
        for t in (c.db.kc, c.db.vc):
            x = torch.zeros((far + t.shape[0],) + tuple(t.shape[1:]), dtype=t.dtype, device=DEV)
            x[far:] = t
            big.append(x)
        c.db.kc, c.db.vc = big
        c.db.tables = torch.where(c.db.tables >= 0, c.db.tables + far, c.db.tables)
        c.out.fill_(9.0)
        assert torch.equal(c.call(pa, varlen), want)
        del big, c
    assert pa.pa_get_error_flags(clear=True) == 0


def test_a_layer_step(pa):
    """Rotary write on several axes, then differential attention on what it wrote, in one graph."""
    c = Diff([130, 40, 300], [1, 40, 60], 16, 4, 128, 16, "bf16", seed=15)
    b = c.b
    c.to_device()
    rng = np.random.default_rng(16)
    pos = rng.integers(0, 500, (3, b.total_q)).astype(np.int32)
    freq = oracle.rotary_frequencies(128)[0].astype(np.float32)
    axes = pa.pa_rotary_pair_axes([16, 24, 24])
    d_pos, d_freq = torch.from_numpy(pos).to(DEV), torch.from_numpy(freq).to(DEV)
    q_in = c.db.q.clone()
    ws = c.workspace(pa, True)

    def layer():
        pa.pa_rotary_axes_and_cache(c.db.q, q_in, c.db.key, c.db.value, c.db.kc, c.db.vc, d_pos, c.db.slots, d_freq, axes)
        c.call(pa, True, ws=ws)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        layer()
    torch.cuda.synchronize()
    eager = c.out.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        layer()
    c.out.fill_(9.0)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(eager, c.out)
    # the oracle from the rows that the write left
    b.q[:] = workloads.torch_to_bits(c.db.q, "bf16")
    b.k_cache, b.v_cache = (workloads.torch_to_bits(x, "bf16") for x in (c.db.kc, c.db.vc))
    c.check()
    key = oracle.rotate_axes(oracle.decode_bits(b.key, "bf16"), pos, freq, axes)
    got = oracle.decode_bits(b.k_cache[b.slot_mapping // 16, :, b.slot_mapping % 16], "bf16")
    e = 2 * np.abs(key).max() * 2.0 ** -20
    assert np.all(np.abs(got - key) <= 2.0 ** -8 * (np.abs(key) + e) + e)

"""GPU: differential attention at its edges: one workspace for batches of many sizes, requests out of
range beside others."""

import pytest
import torch

from tests.diff_harness import Diff

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def pa():
    import paged_kv_cache_pagedattention_gb300 as lib
    lib.pa_get_error_flags(clear=True)
    return lib


@pytest.mark.parametrize("kv,d", [("bf16", 128), ("f16", 64), ("f32", 64)])
def test_one_workspace_for_every_batch(pa, kv, d):
    """The largest batch's workspace, full of NaN, takes smaller ones, which are split more finely."""
    ws = None
    for lens, new in (([900] * 12, [40, 100, 300] + [1] * 9), ([900, 700, 1, 33], [5, 1, 1, 20]), ([900], [37]),
                      ([333, 900], [1, 1]), ([900] * 11, [1] * 10 + [2])):
        c = Diff(lens, new, 8, 4, d, 16, kv, seed=len(lens))
        c.to_device()
        for varlen in (True, False) if max(new) == 1 else (True,):
            if ws is None:
                ws = torch.full_like(c.workspace(pa, varlen), 0xff)
            assert c.workspace(pa, varlen).nbytes <= ws.nbytes
            c.out.fill_(9.0)
            c.call(pa, varlen, ws=ws)
            c.check()
    assert pa.pa_get_error_flags(clear=True) == 0


def test_few_tokens_of_chunks_beside_many_single_tokens(pa):
    """The chunk's context is split less finely than alone: its states count every row of the batch."""
    c = Diff([3000] + [20] * 600, [4] + [1] * 600, 32, 8, 128, 16, "bf16", seed=41)
    c.to_device()
    c.call(pa, True)
    assert pa.pa_get_error_flags(clear=True) == 0
    c.check(rows={0, 1, 2, 3, 4, 5, 300, 603})


@pytest.mark.parametrize("kv,qd,d,bs", [("bf16", None, 128, 16), ("f16", None, 64, 32), ("fp8_e4m3", "bf16", 128, 32),
                                        ("f32", None, 64, 16), ("bf16", None, 96, 16), ("nvfp4", "bf16", 128, 16),
                                        ("bf16", None, 128, 48)])
@pytest.mark.parametrize("part", [0, 2])
def test_requests_out_of_range_beside_others(pa, kv, qd, d, bs, part):
    """Rows of several tokens are left as they were, single tokens are 0, whichever kernel serves the shape."""
    lens, new = [90, 200, 70, 300, 40], [40, 30, 1, 60, 1]
    start = [0, 40, 70, 71, 131]
    c = Diff(lens, new, 8, 4, d, bs, kv, qd, seed=42)
    c.to_device()
    rows = set(range(132))
    ws = torch.full_like(c.workspace(pa, True, part * bs), 0xff)
    query, length = pa.PA_ERRFLAG_QUERY, pa.PA_ERRFLAG_SEQ_LEN
    for r, wrong, flag in ((0, 39, query), (0, 301, length), (1, 0, query), (3, -5, query), (3, 2 ** 31 - 1, length),
                           (2, 0, query), (2, 301, length), (4, 2 ** 31 - 1, length), (4, -1, query)):
        c.db.lens[r] = wrong
        c.out.fill_(9.0)
        c.call(pa, True, part * bs, ws)
        assert pa.pa_get_error_flags(clear=True) & flag, (r, wrong)
        own = set(range(start[r], start[r] + new[r]))
        c.check(rows=rows - own)
        assert bool((c.out[sorted(own)] == (0.0 if new[r] == 1 else 9.0)).all()), (r, wrong)
        c.db.lens[r] = lens[r]
    # more tokens than told, by some of the requests and by all of several tokens
    for told, over in ((40, (3,)), (30, (0, 3)), (1, (0, 1, 3))):
        c.b.__class__.max_query_len, keep = property(lambda b, told=told: told), c.b.__class__.max_query_len
        try:
            ws = c.workspace(pa, True, part * bs)
            c.out.fill_(9.0)
            c.call(pa, True, part * bs, ws)
        finally:
            c.b.__class__.max_query_len = keep
        assert pa.pa_get_error_flags(clear=True) == query
        own = {t for r in over for t in range(start[r], start[r] + new[r])}
        c.check(rows=rows - own)
        assert bool((c.out[sorted(own)] == 9.0).all()), told
    c.call(pa, True, part * bs)
    assert pa.pa_get_error_flags(clear=True) == 0
    c.check()


@pytest.mark.parametrize("kv,d", [("bf16", 128), ("f32", 64), ("bf16", 96)])
def test_one_request_longer_than_told(pa, kv, d):
    c = Diff([50], [20], 8, 4, d, 16, kv, seed=43)
    c.to_device()
    for told in (1, 19):
        c.b.__class__.max_query_len, keep = property(lambda b, told=told: told), c.b.__class__.max_query_len
        try:
            c.call(pa, True)
        finally:
            c.b.__class__.max_query_len = keep
        assert pa.pa_get_error_flags(clear=True) == pa.PA_ERRFLAG_QUERY
        assert bool((c.out == 9.0).all())

"""GPU: the plan of flattened batches.  A request's row tiles are listed by its own thread or by warps,
as their number and the other requests' decide; every tile is listed once either way, and a batch of
many short requests is planned in a few times what one request takes."""

import numpy as np
import pytest
import torch

import workloads
from tests.diff_harness import Diff
from tests.test_gpu_varlen import _varlen_parity

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def pa():
    import paged_kv_cache_pagedattention_gb300 as lib
    lib.pa_get_error_flags(clear=True)
    return lib


BATCHES = [  # new tokens, contexts, partition
    ([3] * 150, [3 + 7 * i % 90 for i in range(150)], 0),              # a tile each, more requests than threads of a warp
    ([2, 1] * 70 + [300], [40] * 140 + [700], 64),                     # one long list beside 70 short ones
    ([9, 600, 1, 5, 0, 257], [400, 600, 30, 900, 12, 1300], 64),       # lists on both sides of a warp's turn
    ([33] * 8 + [34], [33 * (i + 1) for i in range(8)] + [520], 32),   # lists of 1 to 17 tiles
]


@pytest.mark.parametrize("case", range(len(BATCHES)))
@pytest.mark.parametrize("kv", ["bf16", "fp8_e4m3"])
def test_every_tile_is_listed_once(pa, case, kv):
    new, lens, part = BATCHES[case]
    _varlen_parity(pa, workloads.build("plan", 500 + case, lens, new, 16, 4, 128, 16, kv), part, True)
    c = Diff(lens, new, 16, 4, 128, 16, kv, "bf16" if kv != "bf16" else None, seed=500 + case)
    c.to_device()
    c.call(pa, True, part)
    assert pa.pa_get_error_flags(clear=True) == 0
    c.check()


def plan_us(pa, requests, tokens, context):
    """The plan kernel's least time in microseconds over some calls of pa_varlen_attn."""
    t, hq, d, bs = requests * tokens, 8, 64, 16
    width = -(-context // bs)
    q = torch.zeros(t, hq, d, dtype=torch.bfloat16, device=DEV)
    cache = torch.zeros(width, 2, bs, d, dtype=torch.bfloat16, device=DEV)
    tables = torch.arange(width, dtype=torch.int32, device=DEV).repeat(requests, 1)
    starts = torch.arange(0, t + 1, tokens, dtype=torch.int32, device=DEV)
    lens = torch.full((requests,), context, dtype=torch.int32, device=DEV)
    ws = pa.workspace_tensor(pa.pa_varlen_workspace_size(requests, t, tokens, hq, 2, d, context, bs), DEV)
    out, times = torch.empty_like(q), []
    pa.pa_trace_enable(True)
    try:
        for _ in range(12):
            pa.pa_trace_read(pa.TRACE_KINDS.index("varlen_plan"), reset=True)
            pa.pa_varlen_attn(out, q, cache, cache, tables, starts, lens, tokens, context, 0.1, ws)
            torch.cuda.synchronize()
            times.append(pa.pa_trace_read(pa.TRACE_KINDS.index("varlen_plan"), reset=True)[1] * 1e3)
    finally:
        pa.pa_trace_enable(False)
    return float(np.min(times))


@pytest.mark.parametrize("requests,tokens,context", [(2000, 3, 64), (256, 4, 1000), (900, 2, 300)])
def test_many_short_requests(pa, requests, tokens, context):
    """Lists of one tile each are written at once, not by warps in turn (which takes 2,000 requests nine
    times the plan of one, and 256 three times)."""
    one, many = plan_us(pa, 1, tokens, context), plan_us(pa, requests, tokens, context)
    assert many <= (2.5 if requests < 1024 else 4.0) * one, (one, many)

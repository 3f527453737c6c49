"""GPU: differential attention at its edges: one workspace for batches of many sizes."""

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

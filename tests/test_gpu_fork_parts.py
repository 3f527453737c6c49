"""pa_fork_blocks by parents where a part holds as many children as it can: the grid of parents and slices
fills the device, so the children are cut into as few parts as there are, of up to 1,024, and all of a part's
children may come from one parent."""

import numpy as np
import pytest
import torch

from test_gpu_sequences import Pool, pa  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("children", [1024, 1025, 2047, 2048, 2049])
def test_parts_full_of_one_parents_children(pa, children):  # noqa: F811
    parents, width, blocks = 200, 8192, 4000     # 200 x 8 blocks of the grid a part, tables of 8 slices
    rng = np.random.default_rng(51)
    p = Pool(parents, width, blocks, 1)
    lens = rng.integers(0, 6, parents)
    lens[7] = 1100                               # a row of two slices
    p.append(pa, lens)
    one = np.full(children, 7)
    some = np.where(rng.random(children) < 0.9, 7, rng.integers(-1, parents, children))
    for chosen in (one, some):
        before = p.refs.copy()
        t2, l2, dt, dl = p.fork(pa, chosen)
        q = Pool(1, width, blocks, 1)
        q.refs, q.d_refs = p.refs, p.d_refs
        q.take((t2, l2, dt, dl))
        q.release(pa)
        p.same()
        assert np.array_equal(p.refs, before)
    assert pa.pa_get_error_flags(clear=True) == 0

"""GPU parity of pa_fork_blocks, pa_append_blocks and pa_release_blocks: every array equal to
the oracle's, row by row and in order, over random histories and at the edges; refused
calls leave everything as it was."""

import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def pa():
    import paged_kv_cache_pagedattention_gb300 as lib
    lib.pa_get_error_flags(clear=True)
    return lib


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


class Pool:
    """The same state on the host (the oracle's) and on the device (the library's)."""

    def __init__(self, rows, width, blocks, bs):
        self.bs, self.rows = bs, rows
        self.tables = np.full((rows, width), -1, np.int32)
        self.lens = np.zeros(rows, np.int32)
        self.refs = np.zeros(blocks, np.int32)
        self.to_device()

    def to_device(self):
        self.d_tables, self.d_lens, self.d_refs = dev(self.tables), dev(self.lens), dev(self.refs)

    def same(self):
        torch.cuda.synchronize()
        assert np.array_equal(self.d_tables.cpu().numpy(), self.tables)
        assert np.array_equal(self.d_lens.cpu().numpy(), self.lens)
        assert np.array_equal(self.d_refs.cpu().numpy(), self.refs)

    def append(self, pa, add, ws=None):
        qsl = np.concatenate([[0], np.cumsum(add)]).astype(np.int32)
        total = int(qsl[-1])
        slots = torch.full((total,), 77, dtype=torch.int64, device=DEV)
        pairs = torch.full((self.rows, 2), 77, dtype=torch.int64, device=DEV)
        if ws is None:
            ws = torch.full((pa.pa_append_workspace_size(self.rows, total, self.bs),), 0xff, dtype=torch.uint8,
                            device=DEV)
        pa.pa_append_blocks(self.d_tables, self.d_lens, dev(qsl), slots, pairs, self.d_refs, self.bs, ws)
        flags = pa.pa_get_error_flags(clear=True)
        want = oracle.append_blocks(self.tables, self.lens, qsl, self.refs, self.bs)
        if want is None:
            want = np.full(total, -1), np.zeros((self.rows, 2))
            assert flags
        else:
            assert flags == 0
        assert np.array_equal(slots.cpu().numpy(), want[0])
        assert np.array_equal(pairs.cpu().numpy(), want[1])
        self.same()
        return flags

    def fork(self, pa, parents):
        parents = np.asarray(parents, np.int32)
        t2, l2 = np.full((len(parents), self.tables.shape[1]), -5, np.int32), np.full(len(parents), -5, np.int32)
        dt, dl = dev(t2), dev(l2)
        pa.pa_fork_blocks(dt, dl, self.d_tables, self.d_lens, dev(parents), self.d_refs, self.bs)
        oracle.fork_blocks(t2, l2, self.tables, self.lens, parents, self.refs, self.bs)
        self.same()
        assert np.array_equal(dt.cpu().numpy(), t2) and np.array_equal(dl.cpu().numpy(), l2)
        return t2, l2, dt, dl

    def release(self, pa, keep=None):
        keep = None if keep is None else np.asarray(keep, np.int32)
        pa.pa_release_blocks(self.d_tables, self.d_lens, self.d_refs, self.bs, None if keep is None else dev(keep))
        oracle.release_blocks(self.tables, self.lens, self.refs, self.bs, keep)
        self.same()

    def take(self, rows):
        self.tables, self.lens, self.d_tables, self.d_lens = rows
        self.rows = len(self.lens)


@pytest.mark.parametrize("rows,width,blocks,bs,most", [(1, 5, 9, 16, 20), (4, 13, 64, 16, 9), (7, 40, 300, 4, 17),
                                                       (33, 9, 4000, 1, 3), (130, 20, 3000, 32, 70)])
def test_random_histories(pa, rows, width, blocks, bs, most):
    rng = np.random.default_rng(31)
    p = Pool(rows, width, blocks, bs)
    for step in range(40):
        op = rng.integers(4) if step else 0
        if op <= 1:
            add = np.minimum(rng.integers(0, most, rows), width * bs - p.lens)
            p.append(pa, add)
        elif op == 2:
            children = p.fork(pa, rng.integers(-1, rows, rows))
            p.release(pa)
            p.take(children)
        else:
            p.release(pa, rng.integers(0, width * bs, rows))
    assert pa.pa_get_error_flags(clear=True) == 0
    p.release(pa)
    assert not p.refs.any()


@pytest.mark.parametrize("rows", [1000, 1024, 1025, 2600, 8192])
def test_many_rows_share_few_tails(pa, rows):
    rng = np.random.default_rng(32)
    p = Pool(5, 6, 4 * rows + 50, 16)
    p.append(pa, [20, 32, 1, 0, 47])
    held = (p.tables, p.lens, p.d_tables, p.d_lens)
    children = p.fork(pa, rng.integers(-1, 5, rows))
    p.take(children)
    p.append(pa, rng.integers(0, 20, rows))     # the parents still hold their tails: every child copies
    p.release(pa)
    p.take(held)
    children = p.fork(pa, rng.integers(0, 5, rows))
    p.release(pa)
    p.take(children)
    p.append(pa, np.ones(rows, int))            # of a tail's holders the last keeps it
    p.release(pa)
    assert not p.refs.any()


def test_long_rows_and_a_large_pool(pa):
    rng = np.random.default_rng(33)
    p = Pool(3, 16400, 150000, 16)
    order = rng.permutation(150000)
    for i, n in enumerate((262144, 262100, 5)):
        k = -(-n // 16)
        p.tables[i, :k] = order[i * 16400:i * 16400 + k]
        p.refs[p.tables[i, :k]] = 1
        p.lens[i] = n
    p.refs[:140000][p.refs[:140000] == 0] = 3   # free blocks only at the pool's end
    p.to_device()
    base = (p.tables, p.lens, p.d_tables, p.d_lens)
    children = p.fork(pa, [0, 1, 1, 2, 0, 1, 2, 0])
    p.take(children)
    p.append(pa, [1, 7, 40, 3, 17, 0, 100, 200])
    p.release(pa, [262144, 100, 0, 5, 262145, 262090, 3, 131072])
    p.release(pa)
    p.take(base)
    p.release(pa)
    assert pa.pa_get_error_flags(clear=True) == 0


def test_prompts_of_one_token_to_thousands(pa):
    p = Pool(6, 600, 2000, 16)
    p.append(pa, [1, 0, 4097, 16, 15, 9000])
    p.append(pa, [0, 8191, 1, 1, 1, 600])
    p.append(pa, [0] * 6)                       # nothing to add
    assert pa.pa_get_error_flags(clear=True) == 0


@pytest.mark.parametrize("bs", [1, 7, 16])
def test_long_prompts_among_short_ones(pa, bs):
    """Rows that grow by nothing, one block and thousands of blocks in one call, and then one
    token each: threads write some blocks alone, others together."""
    rng = np.random.default_rng(34)
    p = Pool(70, 9100, 40000, bs)
    add = rng.integers(0, 4, 70) * bs
    add[[3, 4, 40, 69]] = [9000 * bs, 33 * bs + 1, 3 * bs, 8191 * bs - 1]
    p.append(pa, add)
    p.append(pa, np.ones(70, int))
    p.append(pa, rng.integers(0, 9, 70))         # slots across block borders, eight tokens at most
    p.release(pa)
    assert pa.pa_get_error_flags(clear=True) == 0 and not p.refs.any()


def test_fork_by_children_and_by_parents(pa):
    """More children than the parents' way takes, more parents than children, none."""
    rng = np.random.default_rng(35)
    p = Pool(40, 30, 3000, 16)
    p.append(pa, rng.integers(0, 480, 40))
    for n in (1, 39, 40, 41, 1024, 1025):
        t2, l2, dt, dl = p.fork(pa, rng.integers(-2, 40, n))
        q = Pool(n, 30, 3000, 16)
        q.refs, q.d_refs = p.refs, p.d_refs
        q.take((t2, l2, dt, dl))
        q.release(pa)
    p.same()
    empty = torch.zeros(0, 30, dtype=torch.int32, device=DEV)
    out, lens = torch.full((3, 30), 5, dtype=torch.int32, device=DEV), torch.full((3,), 5, dtype=torch.int32, device=DEV)
    pa.pa_fork_blocks(out, lens, empty, empty[:, 0].contiguous(), dev(np.array([-1, -7, -1], np.int32)), p.d_refs, 16)
    assert lens.tolist() == [0, 0, 0] and bool((out == 5).all())
    assert pa.pa_get_error_flags(clear=True) == 0


@pytest.mark.parametrize("parents,children", [(1, 70), (1, 1100), (5, 300), (5, 2500), (150, 300), (151, 300)])
def test_fork_of_long_tables(pa, parents, children):
    """Tables wide enough that children are dealt with by their parents."""
    rng = np.random.default_rng(36)
    width = 8000
    p = Pool(parents, width, 40000, 1)
    lens = rng.integers(0, 100, parents)
    lens[0] = 1200 if children <= 300 else 300
    p.append(pa, lens)
    for low, high in ((-1, parents), (parents - 1, parents), (-3, -1), (-1, parents + 2)):
        chosen = rng.integers(low, high, children)
        t2, l2, dt, dl = p.fork(pa, chosen)
        assert pa.pa_get_error_flags(clear=True) == (pa.PA_ERRFLAG_PARENT if (chosen >= parents).any() else 0)
        q = Pool(children, width, 40000, 1)
        q.refs, q.d_refs = p.refs, p.d_refs
        q.take((t2, l2, dt, dl))
        q.release(pa)
        p.same()


def test_too_few_free_blocks_change_nothing(pa):
    p = Pool(4, 8, 10, 16)
    assert p.append(pa, [40, 40, 40, 0]) == 0    # nine of ten
    assert p.append(pa, [16, 0, 16, 0]) == pa.PA_ERRFLAG_POOL
    children = p.fork(pa, [0, 0, 0, 0])
    parent = (p.tables, p.lens, p.d_tables, p.d_lens)
    p.take(children)
    assert p.append(pa, [1, 1, 1, 1]) == pa.PA_ERRFLAG_POOL   # four copies of the tail, one free block
    assert p.append(pa, [1, 0, 0, 0]) == 0
    p.release(pa)
    p.take(parent)
    p.release(pa)
    assert not p.refs.any()


def test_inputs_out_of_range_change_nothing(pa):
    p = Pool(3, 4, 20, 16)
    p.append(pa, [10, 20, 0])

    def refused(flag, qsl=(0, 1, 2, 3), total=3, **edits):
        saved = p.tables.copy(), p.lens.copy(), p.refs.copy()
        for name, (at, v) in edits.items():
            getattr(p, name)[at] = v
        p.to_device()
        slots = torch.full((total,), 77, dtype=torch.int64, device=DEV)
        pairs = torch.full((3, 2), 77, dtype=torch.int64, device=DEV)
        ws = pa.workspace_tensor(pa.pa_append_workspace_size(3, total, 16))
        pa.pa_append_blocks(p.d_tables, p.d_lens, dev(np.array(qsl, np.int32)), slots, pairs, p.d_refs, 16, ws)
        assert pa.pa_get_error_flags(clear=True) == flag
        assert bool((slots == -1).all()) and not bool(pairs.any())
        p.same()
        p.tables, p.lens, p.refs = saved
        p.to_device()

    refused(pa.PA_ERRFLAG_QUERY, qsl=(1, 1, 2, 3))
    refused(pa.PA_ERRFLAG_QUERY, qsl=(0, 1, 2, 4))
    refused(pa.PA_ERRFLAG_QUERY, qsl=(0, 2, 1, 3))
    refused(pa.PA_ERRFLAG_QUERY | pa.PA_ERRFLAG_SEQ_LEN, qsl=(0, 2 ** 31 - 1, -2 ** 31, 3))
    refused(pa.PA_ERRFLAG_SEQ_LEN, lens=(0, -1))
    refused(pa.PA_ERRFLAG_SEQ_LEN, lens=(0, 64))
    refused(pa.PA_ERRFLAG_SEQ_LEN, lens=(2, 2 ** 31 - 1))
    refused(pa.PA_ERRFLAG_BLOCK_TABLE, tables=((1, 1), 20))
    refused(pa.PA_ERRFLAG_BLOCK_TABLE, tables=((0, 0), -1))
    refused(pa.PA_ERRFLAG_REF_COUNT, refs=(int(p.tables[1, 1]), 0))
    assert p.append(pa, [1, 1, 1]) == 0


def test_fork_edges(pa):
    p = Pool(3, 6, 30, 16)
    p.append(pa, [96, 0, 17])                    # a full row, an empty one
    p.fork(pa, [0, 1, 2, -1, -2 ** 31, 2, 2])
    assert pa.pa_get_error_flags(clear=True) == 0
    p.fork(pa, [3, 0, 2 ** 31 - 1])
    assert pa.pa_get_error_flags(clear=True) == pa.PA_ERRFLAG_PARENT
    p.lens[0], p.lens[1] = 97, -4                # lengths that are none
    p.to_device()
    p.fork(pa, [0, 1, 2])
    assert pa.pa_get_error_flags(clear=True) == pa.PA_ERRFLAG_SEQ_LEN
    p.lens[0], p.lens[1] = 96, 0
    p.tables[0, :3] = [-1, -1, 30]               # released before a window; out of range
    p.to_device()
    p.fork(pa, [0, 0])
    assert pa.pa_get_error_flags(clear=True) == pa.PA_ERRFLAG_BLOCK_TABLE
    p.release(pa, [40, 0, 0])
    assert pa.pa_get_error_flags(clear=True) == 0
    p.release(pa)
    assert pa.pa_get_error_flags(clear=True) == pa.PA_ERRFLAG_BLOCK_TABLE


def test_release_edges(pa):
    p = Pool(4, 5, 30, 16)
    p.append(pa, [80, 33, 1, 16])
    p.release(pa, [80, 33, 5, 2 ** 31 - 1])      # nothing to give up
    p.release(pa, [79, 32, 0, 0])
    p.release(pa, [79, 32, 0, 0])                # again: harmless
    assert pa.pa_get_error_flags(clear=True) == 0
    p.release(pa, [-1, 16, 0, 0])
    assert pa.pa_get_error_flags(clear=True) == pa.PA_ERRFLAG_SEQ_LEN
    p.refs[p.tables[0, 1]] = 0                   # books that do not balance
    p.to_device()
    p.release(pa)
    assert pa.pa_get_error_flags(clear=True) == pa.PA_ERRFLAG_REF_COUNT
    p.lens[2] = 81
    p.to_device()
    p.release(pa)
    assert pa.pa_get_error_flags(clear=True) == pa.PA_ERRFLAG_SEQ_LEN


def test_forking_into_other_rows_of_the_same_arrays(pa):
    p = Pool(8, 4, 40, 16)
    p.append(pa, [20, 30, 0, 0, 0, 0, 0, 0])
    want_t, want_l = p.tables.copy(), p.lens.copy()
    oracle.fork_blocks(want_t[2:], want_l[2:], p.tables[:2], p.lens[:2], [0, 1, 1, 0, 1, -1], p.refs, 16)
    pa.pa_fork_blocks(p.d_tables[2:], p.d_lens[2:], p.d_tables[:2], p.d_lens[:2],
                      dev(np.array([0, 1, 1, 0, 1, -1], np.int32)), p.d_refs, 16)
    p.tables, p.lens = want_t, want_l
    p.same()
    with pytest.raises(pa.PAError):
        pa.pa_fork_blocks(p.d_tables[1:3], p.d_lens[1:3], p.d_tables[:2], p.d_lens[:2],
                          dev(np.array([0, 1], np.int32)), p.d_refs, 16)


def test_replayed_from_a_graph_on_another_stream(pa):
    p = Pool(6, 30, 400, 16)
    p.append(pa, [100, 33, 64, 1, 0, 200])
    refs0 = p.d_refs.clone()
    tables = torch.full((9, 30), -1, dtype=torch.int32, device=DEV)
    lens = torch.zeros(9, dtype=torch.int32, device=DEV)
    parents = dev(np.array([0, 0, 1, 5, 5, 5, 3, 2, 4], np.int32))
    qsl = dev(np.arange(0, 28, 3, dtype=np.int32))
    slots = torch.zeros(27, dtype=torch.int64, device=DEV)
    pairs = torch.zeros(9, 2, dtype=torch.int64, device=DEV)
    ws = pa.workspace_tensor(pa.pa_append_workspace_size(9, 27, 16))
    between = torch.zeros_like(refs0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())

    def life():
        pa.pa_fork_blocks(tables, lens, p.d_tables, p.d_lens, parents, p.d_refs, 16)
        pa.pa_append_blocks(tables, lens, qsl, slots, pairs, p.d_refs, 16, ws)
        between.copy_(p.d_refs)
        pa.pa_release_blocks(tables, lens, p.d_refs, 16)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        life()
    t2, l2, r2 = np.full((9, 30), -1, np.int32), np.zeros(9, np.int32), p.refs.copy()
    oracle.fork_blocks(t2, l2, p.tables, p.lens, parents.cpu().numpy(), r2, 16)
    want = oracle.append_blocks(t2, l2, qsl.cpu().numpy(), r2, 16)
    for _ in range(3):
        for t in (slots, pairs, between):
            t.fill_(-3)
        graph.replay()
        torch.cuda.synchronize()
        assert pa.pa_get_error_flags(clear=True) == 0
        assert np.array_equal(slots.cpu().numpy(), want[0]) and np.array_equal(pairs.cpu().numpy(), want[1])
        assert np.array_equal(between.cpu().numpy(), r2)
        assert torch.equal(p.d_refs, refs0) and not bool(lens.any())


def test_slots_behind_2_to_32(pa):
    """A pool whose last blocks alone are free, their slots behind 2^32."""
    blocks, bs = 2 ** 27 + 5, 64
    refs = torch.ones(blocks, dtype=torch.int32, device=DEV)
    refs[-3:] = 0
    tables, lens = torch.full((2, 4), -1, dtype=torch.int32, device=DEV), torch.zeros(2, dtype=torch.int32, device=DEV)
    slots, pairs = torch.zeros(80, dtype=torch.int64, device=DEV), torch.zeros(2, 2, dtype=torch.int64, device=DEV)
    ws = pa.workspace_tensor(pa.pa_append_workspace_size(2, 80, bs))
    pa.pa_append_blocks(tables, lens, dev(np.array([0, 70, 80], np.int32)), slots, pairs, refs, bs, ws)
    first = (blocks - 3) * bs
    assert slots.tolist() == list(range(first, first + 70)) + list(range(first + 2 * bs, first + 2 * bs + 10))
    assert refs[-4:].tolist() == [1, 1, 1, 1] and not bool(pairs.any())
    pa.pa_release_blocks(tables, lens, refs, bs)
    assert refs[-4:].tolist() == [1, 0, 0, 0] and pa.pa_get_error_flags(clear=True) == 0

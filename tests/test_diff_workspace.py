"""CPU: one workspace serves every smaller batch.  The default partitions of differential attention grow
finer as a batch shrinks; the sizes that the library names are bounds over all of that.

Whether a call takes a size is seen from its refusal: the output lies in the workspace, which is
PA_ERR_WORKSPACE where the workspace is too small and PA_ERR_INVALID_ARG where it is not.  Nothing is
launched, and no address is touched."""

import random

import pytest

WS = 1 << 44


@pytest.fixture(scope="module")
def pa():
    import __graft_entry__ as g
    g.build()
    import paged_kv_cache_pagedattention_gb300 as lib
    return lib


SHAPES = [(32, 8, 128, 16), (64, 8, 128, 32), (16, 16, 64, 16), (8, 4, 64, 64), (2, 2, 256, 16), (24, 4, 128, 48),
          (144, 8, 64, 16), (6, 2, 80, 5)]


def decode(pa, shape, n, longest, size, window=0):
    hq, hkv, d, bs = shape
    return pa._lib.pa_diff_decode(WS, 1 << 40, 2 << 40, 3 << 40, 10, 1 << 20, 4, 1 << 20, n, longest, hq, hkv, d, bs,
                                  0.1, 4 << 40, hq // 2, 1, None, 1e-5, window, 2, 2, None, None, 0, WS, size, None)


def varlen(pa, shape, n, t, most, longest, size, window=0):
    hq, hkv, d, bs = shape
    return pa._lib.pa_diff_varlen_attn(WS, 1 << 40, 2 << 40, 3 << 40, 10, 1 << 20, 4, 1 << 20, 1 << 20, n, t, most,
                                       longest, hq, hkv, d, bs, 0.1, 4 << 40, hq // 2, 1, None, 1e-5, window, 1, 2, 2,
                                       None, None, 0, WS, size, None)


def decode_size(pa, shape, n, longest, part=0):
    hq, hkv, d, bs = shape
    return pa.pa_diff_decode_workspace_size(n, hq, hkv, d, longest, bs, part)


def varlen_size(pa, shape, n, t, most, longest, part=0):
    hq, hkv, d, bs = shape
    return pa.pa_diff_varlen_workspace_size(n, t, most, hq, hkv, d, longest, bs, part)


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("longest", [100, 4096, 32768, 131072, 5_000_000])
def test_decode_sizes_hold_for_smaller_batches(pa, shape, longest):
    rng = random.Random(f"{shape}{longest}")
    size = decode_size(pa, shape, 512, longest)
    last = 0
    for n in range(1, 513):
        own = decode_size(pa, shape, n, longest)
        assert last <= own <= size
        last = own
        shorter = rng.randint(1, longest)
        assert decode_size(pa, shape, n, shorter) <= own
        for at in (longest, shorter):
            assert decode(pa, shape, n, at, decode_size(pa, shape, n, at)) == pa.PA_ERR_INVALID_ARG, (n, at)
            assert decode(pa, shape, n, at, size, rng.choice([0, 1, 1000])) == pa.PA_ERR_INVALID_ARG, (n, at)
    assert decode(pa, shape, 512, longest, 512) == pa.PA_ERR_WORKSPACE


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_varlen_sizes_hold_for_smaller_batches(pa, shape):
    rng = random.Random(str(shape))
    log = lambda lo, hi: max(lo, min(hi, int(lo * (hi / lo) ** rng.random() + 0.5)))  # noqa: E731
    for _ in range(300):
        n, longest = log(1, 2000), log(1, 200_000)
        t = n + log(1, 8192)
        most = rng.randint(1, t)
        size = varlen_size(pa, shape, n, t, most, longest)
        for _ in range(12):
            n2, longest2 = log(1, n), log(1, longest)
            t2 = log(1, t)
            most2 = rng.randint(1, most)
            own = varlen_size(pa, shape, n2, t2, most2, longest2)
            assert own <= size
            assert varlen(pa, shape, n2, t2, most2, longest2, own) == pa.PA_ERR_INVALID_ARG, (n2, t2, most2, longest2)
            assert varlen(pa, shape, n2, t2, most2, longest2, size) == pa.PA_ERR_INVALID_ARG
    assert varlen(pa, shape, 4, 50, 20, 4096, 1024) == pa.PA_ERR_WORKSPACE


def test_batches_that_asked_for_more_when_smaller(pa):
    """32/8 heads of 128: 455 sequences of 32,768 tokens, 300 new tokens, 64 requests of up to 5 tokens."""
    shape = SHAPES[0]
    assert decode(pa, shape, 455, 32768, decode_size(pa, shape, 512, 32768)) == pa.PA_ERR_INVALID_ARG
    assert varlen(pa, shape, 1, 300, 300, 32768, varlen_size(pa, shape, 1, 512, 512, 32768)) == pa.PA_ERR_INVALID_ARG
    assert varlen(pa, shape, 64, 68, 5, 65536, varlen_size(pa, shape, 64, 320, 256, 65536)) == pa.PA_ERR_INVALID_ARG


def test_partitions_of_the_caller(pa):
    for shape in SHAPES:
        part = 64 * shape[3]
        sizes = [varlen_size(pa, shape, n, t, 9, longest, part)
                 for n, t, longest in ((1, 9, 700), (3, 9, 700), (3, 30, 700), (3, 30, 70000))]
        assert sizes == sorted(sizes)
        sizes = [decode_size(pa, shape, n, longest, part) for n, longest in ((1, 700), (9, 700), (9, 70000))]
        assert sizes == sorted(sizes)


def test_few_tokens_of_chunks_beside_many_single_tokens(pa):
    """States of every row at the finest split of a chunk would take gigabytes."""
    assert varlen_size(pa, SHAPES[0], 1001, 1004, 4, 32768) < 400 << 20
    assert varlen_size(pa, SHAPES[0], 4097, 4100, 4, 32768) < 800 << 20

"""GPU: differential attention within its counted roundings (see diff_roundings): single-token rows whose
weights keep two 16-bit numbers, maxima that rise, FP8 caches by the values that they hold."""

import pytest

from tests.diff_roundings import CountedDiff, short_contexts
from tests.test_gpu_diff import growing, poison

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pa():
    import paged_kv_cache_pagedattention_gb300 as lib
    lib.pa_get_error_flags(clear=True)
    return lib


@pytest.mark.parametrize("kv,qd", [("bf16", None), ("f16", None), ("fp8_e4m3", "f16"), ("fp8_e5m2", "f16"),
                                   ("fp8_e4m3", "bf16"), ("fp8_e5m2", "bf16")])
@pytest.mark.parametrize("hq", [16, 64, 88])
def test_weights_of_single_tokens(pa, kv, qd, hq):
    """Up to four heads a group, eight, eleven: both ways of placing the columns."""
    c = short_contexts(kv, qd, hq, seed=70 + hq)
    c.dev = "cuda:0"
    poison(c)
    c.to_device()
    for varlen in (False, True):
        c.out.fill_(9.0)
        c.call(pa, varlen)
        c.check()
    assert pa.pa_get_error_flags(clear=True) == 0


@pytest.mark.parametrize("kv,qd,hq,d,bs", [
    ("bf16", None, 16, 128, 16), ("f16", None, 16, 128, 32), ("bf16", None, 40, 128, 64), ("f16", None, 16, 64, 16),
    ("bf16", None, 8, 64, 64), ("fp8_e4m3", "bf16", 16, 128, 16), ("fp8_e4m3", "f16", 64, 128, 64),
    ("fp8_e5m2", "f16", 64, 128, 32), ("fp8_e5m2", "bf16", 24, 128, 16), ("f32", None, 8, 64, 16),
    ("fp8_e5m2", "bf16", 8, 64, 16), ("fp8_e4m3", "f32", 8, 128, 16), ("f16", None, 8, 128, 48)])
@pytest.mark.parametrize("part", [0, 192])
@pytest.mark.parametrize("norm", [False, True])
def test_maxima_that_rise(pa, kv, qd, hq, d, bs, part, norm):
    for new in ([1, 1, 1], [300, 1, 90], [129, 40, 200]):
        c = CountedDiff([900, 333, 600], new, hq, 4, d, bs, kv, qd, norm=norm, seed=31,
                        cache_scale=0.25 if kv[:3] == "fp8" else None)
        growing(c)
        poison(c)
        c.to_device()
        for varlen in (True, False) if max(new) == 1 else (True,):
            c.out.fill_(9.0)
            c.call(pa, varlen, part)
            c.check()
    assert pa.pa_get_error_flags(clear=True) == 0


@pytest.mark.parametrize("kv,qd,d,bs", [("bf16", None, 128, 32), ("f16", None, 64, 16), ("fp8_e5m2", "bf16", 128, 16),
                                        ("nvfp4", "bf16", 128, 16), ("f32", None, 64, 16)])
@pytest.mark.parametrize("window", [0, 100])
def test_contexts_of_many_partitions(pa, kv, qd, d, bs, window):
    lens, new = [2500, 1, 700, 1300], [1, 1, 1, 70]
    c = CountedDiff(lens, new, 16, 4, d, bs, kv, qd, window, seed=32, per_token=True)
    c.to_device()
    c.call(pa, True)
    c.check()
    c.call(pa, True, 128 if 128 % bs == 0 else bs)
    c.check()
    assert pa.pa_get_error_flags(clear=True) == 0

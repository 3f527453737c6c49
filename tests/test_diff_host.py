"""CPU: the differential-attention oracle against closed forms and the plain attention oracle, its
tolerance against plain fp32 roundings, and what pa_diff_decode and pa_diff_varlen_attn refuse."""

import numpy as np
import pytest
import torch

import oracle
import workloads
from tests.diff_harness import Diff


@pytest.fixture(scope="module")
def pa():
    import __graft_entry__ as g
    g.build()
    import paged_kv_cache_pagedattention_gb300 as lib
    return lib


def test_by_hand():
    """Two keys, equal scores in map 2: one softmax minus a mean."""
    q, k = np.array([[1.0]]), np.array([[0.0], [np.log(3.0)]])
    v = np.array([[1.0, 0.0], [5.0, 4.0]])
    a, _, _ = oracle.diff_map(q, k, v, [1], 1.0)
    assert np.allclose(a, [[4.0, 3.0]])                                # weights 1/4, 3/4
    b, _, _ = oracle.diff_map(q * 0, k, v, [1], 1.0)
    assert np.allclose(b, [[3.0, 2.0]])
    o = a - 0.5 * b
    assert np.allclose(o, [[2.5, 2.0]])
    assert np.allclose(oracle.diff_norm(o, [1.0, 2.0], 0.0), o / np.sqrt((2.5 ** 2 + 2.0 ** 2) / 2) * [1.0, 2.0])
    assert oracle.diff_norm(o, None, 0.0) is o
    first, _, _ = oracle.diff_map(np.array([[1.0], [1.0]]), k, v, [0, 1], 1.0)
    assert np.allclose(first[0], v[0])                                 # one key: its value
    none, _, _ = oracle.diff_map(q, k, v, [1], 1.0, readable=[False, False])
    assert np.array_equal(none, [[0.0, 0.0]])


@pytest.mark.parametrize("window", [0, 7])
@pytest.mark.parametrize("per_token", [False, True])
def test_against_plain_attention(window, per_token):
    """Four plain attentions, one for each map and value half, make the difference."""
    c = Diff([40, 9, 33], [12, 1, 33], 12, 4, 16, 8, "f32", window=window, norm=False, per_token=per_token, dev="cpu")
    b = c.b
    out, diff, spread, reach, keys = c.oracle()
    assert np.array_equal(out, diff) and np.all(spread >= np.abs(diff) - 1e-12) and np.all(reach > 0)
    lam = np.broadcast_to(c.lam.astype(np.float64), (b.total_q, 6))
    plain = lambda q, k, v: oracle.paged_varlen(q, "f32", k, v, "f32", b.block_tables, b.query_start_loc,  # noqa: E731
                                                b.seq_lens, 8, b.scale, True, window=window)
    for h in range(6):
        g = h // 3
        halves = []
        for half in (0, 1):
            a = [plain(b.q[:, 2 * h + j:2 * h + j + 1], b.k_cache[:, 2 * g + j:2 * g + j + 1],
                       b.v_cache[:, 2 * g + half:2 * g + half + 1])[:, 0] for j in (0, 1)]
            halves.append(a[0] - lam[:, h, None] * a[1])
        assert np.allclose(np.concatenate(halves, 1), out[:, h], rtol=0, atol=1e-12)


@pytest.mark.parametrize("kv", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("norm", [False, True])
def test_the_tolerance_holds_for_plain_roundings(kv, norm):
    """fp32 tensor operations with the weights rounded as the kernels round them stay inside."""
    c = Diff([300, 61], [1, 20], 8, 4, 64, 16, kv, norm=norm, dev="cpu")
    b = c.b
    want = c.oracle()
    got = np.zeros_like(want[0])
    q = workloads.bits_to_torch(b.q, kv).float()
    wt = workloads.torch_dtype(kv)
    for r in range(2):
        lo, hi, n = int(b.query_start_loc[r]), int(b.query_start_loc[r + 1]), int(b.seq_lens[r])
        K, V = (torch.from_numpy(oracle.gather_kv(x, b.block_tables[r], n, 16, kv)).float() for x in (b.k_cache, b.v_cache))
        keep = torch.arange(n)[None] <= torch.arange(n - (hi - lo), n)[:, None]
        for h in range(4):
            g = h // 2
            v = torch.cat((V[:, 2 * g], V[:, 2 * g + 1]), 1)
            o = []
            for j in (0, 1):
                s = (q[lo:hi, 2 * h + j] @ K[:, 2 * g + j].T * b.scale).masked_fill(~keep, -np.inf)
                w = (s - s.amax(1, keepdim=True)).exp().to(wt).float()
                o.append(w @ v / w.sum(1, keepdim=True))
            x = o[0] - float(c.lam[h]) * o[1]
            if norm:
                x = x * torch.rsqrt((x * x).mean(1, keepdim=True) + 1e-5) * torch.from_numpy(c.norm)
            got[lo:hi, h] = x.to(wt).double().numpy()
    assert np.all(np.abs(got - want[0]) <= c.tolerance(*want))


F = 1 << 20  # an aligned address that no refused call touches


def decode(pa, **kw):
    a = dict(out=F, q=F + (1 << 20), k=F + (2 << 20), v=F + (3 << 20), nb=10, tables=F, width=4, lens=F, n=2, longest=64,
             hq=8, hkv=4, d=128, bs=16, scale=0.1, lam=F + (9 << 20), ls=4, lh=1, norm=None, eps=1e-5, window=0, qd=2, kd=2,
             ks=None, vs=None, part=0, ws=F + (16 << 20), size=1 << 40, stream=None)
    a.update(kw)
    return pa._lib.pa_diff_decode(*a.values())


def varlen(pa, **kw):
    a = dict(out=F, q=F + (1 << 20), k=F + (2 << 20), v=F + (3 << 20), nb=10, tables=F, width=4, qsl=F, lens=F, n=2, t=5,
             most=4, longest=64, hq=8, hkv=4, d=128, bs=16, scale=0.1, lam=F + (9 << 20), ls=4, lh=1, norm=None, eps=1e-5,
             window=0, causal=1, qd=2, kd=2, ks=None, vs=None, part=0, ws=F + (16 << 20), size=1 << 40, stream=None)
    a.update(kw)
    return pa._lib.pa_diff_varlen_attn(*a.values())


@pytest.mark.parametrize("fn", [decode, varlen])
def test_refusals(pa, fn):
    bad, no, small = pa.PA_ERR_INVALID_ARG, pa.PA_ERR_UNSUPPORTED, pa.PA_ERR_WORKSPACE
    assert fn(pa, n=0) == pa.PA_OK
    for kw in (dict(n=-1), dict(hq=7), dict(hq=6, hkv=3), dict(hq=9, hkv=3), dict(hkv=3), dict(hq=10), dict(hkv=1, hq=2),
               dict(lam=None), dict(ls=-1), dict(lh=-1), dict(scale=0.0), dict(scale=float("nan")), dict(window=-1),
               dict(norm=F + (11 << 20), eps=0.0), dict(norm=F + (11 << 20), eps=float("inf")), dict(out=F + 8),
               dict(q=F + (1 << 20) + 2), dict(lam=F + (9 << 20) + 1), dict(out=None), dict(q=None), dict(k=None),
               dict(ws=None), dict(part=8), dict(bs=0), dict(d=0), dict(longest=0), dict(kd=3)):
        assert fn(pa, **kw) == bad, kw
    # written over what is read
    for kw in (dict(out=F + (1 << 20)), dict(out=F + (1 << 20) - 16), dict(out=F + (2 << 20) + 4096), dict(out=F + (3 << 20)),
               dict(out=F + (9 << 20)), dict(norm=F + 16), dict(out=F + (16 << 20) + 256)):
        assert fn(pa, **kw) == bad, kw
    for kw in (dict(longest=(1 << 30) + 1), dict(part=(1 << 30) + 16), dict(hq=131072, hkv=2), dict(d=264), dict(qd=3), dict(kd=1), dict(kd=99), dict(kd=7, d=24, ks=F, vs=F), dict(ls=1 << 61),
               dict(lh=1 << 61)):
        assert fn(pa, **kw) == no, kw
    assert fn(pa, ws=F + (16 << 20) + 16) == small
    assert fn(pa, size=255) == small
    if fn is varlen:
        assert fn(pa, t=0) == pa.PA_OK
        assert fn(pa, t=-1) == fn(pa, qsl=None) == fn(pa, most=0) == bad
        assert fn(pa, window=4, causal=0) == no


def test_workspace_sizes(pa):
    size = lambda part, n=4: pa.pa_diff_decode_workspace_size(n, 8, 4, 128, 4096, 16, part)  # noqa: E731
    assert pa.pa_diff_decode_workspace_size(0, 8, 4, 128, 4096, 16) == 256
    # a partial state: a maximum and a sum, and twice the head's elements, for each query head
    assert size(512) == 256 + 4 * 8 * 8 * 8 + 4 * 8 * 8 * 256 * 4
    assert size(256) > size(512) and size(512, 5) > size(512)
    v = lambda t: pa.pa_diff_varlen_workspace_size(4, t, 9, 8, 4, 128, 4096, 16)  # noqa: E731
    assert v(0) == 256 and v(50) > v(20) > 256


def test_binding_refusals(pa):
    z = torch.zeros
    good = dict(out=z(2, 4, 256), q=z(2, 8, 128), k_cache=z(3, 4, 16, 128), v_cache=z(3, 4, 16, 128),
                block_tables=z(2, 5, dtype=torch.int32), seq_lens=z(2, dtype=torch.int32), max_seq_len=64, scale=0.1,
                lambda_=z(4), workspace=z(64, dtype=torch.uint8))
    for kw in (dict(out=z(2, 8, 128)), dict(out=z(2, 4, 256).half()), dict(q=z(2, 8, 64)), dict(q=z(2, 7, 128)),
               dict(q=z(16, 128)), dict(lambda_=z(3)), dict(lambda_=z(3, 4)), dict(lambda_=z(1, 1, 4)),
               dict(lambda_=z(4).double()), dict(norm_weight=z(128)), dict(norm_weight=z(256).half()),
               dict(seq_lens=z(2)), dict(block_tables=z(3, 5, dtype=torch.int32)), dict(v_cache=z(3, 4, 16, 64)),
               dict(k_cache=z(3, 3, 16, 128), v_cache=z(3, 3, 16, 128)), dict(q=z(8, 2, 128).transpose(0, 1)),
               dict(k_scale=z(3), v_scale=z(3)), dict(k_scale=z(1)), dict()):
        with pytest.raises(ValueError):
            pa.pa_diff_decode(**{**good, **kw})                        # the last: not on a CUDA device
        with pytest.raises(ValueError):
            args = {**good, **kw}
            pa.pa_diff_varlen_attn(query_start_loc=z(3, dtype=torch.int32), max_query_len=1, **args)

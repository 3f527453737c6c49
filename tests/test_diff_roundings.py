"""CPU: the counted tolerance of differential attention holds for the roundings that the kernels state,
and not for coarser ones: weights of single-token rows as one 16-bit number, a map's sums a fraction off."""

import numpy as np
import pytest
import torch

import oracle
import workloads
from tests.diff_roundings import CountedDiff, half_step, short_contexts
from tests.test_gpu_diff import growing


def attend(c, split, plant=None):
    """c's outputs by fp32 operations with the weights rounded as the kernels round them, to one 16-bit number or
    two; `plant` spoils a map's sums."""
    b = c.b
    fp8 = b.kv_dtype in workloads.FP8
    wt = torch.float16 if fp8 else workloads.torch_dtype(b.q_dtype)
    q = workloads.bits_to_torch(b.q, b.q_dtype).float()
    lam = np.broadcast_to(c.lam, (b.total_q, c.heads))
    got = np.zeros((b.total_q, c.heads, 2 * b.head_size))
    per = b.num_q_heads // b.num_kv_heads
    for r, n in enumerate(b.seq_lens):
        lo, hi, n = int(b.query_start_loc[r]), int(b.query_start_loc[r + 1]), int(n)
        K, V = (torch.from_numpy(oracle.gather_kv(x, b.block_tables[r], n, b.block_size, b.kv_dtype, s)).float()
                for x, s in ((b.k_cache, b.k_scale), (b.v_cache, b.v_scale)))
        keep = torch.arange(n)[None] <= torch.arange(n - (hi - lo), n)[:, None]
        for h in range(c.heads):
            g, o = h // per, []
            v = torch.cat((V[:, 2 * g], V[:, 2 * g + 1]), 1)
            for j in (0, 1):
                s = (q[lo:hi, 2 * h + j] @ K[:, 2 * g + j].T * b.scale).masked_fill(~keep, -np.inf)
                e = (s - s.amax(1, keepdim=True)).exp()
                w = e.to(wt).float()
                if split:
                    w = w + (e - w).to(wt).float()
                l = w.sum(1, keepdim=True) if fp8 and b.q_dtype == "bf16" and not split else e.sum(1, keepdim=True)
                o.append(w @ v / l if plant is None else plant(w, v, l, j))
            x = o[0] - torch.from_numpy(lam[lo:hi, h, None].astype(np.float32)) * o[1]
            got[lo:hi, h] = x.to(workloads.torch_dtype(b.q_dtype)).double().numpy()
    return torch.from_numpy(got)


@pytest.mark.parametrize("kv,qd", [("bf16", None), ("f16", None), ("fp8_e4m3", "f16"), ("fp8_e5m2", "f16")])
def test_one_number_a_weight_shows(kv, qd):
    c = short_contexts(kv, qd)
    assert c.check(attend(c, True)) <= 1.0
    with pytest.raises(AssertionError):
        c.check(attend(c, False))


@pytest.mark.parametrize("kv", ["fp8_e4m3", "fp8_e5m2"])
def test_one_number_where_it_is_stated(kv):
    c = short_contexts(kv, "bf16")
    assert c.check(attend(c, False)) <= 1.0


@pytest.mark.parametrize("kv,qd,hq", [("bf16", None, 8), ("fp8_e5m2", "f16", 8), ("fp8_e5m2", "bf16", 8), ("fp8_e4m3", "bf16", 8)])
@pytest.mark.parametrize("new", [[1, 1, 1], [129, 40, 200]])
def test_growing_maxima_leave_no_room(kv, qd, hq, new):
    """What an output may be off is a small part of it, and sums rescaled by a fiftieth too much show."""
    c = CountedDiff([900, 333, 600], new, hq, 4, 128, 32, kv, qd, norm=False, seed=31, dev="cpu",
                    cache_scale=0.25 if kv[:3] == "fp8" else None)
    growing(c)
    want = c.oracle()
    tol = c.tolerance(*want)
    assert np.median(tol) <= 0.03 * np.sqrt((want[0] ** 2).mean())
    single = new[0] == 1
    got = attend(c, single and not (kv[:3] == "fp8" and qd == "bf16"))
    assert c.check(got) <= 1.0

    def plant(w, v, l, j):  # of map 2, the keys that hold the first half of a row's weight
        early = w.cumsum(1) < w.sum(1, keepdim=True) / 2
        return (w * torch.where(early, 1.02 if j else 1.0, 1.0)) @ v / l
    with pytest.raises(AssertionError):
        c.check(attend(c, single, plant))


def test_half_steps():
    for dtype in ("f32", "f16", "bf16"):
        t = workloads.torch_dtype(dtype)
        x = torch.tensor([1.0, 1.5, 3.75, 1e-3, 6e-5, 3e-6, 1000.0]).to(t)
        up = torch.nextafter(x, torch.full_like(x, float("inf")))
        assert np.array_equal(half_step(x.double().numpy(), dtype), (up.double() - x.double()).numpy() / 2)

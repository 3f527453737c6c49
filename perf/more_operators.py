"""Cases of the operators for sequences of text and media, and of differential attention, on a
paged KV cache.

Three kinds of case, named by ``case["op"]``:

* ``positions``  a step's request lengths, block tables and media grids become the new tokens'
                 positions on three axes (time, height, width) and their cache slots.
* ``axes``       the new tokens' q and k are rotated, every pair by the position on its own axis;
                 k and v are written to their slots of the paged cache.
* ``diff``       differential attention over the paged cache: each head is the difference of two
                 softmax maps over one value row, single-token rows and chunks of new tokens alike,
                 with the heads' root-mean-square norm where the model has one.

``run`` computes a case with elementary torch operations, or, where ``own`` is true, with the
library's calls.
"""

import math

import numpy as np
import torch

own = False

_FLOAT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_CACHE = dict(_FLOAT, fp8_e4m3=torch.float8_e4m3fn, fp8_e5m2=torch.float8_e5m2)
_SIZE = {"f32": 4, "f16": 2, "bf16": 2, "fp8_e4m3": 1, "fp8_e5m2": 1}
_FP8_MAX = {"fp8_e4m3": 448.0, "fp8_e5m2": 57344.0}


def _positions(name, decodes, chunks, chunk, longest, media, block):
    return {"name": name, "op": "positions", "decodes": decodes, "chunks": chunks, "chunk": chunk, "longest": longest,
            "media": media, "block": block}


def _axes(name, tokens, q_heads, kv_heads, head, rot, cycled, layout, dtype, cache, block, far, pad):
    return {"name": name, "op": "axes", "tokens": tokens, "q_heads": q_heads, "kv_heads": kv_heads, "head": head,
            "rot": rot, "cycled": cycled, "layout": layout, "dtype": dtype, "cache": cache, "block": block, "far": far,
            "pad": pad}


def _diff(name, decodes, shortest, longest, chunks, chunk, before, q_heads, kv_heads, head, block, dtype, cache,
          window=0, norm=True, per_token=False):
    return {"name": name, "op": "diff", "decodes": decodes, "shortest": shortest, "longest": longest,
            "chunks": chunks, "chunk": chunk, "before": before, "q_heads": q_heads, "kv_heads": kv_heads,
            "head": head, "block": block, "dtype": dtype, "cache": cache, "window": window, "norm": norm,
            "per_token": per_token}


def listed():
    return [
        # a decode batch of conversations with up to 64 images each: the call's latency
        _positions("positions decode", 256, 0, 0, 32768, 64, 16),
        # prompts of long videos, up to 700 frames in each, and some decodes beside them
        _positions("positions videos", 33, 15, 8191, 131072, 700, 16),
        # one sequence decoding alone
        _axes("axes one token", 1, 28, 4, 128, 128, False, "half", "bf16", "bf16", 16, 4096, 0),
        # a mixed step onto an FP8 cache, axes dealt round pair by pair
        _axes("axes mixed fp8", 2176, 32, 8, 128, 128, True, "half", "bf16", "fp8_e4m3", 32, 65536, 0),
        # long video prefill of a large model, half of the head rotated, pairs side by side, padded at its end
        _axes("axes video prefill", 8192, 64, 8, 128, 64, False, "interleaved", "f16", "f16", 16, 262144, 61),
        # four short sequences of a small fp32 model: the call's latency
        _diff("diff f32 tiny", 4, 17, 200, 0, 0, 0, 8, 4, 64, 16, "f32", "f32"),
        # an ordinary decode batch
        _diff("diff decode batch", 64, 512, 4096, 0, 0, 0, 32, 8, 128, 16, "bf16", "bf16"),
        # a few long contexts, eight heads to a pair of KV heads: the work has to be split over the context
        _diff("diff decode long", 3, 98304, 131072, 0, 0, 0, 64, 8, 128, 16, "f16", "f16", 0, True, True),
        # a large decode batch with a sliding window on an FP8 cache; blocks before the window are given back
        _diff("diff decode fp8 window", 256, 1024, 32768, 0, 0, 0, 32, 8, 128, 32, "bf16", "fp8_e4m3", 4096, False),
        # one short question on a cached prompt, small heads
        _diff("diff question", 0, 0, 0, 1, 37, 1000, 16, 8, 64, 16, "bf16", "bf16"),
        # a mixed step: four prefill chunks of 512 tokens on prefixes of up to 64K, and 128 decodes
        _diff("diff mixed step", 128, 512, 8192, 4, 512, 65536, 32, 8, 128, 16, "bf16", "bf16", 0, True, True),
        # a long prompt in one piece
        _diff("diff long prefill", 0, 0, 0, 1, 8192, 0, 32, 8, 128, 16, "bf16", "bf16"),
    ]


def _log_range(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["positions", "axes", "diff", "diff"])
    if op == "positions":
        longest = _log_range(rng, 256, 131072)
        chunks = rng.choice([0, 1, 2, 7, 15])
        chunk = _log_range(rng, 2, min(8191, longest)) if chunks else 0
        decodes = _log_range(rng, 1, 256) if not chunks or rng.random() < 0.5 else 0
        case = _positions("", decodes, chunks, chunk, longest, _log_range(rng, 1, max(1, min(700, longest // 64))),
                          rng.choice([16, 32, 64]))
    elif op == "axes":
        q_heads, kv_heads = rng.choice([(8, 2), (16, 2), (28, 4), (32, 8), (40, 8), (64, 8)])
        head = rng.choice([64, 128])
        dtype = rng.choice(["f32", "f16", "bf16", "bf16"])
        tokens = _log_range(rng, 1, min(8192, 8192 * 64 * 128 // (q_heads * head)) // (2 if dtype == "f32" else 1))
        case = _axes("", tokens, q_heads, kv_heads, head, rng.choice([head, head, head // 2]), rng.random() < 0.5,
                     rng.choice(["half", "interleaved"]), dtype, rng.choice([dtype, dtype, "fp8_e4m3", "fp8_e5m2"]),
                     rng.choice([16, 32, 64]), _log_range(rng, 2048, 262144), rng.randrange(0, 1 + tokens // 8))
    else:
        q_heads, kv_heads = rng.choice([(8, 4), (16, 4), (16, 16), (24, 4), (32, 8), (64, 8)])
        head = rng.choice([64, 128, 128])
        block = rng.choice([16, 32])
        dtype = rng.choice(["f16", "bf16"])
        cache = rng.choice([dtype, dtype, "fp8_e4m3", "fp8_e5m2"]) if head == 128 else dtype
        window = rng.choice([0, 0, 0, 333, 1024])
        norm, per_token = rng.random() < 0.7, rng.random() < 0.5
        decodes = shortest = longest = chunks = chunk = before = 0
        kind = rng.choice(["decode", "prefill", "mixed"])
        if kind != "prefill":
            longest = _log_range(rng, 64, 65536)
            shortest = max(1, longest // rng.randint(2, 16))
            decodes = _log_range(rng, 1, max(1, min(256, (1 << 19) * 8 * 128 // (longest * kv_heads * head))))
        if kind != "decode":
            chunks = rng.choice([1, 1, 2, 3, 4])
            chunk = _log_range(rng, 2, 4096 // chunks)
            before = _log_range(rng, 1, 32768) if rng.random() < 0.7 else 0
        case = _diff("", decodes, shortest, longest, chunks, chunk, before, q_heads, kv_heads, head, block, dtype,
                     cache, window, norm, per_token)
        while work(case)["flops"] > 1.5e12:  # no dearer than the largest listed one
            case["chunk"] = case["chunk"] * 2 // 3
    del case["name"]
    return case


# ---------------------------------------------------------------- inputs


def _spread(low, high, n):
    """n whole numbers from low to high, evenly apart."""
    if n == 1:
        return [high]
    return [low + (high - low) * i // (n - 1) for i in range(n)]


def _step_lengths(case, mix):
    """(context lengths, new tokens) of a step's requests, chunks first; ``mix`` shuffles the decodes."""
    if case["op"] == "positions":
        low = max(case["chunk"], case["longest"] // 8, 1)
        long = _spread(low, max(low, case["longest"]), case["chunks"]) if case["chunks"] else []
        short = _spread(max(1, case["longest"] // 16), case["longest"], case["decodes"]) if case["decodes"] else []
    else:
        # prefixes of an eighth to all of `before`
        long = [b + case["chunk"] for b in _spread(case["before"] // 8, case["before"], case["chunks"])] \
            if case["chunks"] else []
        short = _spread(case["shortest"], case["longest"], case["decodes"]) if case["decodes"] else []
    short = [short[i] for i in mix(len(short))]
    return long + short, [case["chunk"]] * len(long) + [1] * len(short)


def _pool(lens, first, bs, dev, gen):
    """Block tables of sequences that hold the blocks of tokens first..len, in a pool in random order
    (entries before them are -1), and the pool's size."""
    lens, first = np.asarray(lens), np.asarray(first)
    blocks, gone = -(-lens // bs), first // bs
    held = blocks - gone
    nb = int(held.sum()) + 3
    width = int(blocks.max()) + 2
    order = torch.randperm(nb, device=dev, generator=gen).int()
    col = torch.arange(width, device=dev)
    lo, hi = torch.from_numpy(gone).to(dev)[:, None], torch.from_numpy(blocks).to(dev)[:, None]
    at = torch.from_numpy(np.cumsum(held) - held).to(dev)[:, None] + col - lo
    return torch.where((col >= lo) & (col < hi), order[at.clamp(0, nb - 1)], -1), nb


def _media_grids(rng, length, most):
    """Media of one sequence, ascending: (first token, frames, rows, columns, positions a frame takes)."""
    found, at = [], int(rng.integers(0, 20))
    room = max(1, length // (most + 1))
    for _ in range(most):
        side = max(1, math.isqrt(room))
        rows, cols = int(rng.integers(1, side + 1)), int(rng.integers(1, side + 1))
        frames = int(rng.integers(1, 5)) if rng.random() < 0.3 else 1
        if at + frames * rows * cols > length + room:  # the last one may still be arriving
            break
        found.append((at, frames, rows, cols, int(rng.integers(1, 4))))
        at += frames * rows * cols + int(rng.integers(0, 12))
    return found


def _prepare_positions(case, gen, dev):
    rng = np.random.default_rng(int(torch.randint(0, 1 << 62, (1,), generator=gen, device=dev)))
    lens, new = _step_lengths(case, rng.permutation)
    tables, nb = _pool(lens, [0] * len(lens), case["block"], dev, gen)
    media = [_media_grids(rng, n, int(rng.integers(case["media"] // 2, case["media"] + 1))) for n in lens]
    flat = [m for one in media for m in one] or [(0, 0, 0, 0, 0)]
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    total = sum(new)
    return {"case": case, "total": total, "num_blocks": nb, "tables": tables, "lens": ints(lens),
            "starts": ints(np.concatenate(([0], np.cumsum(new)))),
            "media_starts": ints(np.concatenate(([0], np.cumsum([len(one) for one in media])))),
            "media": ints(flat)[:sum(len(one) for one in media)],
            "positions": torch.zeros(3, total, dtype=torch.int32, device=dev),
            "slots": torch.zeros(total, dtype=torch.int64, device=dev)}


def _sections(half):
    """Pairs of the time, height and width axes: a quarter, and the rest in two."""
    time = half - 2 * (3 * half // 8)
    return [time, 3 * half // 8, 3 * half // 8]


def _pair_axes(half, cycled):
    """The axis of every pair: axes one after the other, or dealt round while an axis has pairs left."""
    n = _sections(half)
    if cycled:
        return [i % 3 if i % 3 and i < 3 * n[i % 3] else 0 for i in range(half)]
    return [a for a in range(3) for _ in range(n[a])]


def _scale(cache, dev):
    """The scale of an FP8 cache."""
    return torch.tensor([2.0 ** -5], device=dev) if cache.startswith("fp8") else None


def _prepare_axes(case, gen, dev):
    t, hq, hkv, d, bs = case["tokens"], case["q_heads"], case["kv_heads"], case["head"], case["block"]
    dt, cdt = _FLOAT[case["dtype"]], _CACHE[case["cache"]]
    qkv = torch.randn(t, (hq + 2 * hkv) * d, device=dev, generator=gen).to(dt)
    nb = -(-2 * t // bs) + 2
    slots = torch.randperm(nb * bs, device=dev, generator=gen)[:t]
    if case["pad"]:
        slots[t - case["pad"]:] = -1
    half = case["rot"] // 2
    freq = 1000000.0 ** (-np.arange(half, dtype=np.float64) / half)
    # time runs far, height and width stay near it
    time = torch.randint(0, case["far"], (t,), device=dev, generator=gen, dtype=torch.int32)
    near = torch.randint(0, 64, (2, t), device=dev, generator=gen, dtype=torch.int32)
    return {
        "case": case,
        "q": qkv[:, :hq * d].view(t, hq, d), "key": qkv[:, hq * d:(hq + hkv) * d].view(t, hkv, d),
        "value": qkv[:, (hq + hkv) * d:].view(t, hkv, d),
        "q_out": torch.zeros(t, hq, d, dtype=dt, device=dev),
        "k_cache": torch.randn(nb, hkv, bs, d, device=dev, generator=gen).to(cdt),
        "v_cache": torch.randn(nb, hkv, bs, d, device=dev, generator=gen).to(cdt),
        "positions": torch.cat((time[None], time + near)), "slots": slots,
        "inv_freq": torch.from_numpy(freq.astype(np.float32)).to(dev),
        "pair_axis": bytes(_pair_axes(half, case["cycled"])),
        "axis_of_pair": torch.tensor(_pair_axes(half, case["cycled"]), device=dev),
        "k_scale": _scale(case["cache"], dev), "v_scale": _scale(case["cache"], dev),
    }


def _prepare_diff(case, gen, dev):
    hq, hkv, d, bs = case["q_heads"], case["kv_heads"], case["head"], case["block"]
    dt, cdt = _FLOAT[case["dtype"]], _CACHE[case["cache"]]
    mix = lambda n: torch.randperm(n, device=dev, generator=gen).tolist()  # noqa: E731
    lens, new = _step_lengths(case, mix)
    w = case["window"]
    first = [max(0, n - q - w + 1) if w else 0 for n, q in zip(lens, new)]  # the first key anyone attends
    tables, nb = _pool(lens, first, bs, dev, gen)
    total = sum(new)
    heads = hq // 2
    # one weight a head, or one a token and head where the model computes it from the token
    lam = torch.rand(total if case["per_token"] else 1, heads, device=dev, generator=gen).mul_(0.6).add_(0.2)
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    cache = lambda: torch.randn(nb, hkv, bs, d, device=dev, generator=gen, dtype=torch.float16 if cdt.itemsize < 4  # noqa: E731
                                else torch.float32).mul_(32.0 if cdt.itemsize == 1 else 1.0).to(cdt)
    return {
        "case": case, "total": total, "lens_host": lens, "new_host": new, "first_host": first,
        "starts_host": [0] + np.cumsum(new).tolist(),
        "q": torch.randn(total, hq, d, device=dev, generator=gen).to(dt),
        "k_cache": cache(), "v_cache": cache(), "tables": tables,
        "lens": ints(lens), "starts": ints([0] + np.cumsum(new).tolist()),
        "lambda": lam if case["per_token"] else lam[0],
        "norm": torch.rand(2 * d, device=dev, generator=gen).add_(0.5).mul_(0.2) if case["norm"] else None,
        "k_scale": _scale(case["cache"], dev), "v_scale": _scale(case["cache"], dev),
        "out": torch.zeros(total, heads, 2 * d, dtype=dt, device=dev),
        "scale": d ** -0.5,
    }


_PREPARE = {"positions": _prepare_positions, "axes": _prepare_axes, "diff": _prepare_diff}


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    return _PREPARE[case["op"]](case, gen, dev)


# ---------------------------------------------------------------- positions and slots


def _plain_positions(s):
    bs, dev = s["case"]["block"], s["lens"].device
    lens, starts, media = s["lens"].long(), s["starts"].long(), s["media"].long()
    new = starts[1:] - starts[:-1]
    owner = torch.repeat_interleave(torch.arange(lens.numel(), device=dev), new, output_size=s["total"])
    at = lens[owner] - new[owner] + torch.arange(s["total"], device=dev) - starts[owner]
    s["slots"].copy_(s["tables"][owner, at // bs].long() * bs + at % bs)
    # the last medium of the token's sequence that starts at or before it
    counts = (s["media_starts"][1:] - s["media_starts"][:-1]).long()
    of = torch.repeat_interleave(torch.arange(lens.numel(), device=dev), counts, output_size=media.shape[0])
    first, frames, rows, cols, step = media.unbind(1)
    size = frames * rows * cols
    extent = torch.maximum((frames - 1) * step + 1, torch.maximum(rows, cols))
    place = torch.searchsorted((of << 32) + first, (owner << 32) + at, right=True) - 1
    some = place >= s["media_starts"].long()[owner]
    place = place.clamp(min=0)
    saved = torch.nn.functional.pad((size - extent).cumsum(0), (1, 0))
    before = saved[place] - saved[s["media_starts"].long()[owner]]  # positions that earlier media leave out
    inside = at - first[place]
    base = first[place] - before
    text = torch.where(some, at - before - (size - extent)[place], at)
    frame, cell = inside // (rows * cols)[place], inside % (rows * cols)[place]
    grid = torch.stack((frame * step[place], cell // cols[place], cell % cols[place])) + base
    s["positions"].copy_(torch.where(some & (inside < size[place]), grid, text))
    return {"positions": s["positions"], "slots": s["slots"]}


def _own_positions(s):
    import paged_kv_cache_pagedattention_gb300 as pa

    pa.pa_positions_and_slots(s["positions"], s["slots"], s["starts"], s["lens"], s["tables"], s["num_blocks"],
                              s["case"]["block"], s["media_starts"], s["media"])
    return {"positions": s["positions"], "slots": s["slots"]}


def _exact_positions(s):
    bs = s["case"]["block"]
    lens, starts, media_starts = (s[k].cpu().numpy().astype(np.int64) for k in ("lens", "starts", "media_starts"))
    media, tables = s["media"].cpu().numpy().astype(np.int64), s["tables"].cpu().numpy().astype(np.int64)
    positions, slots = np.zeros((3, s["total"]), np.int32), np.zeros(s["total"], np.int64)
    for r in range(len(lens)):
        # the whole sequence's positions, piece after piece
        every, token, place = [], 0, 0
        for first, frames, rows, cols, step in media[media_starts[r]:media_starts[r + 1]]:
            every.append(np.tile(place + np.arange(first - token), (3, 1)))
            place += first - token
            f, y, x = np.meshgrid(np.arange(frames) * step, np.arange(rows), np.arange(cols), indexing="ij")
            every.append(place + np.stack([f.ravel(), y.ravel(), x.ravel()]))
            token = first + frames * rows * cols
            place = every[-1].max() + 1
        every.append(np.tile(place + np.arange(max(0, lens[r] - token)), (3, 1)))
        n = starts[r + 1] - starts[r]
        at = np.arange(lens[r] - n, lens[r])
        positions[:, starts[r]:starts[r + 1]] = np.concatenate(every, 1)[:, at]
        slots[starts[r]:starts[r + 1]] = tables[r, at // bs] * bs + at % bs
    return {"positions": positions, "slots": slots}


# ---------------------------------------------------------------- rotary positions on several axes


def _rotated(x, cos, sin, rot, layout):
    x = x.float()
    r = x[..., :rot]
    if layout == "half":
        a, b = r[..., :rot // 2], r[..., rot // 2:]
        r = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    else:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    return torch.cat((r, x[..., rot:]), -1)


def _store(cache, kind, rows, scale, block, offset):
    if scale is not None:
        top = _FP8_MAX[kind]
        rows = (rows / scale).clamp(-top, top).to(cache.dtype).view(torch.uint8)
        cache = cache.view(torch.uint8)
    cache[block, :, offset] = rows.to(cache.dtype)


def _plain_axes(s):
    case = s["case"]
    rot, layout, bs = case["rot"], case["layout"], case["block"]
    angle = s["positions"].double()[s["axis_of_pair"]].t() * s["inv_freq"].double()
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    q = _rotated(s["q"], cos, sin, rot, layout).to(s["q"].dtype)
    s["q_out"].copy_(torch.where((s["slots"] >= 0)[:, None, None], q, s["q_out"]))
    row = (s["slots"] >= 0).nonzero()[:, 0]
    block, offset = s["slots"][row] // bs, s["slots"][row] % bs
    key = _rotated(s["key"], cos, sin, rot, layout)[row]
    _store(s["k_cache"], case["cache"], key, s["k_scale"], block, offset)
    _store(s["v_cache"], case["cache"], s["value"][row].float(), s["v_scale"], block, offset)
    return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _own_axes(s):
    import paged_kv_cache_pagedattention_gb300 as pa

    pa.pa_rotary_axes_and_cache(s["q_out"], s["q"], s["key"], s["value"], s["k_cache"], s["v_cache"], s["positions"],
                                s["slots"], s["inv_freq"], s["pair_axis"],
                                interleaved=s["case"]["layout"] == "interleaved", k_scale=s["k_scale"],
                                v_scale=s["v_scale"])
    return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _exact_axes(s):
    case = s["case"]
    rot, bs, half = case["rot"], case["block"], case["rot"] // 2
    axis = torch.tensor(list(s["pair_axis"]), device=s["q"].device)
    turn = s["positions"].double().index_select(0, axis).transpose(0, 1) * s["inv_freq"].double()[None]
    phase = torch.polar(torch.ones_like(turn), turn)[:, None]  # a rotation is a complex product
    first, second = (slice(0, half), slice(half, rot)) if case["layout"] == "half" else (slice(0, rot, 2),
                                                                                        slice(1, rot, 2))
    out = []
    for x in (s["q"], s["key"]):
        y = x.double().clone()
        z = torch.complex(y[..., first], y[..., second]) * phase
        y[..., first], y[..., second] = z.real, z.imag
        out.append(y)
    out.append(s["value"].double())
    keep = s["slots"] >= 0
    q = s["q_out"].double()
    q[keep] = out[0][keep]
    got = {"q": q}
    for name, rows, scale in (("k_cache", out[1], s["k_scale"]), ("v_cache", out[2], s["v_scale"])):
        cache = s[name].double().permute(0, 2, 1, 3).reshape(-1, case["kv_heads"], case["head"])
        rows = rows[keep]
        if scale is not None:  # an FP8 cache holds the nearest code of value / scale
            rows = (rows / scale.double()).clamp(-_FP8_MAX[case["cache"]], _FP8_MAX[case["cache"]])
        cache[s["slots"][keep]] = rows
        got[name] = cache.view(-1, bs, case["kv_heads"], case["head"]).permute(0, 2, 1, 3).contiguous()
    return got


# ---------------------------------------------------------------- differential attention
#
# q head 2h + j is map j of head h; K head 2g + j is map j of its KV group g, and V heads 2g, 2g + 1 are the two
# halves of the group's value row.


def _cached(cache, scale, tables, at, bs):
    """Rows of the cache at token places ``at`` of the tables' sequences, heads first, as fp32."""
    block = torch.gather(tables.long(), 1, (at // bs).clamp(max=tables.shape[1] - 1)).clamp(min=0)
    rows = cache[block, :, at % bs].float()
    return (rows if scale is None else rows * scale).transpose(1, 2)


def _plain_maps(s, rows, seqs, first, span, new):
    """Rows ``rows`` (``new`` for each of the sequences ``seqs``) attend keys first .. first + span."""
    case = s["case"]
    d, bs, groups = case["head"], case["block"], case["kv_heads"] // 2
    n, dev = seqs.numel(), s["q"].device
    at = first[:, None] + torch.arange(span, device=dev)
    tables = s["tables"][seqs]
    k = _cached(s["k_cache"], s["k_scale"], tables, at, bs).reshape(n, groups, 2, 1, span, d)
    v = _cached(s["v_cache"], s["v_scale"], tables, at, bs).reshape(n, groups, 2, span, d)
    v = v.transpose(2, 3).reshape(n, groups, 1, 1, span, 2 * d)
    # [sequence][group][map][head of the group][row][head_size]
    q = s["q"][rows].float().view(n, new, groups, -1, 2, d).permute(0, 2, 4, 3, 1, 5)
    pos = s["lens"].long()[seqs][:, None] - new + torch.arange(new, device=dev)
    keep = at[:, None] <= pos[..., None]
    if case["window"]:
        keep &= at[:, None] > pos[..., None] - case["window"]
    score = (q * s["scale"]) @ k.transpose(-1, -2)
    score = score.masked_fill(~keep[:, None, None, None], -math.inf)
    weight = (score - score.amax(-1, keepdim=True)).exp()
    out = weight @ v / weight.sum(-1, keepdim=True)
    out = out.permute(0, 4, 1, 3, 2, 5).reshape(rows.numel(), groups * q.shape[3], 2, 2 * d)
    lam = s["lambda"] if s["lambda"].dim() == 1 else s["lambda"][rows]
    out = out[:, :, 0] - lam[..., None] * out[:, :, 1]
    if s["norm"] is not None:
        out = out * torch.rsqrt((out * out).mean(-1, keepdim=True) + 1e-5) * s["norm"]
    s["out"][rows] = out.to(s["out"].dtype)


def _plain_diff(s):
    case, dev = s["case"], s["q"].device
    for r in range(case["chunks"]):  # chunks of one size on contexts of very different lengths: one by one
        rows = torch.arange(s["starts_host"][r], s["starts_host"][r + 1], device=dev)
        first = s["first_host"][r]
        _plain_maps(s, rows, torch.tensor([r], device=dev), torch.tensor([first], device=dev),
                    s["lens_host"][r] - first, case["chunk"])
    if case["decodes"]:  # all single-token rows together
        seqs = torch.arange(case["chunks"], len(s["lens_host"]), device=dev)
        rows = seqs - case["chunks"] + case["chunks"] * case["chunk"]
        lens = s["lens"].long()[seqs]
        first = (lens - case["window"]).clamp(min=0) if case["window"] else torch.zeros_like(lens)
        _plain_maps(s, rows, seqs, first, min(case["longest"], case["window"] or case["longest"]), 1)
    return {"out": s["out"]}


def _own_diff(s):
    import paged_kv_cache_pagedattention_gb300 as pa

    case = s["case"]
    hq, hkv, d, bs = case["q_heads"], case["kv_heads"], case["head"], case["block"]
    longest, n = max(s["lens_host"]), len(s["lens_host"])
    if case["chunks"] == 0:
        if "workspace" not in s:
            s["workspace"] = pa.workspace_tensor(pa.pa_diff_decode_workspace_size(n, hq, hkv, d, longest, bs))
        pa.pa_diff_decode(s["out"], s["q"], s["k_cache"], s["v_cache"], s["tables"], s["lens"], longest, s["scale"],
                          s["lambda"], s["workspace"], norm_weight=s["norm"], norm_eps=1e-5, k_scale=s["k_scale"],
                          v_scale=s["v_scale"], window=case["window"])
    else:
        if "workspace" not in s:
            s["workspace"] = pa.workspace_tensor(pa.pa_diff_varlen_workspace_size(n, s["total"], case["chunk"], hq,
                                                                                  hkv, d, longest, bs))
        pa.pa_diff_varlen_attn(s["out"], s["q"], s["k_cache"], s["v_cache"], s["tables"], s["starts"], s["lens"],
                               case["chunk"], longest, s["scale"], s["lambda"], s["workspace"],
                               norm_weight=s["norm"], norm_eps=1e-5, k_scale=s["k_scale"], v_scale=s["v_scale"],
                               window=case["window"])
    return {"out": s["out"]}


def _exact_diff(s):
    case = s["case"]
    d, bs, w = case["head"], case["block"], case["window"]
    per = case["q_heads"] // case["kv_heads"]
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=s["q"].device)
    lam = s["lambda"].double().expand(s["total"], -1)
    for r, (n, q_len) in enumerate(zip(s["lens_host"], s["new_host"])):
        base = s["first_host"][r] // bs * bs
        rows = slice(s["starts_host"][r], s["starts_host"][r] + q_len)
        held = s["tables"][r, base // bs:-(-n // bs)].long()
        key = torch.arange(base, n, device=out.device)
        query = torch.arange(n - q_len, n, device=out.device)
        off = key[None] > query[:, None]
        if w:
            off |= key[None] <= query[:, None] - w
        for g in range(case["kv_heads"] // 2):
            k, v = (c[held][:, 2 * g:2 * g + 2].double().transpose(0, 1).reshape(2, -1, d)[:, :n - base]
                    for c in (s["k_cache"], s["v_cache"]))
            if s["k_scale"] is not None:
                k, v = k * s["k_scale"].double(), v * s["v_scale"].double()
            v = torch.cat((v[0], v[1]), -1)
            for h in range(g * per, (g + 1) * per):
                a, b = (torch.softmax((s["q"][rows, 2 * h + j].double() @ k[j].T * s["scale"])
                                      .masked_fill(off, -math.inf), -1) for j in (0, 1))
                o = (a - lam[rows, h, None] * b) @ v
                if s["norm"] is not None:
                    o = o / (o.square().mean(-1, keepdim=True) + 1e-5).sqrt() * s["norm"].double()
                out[rows, h] = o
    return {"out": out}


# ---------------------------------------------------------------- entry points


_PLAIN = {"positions": _plain_positions, "axes": _plain_axes, "diff": _plain_diff}
_OWN = {"positions": _own_positions, "axes": _own_axes, "diff": _own_diff}
_EXACT = {"positions": _exact_positions, "axes": _exact_axes, "diff": _exact_diff}


def run(state):
    return (_OWN if own else _PLAIN)[state["case"]["op"]](state)


def exact(case, seed):
    return _EXACT[case["op"]](prepare(case, seed))


def work(case):
    if case["op"] == "positions":
        n, t = case["decodes"] + case["chunks"], case["decodes"] + case["chunks"] * case["chunk"]
        # lengths, starts and media records in, a table entry for each new block, positions and slots out
        return {"bytes": 12 * n + n * 20 * 3 * case["media"] // 4 + 4 * (n + t // case["block"]) + 20 * t,
                "flops": 16 * t}
    if case["op"] == "axes":
        t, d, e = case["tokens"], case["head"], _SIZE[case["dtype"]]
        real = t - case["pad"]
        read = real * (case["q_heads"] + 2 * case["kv_heads"]) * d * e + real * 12 + t * 8
        wrote = real * (case["q_heads"] * e + 2 * case["kv_heads"] * _SIZE[case["cache"]]) * d
        return {"bytes": read + wrote, "flops": real * 3 * case["rot"] * (case["q_heads"] + case["kv_heads"])}
    lens, new = _step_lengths(case, range)
    w, heads, d, bs = case["window"], case["q_heads"] // 2, case["head"], case["block"]
    seen = pairs = 0
    for n, q in zip(lens, new):
        seen += min(n, w + q - 1) if w else n
        pairs += sum(min(p + 1, w) for p in range(n - q, n)) if w else q * (n - q) + q * (q + 1) // 2
    t = sum(new)
    return {"bytes": seen * 2 * case["kv_heads"] * d * _SIZE[case["cache"]] + 4 * seen // bs +
            2 * t * case["q_heads"] * d * _SIZE[case["dtype"]],
            # two maps of 2 d operations a key, and two sums over 2 d values
            "flops": 12 * d * heads * pairs}

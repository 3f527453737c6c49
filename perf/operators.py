"""Cases of the decoding-step operators: rotary positions written into a paged KV cache,
beam selection over beams and vocabulary, and the pages of forked sequences.

Three kinds of case, named by ``case["op"]``:

* ``rotary``  the new tokens' q, k and v come as slices of one QKV product; q is rotated
              into a buffer of its own, k is rotated and written to its slot of the paged
              cache with v.
* ``beam``    logits of every beam and the beams' scores become the next hypotheses.
* ``branch``  the life of a set of branches: they are forked from parent sequences, extended
              by a few tokens (free pages, copy-on-write of shared tails, slots), and
              released again.

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


def _rotary(name, tokens, q_heads, kv_heads, head, rot, layout, dtype, cache, block, far, factor, pad):
    return {"name": name, "op": "rotary", "tokens": tokens, "q_heads": q_heads, "kv_heads": kv_heads, "head": head,
            "rot": rot, "layout": layout, "dtype": dtype, "cache": cache, "block": block, "far": far,
            "factor": factor, "pad": pad}


def _beam(name, seqs, beams, vocab, keep, dtype, masked):
    return {"name": name, "op": "beam", "seqs": seqs, "beams": beams, "vocab": vocab, "keep": keep, "dtype": dtype,
            "masked": masked}


def _branch(name, parents, children, shortest, longest, grow, kv_heads, head, block, dtype):
    return {"name": name, "op": "branch", "parents": parents, "children": children, "shortest": shortest,
            "longest": longest, "grow": grow, "kv_heads": kv_heads, "head": head, "block": block, "dtype": dtype}


def listed():
    return [
        # one sequence decoding alone: the call's latency
        _rotary("rotary one token", 1, 32, 8, 128, 128, "half", "bf16", "bf16", 16, 4096, 1.0, 0),
        # a small fp32 model, ragged count, pairs side by side, half of the head rotated
        _rotary("rotary f32 partial", 37, 8, 2, 64, 32, "interleaved", "f32", "f32", 16, 2048, 1.0, 3),
        # a decode batch on an FP8 cache, contexts stretched to 32K (scaled frequencies and attention factor)
        _rotary("rotary fp8 decode", 256, 32, 8, 128, 128, "half", "bf16", "fp8_e4m3", 32, 32768, 8.0, 0),
        # a mixed step: four prefill chunks of 512 tokens and 128 decodes
        _rotary("rotary mixed step", 2176, 32, 8, 128, 128, "half", "bf16", "bf16", 16, 65536, 4.0, 0),
        # long-context prefill of a large model, far positions, part of the head, padded at its end
        _rotary("rotary long prefill", 8192, 64, 8, 128, 64, "interleaved", "f16", "f16", 16, 262144, 16.0, 61),
        # one request of four beams, fp32 logits: the call's latency
        _beam("beam one request", 1, 4, 32000, 8, "f32", 0.0),
        # a few requests, an odd vocabulary (rows start off any vector boundary), constrained decoding masks a third
        _beam("beam odd masked", 7, 5, 65537, 10, "bf16", 0.34),
        # an ordinary batch of wide beams
        _beam("beam wide", 16, 8, 131072, 16, "bf16", 0.0),
        # the largest: many requests, a large vocabulary, fp32 logits
        _beam("beam large", 64, 4, 262144, 8, "f32", 0.02),
        # four samples of one short prompt in a pool of a few dozen pages
        _branch("branch one prompt", 1, 4, 17, 200, 1, 2, 64, 16, "f32"),
        # beams of a decode batch: 64 sequences of 512 to 4096 tokens, four branches each
        _branch("branch batch", 64, 256, 512, 4096, 1, 8, 128, 16, "bf16"),
        # agents forked from long contexts, each with a few drafted tokens; one KV head of a split cache
        _branch("branch long forks", 32, 256, 32768, 131072, 7, 1, 64, 16, "bf16"),
    ]


def _log_range(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["rotary", "beam", "branch"])
    if op == "rotary":
        q_heads, kv_heads = rng.choice([(8, 2), (10, 10), (16, 2), (28, 4), (32, 8), (40, 8), (64, 8)])
        head = rng.choice([64, 96, 128, 160, 256])
        most = min(8192, 8192 * 64 * 128 // (q_heads * head))
        tokens = _log_range(rng, 1, most)
        dtype = rng.choice(["f32", "f16", "bf16", "bf16"])
        if dtype == "f32":
            tokens = max(1, tokens // 2)
        rot = rng.choice([head, head, head // 2, head // 4])
        case = _rotary("", tokens, q_heads, kv_heads, head, rot, rng.choice(["half", "interleaved"]), dtype,
                       rng.choice([dtype, dtype, "fp8_e4m3", "fp8_e5m2"]), rng.choice([16, 32, 64]),
                       _log_range(rng, 2048, 262144), rng.choice([1.0, 2.0, 4.0, 8.0, 16.0]),
                       rng.randrange(0, 1 + tokens // 8))
    elif op == "beam":
        vocab = _log_range(rng, 1000, 262144)
        beams = rng.choice([1, 2, 3, 4, 5, 8, 16])
        seqs = _log_range(rng, 1, min(64, max(1, 64 * 4 * 262144 // (vocab * beams))))
        keep = min(32, rng.choice([beams, 2 * beams]))
        case = _beam("", seqs, beams, vocab, keep, rng.choice(["f32", "f16", "bf16"]),
                     rng.choice([0.0, 0.0, 0.1, 0.5, 0.9]))
    else:
        parents = _log_range(rng, 1, 64)
        children = min(256, parents * rng.randint(1, 8))
        longest = _log_range(rng, 64, min(131072, 32 * 131072 // max(parents, children // 8)))
        block = rng.choice([16, 32])
        case = _branch("", parents, children, max(1, longest // rng.randint(2, 16)), longest, rng.randint(1, 9),
                       1 if longest > 8192 else rng.choice([1, 2, 4]), rng.choice([64, 128]) if longest <= 65536 else 64,
                       block, rng.choice(["bf16", "f16"]))
    del case["name"]
    return case


# ---------------------------------------------------------------- inputs


def _prepare_rotary(case, gen, dev):
    t, hq, hkv, d, bs = case["tokens"], case["q_heads"], case["kv_heads"], case["head"], case["block"]
    dt, cdt = _FLOAT[case["dtype"]], _CACHE[case["cache"]]
    qkv = torch.randn(t, (hq + 2 * hkv) * d, device=dev, generator=gen).to(dt)
    nb = -(-2 * t // bs) + 2
    scaled = cdt.itemsize == 1

    def cache():
        return torch.randn(nb, hkv, bs, d, device=dev, generator=gen).mul_(0.5 if scaled else 1.0).to(cdt)

    slots = torch.randperm(nb * bs, device=dev, generator=gen)[:t]
    if case["pad"]:
        slots[t - case["pad"]:] = -1
    half = case["rot"] // 2
    freq = 10000.0 ** (-np.arange(half, dtype=np.float64) / half)
    if case["factor"] > 1:  # scaled by parts: wavelengths that fit 8192 positions less than once are stretched
        ramp = np.clip((8192 * freq / (2 * math.pi) - 1.0) / 31.0, 0.0, 1.0)
        freq = freq * ramp + freq / case["factor"] * (1.0 - ramp)
    return {
        "case": case,
        "q": qkv[:, :hq * d].view(t, hq, d), "key": qkv[:, hq * d:(hq + hkv) * d].view(t, hkv, d),
        "value": qkv[:, (hq + hkv) * d:].view(t, hkv, d),
        "q_out": torch.zeros(t, hq, d, dtype=dt, device=dev),
        "k_cache": cache(), "v_cache": cache(),
        "positions": torch.randint(0, case["far"], (t,), device=dev, generator=gen, dtype=torch.int32),
        "slots": slots,
        "inv_freq": torch.from_numpy(freq.astype(np.float32)).to(dev),
        "attn_factor": 0.1 * math.log(case["factor"]) + 1.0,
        # per-tensor scales of an FP8 cache
        "k_scale": torch.tensor([2.0 ** -6], device=dev) if scaled else None,
        "v_scale": torch.tensor([2.0 ** -5], device=dev) if scaled else None,
    }


def _prepare_beam(case, gen, dev):
    b, w, v = case["seqs"], case["beams"], case["vocab"]
    logits = torch.randn(b * w, v, device=dev, generator=gen).mul_(2.5)
    if case["masked"]:
        logits.masked_fill_(torch.rand(b * w, v, device=dev, generator=gen) < case["masked"], -math.inf)
    scores = -torch.rand(b, w, device=dev, generator=gen).mul_(6.0).cumsum(1)
    if w > 2:
        scores[b // 2, w - 1] = -math.inf  # a beam that has ended
    return {"case": case, "logits": logits.to(_FLOAT[case["dtype"]]), "scores": scores,
            "out": [torch.empty(b, case["keep"], dtype=dt, device=dev)
                    for dt in (torch.float32, torch.int32, torch.int32)]}


def _prepare_branch(case, gen, dev):
    m, n, bs, grow = case["parents"], case["children"], case["block"], case["grow"]
    lens = torch.randint(case["shortest"], case["longest"] + 1, (m,), device=dev, generator=gen, dtype=torch.int32)
    width = -(-(case["longest"] + grow) // bs) + 1
    blocks = (lens + bs - 1) // bs
    # the pool: room for every parent at its longest, and for the branches' own pages
    nb = m * -(-case["longest"] // bs) + n * (2 + grow // bs) + 8
    order = torch.randperm(nb, device=dev, generator=gen).int()
    col = torch.arange(width, device=dev, dtype=torch.int32)
    live = col < blocks[:, None]
    at = (blocks.cumsum(0).int() - blocks)[:, None] + col
    tables = torch.where(live, order[at.clamp(max=nb - 1).long()], -1)
    refs = torch.zeros(nb, dtype=torch.int32, device=dev)
    refs[tables[live].long()] = 1
    new = torch.randperm(n, device=dev, generator=gen) % grow + 1
    starts = torch.zeros(n + 1, dtype=torch.int32, device=dev)
    starts[1:] = new.cumsum(0)
    total = int(starts[-1])
    shape = (nb, case["kv_heads"], bs, case["head"])
    dt = _FLOAT[case["dtype"]]
    return {
        "case": case, "total": total,
        "tables": tables, "lens": lens, "refs": refs,
        "parents": torch.randint(0, m, (n,), device=dev, generator=gen, dtype=torch.int32),
        "child_tables": torch.full((n, width), -1, dtype=torch.int32, device=dev),
        "child_lens": torch.zeros(n, dtype=torch.int32, device=dev),
        "starts": starts,
        "slots": torch.empty(total, dtype=torch.int64, device=dev),
        "pairs": torch.empty(n, 2, dtype=torch.int64, device=dev),
        "k_cache": torch.randn(shape, device=dev, generator=gen).to(dt),
        "v_cache": torch.randn(shape, device=dev, generator=gen).to(dt),
    }


_PREPARE = {"rotary": _prepare_rotary, "beam": _prepare_beam, "branch": _prepare_branch}


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    return _PREPARE[case["op"]](case, gen, dev)


# ---------------------------------------------------------------- rotary positions


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


def _plain_rotary(s):
    case = s["case"]
    rot, layout, bs = case["rot"], case["layout"], case["block"]
    angle = s["positions"].double()[:, None] * s["inv_freq"].double()
    cos = (angle.cos() * s["attn_factor"]).float()[:, None]
    sin = (angle.sin() * s["attn_factor"]).float()[:, None]
    q = _rotated(s["q"], cos, sin, rot, layout).to(s["q"].dtype)
    s["q_out"].copy_(torch.where((s["slots"] >= 0)[:, None, None], q, s["q_out"]))
    row = (s["slots"] >= 0).nonzero()[:, 0]
    block, offset = s["slots"][row] // bs, s["slots"][row] % bs
    key = _rotated(s["key"], cos, sin, rot, layout)[row]
    _store(s["k_cache"], case["cache"], key, s["k_scale"], block, offset)
    _store(s["v_cache"], case["cache"], s["value"][row].float(), s["v_scale"], block, offset)
    return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _own_rotary(s):
    import paged_kv_cache_pagedattention_gb300 as pa

    pa.pa_rotary_and_cache(s["q_out"], s["q"], s["key"], s["value"], s["k_cache"], s["v_cache"], s["positions"],
                           s["slots"], s["inv_freq"], interleaved=s["case"]["layout"] == "interleaved",
                           attn_factor=s["attn_factor"], k_scale=s["k_scale"], v_scale=s["v_scale"])
    return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _exact_rotary(s):
    case = s["case"]
    rot, bs, half = case["rot"], case["block"], case["rot"] // 2
    turn = torch.outer(s["positions"].double(), s["inv_freq"].double())
    phase = torch.polar(torch.full_like(turn, s["attn_factor"]), turn)[:, None]  # a rotation is a complex product
    out = []
    for x in (s["q"], s["key"]):
        y = x.double().clone()
        first, second = (slice(0, half), slice(half, rot)) if case["layout"] == "half" else (slice(0, rot, 2),
                                                                                            slice(1, rot, 2))
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
            top = _FP8_MAX[case["cache"]]
            rows = (rows / scale.double()).clamp(-top, top)
        cache[s["slots"][keep]] = rows
        got[name] = cache.view(-1, bs, case["kv_heads"], case["head"]).permute(0, 2, 1, 3).contiguous()
    return got


# ---------------------------------------------------------------- beam selection


def _plain_beam(s):
    case = s["case"]
    b, w, v, k = case["seqs"], case["beams"], case["vocab"], case["keep"]
    x = s["logits"].double()
    x = torch.where(x.isnan(), -math.inf, x).clamp(max=torch.finfo(s["logits"].dtype).max)
    top = x.amax(1, keepdim=True)
    top = torch.where(top.isinf(), 0.0, top)
    x = x - top
    logp = torch.where(x.isinf(), -math.inf, x - x.exp().sum(1, keepdim=True).log())
    flat = (s["scores"].double()[..., None] + logp.view(b, w, v)).view(b, w * v)
    # the k largest, ties to the lowest index: what is above the k-th value, then its equals in order
    kth = flat.topk(k).values[:, -1:]
    place = torch.arange(w * v, device=flat.device)
    rank = torch.where(flat > kth, 1, torch.where(flat == kth, -place, -w * v - 1))
    at = rank.topk(k).indices.sort().values
    best, order = flat.gather(1, at).sort(descending=True, stable=True)
    at = at.gather(1, order)
    row = torch.arange(b, device=at.device)[:, None] * w + at // v
    none = best.isinf()
    return {"scores": best.float(), "tokens": torch.where(none, -1, at % v).int(),
            "parents": torch.where(none, -1, row).int()}


def _own_beam(s):
    import paged_kv_cache_pagedattention_gb300 as pa

    case = s["case"]
    if "workspace" not in s:
        s["workspace"] = pa.workspace_tensor(pa.pa_beam_select_workspace_size(case["seqs"], case["beams"],
                                                                              case["vocab"], case["keep"]))
    scores, tokens, parents = s["out"]
    pa.pa_beam_select(scores, tokens, parents, s["logits"], s["scores"], s["workspace"])
    return {"scores": scores, "tokens": tokens, "parents": parents}


def _exact_beam(s):
    case = s["case"]
    b, w, v, k = case["seqs"], case["beams"], case["vocab"], case["keep"]
    scores, tokens, parents = [], [], []
    for i in range(b):
        x = s["logits"][i * w:(i + 1) * w].double()
        logp = torch.log_softmax(x, -1)
        every = (s["scores"][i].double()[:, None] + logp).reshape(-1)
        value, at = torch.sort(every, descending=True, stable=True)
        value, at = value[:k], at[:k]
        lost = torch.isneginf(value)
        scores.append(value)
        tokens.append(at.remainder(v).masked_fill(lost, -1))
        parents.append((i * w + at.div(v, rounding_mode="floor")).masked_fill(lost, -1))
    return {"scores": torch.stack(scores), "tokens": torch.stack(tokens).int(), "parents": torch.stack(parents).int()}


# ---------------------------------------------------------------- pages of branches


def _plain_fork(s, bs):
    parent = s["parents"].long()
    lens = s["lens"][parent]
    taken = s["tables"][parent]
    live = torch.arange(taken.shape[1], device=taken.device) < ((lens + bs - 1) // bs)[:, None]
    s["child_tables"].copy_(torch.where(live, taken, s["child_tables"]))
    s["child_lens"].copy_(lens)
    s["refs"].scatter_add_(0, torch.where(live, taken, 0).flatten().long(), live.flatten().int())


def _plain_append(s, bs, most):
    tables, lens, refs, starts = s["child_tables"], s["child_lens"], s["refs"], s["starts"]
    n, dev = lens.numel(), lens.device
    new = starts[1:] - starts[:-1]
    after = lens + new
    old_blocks, new_blocks = (lens + bs - 1) // bs, (after + bs - 1) // bs
    # shared tails that would be written: every holder but the last copies
    tail_at = (lens // bs).long()[:, None]
    tail = tables.gather(1, tail_at)[:, 0].long()
    partial = (new > 0) & (lens % bs > 0)
    row = torch.arange(n, device=dev)
    lower = (tail[:, None] == tail[None]) & partial[:, None] & partial[None] & (row[:, None] > row[None])
    held = torch.where(partial, refs[torch.where(partial, tail, 0)], 0)
    copies = partial & (lower.sum(1) < held - 1)
    need = copies.int() + new_blocks - old_blocks
    first = need.cumsum(0) - need
    # the lowest-numbered free pages, in row order
    free = refs == 0
    nb = refs.numel()
    ids = torch.zeros(nb + 1, dtype=torch.int32, device=dev)
    ids[torch.where(free, free.cumsum(0) - 1, nb)] = torch.arange(nb, device=dev, dtype=torch.int32)
    head = ids[first.long()].long()
    fresh = torch.where(copies, head, tail)
    tables.scatter_(1, tail_at, torch.where(partial, fresh, tables.gather(1, tail_at)[:, 0].long()).int()[:, None])
    col = old_blocks[:, None] + torch.arange(-(-most // bs) + 1, device=dev)
    col = col.clamp(max=tables.shape[1] - 1).long()
    grown = col < new_blocks[:, None]
    more = ids[(first + copies.int())[:, None] + col - old_blocks[:, None]]
    spot = (row[:, None] * tables.shape[1] + col)[grown]
    tables.view(-1)[spot] = more[grown]
    refs.scatter_add_(0, torch.where(copies, tail, 0), -copies.int())
    refs[head[copies]] = 1
    refs[more[grown].long()] = 1
    s["pairs"].copy_(torch.where(copies[:, None], torch.stack((tail, head), 1), 0))
    owner = torch.repeat_interleave(row, new, output_size=s["total"])
    pos = (lens[owner] + torch.arange(s["total"], device=dev) - starts[owner]).long()
    s["slots"].copy_(tables[owner, pos // bs].long() * bs + pos % bs)
    lens.copy_(after)
    src, dst = tail[copies], head[copies]
    s["k_cache"][dst] = s["k_cache"][src]
    s["v_cache"][dst] = s["v_cache"][src]


def _plain_release(s, bs):
    tables, lens = s["child_tables"], s["child_lens"]
    live = torch.arange(tables.shape[1], device=lens.device) < ((lens + bs - 1) // bs)[:, None]
    s["refs"].scatter_add_(0, torch.where(live, tables, 0).flatten().long(), -live.flatten().int())
    lens.zero_()


def _branch_out(s):
    return {"tables": s["child_tables"], "lens": s["child_lens"], "refs": s["refs"], "slots": s["slots"],
            "pairs": s["pairs"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_branch(s):
    bs = s["case"]["block"]
    _plain_fork(s, bs)
    _plain_append(s, bs, s["case"]["grow"])
    _plain_release(s, bs)
    return _branch_out(s)


def _own_branch(s):
    import paged_kv_cache_pagedattention_gb300 as pa

    bs = s["case"]["block"]
    if "workspace" not in s:
        s["workspace"] = pa.workspace_tensor(pa.pa_append_workspace_size(s["case"]["children"], s["total"], bs))
    pa.pa_fork_blocks(s["child_tables"], s["child_lens"], s["tables"], s["lens"], s["parents"], s["refs"], bs)
    pa.pa_append_blocks(s["child_tables"], s["child_lens"], s["starts"], s["slots"], s["pairs"], s["refs"], bs,
                        s["workspace"])
    pa.pa_copy_blocks(s["k_cache"], s["v_cache"], s["pairs"])
    pa.pa_release_blocks(s["child_tables"], s["child_lens"], s["refs"], bs)
    return _branch_out(s)


def _exact_branch(s):
    bs = s["case"]["block"]
    host = {k: s[k].cpu().numpy() for k in ("tables", "lens", "refs", "parents", "starts", "child_tables")}
    refs, table = host["refs"].copy(), host["child_tables"].copy()
    size = [int(host["lens"][p]) for p in host["parents"]]
    k_cache, v_cache = s["k_cache"].double(), s["v_cache"].double()
    for i, p in enumerate(host["parents"]):
        held = host["tables"][p, :-(-size[i] // bs)]
        table[i, :held.size] = held
        refs[held] += 1
    unused = iter(np.flatnonzero(refs == 0).tolist())
    slots, pairs, moved = [], [], []
    for i in range(len(size)):
        pair = [0, 0]
        for pos in range(size[i], size[i] + int(host["starts"][i + 1] - host["starts"][i])):
            j = pos // bs
            if pos % bs == 0:
                table[i, j] = next(unused)
                refs[table[i, j]] = 1
            elif pos == size[i] and refs[table[i, j]] > 1:
                pair = [int(table[i, j]), next(unused)]
                refs[pair[0]] -= 1
                refs[pair[1]] = 1
                table[i, j] = pair[1]
                moved.append(pair)
            slots.append(int(table[i, j]) * bs + pos % bs)
        pairs.append(pair)
    for i in range(len(size)):
        size[i] += int(host["starts"][i + 1] - host["starts"][i])
        refs[table[i, :-(-size[i] // bs)]] -= 1
    for src, dst in moved:
        k_cache[dst], v_cache[dst] = k_cache[src], v_cache[src]
    return {"tables": table, "lens": np.zeros(len(size), np.int32), "refs": refs, "slots": np.array(slots, np.int64),
            "pairs": np.array(pairs, np.int64), "k_cache": k_cache, "v_cache": v_cache}


# ---------------------------------------------------------------- entry points


_PLAIN = {"rotary": _plain_rotary, "beam": _plain_beam, "branch": _plain_branch}
_OWN = {"rotary": _own_rotary, "beam": _own_beam, "branch": _own_branch}
_EXACT = {"rotary": _exact_rotary, "beam": _exact_beam, "branch": _exact_branch}


def run(state):
    return (_OWN if own else _PLAIN)[state["case"]["op"]](state)


def exact(case, seed):
    return _EXACT[case["op"]](prepare(case, seed))


def work(case):
    if case["op"] == "rotary":
        t, d, e = case["tokens"], case["head"], _SIZE[case["dtype"]]
        real = t - case["pad"]
        read = real * (case["q_heads"] + 2 * case["kv_heads"]) * d * e + real * 4 + t * 8
        wrote = real * (case["q_heads"] * e + 2 * case["kv_heads"] * _SIZE[case["cache"]]) * d
        return {"bytes": read + wrote, "flops": real * 3 * case["rot"] * (case["q_heads"] + case["kv_heads"])}
    if case["op"] == "beam":
        rows = case["seqs"] * case["beams"]
        return {"bytes": rows * (case["vocab"] * _SIZE[case["dtype"]] + 4) + 12 * case["seqs"] * case["keep"],
                "flops": 4 * rows * case["vocab"]}
    # a table entry is 4 bytes, a count is read and written; tails part-filled in (block - 1) of block cases are copied
    m, n, bs = case["parents"], case["children"], case["block"]
    held = (case["shortest"] + case["longest"]) / 2 / bs
    new = n * (1 + case["grow"]) / 2
    page = 2 * case["kv_heads"] * bs * case["head"] * _SIZE[case["dtype"]]
    fork = m * held * 12 + n * held * 4
    append = new * 8 + n * (24 + 16) + n * (bs - 1) / bs * 2 * page
    release = n * held * 4 + m * held * 8
    return {"bytes": fork + append + release, "flops": 2 * n * held}

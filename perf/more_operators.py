"""Sparse attention over the 8-bit paged cache as workloads: what each operator is given, its plain form, and what it
has to move.

The cache.  ``k`` (and ``v``; a latent cache uses ``k`` as both) is a pool ``[num_blocks, n_kv_heads, T, head_dim]``
of e4m3 values with one fp32 scale for each (block, head): the value held is ``e4m3 * scale``, and every scale is a
power of two.  A request's entry ``p`` sits in slot ``p % T`` of block ``block_table[rid, p // T]``.

Five operators work on it:

``rope``    appends new rows with their norm and their positions' rotation on the way;
``bounds``  the largest and smallest code of each channel of the blocks that a step touched;
``score``   for each query, kv head and block the bound ``max(q . k)`` that the block's bounds give;
``select``  for each query and kv head the blocks to read: the first, the newest and those of largest score;
``attn``    softmax attention of each query over the entries that it sees in its listed blocks.
"""
import math

import numpy as np
import torch

own = False

E_MIN, E_MAX = -48, 48  # exponents of the scales
E4M3 = torch.float8_e4m3fn
DEV = "cuda"
EPS = 1e-6


# ----------------------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one decode step's compressed rows into a latent cache: normalised, their last 64 channels rotated in pairs;
        # most of the 256 requests have no new row
        dict(name="rope_decode", op="rope", batch=256, new_min=0, new_max=1, len_max=8192, kv_heads=1, head_dim=512,
             block=64, shared=True, dtype="bf16", norm=True, halves=False, rope_dim=64, heads=0),
        # ragged prefill rows of eight heads, rotated over all channels, as they lie in a fused projection beside the
        # 32 query heads; some continue a block that is partly filled
        dict(name="rope_prefill", op="rope", batch=16, new_min=1, new_max=4096, len_max=8192, kv_heads=8,
             head_dim=128, block=32, shared=False, dtype="bf16", norm=False, halves=True, rope_dim=128, heads=32),
        # the one block of each request that a decode step stored into
        dict(name="bounds_decode", op="bounds", batch=64, new_min=1, new_max=1, len_max=16384, kv_heads=8, head_dim=128,
             block=64),
        # every block of a batch of prompts
        dict(name="bounds_prefill", op="bounds", batch=32, new_min=1, new_max=16384, len_max=16384, kv_heads=8,
             head_dim=128, block=64),
        # scores of a decode batch over long contexts: the bounds' bytes set the time
        dict(name="score_decode", op="score", batch=64, q_min=1, q_max=1, len_max=65536, heads=32, kv_heads=8,
             head_dim=128, block=64, ratio=1),
        # scores of chunked prefill: the products and the scores themselves count
        dict(name="score_chunk", op="score", batch=3, q_min=500, q_max=1024, len_max=32768, heads=32, kv_heads=8,
             head_dim=128, block=64, ratio=1),
        # one decode step's choice of 32 blocks of up to 1024, for 64 requests and eight heads
        dict(name="select_decode", op="select", batch=64, q_min=1, q_max=1, len_max=65536, kv_heads=8, block=64, ratio=1,
             budget=32, sinks=1, recent=2),
        # the choices of a few thousand queries
        dict(name="select_chunk", op="select", batch=3, q_min=500, q_max=1024, len_max=32768, kv_heads=8, block=64,
             ratio=1, budget=32, sinks=1, recent=2),
        # the smallest attention: one request, one token, an odd length; latency is all
        dict(name="attn_one", op="attn", batch=1, q_min=1, q_max=1, len_max=5003, heads=8, kv_heads=1, head_dim=128,
             block=16, shared=False, ratio=1, budget=16),
        # an ordinary decode batch of grouped heads, 2048 entries for each query and kv head
        dict(name="attn_decode", op="attn", batch=64, q_min=1, q_max=1, len_max=32768, heads=32, kv_heads=8,
             head_dim=128, block=64, shared=False, ratio=1, budget=32),
        # decode over a latent cache compressed four to one: 64 heads share 2048 of the 512-wide entries
        dict(name="attn_latent", op="attn", batch=64, q_min=1, q_max=1, len_max=16384, heads=64, kv_heads=1,
             head_dim=512, block=64, shared=True, ratio=4, budget=32),
        # chunked prefill, each query with blocks of its own
        dict(name="attn_chunk", op="attn", batch=2, q_min=300, q_max=512, len_max=16384, heads=16, kv_heads=4,
             head_dim=128, block=64, shared=False, ratio=1, budget=24),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["rope", "rope", "bounds", "score", "score", "select", "attn", "attn", "attn"])
    most = max(_cost(c) for c in listed() if c["op"] == op)
    while True:
        shared = rng.random() < 0.3
        kv = 1 if shared else rng.choice([1, 2, 4, 8])
        c = dict(op=op, batch=_log_int(rng, 1, 256), len_max=_log_int(rng, 1, 140000), kv_heads=kv,
                 head_dim=rng.choice([128, 512] if shared else [64, 128, 256]), block=rng.choice([16, 32, 64, 128]))
        if op in ("rope", "bounds"):
            c.update(new_min=rng.choice([0, 1]), new_max=_log_int(rng, 1, 4096 if op == "rope" else 16384))
            c["len_max"] = max(c["len_max"], c["new_max"])
        else:
            c["ratio"] = rng.choice([1, 4, 128] if shared else [1, 1, 4])
            c["q_max"] = min(c["len_max"], rng.choice([1, 1, 1, 4, _log_int(rng, 2, 1024)]))
            c["q_min"] = rng.randint(1, c["q_max"])
            c["heads"] = kv * rng.choice([1, 2, 4, 7, 8, 16] + ([64, 128] if shared else []))
        if op == "rope":
            c.update(shared=shared, dtype=rng.choice(["bf16", "bf16", "f32"]), norm=rng.random() < 0.5,
                     halves=rng.random() < 0.5, heads=rng.choice([0, kv, 4 * kv]),
                     rope_dim=rng.choice([r for r in (32, 64, 128, 192, 512) if r <= c["head_dim"]]))
        elif op == "select":
            c["budget"] = _log_int(rng, 1, 512)
            c["sinks"] = rng.randint(0, min(4, c["budget"] // 2))
            c["recent"] = rng.randint(0, min(8, c["budget"] - c["sinks"]))
        elif op == "attn":
            c.update(shared=shared, budget=_log_int(rng, 1, max(1, 4096 // c["block"])))
        # the plain form holds what it gathers in fp32
        n, width, G = c["batch"] * c.get("q_max", 1), -(-c["len_max"] // c["block"]), max(1, c.get("heads", 0) // kv)
        held = {"rope": 0, "bounds": 0, "score": c["batch"] * kv * width * (8 * c["head_dim"] + 8 * G * c.get("q_max", 1)),
                "select": 40 * n * kv * width,
                "attn": n * kv * c.get("budget", 0) * c["block"] * (8 * c["head_dim"] + 16 * G)}[op]
        if _cost(c) <= most and held < 20e9:
            return c


def _cost(case):
    """Seconds at round rates: the order in which cases are compared."""
    w = work(case)
    return w["bytes"] / 6.8e12 + w["flops"] / 1.9e15


def _lengths(case):
    """The requests' numbers, from the case alone so that its work is known: (kv_lens, new or query lengths)."""
    r = np.random.RandomState(case["batch"] * 31 + case["len_max"] * 7 + case["block"])
    B, most = case["batch"], case["len_max"]
    kv = np.sort(r.randint(0 if B >= 8 else 1, most + 1, B))[r.permutation(B)]
    kv[r.randint(0, B)] = most
    if "new_max" in case:
        n = r.randint(case["new_min"], case["new_max"] + 1, B)
        if n.sum() == 0:
            n[:] = 1
        return np.maximum(kv, n), n
    return kv, r.randint(case["q_min"], case["q_max"] + 1, B)


def _seq_lens(case, kv, n):
    """Token counts whose whole groups of ``ratio`` are the cached entries, and never under the query count."""
    ratio = case["ratio"]
    phase = np.arange(len(kv)) * 5 % ratio
    return np.maximum(kv * ratio + phase, n)


def _seen(case):
    """For each request the entries that each of its queries sees."""
    kv, n = _lengths(case)
    seq, ratio = _seq_lens(case, kv, n), case["ratio"]
    return [np.maximum(0, kv[b] - (seq[b] // ratio - (seq[b] - n[b] + 1 + np.arange(n[b])) // ratio)) for b in range(len(kv))]


def work(case):
    kv, n = _lengths(case)
    H, D, T = case["kv_heads"], case.get("head_dim"), case["block"]
    if case["op"] == "rope":
        # rows in, their 8-bit values and the touched blocks' scales out, one table row of (cos, sin) a position
        sides, rows = 1 if case["shared"] else 2, int(n.sum())
        entry = H * D * sides
        return {"bytes": float(rows * (entry * (1 + (2 if case["dtype"] == "bf16" else 4)) + 4 * case["rope_dim"]) + rows // T * H * sides * 4),
                "flops": float(rows * (entry * 2 + H * (3 * case["rope_dim"] + (4 * D if case["norm"] else 0))))}
    if case["op"] == "bounds":
        # the touched blocks' entries in, two rows out for each
        first = (kv - n) // T
        blocks, entries = (-(-kv // T) - first)[n > 0].sum(), (kv - first * T)[n > 0].sum()
        return {"bytes": float(H * D * (entries + 2 * blocks)), "flops": float(2 * H * D * entries)}
    seen = _seen(case)
    blocks = [-(-s // T) for s in seen]
    rows = int(n.sum())
    total, tops = sum(int(b.sum()) for b in blocks), sum(int(b.max()) for b in blocks)
    if case["op"] == "score":
        # bounds and scales in, queries in, scores out
        return {"bytes": float(H * tops * (2 * D + 4) + rows * case["heads"] * D * 2 + H * total * 4),
                "flops": 4.0 * total * case["heads"] * D}
    if case["op"] == "select":
        return {"bytes": float(H * (total * 4 + rows * case["budget"] * 4)), "flops": float(H * total)}
    # attention: the entries that a request's queries list between them, each read once (lists are independent choices)
    entry, listed_entries, read = D * (1 if case["shared"] else 2), 0.0, 0.0
    for s, b in zip(seen, blocks):
        k = np.minimum(b, case["budget"])
        listed_entries += float(np.minimum(s, k * T).sum())
        if b.max() > 0:
            share = k / np.maximum(1, b.max())
            read += float(s.max()) * (1.0 - float(np.exp(np.log1p(-np.minimum(share, 1 - 1e-12)).sum())))
    q = rows * case["heads"] * D
    return {"bytes": H * entry * read + q * 4.0 + rows * H * case["budget"] * 4.0 + rows * case["heads"] * 4.0,
            "flops": 4.0 * listed_entries * case["heads"] * D}


# ------------------------------------------------------------------------------------------------------------ inputs
def _need_exp(amax):
    """The smallest e with amax <= 448 * 2^e, within the scales' range."""
    m, x = torch.frexp(amax)
    return (x - 9 + (m > 0.875).to(x.dtype)).clamp(E_MIN, E_MAX)


def _pow2(e):
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _fill(g, blocks, H, T, D):
    """A pool of e4m3 values and its scales: normal entries, some channels larger, blocks of different size."""
    pool = torch.empty(blocks, H, T, D, dtype=torch.uint8, device=DEV)
    scale = torch.empty(blocks, H, device=DEV)
    channel = torch.exp(0.5 * torch.randn(H, 1, D, device=DEV, generator=g))
    channel = channel / channel.square().mean(-1, keepdim=True).sqrt()
    step = max(1, (1 << 27) // (H * T * D))
    for i in range(0, blocks, step):
        n = min(step, blocks - i)
        x = torch.randn(n, H, T, D, device=DEV, generator=g) * channel
        x += 0.5 * torch.randn(n, H, 1, D, device=DEV, generator=g)  # neighbours are alike
        x *= torch.exp(0.3 * torch.randn(n, H, 1, 1, device=DEV, generator=g))
        s = _pow2(_need_exp(x.abs().amax((2, 3))))
        pool[i:i + n] = (x / s[:, :, None, None]).to(E4M3).view(torch.uint8)
        scale[i:i + n] = s
    return pool.view(E4M3), scale


def _extremes(pool):
    """Every block's bounds, piece by piece."""
    out = torch.empty(pool.shape[0], pool.shape[1], 2, pool.shape[3], dtype=torch.uint8, device=DEV)
    step = max(1, (1 << 27) // pool[0].numel())
    for i in range(0, pool.shape[0], step):
        x = pool.view(torch.uint8)[i:i + step].view(E4M3).float()
        out[i:i + step] = torch.stack((x.amax(2), x.amin(2)), 2).to(E4M3).view(torch.uint8)
    return out.view(E4M3)


def _i64(a):
    return torch.as_tensor(np.asarray(a, np.int64), device=DEV)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    r = np.random.RandomState(seed % (1 << 31))
    kv, n = _lengths(case)
    B, T, H, D, op = case["batch"], case["block"], case["kv_heads"], case.get("head_dim"), case["op"]
    per = -(-kv // T)
    blocks = int(per.sum()) + 3
    order, at = r.permutation(blocks), 0
    rid = r.permutation(B + 2)[:B]
    table = np.full((B + 2, max(1, int(per.max()))), -1, np.int32)
    for b in range(B):
        table[rid[b], :per[b]] = order[at:at + per[b]]
        at += per[b]
    rows = int(n.sum())
    s = dict(case=case, rid=_i64(rid), kv_lens=_i64(kv), new_lens=_i64(n), rows=rows,
             table=torch.as_tensor(table, device=DEV))
    if op != "select":
        s["k"], s["k_scale"] = _fill(g, blocks, H, T, D)
        s["v"], s["v_scale"] = (None, None) if case.get("shared", True) else _fill(g, blocks, H, T, D)
    if op == "rope":
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        # rows as they lie in a projection: query heads, then keys, then values
        sides = 1 if case["shared"] else 2
        size = torch.exp(torch.randn(rows, 1, 1, device=DEV, generator=g))
        fused = (torch.randn(rows, case["heads"] + sides * H, D, device=DEV, generator=g) * size).to(dt)
        s["k_rows"] = fused[:, case["heads"]:case["heads"] + H]
        s["v_rows"] = None if case["shared"] else fused[:, case["heads"] + H:]
        R = case["rope_dim"]
        most = int(kv.max())
        angle = torch.arange(most, device=DEV, dtype=torch.float64)[:, None] * \
            10000.0 ** (-torch.arange(R // 2, device=DEV, dtype=torch.float64) / (R // 2))
        s["freqs"] = torch.stack((angle.cos(), angle.sin()), -1).float()
        b, i = _rows_of(s["new_lens"])
        s["positions"] = (s["kv_lens"] - s["new_lens"])[b] + i
        s["begin"] = 0 if case["halves"] else D - R
        s["weight"] = 1 + 0.1 * torch.randn(D, device=DEV, generator=g) if case["norm"] else None
    elif op == "bounds":
        s["bounds"] = torch.zeros(blocks, H, 2, D, dtype=torch.uint8, device=DEV).view(E4M3)
    else:
        s["seq_lens"] = _i64(_seq_lens(case, kv, n))
        if op != "select":
            s["scale"] = 1.0 / math.sqrt(D)
            s["q"] = (torch.randn(rows, case["heads"], D, device=DEV, generator=g) * 1.5).bfloat16()
        if op == "score":
            s["bounds"] = _extremes(s["k"])
        else:
            _, _, seen = _seen_plain(s)
            count = (seen + T - 1) // T
            width = table.shape[1]
            # scores on a coarse grid, as those of repeated text are: some are equal
            x = (torch.randn(rows, H, width, device=DEV, generator=g) * 3).bfloat16().float()
            x = x.masked_fill_(torch.arange(width, device=DEV) >= count[:, None, None], -math.inf)
            if op == "select":
                s["scores"] = x
            else:
                s["blocks"] = _choose(x, count, case["budget"], min(1, case["budget"] // 2), case["budget"] // 2 and 1)
    return s


# ------------------------------------------------------------------------------------------------------- plain forms
def _rows_of(lens):
    """For each ragged row: its request and its number within it."""
    b = torch.repeat_interleave(torch.arange(lens.numel(), device=lens.device), lens)
    first = torch.cumsum(lens, 0) - lens
    return b, torch.arange(b.numel(), device=lens.device) - first[b]


def _seen_plain(s):
    """For each query: its request, its number there, and how many entries it sees."""
    b, i = _rows_of(s["new_lens"])
    seq, ratio = s["seq_lens"][b], s["case"]["ratio"]
    after = seq // ratio - (seq - s["new_lens"][b] + i + 1) // ratio
    return b, i, (s["kv_lens"][b] - after).clamp(min=0)


def _round8(x):
    return x.clamp(-448.0, 448.0).to(E4M3).view(torch.uint8)


def _rotated(s):
    """The key rows in fp32, normalised and rotated."""
    c = s["case"]
    x = s["k_rows"].float()
    if s["weight"] is not None:
        x = x * s["weight"] / (x.square().mean(-1, keepdim=True) + EPS).sqrt()
    R, at = c["rope_dim"], s["begin"]
    cos, sin = s["freqs"][s["positions"]].unsqueeze(1).unbind(-1)
    y = x[..., at:at + R].unflatten(-1, (2, R // 2) if c["halves"] else (R // 2, 2))
    a, b = y.unbind(-2 if c["halves"] else -1)
    y = torch.stack((a * cos - b * sin, a * sin + b * cos), -2 if c["halves"] else -1).flatten(-2)
    return torch.cat((x[..., :at], y, x[..., at + R:]), -1)


def _store_side(pool, scale, x, s):
    c = s["case"]
    T, n = c["block"], s["new_lens"]
    b, i = _rows_of(n)
    start = s["kv_lens"] - n
    pos = start[b] + i
    block, slot = s["table"][s["rid"][b], pos // T].long(), pos % T
    need = _need_exp(torch.where(x.isfinite(), x.abs(), torch.zeros_like(x)).amax(-1))
    top = torch.full(scale.shape, E_MIN, dtype=need.dtype, device=DEV)
    top.scatter_reduce_(0, block[:, None].expand_as(need), need, "amax")
    new = _pow2(top)
    # the block that a request had begun keeps its scale where that is the larger one; its entries follow it
    begun = (n > 0) & (start % T > 0)
    first = s["table"][s["rid"], torch.where(begun, start // T, torch.zeros_like(start))].long()[begun]
    new[first] = torch.maximum(new[first], scale[first])
    bytes_ = pool.view(torch.uint8)
    old = bytes_[first]
    again = _round8(old.view(E4M3).float() * (scale[first] / new[first])[..., None, None])
    held = torch.arange(T, device=DEV) < (start[begun] % T)[:, None]
    bytes_[first] = torch.where(held[:, None, :, None], again, old)
    bytes_[block, :, slot] = _round8(x / new[block][..., None])
    scale[block] = new[block]
    return pool, scale


def _rope_plain(s):
    out = _store_side(s["k"], s["k_scale"], _rotated(s), s)
    return out if s["v"] is None else out + _store_side(s["v"], s["v_scale"], s["v_rows"].float(), s)


def _bounds_plain(s):
    T, n = s["case"]["block"], s["new_lens"]
    first = (s["kv_lens"] - n) // T
    b, j = _rows_of(torch.where(n > 0, (s["kv_lens"] + T - 1) // T - first, torch.zeros_like(n)))
    j = j + first[b]
    block = s["table"][s["rid"][b], j].long()
    here = (torch.arange(T, device=DEV) < (s["kv_lens"][b] - j * T)[:, None])[:, None, :, None]
    x = s["k"].view(torch.uint8)[block].view(E4M3).float()
    hi = x.masked_fill(~here, -math.inf).amax(2)
    lo = x.masked_fill(~here, math.inf).amin(2)
    s["bounds"].view(torch.uint8)[block] = torch.stack((hi, lo), 2).to(E4M3).view(torch.uint8)
    return s["bounds"]


def _score_plain(s):
    c = s["case"]
    H, G, D, T = c["kv_heads"], c["heads"] // c["kv_heads"], c["head_dim"], c["block"]
    b, i, seen = _seen_plain(s)
    at = s["table"][s["rid"]].clamp(min=0).long()
    k = s["bounds"].view(torch.uint8)[at].view(E4M3).float() * s["k_scale"][at][..., None, None]
    k = k.permute(0, 2, 1, 3, 4).flatten(3)  # [B, H, width, hi and lo]
    q = torch.zeros(c["batch"], c["q_max"], H, G, D, device=DEV)
    q[b, i] = s["q"].float().view(-1, H, G, D)
    q = q.permute(0, 2, 3, 1, 4).flatten(2, 3)
    z = torch.cat((q.clamp(min=0), q.clamp(max=0)), -1) @ k.transpose(2, 3) * s["scale"]
    z = z.unflatten(2, (G, c["q_max"])).amax(2).permute(0, 2, 1, 3)[b, i]
    return z.masked_fill_(torch.arange(z.shape[-1], device=DEV) >= ((seen + T - 1) // T)[:, None, None], -math.inf)


def _choose(scores, count, budget, sinks, recent):
    """[rows, H, budget] int32: block numbers in ascending order, -1 behind."""
    rows, H, width = scores.shape
    j = torch.arange(width, device=DEV)
    count = count[:, None, None]
    x = torch.where((j < sinks) | (j >= count - recent), torch.full_like(scores, math.inf), scores)
    # what a query does not see comes after everything, a score of minus infinity among it
    order = torch.sort(x, dim=-1, descending=True, stable=True).indices
    order = torch.gather(order, -1, torch.sort((order >= count).int(), dim=-1, stable=True).indices)[..., :budget]
    order = torch.where(order < count, order, torch.full_like(order, width))
    order = torch.sort(order, dim=-1).values
    out = torch.full((rows, H, budget), -1, dtype=torch.int32, device=DEV)
    out[..., :order.shape[-1]] = torch.where(order < width, order, torch.full_like(order, -1)).int()
    return out


def _select_plain(s):
    c = s["case"]
    _, _, seen = _seen_plain(s)
    return _choose(s["scores"], (seen + c["block"] - 1) // c["block"], c["budget"], c["sinks"], c["recent"])


def _attn_plain(s):
    c = s["case"]
    H, G, T = c["kv_heads"], c["heads"] // c["kv_heads"], c["block"]
    b, _, seen = _seen_plain(s)
    rows, width = s["rows"], s["table"].shape[1]
    at = torch.where(s["blocks"] >= 0, s["table"][s["rid"][b]].gather(1, s["blocks"].long().clamp(0, width - 1).flatten(1)).view_as(s["blocks"]), s["blocks"]).long()
    entry = s["blocks"].long()[..., None] * T + torch.arange(T, device=DEV)
    see = ((at >= 0)[..., None] & (entry < seen[:, None, None, None])).flatten(2)
    at, h = at.clamp(min=0), torch.arange(H, device=DEV)[:, None]

    def values(pool, scale):
        x = pool.view(torch.uint8)[at, h].view(E4M3).float()
        return x.mul_(scale[at, h][..., None, None]).flatten(2, 3)

    k = values(s["k"], s["k_scale"])
    z = (s["q"].float().view(rows, H, G, -1) @ k.transpose(2, 3)) * s["scale"]
    z = z.masked_fill_(~see[:, :, None], -math.inf)
    top = z.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = z.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    v = k if s["v"] is None else values(s["v"], s["v_scale"])
    v = torch.where(see[..., None], v, torch.zeros_like(v))
    o = (p @ v) / torch.where(total == 0, torch.ones_like(total), total)
    return o.flatten(1, 2).bfloat16(), (total.log() + top).squeeze(-1).flatten(1, 2)


# --------------------------------------------------------------------------------------------------------- one pass
def run(state):
    op = state["case"]["op"]
    if own:
        return _OWN[op](state)
    if op == "rope":
        return _rope_plain(state)
    if op == "bounds":
        return _bounds_plain(state)
    if op == "score":
        return _score_plain(state)
    if op == "select":
        return _select_plain(state)
    return _attn_plain(state)


def _rope_own(s):
    from compressed_kv_attention_compressplan_gb300 import ckv
    cache, c = ckv.Q8Cache(s["k"], s["k_scale"], s["v"], s["v_scale"]), s["case"]
    plan, counts = ckv.plan_q8_store(cache, s["rid"], s["kv_lens"], s["new_lens"], s["rows"], s["table"])
    ckv.q8_rope_store(cache, s["k_rows"], s["v_rows"], plan, s["positions"], s["freqs"], counts, rope_begin=s["begin"],
                      halves=c["halves"], norm_weight=s["weight"], eps=EPS)
    return [x for x in cache if x is not None]


def _bounds_own(s):
    from compressed_kv_attention_compressplan_gb300 import ckv
    cache = ckv.Q8Cache(s["k"], s["k_scale"])
    return ckv.q8_bounds(cache, s["bounds"], s["rid"], s["kv_lens"], s["new_lens"], s["table"])


def _score_own(s):
    from compressed_kv_attention_compressplan_gb300 import ckv
    cache = ckv.Q8Cache(s["k"], s["k_scale"])
    return ckv.q8_block_scores(cache, s["bounds"], s["q"], s["case"]["ratio"], s["rid"], s["seq_lens"], s["new_lens"],
                               s["kv_lens"], s["table"], s["scale"])


def _select_own(s):
    from compressed_kv_attention_compressplan_gb300 import ckv
    c = s["case"]
    return ckv.q8_block_select(s["scores"], c["block"], c["ratio"], s["seq_lens"], s["new_lens"], s["kv_lens"],
                               c["budget"], c["sinks"], c["recent"])


def _attn_own(s):
    from compressed_kv_attention_compressplan_gb300 import ckv
    cache = ckv.Q8Cache(s["k"], s["k_scale"], s["v"], s["v_scale"])
    return ckv.q8_attn_blocks(cache, s["q"], s["blocks"], s["case"]["ratio"], s["rid"], s["seq_lens"], s["new_lens"],
                              s["kv_lens"], s["table"], s["scale"])


_OWN = {"rope": _rope_own, "bounds": _bounds_own, "score": _score_own, "select": _select_own, "attn": _attn_own}


# ------------------------------------------------------------------------------------------------- the definition
def exact(case, seed):
    """The definitions in 64 bits, request by request."""
    if case["op"] == "select":
        return None  # block numbers: nothing is computed
    s = prepare(case, seed)
    return {"rope": _exact_rope, "bounds": _exact_bounds, "score": _exact_score, "attn": _exact_attn}[case["op"]](s)


def _exact_rows(s):
    """The key rows, normalised and turned as complex numbers."""
    c = s["case"]
    x = s["k_rows"].double()
    if s["weight"] is not None:
        x = x * torch.rsqrt(torch.linalg.vector_norm(x, dim=-1, keepdim=True) ** 2 / x.shape[-1] + EPS) * s["weight"].double()
    R, at = c["rope_dim"], s["begin"]
    turn = torch.view_as_complex(s["freqs"][s["positions"]].double())[:, None]
    one = torch.arange(R // 2, device=DEV) if c["halves"] else torch.arange(0, R, 2, device=DEV)
    two = one + (R // 2 if c["halves"] else 1)
    z = torch.complex(x[..., at + one], x[..., at + two]) * turn
    y = x.clone()
    y[..., at + one], y[..., at + two] = z.real, z.imag
    return y


def _exact_rope(s):
    c = s["case"]
    T, out = c["block"], []
    powers = torch.tensor([math.ldexp(1.0, e) for e in range(E_MIN, E_MAX + 1)], dtype=torch.float64, device=DEV)
    for pool, scale, rows in ((s["k"], s["k_scale"], _exact_rows(s)),
                              (s["v"], s["v_scale"], None if s["v"] is None else s["v_rows"].double())):
        if pool is None:
            continue
        held, sc = pool.double(), scale.double()
        first = 0
        for b in range(c["batch"]):
            n, kv = int(s["new_lens"][b]), int(s["kv_lens"][b])
            start, table = kv - n, s["table"][int(s["rid"][b])].tolist()
            for j in range(start // T, -(-kv // T) if n else 0):
                lo, hi = max(start, j * T), min(kv, j * T + T)
                x = rows[first + lo - start:first + hi - start]
                top = x.abs().amax((0, 2))  # the first power of two that 448 times is not under it
                new = powers[(top[:, None] > 448.0 * powers[:-1]).sum(1)]
                block, off = table[j], lo - j * T
                if off:
                    new = torch.maximum(new, sc[block])
                    held[block, :, :off] *= (sc[block] / new)[:, None, None]
                held[block, :, off:off + hi - lo] = (x / new[:, None]).transpose(0, 1)
                sc[block] = new
            first += n
        out += [held, sc]
    return out


def _exact_bounds(s):
    T = s["case"]["block"]
    out = s["bounds"].double()
    for b in range(s["case"]["batch"]):
        kv, n = int(s["kv_lens"][b]), int(s["new_lens"][b])
        table = s["table"][int(s["rid"][b])].long()
        first = (kv - n) // T
        if n == 0:
            continue
        whole = table[first:kv // T]
        if len(whole):
            x = s["k"].view(torch.uint8)[whole].view(E4M3).double()
            out[whole] = torch.stack((x.max(2).values, x.min(2).values), 2)
        if kv % T:
            x = s["k"][table[kv // T]].double()[:, :kv % T]
            out[table[kv // T]] = torch.stack((x.max(1).values, x.min(1).values), 1)
    return out


def _exact_score(s):
    c = s["case"]
    H, G, T, R = c["kv_heads"], c["heads"] // c["kv_heads"], c["block"], c["ratio"]
    if work(c)["flops"] > 2e11:
        return None
    out = torch.full((s["rows"], H, s["table"].shape[1]), -math.inf, dtype=torch.float64, device=DEV)
    first = 0
    for b in range(c["batch"]):
        n, kv, seq = int(s["new_lens"][b]), int(s["kv_lens"][b]), int(s["seq_lens"][b])
        at = s["table"][int(s["rid"][b]), :-(-kv // T)].long()
        k = s["bounds"].view(torch.uint8)[at].view(E4M3).double() * s["k_scale"][at].double()[..., None, None]
        step = max(1, int(2e8 // max(1, len(at) * c["heads"] * c["head_dim"])))
        for lo in range(0, n if kv else 0, step):
            hi = min(n, lo + step)
            q = s["q"][first + lo:first + hi].double().view(hi - lo, H, G, 1, -1)
            z = torch.maximum(q * k[:, :, 0].transpose(0, 1)[:, None], q * k[:, :, 1].transpose(0, 1)[:, None])
            z = z.sum(-1).max(2).values * s["scale"]
            pos = seq - n + 1 + torch.arange(lo, hi, device=DEV)
            seen = (kv - (seq // R - pos // R)).clamp(min=0)
            see = torch.arange(len(at), device=DEV) * T < seen[:, None]
            out[first + lo:first + hi, :, :len(at)] = torch.where(see[:, None], z, torch.full_like(z, -math.inf))
        first += n
    return out


def _exact_attn(s):
    c = s["case"]
    H, G, T, R = c["kv_heads"], c["heads"] // c["kv_heads"], c["block"], c["ratio"]
    if work(c)["flops"] > 1e12:
        return None
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device=DEV)
    first = 0
    for b in range(c["batch"]):
        n, kv, seq = int(s["new_lens"][b]), int(s["kv_lens"][b]), int(s["seq_lens"][b])
        at = s["table"][int(s["rid"][b]), :-(-kv // T)].long()
        sides = [(s["k"], s["k_scale"]), (s["k"], s["k_scale"]) if s["v"] is None else (s["v"], s["v_scale"])]
        held = [p.view(torch.uint8)[at].view(E4M3).double() * sc[at].double()[..., None, None] for p, sc in sides]
        held = [x.transpose(0, 1).flatten(1, 2) for x in held]  # [H, entries, D]
        step = max(1, int(1e8 // max(1, kv * c["heads"])))
        for lo in range(0, n if kv else 0, step):
            hi = min(n, lo + step)
            q = s["q"][first + lo:first + hi].double().view(hi - lo, H, G, -1)
            z = torch.einsum("nhgd,hsd->nhgs", q, held[0]) * s["scale"]
            # which blocks each query lists: a place of its own behind them takes the -1s
            chosen = torch.zeros(hi - lo, H, len(at) + 1, dtype=torch.bool, device=DEV)
            lists = s["blocks"][first + lo:first + hi].long()
            chosen.scatter_(2, torch.where(lists < 0, torch.full_like(lists, len(at)), lists), True)
            pos = seq - n + 1 + torch.arange(lo, hi, device=DEV)
            entry = torch.arange(z.shape[-1], device=DEV)
            see = chosen[..., entry // T] & (entry < (kv - (seq // R - pos // R))[:, None, None])
            z = torch.where(see[:, :, None], z, torch.full_like(z, -math.inf))
            l = torch.logsumexp(z, -1)
            p = torch.where(see[:, :, None], torch.exp(z - l[..., None]), torch.zeros_like(z))
            out[first + lo:first + hi] = torch.einsum("nhgs,hsd->nhgd", p, held[1]).flatten(1, 2)
            lse[first + lo:first + hi] = l.flatten(1, 2)
        first += n
    return out, lse

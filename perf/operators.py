"""The 8-bit paged cache's operators as workloads: what each one is given, its plain form, and what it has to move.

The cache.  ``k`` (and ``v``; a latent cache uses ``k`` as both) is a pool ``[num_blocks, n_kv_heads, T, head_dim]``
of e4m3 values with one fp32 scale for each (block, head): the value held is ``e4m3 * scale``, and every scale is a
power of two.  A request's entry ``p`` sits in slot ``p % T`` of block ``block_table[rid, p // T]``.

Four operators work on it:

``store``  appends new rows, choosing each touched block's scale from its largest finite value;
``attn``   softmax attention of the queries over the cache, with the number of entries that a query sees counted in
           whole groups of ``ratio`` tokens (ratio 1: causal attention; 4 or 128: a compressed cache);
``weigh``  adds the attention weight that each cached entry received to its running sum;
``evict``  keeps the ``budget`` entries of largest sum, besides the first and the newest ones, and moves them into
           blocks of their own.
"""
import math

import numpy as np
import torch

own = False

E_MIN, E_MAX = -48, 48  # exponents of the scales
E4M3 = torch.float8_e4m3fn
DEV = "cuda"


# ----------------------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one decode step's compressed rows into a latent cache: 256 requests, most of them without a new row
        dict(name="store_decode", op="store", batch=256, new_min=0, new_max=1, len_max=8192, kv_heads=1, head_dim=512,
             block=64, shared=True, dtype="bf16"),
        # ragged prefill rows of a cache of eight heads, some continuing a block that is partly filled
        dict(name="store_prefill", op="store", batch=16, new_min=1, new_max=4096, len_max=8192, kv_heads=8,
             head_dim=128, block=32, shared=False, dtype="bf16"),
        # the smallest call: one request, one token, an odd length; latency is all
        dict(name="attn_one", op="attn", batch=1, q_min=1, q_max=1, len_max=777, heads=8, kv_heads=1, head_dim=128,
             block=16, shared=False, ratio=1),
        # an ordinary decode batch of grouped heads, lengths spread from nothing to the longest
        dict(name="attn_decode", op="attn", batch=64, q_min=1, q_max=1, len_max=16384, heads=32, kv_heads=8,
             head_dim=128, block=64, shared=False, ratio=1),
        # decode over a latent cache compressed four to one: every head reads the same 512-wide entries
        dict(name="attn_latent", op="attn", batch=64, q_min=1, q_max=1, len_max=8192, heads=64, kv_heads=1,
             head_dim=512, block=64, shared=True, ratio=4),
        # two requests with long contexts: the work of one row is split over the whole card
        dict(name="attn_long", op="attn", batch=2, q_min=1, q_max=1, len_max=140001, heads=32, kv_heads=4,
             head_dim=128, block=128, shared=False, ratio=1),
        # a speculative verify step: one to four tokens a request, narrow heads, small blocks, odd lengths
        dict(name="attn_verify", op="attn", batch=48, q_min=1, q_max=4, len_max=5003, heads=16, kv_heads=2,
             head_dim=64, block=16, shared=False, ratio=1),
        # chunked prefill: a few thousand queries over long cached contexts; the matrix products set the time
        dict(name="attn_chunk", op="attn", batch=3, q_min=1000, q_max=2048, len_max=16384, heads=32, kv_heads=8,
             head_dim=128, block=64, shared=False, ratio=1),
        # the weights of one decode step, for eviction later
        dict(name="weigh_decode", op="weigh", batch=32, q_min=1, q_max=1, len_max=8192, heads=32, kv_heads=8,
             head_dim=128, block=64, shared=False, ratio=1),
        # the weights that a prefill's last window of queries gives to the prompt
        dict(name="weigh_window", op="weigh", batch=4, q_min=32, q_max=32, len_max=32768, heads=16, kv_heads=2,
             head_dim=128, block=32, shared=False, ratio=1),
        # one request cut down to a third
        dict(name="evict_one", op="evict", batch=1, len_max=1500, budget=512, sinks=4, recent=128, kv_heads=1,
             head_dim=512, block=64, shared=True),
        # a serving batch cut down to 4096 entries each; short requests are moved whole
        dict(name="evict_batch", op="evict", batch=32, len_max=16384, budget=4096, sinks=4, recent=512, kv_heads=8,
             head_dim=128, block=64, shared=False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["store", "attn", "attn", "attn", "weigh", "evict"])
    most = {c["op"]: 0.0 for c in listed()}
    for c in listed():
        most[c["op"]] = max(most[c["op"]], _cost(c))
    while True:
        shared = rng.random() < 0.3
        kv = 1 if shared else rng.choice([1, 2, 4, 8])
        c = dict(op=op, batch=_log_int(rng, 1, 256), len_max=_log_int(rng, 1, 140000), kv_heads=kv,
                 head_dim=rng.choice([128, 512] if shared else [64, 128, 256]), block=rng.choice([16, 32, 64, 128]),
                 shared=shared)
        if op == "store":
            c.update(new_min=rng.choice([0, 1]), new_max=_log_int(rng, 1, 4096), dtype=rng.choice(["bf16", "bf16", "f32"]))
            c["len_max"] = max(c["len_max"], c["new_max"])
        elif op == "evict":
            c["len_max"] = max(16, c["len_max"])
            c["budget"] = _log_int(rng, 8, min(8192, c["len_max"]))
            c["sinks"] = rng.randint(0, min(8, c["budget"] // 4))
            c["recent"] = rng.randint(0, c["budget"] // 2)
        else:
            group = rng.choice([1, 2, 4, 7, 8, 16] + ([64, 128] if shared else []))
            c["heads"] = kv * group
            c["ratio"] = rng.choice([1, 4, 128] if shared else [1, 1, 4])
            c["q_max"] = rng.choice([1, 1, 1, 4, _log_int(rng, 2, 2048)])
            if op == "weigh":
                c["q_max"] = min(c["q_max"], 64)
            c["q_max"] = min(c["q_max"], c["len_max"])
            c["q_min"] = rng.randint(1, c["q_max"])
        # the plain form holds the padded scores and an fp32 copy of the padded cache
        padded = c["batch"] * c["len_max"] * (4 * 2 * kv * c["head_dim"] + 12 * c.get("heads", 0) * c.get("q_max", 0))
        if _cost(c) <= most[op] and padded < 40e9:
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
    if case["op"] == "store":
        n = r.randint(case["new_min"], case["new_max"] + 1, B)
        if n.sum() == 0:
            n[:] = 1
        return np.maximum(kv, n), n
    if case["op"] == "evict":
        return kv, np.zeros(B, np.int64)
    return kv, r.randint(case["q_min"], case["q_max"] + 1, B)


def _seq_lens(case, kv, n):
    """Token counts whose whole groups of ``ratio`` are the cached entries, and never under the query count."""
    ratio = case.get("ratio", 1)
    phase = np.arange(len(kv)) * 5 % ratio
    return np.maximum(kv * ratio + phase, n)


def _seen(case):
    """Sum over queries of the entries each sees, and the largest such number for each request."""
    kv, n = _lengths(case)
    seq, ratio = _seq_lens(case, kv, n), case["ratio"]
    total, tops = 0, []
    for b in range(len(kv)):
        pos = seq[b] - n[b] + 1 + np.arange(n[b])
        vis = np.maximum(0, kv[b] - (seq[b] // ratio - pos // ratio))
        total += int(vis.sum())
        tops.append(int(vis.max()))
    return total, tops


def work(case):
    kv, n = _lengths(case)
    H, D, sides = case["kv_heads"], case["head_dim"], 1 if case["shared"] else 2
    entry = H * D * sides  # bytes of a cached entry
    if case["op"] == "store":
        # rows in, their 8-bit values out, one scale a touched block; a block begun earlier is read and written
        # only where its scale grows, which is left out
        rows = int(n.sum())
        return {"bytes": float(rows * entry * (1 + (2 if case["dtype"] == "bf16" else 4)) + rows // case["block"] * H * sides * 4),
                "flops": float(rows * entry * 2)}
    if case["op"] == "evict":
        kept = np.minimum(kv, case["budget"])
        return {"bytes": float(kept.sum() * entry * 2 + kv.sum() * 4 + kept.sum() * 8), "flops": float(kv.sum() * 4)}
    total, tops = _seen(case)
    q = int(n.sum()) * case["heads"] * D
    if case["op"] == "attn":
        return {"bytes": float(sum(tops) * entry + q * 4 + int(n.sum()) * case["heads"] * 4),
                "flops": 4.0 * total * case["heads"] * D}
    return {"bytes": float(sum(tops) * H * D + q * 2 + int(n.sum()) * case["heads"] * 4 + sum(tops) * 8),
            "flops": 2.0 * total * case["heads"] * D}


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
        x *= torch.exp(0.3 * torch.randn(n, H, 1, 1, device=DEV, generator=g))
        s = _pow2(_need_exp(x.abs().amax((2, 3))))
        pool[i:i + n] = (x / s[:, :, None, None]).to(E4M3).view(torch.uint8)
        scale[i:i + n] = s
    return pool.view(E4M3), scale


def _i64(a):
    return torch.as_tensor(np.asarray(a, np.int64), device=DEV)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    r = np.random.RandomState(seed % (1 << 31))
    kv, n = _lengths(case)
    B, T, H, D = case["batch"], case["block"], case["kv_heads"], case["head_dim"]
    per = -(-kv // T)
    out_per = -(-np.minimum(kv, case["budget"]) // T) if case["op"] == "evict" else np.zeros(B, np.int64)
    blocks = int(per.sum() + out_per.sum()) + 3
    order = r.permutation(blocks)
    rid = r.permutation(B + 2)[:B]

    def table(counts, at):
        t = np.full((B + 2, max(1, int(counts.max()))), -1, np.int32)
        for b in range(B):
            t[rid[b], :counts[b]] = order[at:at + counts[b]]
            at += counts[b]
        return torch.as_tensor(t, device=DEV)

    s = dict(case=case, rid=_i64(rid), kv_lens=_i64(kv), table=table(per, 0))
    s["k"], s["k_scale"] = _fill(g, blocks, H, T, D)
    s["v"], s["v_scale"] = (None, None) if case["shared"] else _fill(g, blocks, H, T, D)
    rows = int(n.sum())
    if case["op"] == "store":
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        s["new_lens"] = _i64(n)
        grow = torch.exp(torch.randn(rows, 1, 1, device=DEV, generator=g))
        s["k_rows"] = (torch.randn(rows, H, D, device=DEV, generator=g) * grow).to(dt)
        s["v_rows"] = None if case["shared"] else torch.randn(rows, H, D, device=DEV, generator=g).to(dt)
    elif case["op"] == "evict":
        s["dst"] = table(out_per, int(per.sum()))
        s["weights"] = torch.exp(2.0 * torch.randn(blocks, T, device=DEV, generator=g))
    else:
        s["new_lens"], s["seq_lens"] = _i64(n), _i64(_seq_lens(case, kv, n))
        s["scale"] = 1.0 / math.sqrt(D)
        s["q"] = (torch.randn(rows, case["heads"], D, device=DEV, generator=g) * 1.5).bfloat16()
        if case["op"] == "weigh":
            s["lse"] = _attn_plain(s, values=False)[1]
            s["weights"] = torch.rand(blocks, T, device=DEV, generator=g)
    return s


# ------------------------------------------------------------------------------------------------------- plain forms
def _rows_of(lens):
    """For each ragged row: its request and its number within it."""
    b = torch.repeat_interleave(torch.arange(lens.numel(), device=lens.device), lens)
    first = torch.cumsum(lens, 0) - lens
    return b, torch.arange(b.numel(), device=lens.device) - first[b]


def _gather(pool, scale, table):
    """[B, H, S, D] fp32 values of the blocks that ``table`` [B, n] names."""
    at = table.clamp(min=0).long()
    x = pool.view(torch.uint8)[at].view(E4M3).float() * scale[at][..., None, None]
    return x.permute(0, 2, 1, 3, 4).flatten(2, 3)


def _seen_plain(s):
    """For each query row: how many entries it sees."""
    b, i = _rows_of(s["new_lens"])
    seq, ratio = s["seq_lens"][b], s["case"]["ratio"]
    after = seq // ratio - (seq - s["new_lens"][b] + i + 1) // ratio
    return b, i, (s["kv_lens"][b] - after).clamp(min=0)


def _scores_plain(s):
    """Padded scores [B, H, group, Q, S] in fp32, -inf where a query does not see an entry."""
    c = s["case"]
    H, G, D = c["kv_heads"], c["heads"] // c["kv_heads"], c["head_dim"]
    b, i, seen = _seen_plain(s)
    B, Q = c["batch"], c["q_max"]
    q = torch.zeros(B, Q, H, G, D, device=DEV)
    q[b, i] = s["q"].float().view(-1, H, G, D)
    vis = torch.zeros(B, Q, dtype=torch.long, device=DEV)
    vis[b, i] = seen
    k = _gather(s["k"], s["k_scale"], s["table"][s["rid"]])
    z = (q.permute(0, 2, 3, 1, 4).flatten(2, 3) @ k.transpose(2, 3)) * s["scale"]
    z = z.unflatten(2, (G, Q))
    hidden = torch.arange(z.shape[-1], device=DEV) >= vis[:, None, None, :, None]
    return z.masked_fill_(hidden, -math.inf), b, i


def _attn_plain(s, values=True):
    z, b, i = _scores_plain(s)
    top = z.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = z.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    lse = (total.log() + top).squeeze(-1).permute(0, 3, 1, 2).flatten(2, 3)[b, i]
    if not values:
        return None, lse
    pool, scale = (s["k"], s["k_scale"]) if s["v"] is None else (s["v"], s["v_scale"])
    v = _gather(pool, scale, s["table"][s["rid"]])
    here = torch.arange(v.shape[2], device=DEV) < s["kv_lens"][:, None]
    v = torch.where(here[:, None, :, None], v, torch.zeros_like(v))
    o = (p.flatten(2, 3) @ v).unflatten(2, p.shape[2:4]) / torch.where(total == 0, torch.ones_like(total), total)
    o = o.permute(0, 3, 1, 2, 4).flatten(2, 3)[b, i]
    return o.bfloat16(), lse


def _weigh_plain(s):
    z, b, i = _scores_plain(s)
    c = s["case"]
    lse = torch.full((c["batch"], c["q_max"], c["heads"]), math.inf, device=DEV)
    lse[b, i] = torch.where(s["lse"] == -math.inf, torch.full_like(s["lse"], math.inf), s["lse"])
    lse = lse.unflatten(2, z.shape[1:3]).permute(0, 2, 3, 1)
    got = z.sub_(lse[..., None]).exp_().sum((1, 2, 3))
    flat, at = s["weights"].view(-1), _slots(s, s["kv_lens"])
    rb, ri = _rows_of(s["kv_lens"])
    flat[at] += got[rb, ri]
    return s["weights"]


def _slots(s, lens):
    """The pool slot of each entry, request after request."""
    b, i = _rows_of(lens)
    T = s["case"]["block"]
    return s["table"][s["rid"][b], i // T].long() * T + i % T


def _round8(x):
    return x.clamp(-448.0, 448.0).to(E4M3).view(torch.uint8)


def _store_side(pool, scale, rows, s):
    c = s["case"]
    T, n = c["block"], s["new_lens"]
    b, i = _rows_of(n)
    start = s["kv_lens"] - n
    pos = start[b] + i
    block, slot = s["table"][s["rid"][b], pos // T].long(), pos % T
    x = rows.float()
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


def _store_plain(s):
    out = _store_side(s["k"], s["k_scale"], s["k_rows"], s)
    return out if s["v"] is None else out + _store_side(s["v"], s["v_scale"], s["v_rows"], s)


def _evict_plain(s):
    c = s["case"]
    T, S = c["block"], s["table"].shape[1] * c["block"]
    lens = s["kv_lens"]
    at = s["table"][s["rid"]].clamp(min=0).long()
    w = s["weights"][at].flatten(1)
    pos = torch.arange(S, device=DEV)
    inside = pos < lens[:, None]
    safe = (pos < c["sinks"]) | (pos >= lens[:, None] - c["recent"])
    w = torch.where(safe, torch.full_like(w, math.inf), w)
    w = torch.where(inside, w, torch.full_like(w, -math.inf))
    keep = min(c["budget"], S)
    chosen = torch.sort(w, dim=1, descending=True, stable=True).indices[:, :keep]
    count = torch.minimum(lens, torch.full_like(lens, keep))
    rank = torch.arange(keep, device=DEV)
    chosen = torch.where(rank < count[:, None], chosen, torch.full_like(chosen, S))
    chosen = torch.sort(chosen, dim=1).values
    b, i = _rows_of(count)
    p = chosen[b, i]
    src, src_slot = s["table"][s["rid"][b], p // T].long(), p % T
    dst, dst_slot = s["dst"][s["rid"][b], i // T].long(), i % T
    out = []
    for pool, scale in ((s["k"], s["k_scale"]), (s["v"], s["v_scale"]))[:1 if s["v"] is None else 2]:
        new = torch.zeros_like(scale).scatter_reduce_(0, dst[:, None].expand(-1, scale.shape[1]), scale[src], "amax")
        x = pool.view(torch.uint8)[src, :, src_slot].view(E4M3).float() * (scale[src] / new[dst])[..., None]
        pool.view(torch.uint8)[dst, :, dst_slot] = _round8(x)
        scale[dst] = new[dst]
        out += [pool, scale]
    s["weights"][dst, dst_slot] = s["weights"][src, src_slot]
    kept = torch.full((c["batch"], c["budget"]), -1, dtype=torch.int32, device=DEV)
    kept[b, i] = p.int()
    return [kept, count, s["weights"]] + out


# --------------------------------------------------------------------------------------------------------- one pass
def run(state):
    s = state
    op = s["case"]["op"]
    if own:
        return _OWN[op](s)
    if op == "store":
        return _store_plain(s)
    if op == "attn":
        return _attn_plain(s)
    if op == "weigh":
        return _weigh_plain(s)
    return _evict_plain(s)


def _store_own(s):
    from compressed_kv_attention_compressplan_gb300 import ckv
    cache = ckv.Q8Cache(s["k"], s["k_scale"], s["v"], s["v_scale"])
    plan, counts = ckv.plan_q8_store(cache, s["rid"], s["kv_lens"], s["new_lens"], s["k_rows"].shape[0], s["table"])
    ckv.q8_store(cache, s["k_rows"], s["v_rows"], plan, counts)
    return [x for x in cache if x is not None]


def _attn_own(s):
    from compressed_kv_attention_compressplan_gb300 import ckv
    cache = ckv.Q8Cache(s["k"], s["k_scale"], s["v"], s["v_scale"])
    plan = ckv.plan_q8_attn(cache, s["case"]["heads"], s["case"]["ratio"], s["rid"], s["seq_lens"], s["new_lens"],
                            s["kv_lens"], s["q"].shape[0])
    return ckv.q8_attn(cache, s["q"], plan, s["table"], s["scale"])


def _weigh_own(s):
    from compressed_kv_attention_compressplan_gb300 import ckv
    cache = ckv.Q8Cache(s["k"], s["k_scale"], s["v"], s["v_scale"])
    return ckv.q8_weigh(cache, s["q"], s["lse"], s["weights"], s["case"]["ratio"], s["rid"], s["seq_lens"],
                        s["new_lens"], s["kv_lens"], s["table"], s["scale"])


def _evict_own(s):
    from compressed_kv_attention_compressplan_gb300 import ckv
    cache, c = ckv.Q8Cache(s["k"], s["k_scale"], s["v"], s["v_scale"]), s["case"]
    kept, count = ckv.q8_evict(cache, s["weights"], s["rid"], s["kv_lens"], s["table"], s["dst"], c["budget"],
                               c["sinks"], c["recent"])
    return [kept, count, s["weights"]] + [x for x in cache if x is not None]


_OWN = {"store": _store_own, "attn": _attn_own, "weigh": _weigh_own, "evict": _evict_own}


# ------------------------------------------------------------------------------------------------- the definition
def exact(case, seed):
    """The definitions in 64 bits, request by request."""
    s = prepare(case, seed)
    return {"store": _exact_store, "attn": _exact_attn, "weigh": _exact_weigh, "evict": _exact_evict}[case["op"]](s)


def _entries(s, b, side):
    """Request b's cached values [H, kv_len, D] in 64 bits."""
    T, L = s["case"]["block"], int(s["kv_lens"][b])
    at = s["table"][int(s["rid"][b]), :-(-L // T)].long()
    pool, scale = (s["k"], s["k_scale"]) if side == "k" or s["v"] is None else (s["v"], s["v_scale"])
    x = pool.view(torch.uint8)[at].view(E4M3).double() * scale[at].double()[:, :, None, None]
    return x.transpose(0, 1).flatten(1, 2)[:, :L]


def _exact_rows(s, b, lo, hi):
    """Scores [H, group, hi - lo, kv_len] of request b's queries lo .. hi, and what each query sees."""
    c = s["case"]
    H, G, R = c["kv_heads"], c["heads"] // c["kv_heads"], c["ratio"]
    n = int(s["new_lens"][b])
    first = int(s["new_lens"][:b].sum())
    q = s["q"][first + lo:first + hi].double().view(-1, H, G, c["head_dim"]).permute(1, 2, 0, 3)
    z = torch.einsum("hgqd,hsd->hgqs", q, _entries(s, b, "k")) * s["scale"]
    seq, kv = int(s["seq_lens"][b]), int(s["kv_lens"][b])
    pos = seq - n + 1 + torch.arange(lo, hi, device=DEV)
    seen = kv - (seq // R - pos // R)
    see = torch.arange(kv, device=DEV) < seen[:, None]
    return z, see, first


def _exact_attn(s):
    c = s["case"]
    if work(c)["flops"] > 3e12:
        return None
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device=DEV)
    for b in range(c["batch"]):
        n, kv = int(s["new_lens"][b]), int(s["kv_lens"][b])
        step = max(1, int(2e8 // max(1, kv * c["heads"])))
        for lo in range(0, n if kv else 0, step):
            hi = min(n, lo + step)
            z, see, first = _exact_rows(s, b, lo, hi)
            z = torch.where(see, z, torch.full_like(z, -math.inf))
            l = torch.logsumexp(z, -1)
            p = torch.where(see, torch.exp(z - l[..., None]), torch.zeros_like(z))
            o = torch.einsum("hgqs,hsd->qhgd", p, _entries(s, b, "v"))
            out[first + lo:first + hi] = o.flatten(1, 2)
            lse[first + lo:first + hi] = l.permute(2, 0, 1).flatten(1, 2)
    return out, lse


def _exact_weigh(s):
    c = s["case"]
    total = s["weights"].double()
    T = c["block"]
    for b in range(c["batch"]):
        n, kv = int(s["new_lens"][b]), int(s["kv_lens"][b])
        at = torch.arange(kv, device=DEV)
        slot = s["table"][int(s["rid"][b])].long()[at // T] * T + at % T
        step = max(1, int(2e8 // max(1, kv * c["heads"])))
        for lo in range(0, n if kv else 0, step):
            hi = min(n, lo + step)
            z, see, first = _exact_rows(s, b, lo, hi)
            l = s["lse"][first + lo:first + hi].double().view(hi - lo, *z.shape[:2]).permute(1, 2, 0)[..., None]
            total.view(-1)[slot] += torch.where(see, torch.exp(z - l), torch.zeros_like(z)).sum((0, 1, 2))
    return total


def _exact_store(s):
    c = s["case"]
    T, out = c["block"], []
    powers = torch.tensor([math.ldexp(1.0, e) for e in range(E_MIN, E_MAX + 1)], dtype=torch.float64, device=DEV)
    for pool, scale, rows in ((s["k"], s["k_scale"], s["k_rows"]), (s["v"], s["v_scale"], s["v_rows"])):
        if pool is None:
            continue
        held, sc = pool.double(), scale.double()
        first = 0
        for b in range(c["batch"]):
            n, kv = int(s["new_lens"][b]), int(s["kv_lens"][b])
            start, table = kv - n, s["table"][int(s["rid"][b])].tolist()
            for j in range(start // T, -(-kv // T) if n else 0):
                lo, hi = max(start, j * T), min(kv, j * T + T)
                x = rows[first + lo - start:first + hi - start].double()
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


def _exact_evict(s):
    c = s["case"]
    T, budget = c["block"], c["budget"]
    kept = torch.full((c["batch"], budget), -1, dtype=torch.int32)
    counts = torch.minimum(s["kv_lens"], torch.full_like(s["kv_lens"], budget))
    weights = s["weights"].double()
    pools = [(s["k"].double(), s["k_scale"].double())] + ([] if s["v"] is None else [(s["v"].double(), s["v_scale"].double())])
    for b in range(c["batch"]):
        L, r = int(s["kv_lens"][b]), int(s["rid"][b])
        src = s["table"][r].long()
        at = np.arange(L)
        w = weights.view(-1)[src[torch.as_tensor(at // T, device=DEV)] * T + torch.as_tensor(at % T, device=DEV)].cpu().numpy() if L else np.zeros(0)
        if L > budget:
            free = at[c["sinks"]:L - c["recent"]]
            best = free[np.lexsort((free, -w[free]))[:budget - c["sinks"] - c["recent"]]]
            at = np.sort(np.concatenate([at[:c["sinks"]], best, at[L - c["recent"]:]]))
        kept[b, :len(at)] = torch.as_tensor(at, dtype=torch.int32)
        p = torch.as_tensor(at, device=DEV)
        for j in range(-(-len(at) // T)):
            q = p[j * T:(j + 1) * T]
            d, blk = int(s["dst"][r, j]), src[q // T]
            for held, sc in pools:
                new = sc[blk].amax(0)
                x = held[blk, :, q % T] * (sc[blk] / new)[..., None]
                held[d, :, :len(q)] = x.transpose(0, 1)
                sc[d] = new
            weights[d, :len(q)] = weights[blk, q % T]
    out = [None, None, weights]  # positions and counts are whole numbers
    for held, sc in pools:
        out += [held, sc]
    return out

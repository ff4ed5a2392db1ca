"""The 8-bit paged cache's operators in plain numpy, 64 bits, request by request: the oracle of their tests.

Pools are uint8 arrays of e4m3 codes; every function works on the arrays it is given, or on copies, as it says."""
import numpy as np

E_MIN, E_MAX = -48, 48


def _codes():
    """The value of each e4m3 code: 4 exponent bits of bias 7, 3 mantissa bits, no infinity, 0x7F / 0xFF NaN."""
    out = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = m / 8.0 * 2.0 ** -6 if e == 0 else (1 + m / 8.0) * 2.0 ** (e - 7)
        out[c] = np.nan if (c & 0x7F) == 0x7F else (-x if c & 0x80 else x)
    return out


E4M3 = _codes()
_POS = E4M3[:0x7F]  # ascending, code = index


def round8(x):
    """Codes of the nearest e4m3 values (ties to the even code), past 448 the largest, NaN to 0x7F."""
    x = np.asarray(x, np.float64)
    a = np.minimum(np.where(np.isnan(x), 0.0, np.abs(x)), 448.0)
    hi = np.searchsorted(_POS, a).clip(0, 0x7E)  # first code not under a
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - _POS[lo], _POS[hi] - a
    pick = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    code = (pick | np.where(np.signbit(x), 0x80, 0)).astype(np.uint8)
    return np.where(np.isnan(x), np.uint8(0x7F), code)


def need_scale(amax):
    """The smallest power of two in range with amax <= 448 * it."""
    for e in range(E_MIN, E_MAX):
        if amax <= 448.0 * 2.0 ** e:
            return 2.0 ** e
    return 2.0 ** E_MAX


def same_codes(a, b):
    """Equal codes, every NaN alike."""
    return np.array_equal(np.where((a & 0x7F) == 0x7F, 0x7F, a), np.where((b & 0x7F) == 0x7F, 0x7F, b))


def store_plan(rid, kv_lens, new_lens, table, T):
    recs, row = [], 0
    for r, kv, n in zip(rid, kv_lens, new_lens):
        p = kv - n
        while p < kv:
            cnt = min(kv - p, T - p % T)
            recs.append((int(table[r, p // T]), row, int(p % T), int(cnt)))
            p += cnt
            row += cnt
    return recs


def store(pool, scale, rows, recs):
    """In place: pool [blocks, H, T, D] codes, scale [blocks, H], rows [N, H, D]."""
    for block, row, off, cnt in recs:
        for h in range(pool.shape[1]):
            x = rows[row:row + cnt, h].astype(np.float64)
            fin = np.abs(x[np.isfinite(x)])
            s = need_scale(fin.max() if fin.size else 0.0)
            if off:
                s = max(s, float(scale[block, h]))
                if s != scale[block, h]:
                    pool[block, h, :off] = round8(E4M3[pool[block, h, :off]] * (float(scale[block, h]) / s))
            pool[block, h, off:off + cnt] = round8(x / s)
            scale[block, h] = s


def visible(kv_len, seq_len, q_len, i, ratio):
    return max(0, kv_len - (seq_len // ratio - (seq_len - q_len + i + 1) // ratio))


def entries(pool, scale, table_row, n):
    """Values [H, n, D] of a request's first n entries."""
    T = pool.shape[2]
    blk = np.asarray(table_row[:-(-n // T)], np.int64)
    x = E4M3[pool[blk]] * scale[blk].astype(np.float64)[:, :, None, None]
    return x.transpose(1, 0, 2, 3).reshape(pool.shape[1], -1, pool.shape[3])[:, :n]


def _scores(q, k, scale):
    """[H, group, S] of one query [heads, D]."""
    H = k.shape[0]
    return np.einsum("hgd,hsd->hgs", q.reshape(H, -1, q.shape[-1]), k) * scale


def attn(k, ks, v, vs, q, rid, seq_lens, q_lens, kv_lens, table, ratio, scale):
    """(out, lse, mag, big, flat), the last three the scales of the output's error bound: sum p |v|, and the largest
    scale * sum |q| |k| and scale * max |q| * sum |k| of a score."""
    out, mag, flat = np.zeros(q.shape), np.zeros(q.shape), np.zeros(q.shape[:2])
    lse, big = np.full(q.shape[:2], -np.inf), np.zeros(q.shape[:2])
    at = 0
    for b in range(len(rid)):
        n = int(kv_lens[b])
        kk = entries(k, ks, table[rid[b]], n)
        vv = kk if v is None else entries(v, vs, table[rid[b]], n)
        for i in range(int(q_lens[b])):
            see = min(n, visible(n, int(seq_lens[b]), int(q_lens[b]), i, ratio))
            if see:
                x = q[at].astype(np.float64)
                z = _scores(x, kk[:, :see], scale)
                top = z.max(-1, keepdims=True)
                p = np.exp(z - top)
                tot = p.sum(-1, keepdims=True)
                lse[at] = (np.log(tot) + top).reshape(-1)
                out[at] = np.einsum("hgs,hsd->hgd", p / tot, vv[:, :see]).reshape(q.shape[1:])
                mag[at] = np.einsum("hgs,hsd->hgd", p / tot, np.abs(vv[:, :see])).reshape(q.shape[1:])
                big[at] = _scores(np.abs(x), np.abs(kk[:, :see]), scale).max(-1).reshape(-1)
                top_q = np.abs(x).max(-1, keepdims=True) * np.ones(x.shape[-1])
                flat[at] = _scores(top_q, np.abs(kk[:, :see]), scale).max(-1).reshape(-1)
            at += 1
    return out, lse, mag, big, flat


def weigh(k, ks, weights, q, lse, rid, seq_lens, q_lens, kv_lens, table, ratio, scale, decay):
    """New weights [blocks, T] (64 bits)."""
    w = weights.astype(np.float64).copy()
    T = k.shape[2]
    at = 0
    for b in range(len(rid)):
        n = int(kv_lens[b])
        got = np.zeros(n)
        kk = entries(k, ks, table[rid[b]], n)
        for i in range(int(q_lens[b])):
            see = min(n, visible(n, int(seq_lens[b]), int(q_lens[b]), i, ratio))
            if see:
                z = _scores(q[at].astype(np.float64), kk[:, :see], scale)
                got[:see] += np.exp(z - lse[at].astype(np.float64).reshape(z.shape[0], -1, 1)).sum((0, 1))
            at += 1
        if q_lens[b]:
            for p in range(n):
                blk = table[rid[b], p // T]
                w[blk, p % T] = got[p] if decay == 0 else decay * w[blk, p % T] + got[p]
    return w


def evict_choice(w, budget, sinks, recent):
    """Kept positions (ascending) of a request with weights w."""
    n = len(w)
    if n <= budget:
        return list(range(n))
    free = sorted(range(sinks, n - recent), key=lambda p: (bool(np.isnan(w[p])), 0.0 if np.isnan(w[p]) else -float(w[p]), p))
    return sorted(list(range(sinks)) + free[:budget - sinks - recent] + list(range(n - recent, n)))


def evict(pools, weights, rid, kv_lens, table, dst, budget, sinks, recent):
    """In place on pools [(codes, scales)] and weights; returns the kept positions of each request."""
    T = pools[0][0].shape[2]
    kept = []
    for b in range(len(rid)):
        row = table[rid[b]]
        w = np.array([weights[row[p // T], p % T] for p in range(int(kv_lens[b]))])
        keep = evict_choice(w, budget, sinks, recent)
        kept.append(keep)
        for j in range(0, len(keep), T):
            d = dst[rid[b], j // T]
            src = [(int(row[p // T]), p % T) for p in keep[j:j + T]]
            for pool, scale in pools:
                for h in range(pool.shape[1]):
                    s = max(float(scale[x, h]) for x, _ in src)
                    for i, (x, slot) in enumerate(src):
                        f = float(scale[x, h]) / s
                        pool[d, h, i] = pool[x, h, slot] if f == 1 else round8(E4M3[pool[x, h, slot]] * f)
                    scale[d, h] = s
            for i, (x, slot) in enumerate(src):
                weights[d, i] = weights[x, slot]
    return kept

"""The rotated append and the sparse attention of the 8-bit paged cache in plain numpy, 64 bits, one query at a time:
the oracle of their tests."""
import numpy as np

from tests import q8_ref as ref


def rope(rows, weight, eps, freqs, pos, begin, halves, dtype=np.float64):
    """Rows [N, H, D], normalised (weight not None) and rotated; in float32 every operation rounds by itself."""
    x = rows.astype(dtype)
    if weight is not None:
        x = x * weight.astype(dtype) * (1 / np.sqrt((x * x).mean(-1, keepdims=True) + dtype(eps)))
    if freqs is None:
        return x
    half = freqs.shape[1]
    i = np.arange(half)
    a, b = (begin + i, begin + half + i) if halves else (begin + 2 * i, begin + 2 * i + 1)
    c, s = (freqs[pos][:, None, :, k].astype(dtype) for k in range(2))
    y = x.copy()
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., a] * s + x[..., b] * c
    return y


def bounds(out, k, rid, kv_lens, new_lens, table):
    """In place: out [blocks, H, 2, D] codes, -0 as 0."""
    T = k.shape[2]
    for r, kv, n in zip(rid, kv_lens, new_lens):
        for j in range((kv - n) // T, -(-kv // T) if n else 0):
            x = ref.E4M3[k[table[r, j], :, :min(T, kv - j * T)]]
            out[table[r, j]] = ref.round8(np.stack((x.max(1), x.min(1)), 1) + 0.0)
    return out


def requests_of(q_lens):
    """(request, its query) of each ragged query."""
    return [(b, i) for b, n in enumerate(q_lens) for i in range(int(n))]


def scores(bnd, ks, q, rid, seq, q_lens, lens, table, T, ratio, scale, width):
    """(scores [N, H, width], the scale of their error: scale * ks * sum |q| max(|hi|, |lo|), and with max |q| for |q|)."""
    H = ks.shape[1]
    out, mag, flat = (np.zeros((len(q), H, width)) for _ in range(3))
    out[:] = -np.inf
    for at, (b, i) in enumerate(requests_of(q_lens)):
        see = ref.visible(int(lens[b]), int(seq[b]), int(q_lens[b]), i, ratio)
        x = q[at].astype(np.float64).reshape(H, -1, q.shape[-1])
        for j in range(-(-see // T)):
            blk = table[rid[b], j]
            if not 0 <= blk < len(bnd):
                continue
            v = ref.E4M3[bnd[blk]] * ks[blk].astype(np.float64)[:, None, None]
            with np.errstate(invalid="ignore"):
                z = np.maximum(x * v[:, None, 0], x * v[:, None, 1]).sum(-1) * scale
            out[at, :, j] = z.max(-1)
            w = np.abs(v).max(1)
            mag[at, :, j] = (np.abs(x) * w[:, None]).sum(-1).max(-1) * scale
            flat[at, :, j] = (np.abs(x).max(-1) * w.sum(-1)[:, None]).max(-1) * scale
    return out, mag, flat


def choose(row, n, budget, sinks, recent):
    """The chosen ones of the first n scores, ascending."""
    if n <= budget:
        return list(range(n))
    free = sorted(range(sinks, n - recent), key=lambda j: (bool(np.isnan(row[j])), 0.0 if np.isnan(row[j]) else -float(row[j]), j))
    return sorted(list(range(sinks)) + free[:budget - sinks - recent] + list(range(n - recent, n)))


def select(s, seq, q_lens, lens, T, ratio, budget, sinks, recent):
    out = np.full((s.shape[0], s.shape[1], budget), -1, np.int32)
    for at, (b, i) in enumerate(requests_of(q_lens)):
        n = -(-ref.visible(int(lens[b]), int(seq[b]), int(q_lens[b]), i, ratio) // T)
        for h in range(s.shape[1]):
            c = choose(s[at, h], n, budget, sinks, recent)
            out[at, h, :len(c)] = c
    return out


def attn(k, ks, v, vs, q, blocks, rid, seq, q_lens, lens, table, ratio, scale, skip=()):
    """As q8_ref.attn, over the listed blocks but those whose number in the pool is in skip."""
    out, mag, flat = np.zeros(q.shape), np.zeros(q.shape), np.zeros(q.shape[:2])
    lse, big = np.full(q.shape[:2], -np.inf), np.zeros(q.shape[:2])
    H, T = ks.shape[1], k.shape[2]
    G = q.shape[1] // H
    for at, (b, i) in enumerate(requests_of(q_lens)):
        see = ref.visible(int(lens[b]), int(seq[b]), int(q_lens[b]), i, ratio)
        for h in range(H):
            kk, vv = [], []
            for j in blocks[at, h]:
                if j < 0 or j * T >= see or table[rid[b], j] in skip:
                    continue
                blk, n = table[rid[b], j], min(T, see - j * T)
                kk.append(ref.E4M3[k[blk, h, :n]] * float(ks[blk, h]))
                vv.append(kk[-1] if v is None else ref.E4M3[v[blk, h, :n]] * float(vs[blk, h]))
            if not kk:
                continue
            kk, vv = np.concatenate(kk), np.concatenate(vv)
            rows = slice(h * G, h * G + G)
            x = q[at, rows].astype(np.float64)
            z = x @ kk.T * scale
            top = z.max(-1, keepdims=True)
            p = np.exp(z - top)
            tot = p.sum(-1, keepdims=True)
            lse[at, rows] = (np.log(tot) + top)[:, 0]
            out[at, rows] = p / tot @ vv
            mag[at, rows] = p / tot @ np.abs(vv)
            big[at, rows] = (np.abs(x) @ np.abs(kk).T).max(-1) * scale
            flat[at, rows] = np.abs(x).max(-1) * np.abs(kk).sum(-1).max() * scale
    return out, lse, mag, big, flat

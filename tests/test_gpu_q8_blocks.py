"""The rotated append and the sparse attention of the 8-bit cache on the GPU against their 64-bit oracle: codes, bounds
and choices exactly, scores and attention within bounds derived from the roundings that the kernels make."""
import math

import numpy as np
import pytest
import torch

from compressed_kv_attention_compressplan_gb300 import ckv
from tests import q8_blocks_ref as bref
from tests import q8_ref as ref
from tests.test_gpu_q8 import World, attn_bounds, codes, i32, i64, status

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ckv.load_library()


def f32(a):
    return torch.as_tensor(np.asarray(a, np.float32), device=DEV)


def table_of_angles(n, dim, base=10000.0):
    ang = np.arange(n)[:, None] * base ** (-np.arange(dim // 2) / max(1, dim // 2))
    return np.stack([np.cos(ang), np.sin(ang)], -1).astype(np.float32)


def up(codes_):
    return torch.as_tensor(codes_, device=DEV).view(torch.float8_e4m3fn)


# ------------------------------------------------------------------------------------------------------ rope store
ROPE = [  # lens before, new, H, D, T, latent, dtype, norm, halves, rope_dim, begin, wider rows
    ([0], [1], 1, 512, 64, True, BF, False, False, 64, 448, 0),
    ([0, 5, 63, 64, 130], [0, 1, 1, 1, 0], 1, 512, 64, True, BF, False, False, 64, 448, 0),
    ([3, 16, 0, 31], [40, 1, 16, 33], 2, 128, 16, False, BF, False, True, 128, 0, 5),
    ([0, 127, 128, 1], [300, 2, 128, 127], 3, 64, 128, False, F32, False, True, 32, 16, 1),
    ([7] * 20, [1] * 20, 2, 256, 32, False, F32, False, False, 96, 80, 0),
    ([0, 0, 9], [0, 0, 5], 8, 128, 32, False, BF, False, True, 64, 64, 2),
    ([1, 30], [130, 3], 1, 512, 128, False, BF, False, True, 512, 0, 0),
    ([0, 2], [70, 61], 2, 64, 64, True, F32, False, False, 64, 0, 3),
    ([5], [40], 4, 256, 16, False, BF, False, True, 256, 0, 0),
    ([0, 3], [128, 200], 2, 512, 128, False, F32, False, False, 64, 448, 0),   # blocks whose rows do not fit the registers
    ([60, 3], [70, 1], 2, 512, 64, False, F32, False, True, 128, 384, 1),
    ([9], [250], 3, 256, 128, False, F32, False, False, 256, 0, 0),
    ([9], [250], 3, 256, 64, True, F32, False, False, 32, 0, 0),
    ([3] * 1024, [2] * 1024, 1, 64, 16, True, BF, False, False, 32, 32, 0),
    ([0, 63, 10], [200, 3, 60], 3, 128, 64, False, BF, False, True, 128, 0, 3),   # four vectors a thread
    ([5, 16], [43, 1], 2, 512, 16, True, BF, False, False, 64, 448, 0),
    ([5, 16], [43, 1], 2, 128, 16, False, F32, False, True, 64, 32, 1),
    ([5, 16], [43, 1], 2, 64, 16, False, F32, False, False, 64, 0, 0),
]


def rope_inputs(r, n, H, D, dt, wider, sides):
    """Rows as they lie in a projection: `wider` heads, then keys, then values."""
    fused = torch.as_tensor(r.standard_normal((n, wider + sides * H, D)) * np.exp(r.standard_normal((n, 1, 1)))).to(dt).to(DEV)
    k = fused[:, wider:wider + H]
    return k, fused[:, wider + H:] if sides == 2 else None


@pytest.mark.parametrize("case", range(len(ROPE)))
def test_rope_store(case):
    """Without a norm every rounding is known: codes and scales bit for bit."""
    before, new, H, D, T, latent, dt, _, halves, dim, begin, wider = ROPE[case]
    w = World(300 + case, before, H, D, T, latent, more=max(new))
    n = sum(new)
    k_rows, v_rows = rope_inputs(w.r, n, H, D, dt, wider, 1 if latent else 2)
    freqs = table_of_angles(700, dim)
    pos = w.r.randint(0, 700, n)
    cache, st, kv = w.cache(), status(), np.asarray(before) + new
    plan, counts = ckv.plan_q8_store(cache, i64(w.rid), i64(kv), i64(new), n, i32(w.table), status=st)
    ckv.q8_rope_store(cache, k_rows, v_rows, plan, i64(pos), f32(freqs), counts, rope_begin=begin, halves=halves, status=st)
    recs = ref.store_plan(w.rid, kv, new, w.table, T)
    ref.store(w.k, w.ks, bref.rope(k_rows.float().cpu().numpy(), None, 0, freqs, pos, begin, halves, np.float32), recs)
    assert ref.same_codes(codes(cache.k), w.k)
    assert np.array_equal(cache.k_scale.cpu().numpy(), w.ks, equal_nan=True)
    if not latent:
        ref.store(w.v, w.vs, v_rows.float().cpu().numpy(), recs)
        assert ref.same_codes(codes(cache.v), w.v)
        assert np.array_equal(cache.v_scale.cpu().numpy(), w.vs, equal_nan=True)
    assert int(st[0]) == 0


@pytest.mark.parametrize("case", range(len(ROPE)))
@pytest.mark.parametrize("turned", [True, False])
def test_rope_store_with_a_norm(case, turned):
    """The norm's sum of D squares is off by (D + 4) 2^-24 of itself, its root by half of that, four products and the
    rotation's sum by 2^-24 each of the pair's length; then half an e4m3 step, 2^-4 of the value or 2^-10 of the scale."""
    before, new, H, D, T, latent, dt, _, halves, dim, begin, wider = ROPE[case]
    w = World(330 + case, [0] * len(before), H, D, T, latent, more=max(new))
    n = sum(new)
    k_rows, v_rows = rope_inputs(w.r, n, H, D, dt, wider, 1 if latent else 2)
    freqs, weight = (table_of_angles(500, dim) if turned else None), (1 + 0.2 * w.r.standard_normal(D)).astype(np.float32)
    pos = w.r.randint(0, 500, n)
    cache, st = w.cache(), status()
    plan, counts = ckv.plan_q8_store(cache, i64(w.rid), i64(new), i64(new), n, i32(w.table), status=st)
    ckv.q8_rope_store(cache, k_rows, v_rows, plan, i64(pos) if turned else None, None if freqs is None else f32(freqs), counts,
                      rope_begin=begin if turned else 0, halves=halves, norm_weight=f32(weight), eps=1e-5, status=st)
    y = bref.rope(k_rows.float().cpu().numpy(), weight, 1e-5, freqs, pos, begin, halves)
    off = ((D + 4) / 2 + 8) * 2.0 ** -24
    got, gs = codes(cache.k), cache.k_scale.cpu().numpy()
    for block, row, slot, cnt in ref.store_plan(w.rid, new, new, w.table, T):
        for h in range(H):
            x = y[row:row + cnt, h]
            s = float(gs[block, h])
            assert s in (ref.need_scale(np.abs(x).max() * (1 - off)), ref.need_scale(np.abs(x).max() * (1 + off)))
            err = np.abs(ref.E4M3[got[block, h, slot:slot + cnt]] * s - x)
            near = off * 2 * np.abs(x).max(-1, keepdims=True)
            assert (err <= np.maximum(np.abs(x) * 2.0 ** -4, s * 2.0 ** -10) + near).all()
    if not latent:
        ref.store(w.v, w.vs, v_rows.float().cpu().numpy(), ref.store_plan(w.rid, new, new, w.table, T))
        assert ref.same_codes(codes(cache.v), w.v)
    assert int(st[0]) == 0


@pytest.mark.parametrize("latent", [False, True])
def test_rope_store_without_norm_and_rotation_is_the_store(latent):
    w = World(360, [5, 0, 31], 2, 128, 32, latent, more=100)
    new = [90, 3, 1]
    k, v = rope_inputs(w.r, 94, 2, 128, BF, 0, 1 if latent else 2)
    k, v = k.contiguous(), None if latent else v.contiguous()
    out = []
    for rotated in (False, True):
        cache, weights = w.cache(), torch.ones(w.blocks, 32, device=DEV)
        plan, counts = ckv.plan_q8_store(cache, i64(w.rid), i64(w.lens + new), i64(new), 94, i32(w.table))
        if rotated:
            ckv.q8_rope_store(cache, k, v, plan, None, None, counts, weights=weights)
        else:
            ckv.q8_store(cache, k, v, plan, counts, weights=weights)
        out.append([x.view(torch.uint8) for x in cache if x is not None] + [weights])
    for x, y in zip(*out):
        assert torch.equal(x, y)


def test_rope_store_leaves_rows_of_positions_outside_the_table():
    w = World(361, [3, 20], 1, 64, 16, False, more=20)
    new, dim = [20, 2], 64
    k, v = rope_inputs(w.r, 22, 1, 64, BF, 1, 2)
    freqs, pos = table_of_angles(100, dim), w.r.randint(0, 100, 22)
    bad = [0, 13, 14, 21]
    pos[bad] = [-1, 100, 1 << 40, -(1 << 40)]
    cache, st, kv = w.cache(), status(), w.lens + new
    weights = torch.full((w.blocks, 16), 5.0, device=DEV)
    plan, counts = ckv.plan_q8_store(cache, i64(w.rid), i64(kv), i64(new), 22, i32(w.table), status=st)
    ckv.q8_rope_store(cache, k, v, plan, i64(pos), f32(freqs), counts, halves=True, weights=weights, status=st)
    assert int(st[0]) == ckv.STATUS_BAD_INDEX
    recs = ref.store_plan(w.rid, kv, new, w.table, 16)
    safe = np.where(np.isin(np.arange(22), bad), 0, pos)
    for pool, scale, rows, got in ((w.k, w.ks, bref.rope(k.float().cpu().numpy(), None, 0, freqs, safe, 0, True, np.float32), cache.k),
                                   (w.v, w.vs, v.float().cpu().numpy(), cache.v)):
        rows = rows.copy()
        rows[bad] = 0  # zeros do not count for a scale
        old = pool.copy()
        ref.store(pool, scale, rows, recs)
        for block, row, slot, cnt in recs:
            for i in range(cnt):
                if row + i in bad:
                    pool[block, :, slot + i] = old[block, :, slot + i]
        assert ref.same_codes(codes(got), pool)
    wn = weights.cpu().numpy()
    for block, row, slot, cnt in recs:
        for i in range(cnt):
            assert wn[block, slot + i] == (5.0 if row + i in bad else 0.0)
    assert (wn == 0).sum() == 18


def test_rope_store_of_infinities_and_nan():
    """They do not count for the scale; NaN is stored as NaN, and so is what a rotation makes of infinities."""
    w = World(362, [0], 1, 64, 16, True, more=8)
    x = w.r.standard_normal((8, 1, 64)).astype(np.float32)
    x[1, 0, 3], x[2, 0, 40], x[3, 0, 5] = np.inf, np.nan, -np.inf
    x[4] = 0
    freqs = table_of_angles(8, 32)
    cache = w.cache()
    plan, counts = ckv.plan_q8_store(cache, i64(w.rid), i64([8]), i64([8]), 8, i32(w.table))
    ckv.q8_rope_store(cache, torch.as_tensor(x, device=DEV), None, plan, i64(np.arange(8)), f32(freqs), counts)
    with np.errstate(invalid="ignore"):
        y = bref.rope(x, None, 0, freqs, np.arange(8), 0, False, np.float32)
    ref.store(w.k, w.ks, y, ref.store_plan(w.rid, [8], [8], w.table, 16))
    assert ref.same_codes(codes(cache.k), w.k)
    assert np.array_equal(cache.k_scale.cpu().numpy(), w.ks, equal_nan=True)


def test_rope_store_of_rows_past_32_bits():
    """Rows 2^22 elements apart: the last one's offset does not fit 32 bits."""
    n, wide = 1100, 1 << 22
    w = World(363, [0], 1, 64, 64, True, more=n)
    big = torch.empty(n, wide // 64, 64, dtype=BF, device=DEV)
    x = torch.as_tensor(w.r.standard_normal((n, 1, 64))).to(BF)
    big[:, 2:3] = x.to(DEV)
    freqs, cache = table_of_angles(n, 64), w.cache()
    plan, counts = ckv.plan_q8_store(cache, i64(w.rid), i64([n]), i64([n]), n, i32(w.table))
    ckv.q8_rope_store(cache, big[:, 2:3], None, plan, i64(np.arange(n)), f32(freqs), counts, halves=True)
    ref.store(w.k, w.ks, bref.rope(x.float().numpy(), None, 0, freqs, np.arange(n), 0, True, np.float32),
              ref.store_plan(w.rid, [n], [n], w.table, 64))
    assert ref.same_codes(codes(cache.k), w.k)


# ---------------------------------------------------------------------------------------------------------- bounds
def same_values(a, b):
    """Equal e4m3 values: the two zeros alike, every NaN alike."""
    return np.array_equal(ref.E4M3[a], ref.E4M3[b], equal_nan=True)


BOUNDS = [  # lens, new, H, D, T, latent
    ([1], [1], 1, 512, 64, True),
    ([100, 0, 33, 64, 300], [1, 0, 2, 64, 300], 2, 128, 16, False),
    ([129, 128, 127], [129, 1, 127], 3, 64, 128, False),
    ([70, 9], [40, 9], 2, 256, 32, True),
    ([5] * 300, [1] * 300, 1, 64, 16, True),
    ([2000], [2000], 8, 128, 64, False),
]


@pytest.mark.parametrize("case", range(len(BOUNDS)))
def test_bounds(case):
    """Slots past a request's end hold NaN codes, and do not count; other blocks' bounds stay."""
    lens, new, H, D, T, latent = BOUNDS[case]
    w = World(400 + case, lens, H, D, T, latent)
    cache, st = w.cache(), status()
    b = up(np.full((w.blocks, H, 2, D), 0x33, np.uint8))
    assert ckv.q8_bounds(cache, b, i64(w.rid), i64(lens), i64(new), i32(w.table), status=st) is b
    want = bref.bounds(np.full((w.blocks, H, 2, D), 0x33, np.uint8), w.k, w.rid, lens, new, w.table)
    assert same_values(codes(b), want)
    assert int(st[0]) == 0


def test_bounds_of_nan_entries_and_shared_blocks():
    w = World(410, [40, 40], 2, 128, 16, True)
    w.k[w.table[w.rid[0], 1], 1, 3, 77] = 0xFF
    w.table[w.rid[1]] = w.table[w.rid[0]]  # the second request is a copy of the first
    cache = w.cache()
    b = ckv.new_q8_bounds(cache)
    ckv.q8_bounds(cache, b, i64(w.rid), i64([40, 40]), i64([40, 40]), i32(w.table))
    got = codes(b)
    want = bref.bounds(np.zeros_like(got), w.k, w.rid[:1], [40], [40], w.table)
    assert same_values(got, want)
    assert (got[w.table[w.rid[0], 1], 1, :, 77] & 0x7F == 0x7F).all() and (got & 0x7F == 0x7F).sum() == 2


def test_bounds_flag_bad_data_and_touch_nothing_for_it():
    w = World(411, [40, 20, 30, 10, 16], 1, 64, 16, True)
    lens, new, rid = [40, 20, 30, 10, 16], [40, 21, 30, 10, -1], w.rid.copy()
    rid[3] = 99
    w.table[w.rid[0], 1] = w.blocks
    cache, st = w.cache(), status()
    b = up(np.full((w.blocks, 1, 2, 64), 0x33, np.uint8))
    ckv.q8_bounds(cache, b, i64(rid), i64(lens), i64(new), i32(w.table), status=st)
    assert int(st[0]) == ckv.STATUS_BAD_LENGTH | ckv.STATUS_BAD_INDEX
    want = np.full((w.blocks, 1, 2, 64), 0x33, np.uint8)
    for blk, n in ((w.table[w.rid[0], 0], 16), (w.table[w.rid[0], 2], 8), (w.table[w.rid[2], 0], 16), (w.table[w.rid[2], 1], 14)):
        x = ref.E4M3[w.k[blk, :, :n]]
        want[blk] = ref.round8(np.stack((x.max(1), x.min(1)), 1))
    assert same_values(codes(b), want)
    st.zero_()
    ckv.q8_bounds(cache, b, i64(w.rid[:1]), i64([w.table.shape[1] * 16 + 1]), i64([1]), i32(w.table), status=st)
    assert int(st[0]) == ckv.STATUS_BAD_LENGTH


# ---------------------------------------------------------------------------------------------------------- scores
def seq_of(lens, q_lens, ratio):
    return np.maximum(np.asarray(lens) * ratio + np.arange(len(lens)) * 3 % ratio, q_lens)


def bounds_of(w):
    return bref.bounds(np.full((w.blocks, w.H, 2, w.D), 0x7F, np.uint8), w.k, w.rid, w.lens, w.lens, w.table)


def check_scores(w, q, seq, q_lens, heads, ratio, width=None, scale=0.07, bnd=None):
    """2 D products of at most |q| max(|hi|, |lo|) summed in fp32 with truncated additions (2^-23 each), three more
    roundings, and query values under 2^-28 of their row's largest off by up to 2^-39 of it."""
    bnd = bounds_of(w) if bnd is None else bnd
    width = w.table.shape[1] if width is None else width
    cache, st = w.cache(), status()
    got = ckv.q8_block_scores(cache, up(bnd), q.to(DEV), ratio, i64(w.rid), i64(seq), i64(q_lens), i64(w.lens), i32(w.table),
                              scale, width=width, status=st)
    want, mag, flat = bref.scores(bnd, w.ks, q.float().numpy(), w.rid, seq, q_lens, w.lens, w.table, w.T, ratio, scale, width)
    got = got.cpu().numpy()
    assert int(st[0]) == 0
    assert np.array_equal(np.isneginf(got), np.isneginf(want))
    fin = np.isfinite(want)
    tol = mag * (2 * w.D + 4) * 2.0 ** -23 + flat * 2.0 ** -38
    assert (np.abs(got[fin] - want[fin]) <= tol[fin]).all()
    return got


SCORES = [  # lens, q_lens, heads, H, D, T, ratio
    ([1], [1], 1, 1, 64, 16, 1),
    ([777], [1], 8, 1, 128, 16, 1),
    ([100, 0, 17, 300, 1], [1, 1, 1, 0, 1], 8, 2, 128, 32, 1),
    ([64, 65, 63], [1, 2, 3], 16, 4, 64, 64, 1),
    ([500, 20], [5, 20], 6, 2, 256, 16, 4),
    ([900, 20], [3, 40], 7, 1, 128, 128, 1),
    ([333], [9], 9, 1, 512, 16, 1),
    ([333, 40], [2, 1], 64, 1, 512, 32, 4),
    ([333], [2], 128, 1, 128, 16, 128),
    ([3000], [1], 12, 2, 64, 16, 1),          # more blocks than a unit's
    ([400, 30], [300, 30], 4, 1, 128, 32, 1),  # more rows than a unit's
    ([200], [150], 2, 1, 64, 16, 1),
    ([200], [37], 3, 1, 256, 16, 1),
    ([160], [4], 256, 1, 128, 16, 1),
    ([160], [2], 136, 1, 256, 32, 1),
    ([50] * 300, [1] * 300, 2, 2, 64, 16, 1),
    ([700, 90], [3, 9], 24, 1, 512, 64, 1),
    ([90, 200], [1, 0], 16, 1, 128, 16, 1),    # fewer queries than requests
    ([90, 200, 30, 30, 30, 30], [0, 1, 0, 0, 0, 2], 12, 1, 512, 16, 1),
    ([40] * 12, [0] * 11 + [1], 72, 1, 256, 16, 1),
    ([90, 0, 30, 700, 30, 30], [0, 1, 0, 5, 0, 0], 6, 2, 64, 16, 4),
    ([17] * 1024, [1] * 1024, 8, 1, 128, 16, 1),   # the largest batch: each kernel's tables of requests
    ([17] * 1024, [2] * 1024, 66, 1, 512, 16, 1),
    ([17] * 1024, [1, 3] * 512, 16, 1, 64, 16, 1),
    ([17] * 1024, [1] * 1024, 2, 1, 512, 16, 1),
]


@pytest.mark.parametrize("case", range(len(SCORES)))
def test_scores(case):
    lens, q_lens, heads, H, D, T, ratio = SCORES[case]
    w = World(500 + case, lens, H, D, T, True)
    check_scores(w, w.queries(q_lens, heads), seq_of(lens, q_lens, ratio), q_lens, heads, ratio)


@pytest.mark.parametrize("width", [7, 130, 200])
def test_scores_of_other_widths(width):
    w = World(530, [100, 112], 2, 128, 16, True)
    check_scores(w, w.queries([2, 1], 4), [100, 112], [2, 1], 4, 1, width=width)


def test_scores_of_large_and_tiny_queries():
    w = World(531, [100], 1, 128, 16, True)
    q = w.queries([4], 4)
    q[0] *= 2.0 ** 60
    q[1] *= 2.0 ** -60
    q[2, :, ::2] *= 2.0 ** -30
    q[3] = 0
    check_scores(w, q, [100], [4], 4, 1)


def test_no_entry_scores_above_its_block():
    w = World(532, [500], 2, 128, 32, True)
    q = w.queries([1], 8)
    got = check_scores(w, q, [500], [1], 8, 1)
    z = np.einsum("hgd,hsd->hgs", q[0].double().numpy().reshape(2, 4, 128), ref.entries(w.k, w.ks, w.table[w.rid[0]], 500)) * 0.07
    for j in range(16):
        part = z[:, :, j * 32:j * 32 + 32].max((1, 2))
        assert (got[0, :, j] >= part - np.abs(part) * 2.0 ** -12 - 1e-4).all()


@pytest.mark.parametrize("heads,D", [(4, 128), (16, 128), (12, 512), (2, 256)])
def test_scores_with_nan_and_infinity(heads, D):
    w = World(533, [100], 1, D, 16, True)
    bnd = bounds_of(w)
    bnd[w.table[w.rid[0], 2], 0, :, 9] = 0x7F
    q = w.queries([3], heads)
    q[1, 1, 5] = float("nan")
    q[2, 0, 7] = float("inf")
    got = ckv.q8_block_scores(w.cache(), up(bnd), q.to(DEV), 1, i64(w.rid), i64([100]), i64([3]), i64([100]), i32(w.table),
                              0.07).cpu().numpy()
    want, _, _ = bref.scores(bnd, w.ks, q.float().numpy(), w.rid, [100], [3], [100], w.table, 16, 1, 0.07, w.table.shape[1])
    assert np.isnan(got[0, 0, 2]) and np.isnan(got[:2]).sum() == 1 + 7
    assert np.array_equal(np.isnan(got), np.isnan(want))
    inf = np.isinf(want)
    assert np.array_equal(got[inf], want[inf])


def test_scores_flag_bad_data():
    w = World(534, [100, 40, 60, 30], 2, 128, 16, True)
    cache, bnd, q = w.cache(), bounds_of(w), w.queries([1, 2, 1, 3], 4)

    def run(rid, seq, q_lens, lens, table=w.table, width=None, n=None):
        st = status()
        out = torch.full((7 if n is None else n, 2, width or w.table.shape[1]), 3.0, device=DEV)
        ckv.q8_block_scores(cache, up(bnd), q[:out.shape[0]].to(DEV), 1, i64(rid), i64(seq), i64(q_lens), i64(lens), i32(table), 0.07,
                            scores=out, status=st)
        return out.cpu().numpy(), int(st[0])

    lens, ql = [100, 40, 60, 30], [1, 2, 1, 3]
    good, st = run(w.rid, lens, ql, lens)
    assert st == 0
    # a request's own lengths
    for bad in (dict(rid=[w.rid[0], 99, *w.rid[2:]]), dict(lens=[100, -1, 60, 30]), dict(seq=[100, 1, 60, 30]),
                dict(lens=[100, w.table.shape[1] * 16 + 1, 60, 30]), dict(seq=[100, 1 << 31, 60, 30])):
        a = dict(rid=w.rid, seq=lens, q_lens=ql, lens=lens)
        a.update(bad)
        got, st = run(**a)
        assert st == ckv.STATUS_BAD_LENGTH
        assert (got[1:3] == 3.0).all() and np.array_equal(got[[0, 3, 4, 5, 6]], good[[0, 3, 4, 5, 6]])
    got, st = run(w.rid, lens, ql, lens, width=4)  # the first has seven blocks
    assert st == ckv.STATUS_BAD_LENGTH and (got[0] == 3.0).all() and np.array_equal(got[1:], good[1:, :, :4])
    # queries that do not all exist, and rows behind the last
    got, st = run(w.rid, lens, ql, lens, n=6)
    assert st == ckv.STATUS_BAD_TOTAL and np.array_equal(got[:4], good[:4]) and (got[4:] == 3.0).all()
    got, st = run(w.rid[:3], lens[:3], ql[:3], lens[:3])
    assert st == ckv.STATUS_BAD_TOTAL and np.array_equal(got[:4], good[:4]) and (got[4:] == 3.0).all()
    # a block outside the pool
    table = w.table.copy()
    table[w.rid[0], 3] = -5
    got, st = run(w.rid, lens, ql, lens, table)
    assert st == ckv.STATUS_BAD_INDEX and np.isneginf(got[0, :, 3]).all()
    got[0, :, 3] = good[0, :, 3]
    assert np.array_equal(got, good)


# ---------------------------------------------------------------------------------------------------------- select
SELECT = [  # lens, q_lens, H, T, ratio, budget, sinks, recent
    ([1], [1], 1, 16, 1, 1, 0, 0),
    ([777], [1], 2, 16, 1, 10, 1, 2),
    ([100, 0, 17, 300, 1], [1, 1, 1, 0, 1], 2, 32, 1, 3, 0, 1),
    ([500, 20], [40, 20], 3, 16, 4, 8, 2, 2),
    ([800, 5000], [3, 2], 2, 16, 1, 64, 0, 0),
    ([5000], [2], 1, 16, 1, 40, 20, 20),      # nothing is left to choose
    ([20000], [3], 2, 16, 1, 33, 1, 4),
    ([70000, 3], [1, 1], 1, 16, 1, 512, 0, 0),
    ([200000], [1], 1, 16, 1, 2000, 1, 1),
    ([530000], [2], 1, 16, 1, 77, 3, 5),
    ([300], [5], 1, 128, 128, 2, 1, 0),
    ([64] * 300, [1] * 300, 2, 16, 1, 2, 0, 0),
    ([1024, 1040, 1008], [1, 1, 1], 2, 16, 1, 1, 0, 0),
    ([4096, 4112], [2, 1], 2, 16, 1, 128, 1, 0),
    ([16384, 16400], [1, 1], 1, 16, 1, 1000, 0, 8),
    ([64] * 1024, [3, 0] * 512, 2, 16, 1, 2, 0, 1),
]


def select(s, lens, q_lens, T, ratio, budget, sinks, recent, **kw):
    st = status()
    got = ckv.q8_block_select(s, T, ratio, i64(seq_of(lens, q_lens, ratio)), i64(q_lens), i64(lens), budget, sinks, recent,
                              status=st, **kw)
    assert int(st[0]) == 0
    return got.cpu().numpy()


@pytest.mark.parametrize("kind", ["plain", "ties", "odd", "equal"])
@pytest.mark.parametrize("case", range(len(SELECT)))
def test_select(case, kind):
    lens, q_lens, H, T, ratio, budget, sinks, recent = SELECT[case]
    r = np.random.RandomState(600 + case)
    s = (r.standard_normal((sum(q_lens), H, max(lens) // T + 2)) * 4).astype(np.float32)
    if kind == "ties":
        s = np.round(s)
        s[s == 0] *= r.choice([-1, 1], (s == 0).sum())  # both zeros
    elif kind == "odd":
        s[r.rand(*s.shape) < 0.3] = np.nan
        s[r.rand(*s.shape) < 0.2] = -np.inf
        s[r.rand(*s.shape) < 0.1] = np.inf
        s[r.rand(*s.shape) < 0.1] *= 1e-42
    elif kind == "equal":
        s[:] = r.choice([-3.4e38, 0, 5]) if case % 2 else -np.inf
    got = select(torch.as_tensor(s, device=DEV), lens, q_lens, T, ratio, budget, sinks, recent)
    assert np.array_equal(got, bref.select(s, seq_of(lens, q_lens, ratio), q_lens, lens, T, ratio, budget, sinks, recent))


def test_select_flags_bad_data_and_leaves_other_rows():
    lens, ql, T = np.array([100, 40, 60]), [1, 2, 1], 16
    s = torch.randn(4, 2, 7, device=DEV)

    def run(seq, q_lens, lens, s=s):
        st, out = status(), torch.full((s.shape[0], 2, 3), 77, dtype=torch.int32, device=DEV)
        ckv.q8_block_select(s, T, 1, i64(seq), i64(q_lens), i64(lens), 3, blocks=out, status=st)
        return out.cpu().numpy(), int(st[0])

    good, st = run(lens, ql, lens)
    assert st == 0
    for seq, ln in ((lens, [100, -1, 60]), ([100, 1, 60], lens), (lens, [100, 113, 60])):
        got, st = run(seq, ql, ln)
        assert st == ckv.STATUS_BAD_LENGTH and (got[1:3] == 77).all() and np.array_equal(got[[0, 3]], good[[0, 3]])
    got, st = run(lens[:2], ql[:2], lens[:2])
    assert st == ckv.STATUS_BAD_TOTAL and np.array_equal(got[:3], good[:3]) and (got[3] == 77).all()
    got, st = run(lens, ql, lens, s[:3])
    assert st == ckv.STATUS_BAD_TOTAL and np.array_equal(got[:3], good[:3])


# ------------------------------------------------------------------------------------------------------- attention
def lists_of(w, seq, q_lens, ratio, budget, r=None, ragged=True):
    """Random ascending lists, of other lengths for each kv head where ragged, -1s behind or between."""
    r = r or w.r
    out = np.full((int(np.sum(q_lens)), w.H, budget), -1, np.int32)
    for at, (b, i) in enumerate(bref.requests_of(q_lens)):
        n = -(-ref.visible(int(w.lens[b]), int(seq[b]), int(q_lens[b]), i, ratio) // w.T)
        for h in range(w.H):
            m = min(n, budget)
            if ragged and m:
                m = r.randint(0 if h % 2 else m, m + 1)
            pick = np.sort(r.permutation(n)[:m])
            place = np.sort(r.permutation(budget)[:m]) if ragged and h % 3 == 2 else np.arange(m)
            out[at, h, place] = pick
    return out


def eight_bit(D, group):
    return group > (32 if D == 256 else 16) and D >= 256


def run_attn(w, q, lists, seq, q_lens, ratio, out_dtype=BF, scale=None, **kw):
    st = status()
    cache = w.cache()
    out, lse = ckv.q8_attn_blocks(cache, q.to(DEV), i32(lists), ratio, i64(w.rid), i64(seq), i64(q_lens), i64(w.lens),
                                  i32(w.table), 1 / math.sqrt(w.D) if scale is None else scale, out_dtype=out_dtype, status=st, **kw)
    return out, lse, int(st[0])


def check_attn(w, q, lists, seq, q_lens, ratio, out_dtype=BF, skip=(), flags=0):
    out, lse, st = run_attn(w, q, lists, seq, q_lens, ratio, out_dtype)
    assert st == flags
    want, wl, mag, big, flat = bref.attn(w.k, w.ks, w.v, w.vs, q.float().numpy(), lists, w.rid, seq, q_lens, w.lens, w.table, ratio,
                                         1 / math.sqrt(w.D), skip)
    pool, sc = (w.k, w.ks) if w.v is None else (w.v, w.vs)
    with np.errstate(invalid="ignore"):
        vmax = np.nanmax(np.abs(np.where(sc[:, :, None, None] > 0, ref.E4M3[pool] * sc[:, :, None, None], 0)))
    tol, ltol = attn_bounds(w.D, max(1, lists.shape[2] * w.T), want, wl, mag, big, flat, vmax, out_dtype == BF,
                            eight_bit(w.D, q.shape[1] // w.H))
    got, gl = out.float().cpu().numpy(), lse.cpu().numpy()
    assert np.isfinite(got).all()
    worst = np.abs(got - want) - tol
    assert (worst <= 0).all(), (worst.max(), np.unravel_index(worst.argmax(), worst.shape))
    assert np.array_equal(np.isneginf(gl), np.isneginf(wl))
    fin = np.isfinite(wl)
    assert (np.abs(gl[fin] - wl[fin]) <= ltol[fin]).all()
    return out, lse


ATTN = [  # lens, q_lens, heads, H, D, T, latent, ratio, budget
    ([1], [1], 1, 1, 64, 16, False, 1, 1),
    ([777], [1], 8, 1, 128, 16, False, 1, 16),
    ([100, 0, 17, 300, 1], [1, 1, 1, 0, 1], 8, 2, 128, 32, False, 1, 5),
    ([64, 65, 63], [1, 2, 3], 16, 4, 64, 64, False, 1, 1),
    ([500, 20], [5, 20], 12, 3, 128, 16, False, 4, 7),
    ([3000], [2], 16, 1, 128, 128, True, 1, 20),
    ([900, 40], [3, 40], 20, 2, 256, 16, True, 1, 30),   # two tiles of eight rows
    ([900, 40], [2, 1], 32, 2, 256, 64, False, 1, 9),
    ([333], [3], 12, 1, 512, 16, True, 1, 12),
    ([333], [3], 24, 2, 512, 32, False, 1, 6),
    # the tensor-core kernels: many heads to a kv head
    ([700, 90, 0], [3, 1, 2], 64, 1, 512, 64, True, 4, 7),
    ([700, 90], [2, 1], 128, 1, 512, 16, True, 1, 33),
    ([700, 90], [2, 2], 80, 2, 256, 32, False, 1, 9),
    ([700], [3], 200, 2, 256, 128, True, 128, 4),
    ([500, 33], [2, 1], 17, 1, 512, 32, False, 1, 10),
    ([700, 90], [2, 1], 72, 1, 128, 16, False, 1, 33),
    ([700, 90], [3, 9], 256, 2, 64, 32, False, 1, 8),
    ([700, 90], [2, 1], 256, 1, 128, 64, True, 4, 5),
    ([400] * 150, [1] * 150, 4, 2, 64, 16, False, 1, 9),
    ([90, 1200], [90, 1100], 2, 2, 64, 16, False, 1, 4),  # more queries than a plan has requests
    ([20] * 1024, [1] * 1024, 8, 2, 128, 16, False, 1, 2),   # the largest batch
    ([20] * 1024, [2, 0] * 512, 64, 1, 512, 16, True, 1, 2),
    ([200] * 40, [0] * 39 + [1], 8, 2, 128, 16, False, 1, 3),
]


@pytest.mark.parametrize("ragged", [False, True])
@pytest.mark.parametrize("case", range(len(ATTN)))
def test_attn_blocks(case, ragged):
    lens, q_lens, heads, H, D, T, latent, ratio, budget = ATTN[case]
    w = World(700 + case, lens, H, D, T, latent)
    seq = seq_of(lens, q_lens, ratio)
    lists = lists_of(w, seq, q_lens, ratio, budget, ragged=ragged)
    check_attn(w, w.queries(q_lens, heads), lists, seq, q_lens, ratio, F32 if (case + ragged) % 2 else BF)


@pytest.mark.parametrize("heads,H,D,latent", [(8, 2, 128, False), (64, 1, 512, True), (96, 1, 256, False), (128, 1, 128, False)])
def test_all_blocks_listed_is_attention(heads, H, D, latent):
    """The two plans cut a row's entries in other places, so that its sums are rounded in another order: each call is within
    attn_bounds of the exact result, hence they are within twice that of one another."""
    w = World(740, [700, 90, 0, 16], H, D, 16, latent)
    q, one = w.queries([1] * 4, heads), [1] * 4
    lists = np.full((4, H, 50), -1, np.int32)
    for b, n in enumerate(w.lens):
        lists[b, :, :-(-n // 16)] = np.arange(-(-n // 16))
    seq = seq_of(w.lens, one, 1)
    out, lse = check_attn(w, q, lists, seq, one, 1, F32)
    cache, args = w.cache(), (i64(w.rid), i64(seq), i64(one), i64(w.lens))
    plan = ckv.plan_q8_attn(cache, heads, 1, *args, 4)
    other, other_lse = ckv.q8_attn(cache, q.to(DEV), plan, i32(w.table), 1 / math.sqrt(D), out_dtype=F32)
    want, wl, mag, big, flat = bref.attn(w.k, w.ks, w.v, w.vs, q.float().numpy(), lists, w.rid, seq, one, w.lens, w.table, 1, 1 / math.sqrt(D))
    tol, ltol = attn_bounds(D, 800, want, wl, mag, big, flat, 448 * np.nanmax(w.ks if latent else w.vs), False, eight_bit(D, heads // H))
    assert (np.abs((out - other).cpu().numpy()) <= 2 * tol).all()
    assert torch.equal(torch.isneginf(lse), torch.isneginf(other_lse))
    fin = np.isfinite(wl)
    assert (np.abs(lse.cpu().numpy()[fin] - other_lse.cpu().numpy()[fin]) <= 2 * ltol[fin]).all()


@pytest.mark.parametrize("heads,D,latent", [(8, 128, False), (64, 512, True), (48, 256, False), (72, 64, False)])
def test_what_is_not_listed_does_not_count(heads, D, latent):
    """NaN in the blocks that are not listed, in hidden entries of the last one and past the end."""
    w = World(741, [500], 1, D, 16, latent)
    seq, q_lens, q = [500], [4], w.queries([4], heads)
    lists = np.array([[[0, 3, 8, 17, 31, -1]]] * 4, np.int32)
    for pool in (w.k, w.v):
        if pool is not None:
            for j in set(range(32)) - {0, 3, 8, 17, 31}:
                pool[w.table[w.rid[0], j]] = 0x7F
            pool[w.table[w.rid[0], 31], :, 1:4] = 0x7F  # entries 497 .. 499: of the queries, only later ones see them
    out, lse, st = run_attn(w, q, lists, seq, q_lens, 1, F32)
    assert st == 0 and torch.isfinite(out[0]).all() and not torch.isfinite(out[1:]).any()
    w.k[w.table[w.rid[0], 31], :, 1:4] = 0x11
    if w.v is not None:
        w.v[w.table[w.rid[0], 31], :, 1:4] = 0x11
    check_attn(w, q, lists, seq, q_lens, 1)


@pytest.mark.parametrize("heads,D,latent", [(4, 128, False), (64, 512, True), (72, 128, False)])
def test_lists_out_of_order_and_blocks_nobody_sees(heads, D, latent):
    w = World(742, [200], 1, D, 16, latent)
    q, seq, q_lens = w.queries([6], heads), [200], [6]
    lists = np.array([[0, 3, 3, 5, 12], [7, 2, 9, 8, 12], [-1, 4, -7, 1, 6], [0, 12, 13, 40, 0x7FFFFFFF],
                      [-1, -1, -1, -1, -1], [13, 14, 15, 16, 17]], np.int32)[:, None]
    kept = np.array([[0, 3, 5, 12, -1], [7, 9, 12, -1, -1], [4, 6, -1, -1, -1], [0, 12, -1, -1, -1], [-1] * 5, [-1] * 5],
                    np.int32)[:, None]
    out, lse, st = run_attn(w, q, lists, seq, q_lens, 1, F32)
    assert st == ckv.STATUS_BAD_INDEX  # rows 0, 1 and 2 do not ascend
    want, want_lse = check_attn(w, q, kept, seq, q_lens, 1, F32)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    out, lse, st = run_attn(w, q, np.where(np.arange(6)[:, None, None] < 3, kept, lists), seq, q_lens, 1, F32)
    assert st == 0 and torch.equal(out, want)


@pytest.mark.parametrize("heads,D,latent", [(4, 128, False), (64, 512, True), (40, 256, False), (72, 64, False)])
def test_missing_blocks_do_not_count(heads, D, latent):
    w = World(743, [300, 60], 1, D, 16, latent)
    gone = {int(w.table[w.rid[0], 0]), int(w.table[w.rid[0], 7])}
    w2 = w.table.copy()
    q, seq, q_lens = w.queries([1, 1], heads), [300, 60], [1, 1]
    lists = np.array([[0, 4, 7, 18], [0, 1, 3, -1]], np.int32)[:, None]
    w.table[w.rid[0], 0], w.table[w.rid[0], 7] = -3, w.blocks
    out, lse, st = run_attn(w, q, lists, seq, q_lens, 1, F32)
    assert st == ckv.STATUS_BAD_INDEX
    ref_out, ref_lse, *_ = bref.attn(w.k, w.ks, w.v, w.vs, q.float().numpy(), lists, w.rid, seq, q_lens, w.lens, w2, 1, 1 / math.sqrt(D), gone)
    assert np.abs(out.cpu().numpy() - ref_out).max() <= 0.02 and np.abs(lse.cpu().numpy() - ref_lse).max() <= 0.01


def test_attn_blocks_flags_bad_data_and_leaves_other_rows():
    w = World(744, [100, 40, 60], 2, 128, 16, False)
    ql, heads = [1, 2, 1], 8
    q = w.queries(ql, heads)
    lists = lists_of(w, w.lens, ql, 1, 3, ragged=False)
    cache, table = w.cache(), i32(w.table)

    def run(rid, seq, q_lens, lens, n=4):
        st = status()
        out, lse = torch.full((n, heads, 128), 5.0, device=DEV), torch.full((n, heads), 5.0, device=DEV)
        ckv.q8_attn_blocks(cache, q[:n].to(DEV), i32(lists[:n]), 1, i64(rid), i64(seq), i64(q_lens), i64(lens), table, 0.1, out=out,
                           lse=lse, status=st)
        return out, lse, int(st[0])

    good, good_lse, st = run(w.rid, w.lens, ql, w.lens)
    assert st == 0
    for rid, seq, lens in ((w.rid, w.lens, [100, -1, 60]), ([w.rid[0], -1, w.rid[2]], w.lens, w.lens),
                           ([w.rid[0], 50, w.rid[2]], w.lens, w.lens), (w.rid, [100, 1, 60], w.lens),
                           (w.rid, w.lens, [100, 16 * w.table.shape[1] + 1, 60])):
        out, lse, st = run(rid, seq, ql, lens)
        assert st == ckv.STATUS_BAD_LENGTH
        assert (out[1:3] == 5).all() and (lse[1:3] == 5).all()
        assert torch.equal(out[[0, 3]], good[[0, 3]]) and torch.equal(lse[[0, 3]], good_lse[[0, 3]])
    out, lse, st = run(w.rid, w.lens, ql, w.lens, 3)
    assert st == ckv.STATUS_BAD_TOTAL and torch.equal(out, good[:3])
    out, lse, st = run(w.rid[:2], w.lens[:2], ql[:2], w.lens[:2])
    assert st == ckv.STATUS_BAD_TOTAL and torch.equal(out[:3], good[:3]) and (out[3] == 5).all() and (lse[3] == 5).all()


@pytest.mark.parametrize("heads,H,D,latent", [(8, 2, 128, False), (64, 1, 512, True)])
def test_results_repeat_bit_for_bit(heads, H, D, latent):
    w = World(745, [3000, 900, 30], H, D, 32, latent)
    q, seq, q_lens = w.queries([2, 1, 1], heads), w.lens, [2, 1, 1]
    lists = lists_of(w, seq, q_lens, 1, 20)
    first = run_attn(w, q, lists, seq, q_lens, 1, F32)
    for _ in range(5):
        again = run_attn(w, q, lists, seq, q_lens, 1, F32)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_offsets_past_32_bits():
    """A pool of more than 2^32 bytes whose last blocks are read by every operator."""
    T, H, D = 64, 8, 128
    blocks = (1 << 32) // (T * H * D) + 70
    cache = ckv.new_q8_cache(blocks, H, T, D, latent=True)
    bounds = ckv.new_q8_bounds(cache)
    w = World(746, [600], H, D, T, True)
    shift = blocks - w.blocks
    cache.k.view(torch.uint8)[shift:] = torch.as_tensor(w.k, device=DEV)
    cache.k_scale[shift:] = torch.as_tensor(w.ks, device=DEV)
    table = i32(np.where(w.table >= 0, w.table + shift, -1))
    args, q = (i64(w.rid), i64([600]), i64([1]), i64([600])), w.queries([1], 32)
    ckv.q8_bounds(cache, bounds, args[0], args[1], args[1], table)
    small = ckv.new_q8_bounds(w.cache())
    ckv.q8_bounds(w.cache(), small, args[0], args[1], args[1], i32(w.table))
    assert torch.equal(bounds.view(torch.uint8)[shift:][w.table[w.rid[0], :10]], small.view(torch.uint8)[w.table[w.rid[0], :10]])
    s = ckv.q8_block_scores(cache, bounds, q.to(DEV), 1, *args, table, 0.1)
    assert torch.equal(s, ckv.q8_block_scores(w.cache(), small, q.to(DEV), 1, *args, i32(w.table), 0.1))
    lists = ckv.q8_block_select(s, T, 1, *args[1:], 4, 1, 1)
    out, lse = ckv.q8_attn_blocks(cache, q.to(DEV), lists, 1, *args, table, 0.1)
    want, want_lse = ckv.q8_attn_blocks(w.cache(), q.to(DEV), lists, 1, *args, i32(w.table), 0.1)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)


# -------------------------------------------------------------------------------------------------------- together
class Serving:
    """A latent cache that grows, its bounds with it, and sparse attention over it, beside the oracle's own."""

    def __init__(self, seed, start, T=16, D=128, heads=16, budget=5, room=200):
        self.r = np.random.RandomState(seed)
        self.T, self.D, self.heads, self.budget, B = T, D, heads, budget, len(start)
        per = -(-(max(start) + room) // T)
        self.rid = self.r.permutation(B + 1)[:B]
        self.table = self.r.permutation((B + 1) * per).reshape(B + 1, per).astype(np.int32)
        blocks = (B + 1) * per + 40
        self.spare = np.arange((B + 1) * per, blocks)
        self.cache, self.st = ckv.new_q8_cache(blocks, 1, T, D, latent=True), status()
        self.bounds = ckv.new_q8_bounds(self.cache)
        self.k, self.ks = np.zeros((blocks, 1, T, D), np.uint8), np.ones((blocks, 1), np.float32)
        self.freqs = table_of_angles(2000, 64)
        self.freqs_dev = f32(self.freqs)
        self.kv = np.zeros(B, np.int64)
        self.weights = torch.zeros(blocks, T, device=DEV)
        self.scale = 1 / math.sqrt(D)
        # what a captured step reads
        self.rid_d, self.table_d = i64(self.rid), i32(self.table)

    def feed(self, new):
        n = int(np.sum(new))
        start = self.kv.copy()
        self.kv = self.kv + new
        pos = np.concatenate([np.arange(a, b) for a, b in zip(start, self.kv)])
        x = torch.as_tensor(self.r.standard_normal((n, 1, self.D))).to(BF)
        q = torch.as_tensor(self.r.standard_normal((n, self.heads, self.D)) * 1.5).to(BF)
        ref.store(self.k, self.ks, bref.rope(x.float().numpy(), None, 0, self.freqs, pos, 64, False, np.float32),
                  ref.store_plan(self.rid, self.kv, new, self.table, self.T))
        return n, pos, x, q

    def step(self, x, q, pos, kv, new, n):
        plan, counts = ckv.plan_q8_store(self.cache, self.rid_d, kv, new, n, self.table_d, status=self.st)
        ckv.q8_rope_store(self.cache, x, None, plan, pos, self.freqs_dev, counts, rope_begin=64, weights=self.weights, status=self.st)
        ckv.q8_bounds(self.cache, self.bounds, self.rid_d, kv, new, self.table_d, status=self.st)
        s = ckv.q8_block_scores(self.cache, self.bounds, q, 1, self.rid_d, kv, new, kv, self.table_d, self.scale, status=self.st)
        lists = ckv.q8_block_select(s, self.T, 1, kv, new, kv, self.budget, 1, 1, status=self.st)
        out, lse = ckv.q8_attn_blocks(self.cache, q, lists, 1, self.rid_d, kv, new, kv, self.table_d, self.scale, status=self.st)
        return s, lists, out, lse

    def check(self, q, new, s, lists, out, lse):
        assert ref.same_codes(codes(self.cache.k), self.k)
        bnd = bref.bounds(np.zeros((len(self.k), 1, 2, self.D), np.uint8), self.k, self.rid, self.kv, self.kv, self.table)
        touched = np.concatenate([self.table[r, :-(-n // self.T)] for r, n in zip(self.rid, self.kv)])
        assert same_values(codes(self.bounds)[touched], bnd[touched])
        qn = q.float().cpu().numpy()
        want, mag, flat = bref.scores(bnd, self.ks, qn, self.rid, self.kv, new, self.kv, self.table, self.T, 1, self.scale, s.shape[2])
        got = s.cpu().numpy()
        fin = np.isfinite(want)
        assert np.array_equal(np.isneginf(got), np.isneginf(want))
        assert (np.abs(got[fin] - want[fin]) <= (mag * (2 * self.D + 4) * 2.0 ** -23 + flat * 2.0 ** -38)[fin]).all()
        ln = lists.cpu().numpy()
        assert np.array_equal(ln, bref.select(got, self.kv, new, self.kv, self.T, 1, self.budget, 1, 1))
        want, wl, mag, big, flat = bref.attn(self.k, self.ks, None, None, qn, ln, self.rid, self.kv, new, self.kv, self.table, 1, self.scale)
        tol, ltol = attn_bounds(self.D, self.budget * self.T, want, wl, mag, big, flat, 448 * self.ks.max(), True)
        assert (np.abs(out.float().cpu().numpy() - want) <= tol).all()
        assert (np.abs(lse.cpu().numpy() - wl) <= ltol).all()
        assert int(self.st[0]) == 0


def test_a_request_s_life_with_sparse_attention():
    """Prompts, decode, an eviction into other blocks with their bounds made anew, and decode over what was kept."""
    s = Serving(801, [150, 70, 33])

    def go(new):
        n, pos, x, q = s.feed(np.asarray(new))
        q = q.to(DEV)
        s.check(q, new, *s.step(x.to(DEV), q, i64(pos), i64(s.kv), i64(new), n))

    go([150, 70, 33])
    for _ in range(4):
        go([1, 1, 1])
    go([3, 0, 2])
    # eviction by weights that the test makes up
    s.weights.copy_(torch.rand(s.weights.shape, device=DEV))
    dst = np.full_like(s.table, -1)
    for b, r in enumerate(s.rid):
        dst[r, :8] = s.spare[8 * b:8 * b + 8]
    kept, lens = ckv.q8_evict(s.cache, s.weights, s.rid_d, i64(s.kv), s.table_d, i32(dst), 60, 2, 8, status=s.st)
    wref = s.weights.cpu().numpy().astype(np.float64)
    ref.evict([(s.k, s.ks)], wref, s.rid, s.kv, s.table, dst, 60, 2, 8)
    s.table, s.table_d, s.kv = dst, i32(dst), lens.cpu().numpy()
    ckv.q8_bounds(s.cache, s.bounds, s.rid_d, lens, lens, s.table_d, status=s.st)
    assert s.kv.tolist() == [60, 60, 39]
    for _ in range(3):
        go([1, 1, 1])


def test_captured_steps_replay_with_new_lengths_and_beside_another():
    sides = [Serving(811, [90, 40]), Serving(812, [17, 130])]
    for s, start in zip(sides, ([90, 40], [17, 130])):
        n, pos, x, q = s.feed(np.asarray(start))
        q = q.to(DEV)
        s.check(q, start, *s.step(x.to(DEV), q, i64(pos), i64(s.kv), i64(start), n))
        s.x, s.q = torch.zeros(2, 1, s.D, dtype=BF, device=DEV), torch.zeros(2, s.heads, s.D, dtype=BF, device=DEV)
        s.pos, s.kv_d, s.one = i64([0, 0]), i64(s.kv + 1), i64([1, 1])
        s.before = [x.clone() for x in (s.cache.k.view(torch.uint8), s.cache.k_scale)]
        t = torch.cuda.Stream()
        t.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(t):
            s.step(s.x, s.q, s.pos, s.kv_d, s.one, 2)
        torch.cuda.current_stream().wait_stream(t)
        torch.cuda.synchronize()
        s.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(s.graph):
            s.got = s.step(s.x, s.q, s.pos, s.kv_d, s.one, 2)
        s.cache.k.view(torch.uint8).copy_(s.before[0])
        s.cache.k_scale.copy_(s.before[1])
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(20):
        for s in sides:
            n, pos, x, q = s.feed(np.array([1, 1]))
            s.x.copy_(x), s.q.copy_(q), s.pos.copy_(i64(pos)), s.kv_d.copy_(i64(s.kv))
        torch.cuda.synchronize()
        for s, t in zip(sides, streams):
            with torch.cuda.stream(t):
                s.graph.replay()
        torch.cuda.synchronize()
        for s in sides:
            s.check(s.q, [1, 1], *s.got)


def test_on_another_stream():
    """Tensors of the current stream's making, calls on another; what a call makes belongs to its stream."""
    w = World(821, [700], 2, 128, 16, False)
    q, one, table, cache = w.queries([1], 8).to(DEV), i64([1]), i32(w.table), w.cache()
    bounds, b2 = ckv.new_q8_bounds(cache), ckv.new_q8_bounds(cache)
    args = i64(w.rid), i64([700]), one, i64([700])

    def go(bounds, **kw):
        ckv.q8_bounds(cache, bounds, args[0], args[1], args[1], table, **kw)
        s = ckv.q8_block_scores(cache, bounds, q, 1, *args, table, 0.1, **kw)
        lists = ckv.q8_block_select(s, 16, 1, *args[1:], 9, 1, 1, **kw)
        return (s, lists) + tuple(ckv.q8_attn_blocks(cache, q, lists, 1, *args, table, 0.1, **kw))

    want = go(bounds)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)  # the current stream still has work to do on memory that it has given back
    junk = [torch.full_like(x, 7) for x in want] + [ckv.q8_attn_blocks_workspace(cache, 8, 1, 9).fill_(0xFF)]
    del junk
    got = go(b2, stream=s)
    torch.cuda.synchronize()
    for x, y in zip(got, want):
        assert torch.equal(x, y)


def test_given_outputs_and_workspaces():
    w = World(822, [700, 300], 2, 128, 16, False)
    q, one, table, cache = w.queries([1, 1], 8).to(DEV), i64([1, 1]), i32(w.table), w.cache()
    args = i64(w.rid), i64(w.lens), one, i64(w.lens)
    bounds = ckv.q8_bounds(cache, ckv.new_q8_bounds(cache), args[0], args[1], args[1], table)
    s = torch.empty(2, 2, 50, device=DEV)
    assert ckv.q8_block_scores(cache, bounds, q, 1, *args, table, 0.1, scores=s) is s
    lists = torch.empty(2, 2, 9, dtype=torch.int32, device=DEV)
    assert ckv.q8_block_select(s, 16, 1, *args[1:], 9, blocks=lists) is lists
    want, want_lse = ckv.q8_attn_blocks(cache, q, lists, 1, *args, table, 0.1, out_dtype=F32)
    out, lse = torch.empty(2, 8, 128, device=DEV), torch.empty(2, 8, device=DEV)
    ws = ckv.q8_attn_blocks_workspace(cache, 8, 2, 9).fill_(0xFF)  # its content does not matter
    got = ckv.q8_attn_blocks(cache, q, lists, 1, *args, table, 0.1, out=out, lse=lse, workspace=ws)
    assert got[0] is out and got[1] is lse and torch.equal(out, want) and torch.equal(lse, want_lse)


def test_shapes_that_the_binding_refuses():
    w = World(823, [20], 2, 128, 16, False)
    cache, q, table = w.cache(), w.queries([1], 4).to(DEV), i32(w.table)
    one, n = i64([1]), i64([20])
    a = (i64(w.rid), n, one, n)
    bounds, s, lists = ckv.new_q8_bounds(cache), torch.zeros(1, 2, 4, device=DEV), torch.zeros(1, 2, 3, dtype=torch.int32, device=DEV)
    rows = torch.zeros(1, 2, 128, dtype=BF, device=DEV)
    plan, freqs, pos = torch.zeros(1, 16, dtype=torch.uint8, device=DEV), torch.zeros(4, 16, 2, device=DEV), i64([0])
    rope = lambda k=rows, v=rows, p=plan, pos=pos, fr=freqs, **kw: ckv.q8_rope_store(cache, k, v, p, pos, fr, **kw)
    bad = [
        lambda: rope(k=rows[:, :, :64]), lambda: rope(v=None), lambda: rope(v=rows.float()), lambda: rope(v=rows.expand(2, 2, 128)),
        lambda: rope(k=rows.transpose(1, 2).contiguous().transpose(1, 2)),
        lambda: rope(p=plan[:, :8]), lambda: rope(pos=None), lambda: rope(pos=pos.int()), lambda: rope(pos=i64([0, 1])),
        lambda: rope(fr=freqs.double()), lambda: rope(fr=freqs[..., :1]), lambda: rope(norm_weight=torch.ones(64, device=DEV)),
        lambda: rope(weights=torch.zeros(3, device=DEV)), lambda: rope(counts=one), lambda: rope(rope_begin=-16),
        lambda: rope(k=rows.half(), v=rows.half()), lambda: rope(k=rows.cpu()),
        lambda: ckv.q8_bounds(cache, bounds[:1], a[0], n, one, table), lambda: ckv.q8_bounds(cache, bounds.view(torch.uint8), a[0], n, one, table),
        lambda: ckv.q8_bounds(cache, bounds, a[0].int(), n, one, table), lambda: ckv.q8_bounds(cache, bounds, a[0], n, one, table.long()),
        lambda: ckv.q8_block_scores(cache, bounds, q.float(), 1, *a, table, 0.1),
        lambda: ckv.q8_block_scores(cache, bounds[:1], q, 1, *a, table, 0.1),
        lambda: ckv.q8_block_scores(cache, bounds, q[0], 1, *a, table, 0.1),
        lambda: ckv.q8_block_scores(cache, bounds, q, 1, *a, table, 0.1, width=-1),
        lambda: ckv.q8_block_scores(cache, bounds, q, 1, *a, table, 0.1, width=5, scores=s),
        lambda: ckv.q8_block_scores(cache, bounds, q, 1, a[0], n, i64([1, 1]), n, table, 0.1),
        lambda: ckv.q8_block_select(s.double(), 16, 1, *a[1:], 3), lambda: ckv.q8_block_select(s[0], 16, 1, *a[1:], 3),
        lambda: ckv.q8_block_select(s, 16, 1, *a[1:], -1), lambda: ckv.q8_block_select(s, 16, 1, *a[1:], 3, blocks=lists[:, :1]),
        lambda: ckv.q8_block_select(s.transpose(1, 2), 16, 1, *a[1:], 3),
        lambda: ckv.q8_attn_blocks(cache, q, lists.long(), 1, *a, table, 0.1),
        lambda: ckv.q8_attn_blocks(cache, q, lists[:, :1], 1, *a, table, 0.1),
        lambda: ckv.q8_attn_blocks(cache, q, lists[..., 0], 1, *a, table, 0.1),
        lambda: ckv.q8_attn_blocks(cache, q, lists, 1 << 32, *a, table, 0.1),
        lambda: ckv.q8_attn_blocks(cache, q, lists, 1, *a, table, 0.1, out=q[:, :2]),
        lambda: ckv.q8_attn_blocks(cache, q, lists, 1, *a, table, 0.1, out_dtype=torch.float16),
        lambda: ckv.q8_attn_blocks(cache, q, lists, 1, *a, table, 0.1, workspace=s),
        lambda: ckv.q8_attn_blocks_workspace(cache, 4, 1 << 32, 3),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            raise AssertionError(i)
    for call in (lambda: rope(fr=torch.zeros(4, 8, 2, device=DEV)), lambda: ckv.q8_block_select(s, 24, 1, *a[1:], 3),
                 lambda: ckv.q8_block_select(s, 16, 1, *a[1:], 3, 2, 2), lambda: ckv.q8_block_scores(cache, bounds, q, 0, *a, table, 0.1),
                 lambda: ckv.q8_attn_blocks(cache, q, lists, 1, *a, table, 0.1, workspace=torch.zeros(64, dtype=torch.uint8, device=DEV))):
        with pytest.raises(ckv.CkvError):
            call()


# ------------------------------------------------------------------------------------------ scores of many query rows
MANY = [  # lens, q_lens, heads, H, D, T, ratio
    ([700], [200], 4, 1, 128, 16, 1),
    ([700, 40, 0], [90, 40, 70], 8, 2, 64, 16, 1),
    ([5000], [130], 1, 1, 128, 32, 1),             # several tiles of blocks
    ([2100, 2048, 2049], [128, 256, 129], 2, 2, 64, 16, 1),
    ([900], [70], 7, 1, 128, 64, 4),
    ([900, 30], [70, 30], 24, 2, 128, 16, 1),      # 12 heads to a kv head: rows of heads that do not exist
    ([900], [40], 64, 1, 128, 128, 1),
    ([900], [33], 33, 1, 64, 16, 1),
    ([3000], [5], 64, 1, 64, 16, 128),
    ([300] * 20, [20] * 20, 16, 1, 128, 16, 1),
    ([600], [300], 3, 1, 256, 16, 1),              # more channels than the tensor-core kernel takes
    ([600], [50], 70, 1, 128, 16, 1),              # and more heads
]


@pytest.mark.parametrize("case", range(len(MANY)))
def test_scores_of_many_rows(case):
    lens, q_lens, heads, H, D, T, ratio = MANY[case]
    w = World(900 + case, lens, H, D, T, True)
    check_scores(w, w.queries(q_lens, heads), seq_of(lens, q_lens, ratio), q_lens, heads, ratio)


def test_scores_of_many_rows_with_nan_missing_blocks_and_other_widths():
    w = World(930, [700, 300], 2, 128, 16, True)
    ql, heads = [150, 100], 8
    bnd, q = bounds_of(w), w.queries(ql, heads)
    bnd[w.table[w.rid[0], 2], 0, :, 9] = 0x7F
    q[7, 5, 3] = float("nan")
    q[200, 0, 7] = float("inf")
    args = i64(w.rid), i64(w.lens), i64(ql), i64(w.lens)
    want, mag, flat = bref.scores(bnd, w.ks, q.float().numpy(), w.rid, w.lens, ql, w.lens, w.table, 16, 1, 0.07, 60)
    st = status()
    got = ckv.q8_block_scores(w.cache(), up(bnd), q.to(DEV), 1, *args, i32(w.table), 0.07, width=60, status=st).cpu().numpy()
    assert int(st[0]) == 0 and np.array_equal(np.isnan(got), np.isnan(want))
    inf = np.isinf(want)
    assert np.array_equal(got[inf], want[inf])
    fin = np.isfinite(want)
    assert (np.abs(got[fin] - want[fin]) <= (mag * 260 * 2.0 ** -23 + flat * 2.0 ** -38)[fin]).all()
    table = w.table.copy()
    table[w.rid[1], 3], table[w.rid[1], 0] = -1, w.blocks
    out = torch.full((260, 2, 60), 3.0, device=DEV)  # ten rows behind the last request's
    more = torch.cat([q, q[:10]]).to(DEV)
    ckv.q8_block_scores(w.cache(), up(bnd), more, 1, *args, i32(table), 0.07, scores=out, status=st)
    assert int(st[0]) == ckv.STATUS_BAD_INDEX | ckv.STATUS_BAD_TOTAL
    assert (out[250:] == 3.0).all() and torch.isneginf(out[150:250, :, [0, 3]]).all()
    again = out[:250].cpu().numpy()
    again[150:, :, [0, 3]] = got[150:, :, [0, 3]]
    assert np.array_equal(again, got, equal_nan=True)


def test_score_waits_that_run_out_are_reported_and_leave_the_context_usable():
    w = World(931, [3000], 2, 128, 16, True)
    q, bnd, cache = w.queries([400], 8).to(DEV), up(bounds_of(w)), w.cache()
    args = i64(w.rid), i64(w.lens), i64([400]), i64(w.lens), i32(w.table)
    want = ckv.q8_block_scores(cache, bnd, q, 1, *args, 0.1)
    torch.cuda.synchronize()
    old = ckv.set_wait_limit_ns(1)
    try:
        st = status()
        ckv.q8_block_scores(cache, bnd, q, 1, *args, 0.1, status=st)
        torch.cuda.synchronize()
    finally:
        ckv.set_wait_limit_ns(old)
    assert int(st[0]) & ckv.STATUS_TIMEOUT
    st.zero_()
    assert torch.equal(ckv.q8_block_scores(cache, bnd, q, 1, *args, 0.1, status=st), want) and int(st[0]) == 0


# ------------------------------------------------------------------------------------------------ scores' range
RANGE = [  # heads, H, D, q_lens: the kernel for few rows, the one for many channels or heads, the tensor cores'
    (1, 1, 64, [2]), (8, 2, 128, [1]), (6, 1, 256, [1]), (4, 2, 512, [1]),
    (12, 1, 512, [2]), (4, 1, 256, [40]), (200, 1, 256, [2]), (70, 1, 128, [5]),
    (4, 1, 128, [40]), (24, 2, 64, [9]), (64, 1, 128, [3]),
]


@pytest.mark.parametrize("q_exp,k_exp,scale", [(124, -38, 0.07), (124, -38, 1e-30), (124, 36, 1e-36), (124, -38, 1e-40),
                                               (-90, 36, 1e29), (-90, -38, 1e29), (0, 36, 1e-44), (0, -38, 0.07)])
@pytest.mark.parametrize("case", range(len(RANGE)))
def test_scores_whose_factors_pass_the_range_that_they_stay_in(case, q_exp, k_exp, scale):
    heads, H, D, q_lens = RANGE[case]
    w = World(960 + case, [100], H, D, 16, True)
    w.ks *= np.float32(2.0) ** k_exp
    q = w.queries(q_lens, heads)
    q[:, ::2] *= 2.0 ** q_exp  # beside heads of ordinary size
    assert torch.isfinite(q).all()
    scale, bnd, st = float(np.float32(scale)), bounds_of(w), status()
    got = ckv.q8_block_scores(w.cache(), up(bnd), q.to(DEV), 1, i64(w.rid), i64([100]), i64(q_lens), i64([100]), i32(w.table),
                              scale, status=st).cpu().numpy().astype(np.float64)
    want, mag, flat = bref.scores(bnd, w.ks, q.float().numpy(), w.rid, [100], q_lens, [100], w.table, 16, 1, scale, got.shape[2])
    assert int(st[0]) == 0
    # as check_scores, but what fp32 does not hold is an infinity: with k_exp 36 and a scale of 1e29 an ordinary head's score is
    # some 2^9 2^29 2^96; below 2^-126 its steps are 2^-149 each, which the row's factor, 2^-18 of the score's, and the block's may add
    most = float(np.finfo(np.float32).max)
    tol = mag * (2 * D + 4) * 2.0 ** -23 + flat * 2.0 ** -38 + 2.0 ** -149
    over = np.abs(want) > most + tol
    assert np.array_equal(got[over], np.sign(want[over]) * np.inf)
    inside = np.abs(want) < most - tol
    assert (over | inside).all() and (np.abs(got[inside] - want[inside]) <= tol[inside]).all()


@pytest.mark.parametrize("q_exp,k_exp", [(122, -36), (-80, 36)])
@pytest.mark.parametrize("heads,H,D,latent", [(4, 1, 64, False), (8, 2, 128, False), (32, 1, 256, True), (8, 1, 512, True), (20, 2, 512, False),
                                              (64, 1, 512, True), (80, 2, 256, False), (72, 1, 128, True)])
def test_attention_whose_factors_pass_the_range_that_its_scores_stay_in(heads, H, D, latent, q_exp, k_exp):
    """Scores of ordinary size, made of queries, entries and a scale that are not."""
    w = World(980, [300, 40], H, D, 16, latent)
    w.ks *= np.float32(2.0) ** k_exp
    seq, q_lens = [300, 40], [2, 1]
    q = w.queries(q_lens, heads) * 2.0 ** q_exp
    assert torch.isfinite(q).all()
    lists = lists_of(w, seq, q_lens, 1, 12, ragged=False)
    scale = float(np.float32(D ** -0.5 * 2.0 ** (-q_exp - k_exp)))
    out, lse, st = run_attn(w, q, lists, seq, q_lens, 1, F32, scale=scale)
    assert st == 0
    want, wl, mag, big, flat = bref.attn(w.k, w.ks, w.v, w.vs, q.float().numpy(), lists, w.rid, seq, q_lens, w.lens, w.table, 1, scale)
    pool, sc = (w.k, w.ks) if latent else (w.v, w.vs)
    vmax = 448 * np.nanmax(sc)
    tol, ltol = attn_bounds(D, 12 * 16, want, wl, mag, big, flat, vmax, False, eight_bit(D, heads // H))
    assert (np.abs(out.cpu().numpy() - want) <= tol).all()
    assert (np.abs(lse.cpu().numpy() - wl) <= ltol).all()


# ----------------------------------------------------------------------------- rotated append: every kernel's special cases
APPEND = [  # T, D: two vectors of sixteen channels to a thread of 32, 64 and 128, four, a unit held by 256 and 512, one read twice
    (16, 64), (16, 128), (32, 128), (64, 128), (64, 256), (64, 512), (128, 512),
]


@pytest.mark.parametrize("dt,latent,halves", [(BF, False, True), (F32, True, False)])
@pytest.mark.parametrize("T,D", APPEND)
def test_every_append_leaves_rows_of_positions_outside_the_table(T, D, dt, latent, halves):
    w = World(1000 + T + D, [3, 0, T + 4], 2, D, T, latent, more=2 * T)
    new = [T + 4, 2 * T, 2]
    n, dim = sum(new), 64
    k, v = rope_inputs(w.r, n, 2, D, dt, 1, 1 if latent else 2)
    freqs, pos = table_of_angles(100, dim), w.r.randint(0, 100, n)
    # single rows, the first and the last of a record, all of one
    bad = np.r_[0, T - 4, T - 3, T + 1, T + 4:2 * T + 4, 3 * T + 3, n - 1]
    pos[bad] = np.resize([-1, 100, 1 << 40, -(1 << 40), 1 << 32], len(bad))
    cache, st, kv = w.cache(), status(), w.lens + new
    weights = torch.full((w.blocks, T), 5.0, device=DEV)
    plan, counts = ckv.plan_q8_store(cache, i64(w.rid), i64(kv), i64(new), n, i32(w.table), status=st)
    ckv.q8_rope_store(cache, k, v, plan, i64(pos), f32(freqs), counts, rope_begin=D - dim, halves=halves, weights=weights, status=st)
    assert int(st[0]) == ckv.STATUS_BAD_INDEX
    recs = ref.store_plan(w.rid, kv, new, w.table, T)
    safe = np.where(np.isin(np.arange(n), bad), 0, pos)
    sides = [(w.k, w.ks, bref.rope(k.float().cpu().numpy(), None, 0, freqs, safe, D - dim, halves, np.float32), cache.k, cache.k_scale)]
    if not latent:
        sides.append((w.v, w.vs, v.float().cpu().numpy(), cache.v, cache.v_scale))
    for pool, scale, rows, got, got_scale in sides:
        rows = rows.copy()
        rows[bad] = 0  # zeros do not count for a scale
        old = pool.copy()
        ref.store(pool, scale, rows, recs)
        for block, row, slot, cnt in recs:
            for i in range(cnt):
                if row + i in bad:
                    pool[block, :, slot + i] = old[block, :, slot + i]
        assert ref.same_codes(codes(got), pool)
        assert np.array_equal(got_scale.cpu().numpy(), scale, equal_nan=True)
    want = np.full((w.blocks, T), 5.0, np.float32)
    for block, row, slot, cnt in recs:
        want[block, slot:slot + cnt] = np.where(np.isin(np.arange(row, row + cnt), bad), 5.0, 0.0)
    assert np.array_equal(weights.cpu().numpy(), want)


@pytest.mark.parametrize("dt,latent", [(BF, True), (F32, False)])
@pytest.mark.parametrize("T,D", APPEND)
def test_every_append_of_infinities_and_nan(T, D, dt, latent):
    """On fresh and on begun blocks; a block of nothing finite among them."""
    w = World(1100 + T + D, [5, 0], 1, D, T, latent, more=2 * T)
    new = [T, T + 3]
    n = sum(new)
    k, v = rope_inputs(w.r, n, 1, D, dt, 0, 1 if latent else 2)
    for x in (k,) if latent else (k, v):
        x[1, 0, 3], x[2, 0, D - 1], x[3, 0, 5] = np.inf, np.nan, -np.inf
        x[4], x[7, 0, :D // 2] = 0, -np.inf
        x[T:T + T] = np.nan
        x[2 * T:, 0, 1::3] = np.inf  # the last block's rows
        x[2 * T:, 0, ::3] = 0
    freqs, pos = table_of_angles(n, 32), np.arange(n)
    cache, kv = w.cache(), w.lens + new
    plan, counts = ckv.plan_q8_store(cache, i64(w.rid), i64(kv), i64(new), n, i32(w.table))
    ckv.q8_rope_store(cache, k, v, plan, i64(pos), f32(freqs), counts)
    recs = ref.store_plan(w.rid, kv, new, w.table, T)
    with np.errstate(invalid="ignore"):
        ref.store(w.k, w.ks, bref.rope(k.float().cpu().numpy(), None, 0, freqs, pos, 0, False, np.float32), recs)
    assert ref.same_codes(codes(cache.k), w.k)
    assert np.array_equal(cache.k_scale.cpu().numpy(), w.ks, equal_nan=True)
    if not latent:
        ref.store(w.v, w.vs, v.float().cpu().numpy(), recs)
        assert ref.same_codes(codes(cache.v), w.v)
        assert np.array_equal(cache.v_scale.cpu().numpy(), w.vs, equal_nan=True)


@pytest.mark.parametrize("dt,latent,halves,dim", [(BF, False, False, 64), (F32, True, True, 32), (BF, True, False, 0)])
@pytest.mark.parametrize("T,D", APPEND)
def test_every_append_with_a_norm_to_begun_blocks(T, D, dt, latent, halves, dim):
    """As test_rope_store_with_a_norm; a begun block keeps the larger scale, and its earlier entries follow it; some rows hold an infinity,
    which its norm makes NaN and the row's others 0, or a NaN, which makes all of it NaN."""
    w = World(1200 + T + D, [3, T + 5, 2 * T - 1], 2, D, T, latent, spread=2, more=T + 9)
    new = [T + 9, 4, 1]
    n = sum(new)
    k, v = rope_inputs(w.r, n, 2, D, dt, 2, 1 if latent else 2)
    k[2, 0, 7], k[6, 1, D - 1], k[5, 0, 0] = np.inf, -np.inf, np.nan
    weight = (1 + 0.2 * w.r.standard_normal(D)).astype(np.float32)
    freqs, pos = table_of_angles(300, dim) if dim else None, w.r.randint(0, 300, n)
    cache, st, kv = w.cache(), status(), w.lens + new
    weights = torch.full((w.blocks, T), 5.0, device=DEV)
    plan, counts = ckv.plan_q8_store(cache, i64(w.rid), i64(kv), i64(new), n, i32(w.table), status=st)
    ckv.q8_rope_store(cache, k, v, plan, i64(pos) if dim else None, f32(freqs) if dim else None, counts, halves=halves,
                      norm_weight=f32(weight), eps=1e-5, weights=weights, status=st)
    with np.errstate(invalid="ignore"):
        y = bref.rope(k.float().cpu().numpy(), weight, 1e-5, freqs, pos, 0, halves)
    off = ((D + 4) / 2 + 8) * 2.0 ** -24
    got, gs, cleared = codes(cache.k), cache.k_scale.cpu().numpy(), weights.cpu().numpy()
    recs = ref.store_plan(w.rid, kv, new, w.table, T)
    for block, row, slot, cnt in recs:
        for h in range(2):
            x, s = y[row:row + cnt, h], float(gs[block, h])
            fin = np.abs(x[np.isfinite(x)]).max()
            old = float(w.ks[block, h]) if slot else 0.0
            assert s in [max(old, ref.need_scale(fin * (1 + d))) for d in (-off, off)]
            e = ref.E4M3[got[block, h, slot:slot + cnt]] * s
            assert np.array_equal(np.isnan(e), np.isnan(x))
            with np.errstate(invalid="ignore"):
                near = off * 2 * np.nanmax(np.abs(np.where(np.isnan(x), 0, x)), -1, keepdims=True)
                assert (np.isnan(x) | (np.abs(e - x) <= np.maximum(np.abs(x) * 2.0 ** -4, s * 2.0 ** -10) + near)).all()
            if slot:
                assert ref.same_codes(got[block, h, :slot], ref.round8(ref.E4M3[w.k[block, h, :slot]] * (old / s)))
        assert (cleared[block, slot:slot + cnt] == 0).all() and (cleared[block, :slot] == 5).all()
    assert (cleared == 0).sum() == n
    if not latent:
        ref.store(w.v, w.vs, v.float().cpu().numpy(), recs)
        assert ref.same_codes(codes(cache.v), w.v)
    assert int(st[0]) == 0


# --------------------------------------------------------------------------------- missing blocks, within the derived bounds
@pytest.mark.parametrize("heads,H,D,latent", [(4, 1, 128, False), (8, 2, 128, False), (64, 1, 512, True), (8, 1, 512, False),
                                              (80, 2, 256, False), (72, 1, 64, False)])
def test_missing_blocks_in_every_part_of_a_list(heads, H, D, latent):
    """Lists long enough to be split; blocks missing at the beginning, in later parts and at the end, and all of a list's."""
    w = World(1300, [1500, 60, 700], H, D, 16, latent)
    q, seq, q_lens = w.queries([1, 2, 1], heads), [1500, 60, 700], [1, 2, 1]
    lists = lists_of(w, seq, q_lens, 1, 90, ragged=False)
    first, last = w.rid[0], w.rid[2]
    w.table[first, [0, 17, 40, 41, 66, 93]] = [-3, w.blocks, -1, 0x7FFFFFFF, -0x80000000, w.blocks + 7]
    w.table[last, :44] = -3
    skip = {-3, -1, w.blocks, 0x7FFFFFFF, -0x80000000, w.blocks + 7}
    assert any(w.table[first, j] in skip for j in lists[0].ravel())
    check_attn(w, q, lists, seq, q_lens, 1, F32, skip=skip, flags=ckv.STATUS_BAD_INDEX)


@pytest.mark.parametrize("T,D", APPEND)
def test_every_append_with_a_norm_of_rows_whose_squares_overflow(T, D):
    """1e20 squared is past fp32: the mean is infinite and the row's factor 0; its neighbours are normed as ever."""
    w = World(1400 + T + D, [0], 1, D, T, True, more=T)
    x = w.r.standard_normal((T, 1, D)).astype(np.float32)
    x[3] *= 1e20
    cache, st = w.cache(), status()
    plan, counts = ckv.plan_q8_store(cache, i64(w.rid), i64([T]), i64([T]), T, i32(w.table), status=st)
    ckv.q8_rope_store(cache, torch.as_tensor(x, device=DEV), None, plan, None, None, counts, norm_weight=torch.ones(D, device=DEV), status=st)
    blk = w.table[w.rid[0], 0]
    got, s = ref.E4M3[codes(cache.k)[blk, 0]], float(cache.k_scale[blk, 0])
    assert (got[3] == 0).all() and int(st[0]) == 0
    y = bref.rope(x, np.ones(D, np.float32), 1e-6, None, None, 0, False)[:, 0]
    y[3] = 0
    off = ((D + 4) / 2 + 8) * 2.0 ** -24
    near = off * 2 * np.abs(y).max(-1, keepdims=True)
    assert (np.abs(got * s - y) <= np.maximum(np.abs(y) * 2.0 ** -4, s * 2.0 ** -10) + near).all()

"""The oracle of the rotated append and the sparse attention against independent facts, and the refusals of their entry
points (no GPU)."""
import ctypes

import numpy as np
import pytest
import torch

from compressed_kv_attention_compressplan_gb300 import build as B
from compressed_kv_attention_compressplan_gb300 import ckv
from tests import q8_blocks_ref as bref
from tests import q8_ref as ref
from tests.test_q8_ref import _arg

vp, f = ctypes.c_void_p, ctypes.c_float


@pytest.fixture(scope="module")
def lib():
    B.build()
    return ckv.load_library()


@pytest.mark.parametrize("halves", [False, True])
def test_rotation_keeps_lengths_and_products_of_equal_distances(halves):
    r = np.random.RandomState(1)
    ang = np.arange(50)[:, None] * 100.0 ** (-np.arange(16) / 16)
    freqs = np.stack([np.cos(ang), np.sin(ang)], -1)
    x, y = r.standard_normal((2, 1, 1, 64))
    at = lambda v, p: bref.rope(v, None, 0, freqs, np.array([p]), 32, halves)[0, 0]
    assert np.allclose(at(x, 0), x[0, 0])
    assert np.allclose(at(x, 33)[:32], x[0, 0, :32]) and not np.allclose(at(x, 33)[32:], x[0, 0, 32:])
    assert np.isclose(np.linalg.norm(at(x, 33)), np.linalg.norm(x))
    assert np.isclose(at(x, 40) @ at(y, 31), at(x, 17) @ at(y, 8))


def test_norm_gives_rows_of_unit_mean_square():
    x = np.random.RandomState(2).standard_normal((3, 2, 64)) * 9
    y = bref.rope(x, np.ones(64), 1e-12, None, None, 0, False)
    assert np.allclose((y * y).mean(-1), 1)


def test_scores_are_above_every_entry_s():
    r = np.random.RandomState(3)
    T, H, D = 16, 2, 64
    k = ref.round8(r.standard_normal((4, H, T, D)))
    ks = np.exp2(r.randint(-3, 3, (4, H))).astype(np.float32)
    table = np.array([[2, 0, 3, 1]])
    b = bref.bounds(np.zeros((4, H, 2, D), np.uint8), k, [0], [60], [60], table)
    q = r.standard_normal((1, 6, D))
    s, _, _ = bref.scores(b, ks, q, [0], [60], [1], [60], table, T, 1, 0.5, 5)
    z = np.einsum("hgd,hsd->hgs", q[0].reshape(H, 3, D), ref.entries(k, ks, table[0], 60)) * 0.5
    for j in range(4):
        assert (s[0, :, j] >= z[:, :, j * T:min(60, j * T + T)].max((1, 2))).all()
    assert np.isneginf(s[0, :, 4]).all()


def test_choice_takes_ties_from_below_and_nan_last():
    row = np.array([1.0, 5, np.nan, 5, -np.inf, 5, 0, 9])
    assert bref.choose(row, 8, 4, 0, 0) == [1, 3, 5, 7]
    assert bref.choose(row, 8, 3, 1, 1) == [0, 1, 7]
    assert bref.choose(row, 8, 7, 0, 0) == [0, 1, 3, 4, 5, 6, 7]
    assert bref.choose(row, 5, 5, 0, 0) == [0, 1, 2, 3, 4]


def test_attention_over_all_blocks_is_attention():
    r = np.random.RandomState(4)
    k, ks = ref.round8(r.standard_normal((3, 2, 16, 64))), np.ones((3, 2), np.float32)
    q, table = r.standard_normal((2, 4, 64)), np.array([[1, 2, 0]])
    lists = np.tile(np.array([0, 1, 2, -1]), (2, 2, 1))
    got = bref.attn(k, ks, None, None, q, lists, [0], [41], [2], [41], table, 1, 0.2)
    want = ref.attn(k, ks, None, None, q, [0], [41], [2], [41], table, 1, 0.2)
    for x, y in zip(got, want):
        assert np.allclose(x, y)


# -------------------------------------------------------------------------------------------------------- refusals
def test_rope_store_refusals(lib):
    def store(dt=1, k=vp(16), ks=256, v=None, vs=0, rows=4, pos=vp(16), w=None, eps=1e-6, fr=vp(16), most=8, begin=0,
              dim=64, plan=vp(16), cnt=None, cap=4, weights=None, cache=None):
        return lib.ckv_q8_rope_store(cache or _arg(), dt, k, ks, v, vs, rows, pos, w, f(eps), fr, most, begin, dim, 1, plan,
                                     cnt, cap, weights, None, None)

    assert store(dt=2) == -5
    assert store(dim=16) == -2
    assert store(dim=160) == -2
    assert store(dim=128, begin=16) == -2
    assert store(begin=8) == -2
    assert store(begin=0xFFFFFFF0) == -2
    assert store(ks=255) == -3      # a row is shorter than two heads of 128
    assert store(ks=257) == -3      # rows would not be aligned
    assert store(ks=1 << 32) == -3
    assert store(dt=0, ks=258) == -3
    assert store(rows=1 << 24) == -3
    assert store(cap=1 << 24) == -3
    assert store(w=vp(16), eps=0.0) == -3
    assert store(w=vp(16), eps=float("nan")) == -3
    assert store(w=vp(8)) == -4
    assert store(k=vp(8)) == -4
    assert store(v=vp(16), vs=256) == -4   # the cache has no values
    assert store(cache=_arg(v=16, vs=16)) == -4
    assert store(cache=_arg(v=16, vs=16), v=vp(16), vs=100) == -3
    assert store(pos=None) == -4
    assert store(pos=vp(4)) == -4
    assert store(fr=None) == -4
    assert store(plan=vp(8)) == -4
    assert store(cnt=vp(2)) == -4
    assert store(weights=vp(2)) == -4
    assert store(cache=_arg(T=8)) == -3
    assert store(rows=0) == 0
    assert store(cap=0) == 0


def test_bounds_refusals(lib):
    def bounds(b=vp(16), rid=vp(16), batch=2, tab=vp(16), stride=4, reqs=2, cache=None):
        return lib.ckv_q8_bounds(cache or _arg(), b, rid, vp(16), vp(16), batch, tab, stride, reqs, None, None)

    assert bounds(b=vp(8)) == -4
    assert bounds(rid=vp(4)) == -4
    assert bounds(tab=None) == -4
    assert bounds(stride=0) == -3
    assert bounds(reqs=0) == -3
    assert bounds(batch=1025) == -3
    assert bounds(cache=_arg(D=96)) == -2
    assert bounds(batch=0) == 0


def test_score_refusals(lib):
    def scores(b=vp(16), heads=8, ratio=1, scale=0.1, q=vp(16), num_q=4, rid=vp(16), seq=vp(16), batch=2, tab=vp(16), stride=4,
               width=4, out=vp(16)):
        return lib.ckv_q8_block_scores(_arg(), b, heads, ratio, f(scale), q, num_q, rid, seq, vp(16), vp(16), batch, tab,
                                       stride, 2, width, out, None, None)

    assert scores(heads=7) == -3
    assert scores(heads=0) == -3
    assert scores(heads=2 * 257) == -3
    assert scores(ratio=0) == -1
    assert scores(ratio=65537) == -1
    assert scores(scale=0.0) == -3
    assert scores(scale=float("nan")) == -3
    assert scores(num_q=1 << 24) == -3
    assert scores(width=0) == -3
    assert scores(width=1 << 31) == -3
    assert scores(batch=1025) == -3
    assert scores(b=vp(8)) == -4
    assert scores(q=vp(8)) == -4
    assert scores(rid=vp(4)) == -4
    assert scores(seq=None) == -4
    assert scores(out=vp(2)) == -4
    assert scores(tab=None) == -4
    assert scores(stride=0) == -3
    assert scores(num_q=0) == 0
    assert scores(batch=0) == 0


def test_select_refusals(lib):
    def select(s=vp(16), heads=2, width=4, T=16, ratio=1, num_q=4, seq=vp(16), batch=2, budget=3, sinks=1, recent=1,
               out=vp(16)):
        return lib.ckv_q8_block_select(s, heads, width, T, ratio, num_q, seq, vp(16), vp(16), batch, budget, sinks, recent,
                                       out, None, None)

    assert select(heads=0) == -3
    assert select(heads=257) == -3
    assert select(T=24) == -3
    assert select(ratio=0) == -1
    assert select(width=0) == -3
    assert select(budget=0) == -3
    assert select(budget=1 << 31) == -3
    assert select(sinks=2, recent=2) == -3
    assert select(sinks=0xFFFFFFFF, recent=5) == -3
    assert select(num_q=1 << 24) == -3
    assert select(batch=1025) == -3
    assert select(s=None) == -4
    assert select(seq=vp(4)) == -4
    assert select(out=vp(2)) == -4
    assert select(num_q=0) == 0
    assert select(batch=0) == 0


def test_attention_over_blocks_refusals(lib):
    size = lib.ckv_q8_attn_blocks_workspace_bytes
    work = size(_arg(), 8, 4, 3)
    assert work > 0
    assert size(_arg(), 7, 4, 3) == 0
    assert size(_arg(), 8, 4, 0) == 0
    assert size(_arg(), 8, 1 << 24, 3) == 0
    assert size(_arg(T=128), 8, 4, 1 << 24) == 0   # 2^31 entries
    assert size(_arg(), 8, 4096, 3) > 0            # more queries than a plan has requests

    def attn(heads=8, ratio=1, scale=0.1, q=vp(16), num_q=4, lists=vp(16), budget=3, rid=vp(16), seq=vp(16), batch=2, tab=vp(16),
             stride=4, dt=1, out=vp(16), lse=None, ws=vp(16), wb=work):
        return lib.ckv_q8_attn_blocks(_arg(), heads, ratio, f(scale), q, num_q, lists, budget, rid, seq, vp(16), vp(16), batch,
                                      tab, stride, 2, dt, out, lse, ws, wb, None, None)

    assert attn(heads=7) == -3
    assert attn(ratio=0) == -1
    assert attn(scale=-1.0) == -3
    assert attn(scale=float("inf")) == -3
    assert attn(dt=2) == -5
    assert attn(budget=0) == -3
    assert attn(batch=1025) == -3
    assert attn(wb=work - 1) == -3
    assert attn(q=vp(8)) == -4
    assert attn(out=vp(8)) == -4
    assert attn(ws=vp(8)) == -4
    assert attn(lse=vp(2)) == -4
    assert attn(lists=vp(2)) == -4
    assert attn(rid=vp(4)) == -4
    assert attn(seq=None) == -4
    assert attn(tab=None) == -4
    assert attn(stride=0) == -3
    assert attn(num_q=0) == 0
    assert attn(batch=0) == 0


def test_the_binding_takes_cuda_tensors_only():
    cpu = ckv.Q8Cache(torch.zeros(2, 1, 16, 64, dtype=torch.uint8).view(torch.float8_e4m3fn), torch.ones(2, 1))
    one, table = torch.zeros(1, dtype=torch.int64), torch.zeros(1, 1, dtype=torch.int32)
    q, lists = torch.zeros(1, 1, 64, dtype=torch.bfloat16), torch.zeros(1, 1, 1, dtype=torch.int32)
    for call in (lambda: ckv.q8_rope_store(cpu, q, None, torch.zeros(1, 16, dtype=torch.uint8), None, None),
                 lambda: ckv.q8_bounds(cpu, ckv.new_q8_bounds(cpu), one, one, one, table),
                 lambda: ckv.q8_block_scores(cpu, ckv.new_q8_bounds(cpu), q, 1, one, one, one, one, table, 0.1),
                 lambda: ckv.q8_block_select(torch.zeros(1, 1, 1), 16, 1, one, one, one, 1),
                 lambda: ckv.q8_attn_blocks(cpu, q, lists, 1, one, one, one, one, table, 0.1)):
        with pytest.raises(ValueError):
            call()

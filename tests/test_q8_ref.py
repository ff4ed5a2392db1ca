"""The oracle of the 8-bit cache's tests against independent facts, and the refusals of its entry points (no GPU)."""
import ctypes

import numpy as np
import pytest
import torch

from compressed_kv_attention_compressplan_gb300 import build as B
from compressed_kv_attention_compressplan_gb300 import ckv
from tests import q8_ref as ref


@pytest.fixture(scope="module")
def lib():
    B.build()
    return ckv.load_library()


def test_round8_is_the_type_s_rounding():
    g = torch.Generator().manual_seed(1)
    x = torch.randn(100000, generator=g) * torch.exp(3 * torch.randn(100000, generator=g))
    x[:600] = torch.arange(-300, 300) / 1024.0  # subnormals and their ties
    want = x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(ref.round8(x.numpy()), want)


def test_scales_are_the_smallest_powers_that_hold():
    for a, want in [(0.0, 2.0 ** -48), (448.0, 1.0), (448.0001, 2.0), (224.0, 0.5), (1e-30, 2.0 ** -48),
                    (1e30, 2.0 ** 48), (7.0, 2.0 ** -6)]:
        assert ref.need_scale(a) == want


def test_growing_a_scale_changes_only_subnormals():
    codes = np.arange(0x7F, dtype=np.uint8)
    for k in range(1, 8):
        back = ref.E4M3[ref.round8(ref.E4M3[codes] * 2.0 ** -k)] * 2.0 ** k
        normal = ref.E4M3[codes] * 2.0 ** -k >= 2.0 ** -6
        assert np.array_equal(back[normal], ref.E4M3[codes][normal])
        assert np.abs(back - ref.E4M3[codes]).max() <= 2.0 ** (k - 10)  # half a subnormal step


@pytest.mark.parametrize("ratio", [1, 4, 128])
def test_visible_counts_whole_groups(ratio):
    for seq in range(1, 300, 7):
        for q in range(1, min(seq, 9) + 1):
            for i in range(q):
                t = seq - q + i  # the query's position: it sees the groups complete by then
                assert ref.visible(seq // ratio, seq, q, i, ratio) == (t + 1) // ratio


def test_capacity_bounds_the_records():
    r = np.random.RandomState(0)
    for _ in range(300):
        T, B_ = int(r.choice([16, 32, 64, 128])), int(r.randint(1, 9))
        new = r.randint(0, 3 * T, B_)
        kv = new + r.randint(0, 5 * T, B_)
        table = np.zeros((B_, 64), np.int64)
        recs = ref.store_plan(range(B_), kv, new, table, T)
        assert len(recs) <= ckv.capacity_q8_store(B_, int(new.sum()), T)


def _arg(k=16, ks=16, v=None, vs=None, nb=8, T=16, H=2, D=128):
    return ckv.Q8CacheArg(k, ks, v, vs, nb, T, H, D)


def test_cache_descriptions_that_are_refused(lib):
    vp = ctypes.c_void_p
    ok = dict(rid=vp(16), kv=vp(16), nl=vp(16), tab=vp(16), plan=vp(16), cnt=vp(16))

    def plan(cache, batch=2, rows=4, stride=4, reqs=2, cap=4, cnt=vp(16), rid=vp(16), tab=vp(16)):
        return lib.ckv_plan_q8_store(cache, rid, ok["kv"], ok["nl"], batch, rows, tab, stride, reqs, cap, 0,
                                     ok["plan"], cnt, None, None)

    assert plan(_arg(D=96)) == -2
    assert plan(_arg(D=1024)) == -2
    assert plan(_arg(T=8)) == -3
    assert plan(_arg(T=256)) == -3
    assert plan(_arg(H=0)) == -3
    assert plan(_arg(H=257)) == -3
    assert plan(_arg(nb=0)) == -3
    assert plan(_arg(k=8)) == -4
    assert plan(_arg(k=None)) == -4
    assert plan(_arg(v=16)) == -4          # v without v_scale
    assert plan(_arg(v=24, vs=16)) == -4
    assert plan(None) == -4
    assert plan(_arg(), batch=1025) == -3
    assert plan(_arg(), rows=1 << 24) == -3
    assert plan(_arg(), stride=0) == -3
    assert plan(_arg(), reqs=0) == -3
    assert plan(_arg(), cnt=vp(8)) == -4
    assert plan(_arg(), rid=vp(12)) == -4
    assert plan(_arg(), tab=vp(2)) == -4


def test_store_refusals(lib):
    vp = ctypes.c_void_p

    def store(cache, dt=1, k=vp(16), v=None, rows=4, plan=vp(16), cap=4):
        return lib.ckv_q8_store(cache, dt, k, v, rows, plan, None, cap, None, None)

    assert store(_arg(), dt=7) == -5
    assert store(_arg(), k=vp(8)) == -4
    assert store(_arg(), v=vp(16)) == -4               # rows for values that the cache does not have
    assert store(_arg(v=16, vs=16)) == -4              # and the other way round
    assert store(_arg(), plan=vp(8)) == -4
    assert store(_arg(), rows=0) == 0
    assert store(_arg(), cap=0) == 0


def test_store_reset_refusals(lib):
    vp = ctypes.c_void_p

    def store(w, dt=1, rows=4, k=vp(16)):
        return lib.ckv_q8_store_reset(_arg(), dt, k, None, rows, vp(16), None, 4, w, None, None)

    assert store(None) == -4
    assert store(vp(18)) == -4
    assert store(vp(16), dt=7) == -5
    assert store(vp(16), k=vp(8)) == -4
    assert store(vp(16), rows=0) == 0


def test_attention_refusals(lib):
    vp, f = ctypes.c_void_p, ctypes.c_float
    need = lib.ckv_q8_attn_plan_bytes(_arg(), 8, 2, 4)
    work = lib.ckv_q8_attn_workspace_bytes(_arg(), 8, 2, 4)
    assert need > 0 and work > 0
    assert lib.ckv_q8_attn_plan_bytes(_arg(), 7, 2, 4) == 0       # 7 heads over 2
    assert lib.ckv_q8_attn_plan_bytes(_arg(D=100), 8, 2, 4) == 0

    def plan(heads=8, ratio=1, batch=2, num_q=4, bytes_=need, p=vp(16), rid=vp(16)):
        return lib.ckv_plan_q8_attn(_arg(), heads, ratio, rid, vp(16), vp(16), vp(16), batch, num_q, p, bytes_, None,
                                    None)

    assert plan(heads=7) == -3
    assert plan(heads=0) == -3
    assert plan(heads=2 * 257) == -3
    assert plan(ratio=0) == -1
    assert plan(ratio=65537) == -1
    assert plan(batch=1025) == -3
    assert plan(bytes_=need - 1) == -3
    assert plan(p=vp(8)) == -4
    assert plan(rid=vp(4)) == -4
    assert plan(num_q=(1 << 24) - 1, heads=512, bytes_=1 << 62) == -3   # 2^32 rows of a kv head

    def attn(heads=8, ratio=1, scale=0.1, q=vp(16), batch=2, num_q=4, tab=vp(16), stride=4, reqs=2, pb=need, dt=1,
             out=vp(16), lse=None, ws=vp(16), wb=work):
        return lib.ckv_q8_attn(_arg(), heads, ratio, f(scale), q, batch, num_q, tab, stride, reqs, vp(16), pb, dt,
                               out, lse, ws, wb, None, None)

    assert attn(heads=9) == -3
    assert attn(ratio=0) == -1
    assert attn(scale=0.0) == -3
    assert attn(scale=float("nan")) == -3
    assert attn(scale=float("inf")) == -3
    assert attn(dt=2) == -5
    assert attn(q=vp(8)) == -4
    assert attn(out=vp(8)) == -4
    assert attn(lse=vp(2)) == -4
    assert attn(ws=vp(8)) == -4
    assert attn(wb=work - 1) == -3
    assert attn(pb=need - 1) == -3
    assert attn(stride=0) == -3
    assert attn(tab=None) == -4
    assert attn(num_q=0) == 0
    assert attn(batch=0) == 0


def test_weigh_and_evict_refusals(lib):
    vp, f = ctypes.c_void_p, ctypes.c_float

    def weigh(heads=8, ratio=1, scale=0.1, decay=1.0, q=vp(16), lse=vp(16), w=vp(16), num_q=4, batch=2):
        return lib.ckv_q8_weigh(_arg(), heads, ratio, f(scale), f(decay), q, lse, num_q, vp(16), vp(16), vp(16),
                                vp(16), batch, vp(16), 4, 2, w, None, None)

    assert weigh(heads=7) == -3
    assert weigh(ratio=0) == -1
    assert weigh(scale=-1.0) == -3
    assert weigh(decay=1.5) == -3
    assert weigh(decay=-0.1) == -3
    assert weigh(decay=float("nan")) == -3
    assert weigh(q=vp(8)) == -4
    assert weigh(lse=None) == -4
    assert weigh(w=None) == -4
    assert weigh(num_q=0) == 0
    assert weigh(batch=0) == 0

    def evict(budget=8, sinks=0, recent=0, batch=2, kept=vp(16), nl=vp(16), dst=vp(16), ds=4):
        return lib.ckv_q8_evict(_arg(), vp(16), vp(16), vp(16), batch, vp(16), 4, dst, ds, 2, budget, sinks, recent,
                                kept, nl, None, None)

    assert evict(budget=0) == -3
    assert evict(sinks=5, recent=4) == -3
    assert evict(sinks=0xFFFFFFFF, recent=2) == -3
    assert evict(budget=1 << 24) == -3
    assert evict(ds=0) == -3
    assert evict(dst=None) == -4
    assert evict(kept=None) == -4
    assert evict(nl=vp(12)) == -4
    assert evict(batch=0) == 0
    assert evict(batch=1025) == -3


def test_record_sizes():
    assert ctypes.sizeof(ckv.Q8CacheArg) == 48


def test_capacity_refuses_counts_past_32_bits(lib):
    for args in ((1 << 32, 4, 16), (1, (1 << 32) + 4, 16), (1, -1, 16), (1, 4, (1 << 32) + 16)):
        with pytest.raises(ValueError):
            ckv.capacity_q8_store(*args)


def test_the_binding_takes_cuda_tensors_only():
    cpu = ckv.Q8Cache(torch.zeros(2, 1, 16, 64, dtype=torch.uint8).view(torch.float8_e4m3fn), torch.ones(2, 1))
    i64 = torch.zeros(1, dtype=torch.int64)
    with pytest.raises(ValueError):
        ckv.plan_q8_store(cpu, i64, i64, i64, 0, torch.zeros(1, 1, dtype=torch.int32))
    with pytest.raises(ValueError):
        ckv.plan_q8_store(cpu._replace(k=torch.zeros(2, 1, 16, 64)), i64, i64, i64, 0,
                          torch.zeros(1, 1, dtype=torch.int32))
    with pytest.raises(ValueError):
        ckv.plan_q8_store(cpu._replace(v=cpu.k), i64, i64, i64, 0, torch.zeros(1, 1, dtype=torch.int32))

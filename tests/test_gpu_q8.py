"""The 8-bit paged cache on the GPU against its 64-bit oracle: plans and codes bit for bit, attention and weights
within bounds derived from the roundings that the kernels make."""
import math

import numpy as np
import pytest
import torch

from compressed_kv_attention_compressplan_gb300 import ckv
from tests import q8_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ckv.load_library()


def i64(a):
    return torch.as_tensor(np.asarray(a, np.int64), device=DEV)


def i32(a):
    return torch.as_tensor(np.asarray(a, np.int32), device=DEV)


class World:
    """A pool and tables of a batch: the requests' blocks in random order, everything unused poisoned."""

    def __init__(self, seed, lens, H, D, T, latent=False, spread=0.3, k_spread=None, extra=3, more=0):
        r = self.r = np.random.RandomState(seed)
        self.T, self.H, self.D, B = T, H, D, len(lens)
        self.lens = np.asarray(lens, np.int64)
        per = np.maximum(1, -(-(self.lens + more) // T))
        self.blocks = int(per.sum()) + extra
        order = r.permutation(self.blocks)
        self.rid = r.permutation(B + 2)[:B]
        self.table = np.full((B + 2, int(per.max()) + 1), -1, np.int32)
        at = 0
        for b in range(B):
            self.table[self.rid[b], :per[b]] = order[at:at + per[b]]
            at += per[b]
        self.spare = [int(x) for x in order[at:]]
        self.k, self.ks = self._side(spread if k_spread is None else k_spread)
        self.v, self.vs = (None, None) if latent else self._side(spread)

    def _side(self, spread):
        pool = np.full((self.blocks, self.H, self.T, self.D), 0x7F, np.uint8)
        scale = np.full((self.blocks, self.H), np.nan, np.float32)
        for b, n in enumerate(self.lens):
            for j in range(-(-int(n) // self.T)):
                blk, cnt = self.table[self.rid[b], j], min(self.T, int(n) - j * self.T)
                x = self.r.standard_normal((self.H, cnt, self.D)) * np.exp2(
                    np.round(spread * self.r.standard_normal((self.H, 1, 1))))
                for h in range(self.H):
                    s = ref.need_scale(np.abs(x[h]).max())
                    scale[blk, h] = s
                    pool[blk, h, :cnt] = ref.round8(x[h] / s)
        return pool, scale

    def cache(self):
        def up(pool, scale):
            return torch.as_tensor(pool, device=DEV).view(torch.float8_e4m3fn), torch.as_tensor(scale, device=DEV)
        return ckv.Q8Cache(*up(self.k, self.ks), *((None, None) if self.v is None else up(self.v, self.vs)))

    def queries(self, q_lens, heads, size=1.5):
        n = int(np.sum(q_lens))
        return torch.as_tensor(self.r.standard_normal((n, heads, self.D)) * size).bfloat16()


def codes(t):
    return t.view(torch.uint8).cpu().numpy()


def status():
    return ckv.new_status(DEV)


def attn_bounds(D, lens_max, out, lse, mag, big, flat, vmax, out_bf16, eight_bit=False):
    """Worst cases: D products and lens_max weighted values summed in fp32 with truncated additions (2^-23 each), the
    exponent's argument a few roundings of its size (2^-22), the weights rounded to fp16 (2^-11), weights under
    2^-31 of the largest dropped (of values up to twice vmax), bf16 output (2^-8).  eight_bit: with more than 32 rows
    at 256 channels, or 16 at 512, the fp16 weights are three e5m2 terms (each leaves 2^-3 of what it is given: 2^-9), dropped under
    2^-17 / 2^6 = 2^-23, and a query value is off by up to 2^-17 of its row's largest."""
    eps = big * (D + 8) * 2.0 ** -23 + (big * 1.5 + 60) * 2.0 ** -22 + (flat * 2.0 ** -17 if eight_bit else 0)
    e = eps[..., None]
    weight, drop = (2.0 ** -9 + 2.0 ** -10, 2.0 ** -23) if eight_bit else (2.0 ** -11, 2.0 ** -31)
    tol = mag * (weight + 2 * e + (lens_max + 32) * 2.0 ** -23) + 2 * lens_max * drop * vmax
    tol = tol + np.abs(out) * (2.0 ** -8 if out_bf16 else 2.0 ** -23) + 1e-30
    with np.errstate(invalid="ignore"):
        return tol, eps + np.where(np.isfinite(lse), np.abs(lse) + 60, 0) * 2.0 ** -22


def eight_bit(w, q_lens, heads):
    return w.D >= 256 and int(np.sum(q_lens)) * (heads // w.H) > (32 if w.D == 256 else 16) * len(q_lens)


def run_attn(w, q, seq, q_lens, heads, ratio, out_dtype=torch.bfloat16, scale=None, lens=None, **kw):
    scale = 1 / math.sqrt(w.D) if scale is None else scale
    lens = w.lens if lens is None else lens
    cache, st = w.cache(), status()
    table = i32(w.table)
    plan = ckv.plan_q8_attn(cache, heads, ratio, i64(w.rid), i64(seq), i64(q_lens), i64(lens), q.shape[0], status=st)
    out, lse = ckv.q8_attn(cache, q.to(DEV), plan, table, scale, out_dtype=out_dtype, status=st, **kw)
    torch.cuda.synchronize()
    return cache, plan, out, lse, int(st[0])


def check_attn(w, q, seq, q_lens, heads, ratio, out_dtype=torch.bfloat16):
    scale = 1 / math.sqrt(w.D)
    cache, plan, out, lse, st = run_attn(w, q, seq, q_lens, heads, ratio, out_dtype)
    assert st == 0
    qn = q.float().numpy()
    want, wl, mag, big, flat = ref.attn(w.k, w.ks, w.v, w.vs, qn, w.rid, seq, q_lens, w.lens, w.table, ratio, scale)
    pool, sc = (w.k, w.ks) if w.v is None else (w.v, w.vs)
    vmax = max([np.abs(ref.entries(pool, sc, w.table[w.rid[b]], int(n))).max() for b, n in enumerate(w.lens) if n] + [0])
    tol, ltol = attn_bounds(w.D, max(1, w.lens.max()), want, wl, mag, big, flat, vmax, out_dtype == torch.bfloat16,
                            eight_bit(w, q_lens, heads))
    got, gl = out.float().cpu().numpy(), lse.cpu().numpy()
    assert np.isfinite(got).all()
    worst = np.abs(got - want) - tol
    assert (worst <= 0).all(), (worst.max(), np.unravel_index(worst.argmax(), worst.shape))
    assert np.array_equal(np.isneginf(gl), np.isneginf(wl))
    fin = np.isfinite(wl)
    assert (np.abs(gl[fin] - wl[fin]) <= ltol[fin]).all()
    return cache, plan, out, lse


# ------------------------------------------------------------------------------------------------------------ store
STORE = [  # lens before, new, H, D, T, latent, dtype
    ([0], [1], 1, 512, 64, True, torch.bfloat16),
    ([0, 5, 63, 64, 130], [0, 1, 1, 1, 0], 1, 512, 64, True, torch.bfloat16),
    ([3, 16, 0, 31], [40, 1, 16, 33], 2, 128, 16, False, torch.bfloat16),
    ([0, 127, 128, 1], [300, 2, 128, 127], 3, 64, 128, False, torch.float32),
    ([7] * 20, [1] * 20, 2, 256, 32, False, torch.float32),
    ([0, 0, 0], [0, 0, 5], 8, 128, 32, False, torch.bfloat16),
]


@pytest.mark.parametrize("case", range(len(STORE)))
def test_store(case):
    before, new, H, D, T, latent, dt = STORE[case]
    w = World(10 + case, before, H, D, T, latent, more=max(new))
    kv = w.lens + np.asarray(new)
    n = int(np.sum(new))
    rows = [torch.as_tensor(w.r.standard_normal((n, H, D)) * np.exp2(np.round(3 * w.r.standard_normal((n, 1, 1))))).to(dt)
            for _ in range(1 if latent else 2)]
    cache, st = w.cache(), status()
    plan, counts = ckv.plan_q8_store(cache, i64(w.rid), i64(kv), i64(new), n, i32(w.table), status=st, pad_invalid=True)
    recs = ref.store_plan(w.rid, kv, new, w.table, T)
    got = plan.cpu().numpy().view(np.uint32).reshape(-1, 4)
    assert counts.cpu().tolist()[:2] == [len(recs), n]
    assert [(int(x[0]), int(x[1]), int(x[2] & 0xFFFF), int(x[2] >> 16)) for x in got[:len(recs)]] == recs
    assert (got[len(recs):] == 0xFFFFFFFF).all()
    ckv.q8_store(cache, rows[0].to(DEV), None if latent else rows[1].to(DEV), plan, counts, status=st)
    torch.cuda.synchronize()
    assert int(st[0]) == 0
    ref.store(w.k, w.ks, rows[0].float().numpy(), recs)
    assert ref.same_codes(codes(cache.k), w.k) and np.array_equal(cache.k_scale.cpu().numpy(), w.ks, equal_nan=True)
    if not latent:
        ref.store(w.v, w.vs, rows[1].float().numpy(), recs)
        assert ref.same_codes(codes(cache.v), w.v) and np.array_equal(cache.v_scale.cpu().numpy(), w.vs, equal_nan=True)


def test_store_token_by_token_equals_one_prefill():
    """Rows whose magnitudes grow, stored one step at a time, against one store: the same scales, and codes that
    differ only where a value was rounded as a subnormal on the way."""
    H, D, T, n = 2, 128, 32, 100
    r = np.random.RandomState(3)
    x = torch.as_tensor(r.standard_normal((n, H, D)) * np.exp2(np.linspace(-6, 6, n))[:, None, None]).bfloat16().to(DEV)
    table = i32(np.arange(4)[None, ::-1].copy())
    one, many = (ckv.new_q8_cache(4, H, T, D, latent=True) for _ in range(2))
    p = ckv.plan_q8_store(one, i64([0]), i64([n]), i64([n]), n, table)
    ckv.q8_store(one, x, None, *p)
    for i in range(n):
        p = ckv.plan_q8_store(many, i64([0]), i64([i + 1]), i64([1]), 1, table)
        ckv.q8_store(many, x[i:i + 1].contiguous(), None, *p)
    torch.cuda.synchronize()
    assert torch.equal(one.k_scale, many.k_scale)
    a, b = (ref.E4M3[codes(c.k)] for c in (one, many))
    normal = np.abs(a) >= 2.0 ** -5
    assert np.array_equal(a[normal], b[normal])
    assert np.abs(a - b).max() <= 2.0 ** -9  # a subnormal step: two roundings of half of one


def test_store_of_infinities_nan_and_extremes():
    x = torch.zeros(4, 1, 64)
    x[0, 0, :6] = torch.tensor([math.inf, -math.inf, math.nan, 448.0, -3.0, 0.0])
    x[1, 0, :2] = torch.tensor([3.0e38, -1e-40])
    x[2, 0, 0] = 1e-30
    cache, st = ckv.new_q8_cache(4, 1, 16, 64, latent=True), status()
    kv = [1, 1, 1, 1]
    plan, counts = ckv.plan_q8_store(cache, i64(range(4)), i64(kv), i64(kv), 4, i32(np.arange(4)[:, None]), status=st)
    ckv.q8_store(cache, x.to(DEV), None, plan, counts, status=st)
    torch.cuda.synchronize()
    k, s = np.full((4, 1, 16, 64), 0, np.uint8), np.ones((4, 1), np.float32)
    ref.store(k, s, x.numpy(), ref.store_plan(range(4), kv, kv, np.arange(4)[:, None], 16))
    assert int(st[0]) == 0
    assert ref.same_codes(codes(cache.k), k) and np.array_equal(cache.k_scale.cpu().numpy(), s)
    assert s[:, 0].tolist() == [1.0, 2.0 ** 48, 2.0 ** -48, 2.0 ** -48]


def test_store_flags_bad_data_and_touches_nothing_for_it():
    w = World(5, [4, 4, 4, 4, 4], 1, 64, 16, True)
    before = w.k.copy()
    kv, new = np.array([5, 3, 5, 5, 999]), np.array([1, 4, -1, 1, 1])
    rid = w.rid.copy()
    rid[3] = 77
    table = w.table.copy()
    table[rid[0], 0] = w.blocks  # past the pool
    cache, st = w.cache(), status()
    plan, counts = ckv.plan_q8_store(cache, i64(rid), i64(kv), i64(new), 7, i32(table), status=st, pad_invalid=True)
    ckv.q8_store(cache, torch.ones(7, 1, 64, device=DEV), None, plan, counts, status=st)
    torch.cuda.synchronize()
    assert int(st[0]) == ckv.STATUS_BAD_LENGTH | ckv.STATUS_BAD_INDEX
    assert np.array_equal(codes(cache.k), before)


def test_store_total_mismatch_and_capacity_are_flagged():
    cache = ckv.new_q8_cache(4, 1, 16, 64, latent=True)
    table = i32([[0, 1], [2, 3]])
    st = status()
    plan, counts = ckv.plan_q8_store(cache, i64([0, 1]), i64([3, 3]), i64([3, 3]), 5, table, status=st)
    ckv.q8_store(cache, torch.ones(5, 1, 64, device=DEV), None, plan, counts, status=st)
    torch.cuda.synchronize()
    assert int(st[0]) == ckv.STATUS_BAD_TOTAL
    assert codes(cache.k)[0].any() and not codes(cache.k)[2].any()  # request 1's rows do not all exist
    st = status()
    ckv.plan_q8_store(cache, i64([0, 1]), i64([3, 3]), i64([3, 3]), 6, table, capacity=1, status=st)
    assert int(st[0]) == ckv.STATUS_CAPACITY


# -------------------------------------------------------------------------------------------------------- attention
ATTN = [  # lens, q_lens, heads, H, D, T, latent, ratio
    ([1], [1], 1, 1, 64, 16, False, 1),
    ([777], [1], 8, 1, 128, 16, False, 1),
    ([0, 1, 15, 16, 17, 300], [1] * 6, 8, 2, 128, 16, False, 1),
    ([5, 129, 640], [1, 4, 3], 16, 2, 64, 16, False, 1),
    ([200, 0, 33], [1, 2, 1], 14, 2, 256, 32, False, 1),
    ([130, 517], [1, 1], 64, 1, 512, 64, True, 4),
    ([260, 64], [2, 5], 20, 1, 512, 128, False, 1),
    ([90, 70], [3, 1], 7, 1, 128, 64, True, 128),
    ([3, 40], [40, 60], 4, 2, 128, 16, False, 1),       # more queries than entries: early ones see nothing
    ([300, 65], [100, 65], 8, 4, 128, 64, False, 1),    # a prefill chunk
    ([50], [33], 12, 4, 64, 16, True, 4),
    ([48], [9], 3, 3, 256, 16, True, 1),
    ([410], [1], 4, 4, 64, 128, False, 1),
    ([600, 33, 128], [200, 33, 1], 16, 1, 64, 32, False, 1),
    ([300, 20], [90, 20], 24, 2, 256, 64, False, 1),
    ([260], [70], 16, 1, 512, 64, True, 4),
    ([257], [40], 16, 1, 512, 32, False, 1),
    ([129], [129], 128, 1, 128, 64, True, 1),
    ([700, 150], [64, 30], 6, 2, 512, 32, False, 1),
    ([1000], [1], 96, 1, 512, 128, True, 1),
    ([390], [300], 4, 4, 128, 16, False, 1),
    # rows on both sides of where another kernel takes over
    ([200], [16], 4, 1, 64, 32, False, 1),
    ([200], [13], 5, 1, 64, 32, False, 1),
    ([170, 30], [12, 12], 8, 2, 128, 16, False, 1),
    ([170], [7], 7, 1, 128, 16, True, 1),
    ([100], [4], 4, 1, 256, 64, True, 1),
    ([100], [17], 1, 1, 256, 64, False, 1),
    ([333], [1], 17, 1, 512, 64, True, 2),
    ([300, 40], [13, 13], 5, 1, 512, 64, True, 1),
    ([300], [13], 5, 1, 256, 32, False, 1),
    # up to eight rows a request on average, some requests with more
    ([300, 1, 70], [1, 2, 1], 4, 1, 256, 64, True, 1),
    ([200, 30], [3, 1], 4, 1, 64, 16, True, 1),
    ([500], [1], 7, 1, 128, 32, True, 4),
    ([90, 60, 0], [5, 1, 0], 4, 1, 512, 32, False, 1),
    ([40, 700], [3, 1], 8, 2, 128, 64, False, 1),
    # more rows on both sides of where another kernel takes over
    ([170], [16], 4, 1, 128, 16, False, 1),
    ([170], [13], 5, 1, 128, 16, True, 1),
    ([100], [8], 4, 1, 256, 64, False, 1),
    ([100], [11], 3, 1, 256, 64, True, 1),
]


def _seq(lens, q_lens, ratio):
    return np.maximum(np.asarray(lens) * ratio + np.arange(len(lens)) * 3 % ratio, q_lens)


@pytest.mark.parametrize("case", range(len(ATTN)))
def test_attn(case):
    lens, q_lens, heads, H, D, T, latent, ratio = ATTN[case]
    w = World(100 + case, lens, H, D, T, latent)
    q = w.queries(q_lens, heads)
    check_attn(w, q, _seq(lens, q_lens, ratio), q_lens, heads, ratio, torch.float32 if case % 2 else torch.bfloat16)


@pytest.mark.parametrize("heads,H,D,latent", [(4, 1, 128, False), (8, 1, 512, True), (2, 2, 64, False), (64, 1, 128, True),
                                                (64, 1, 512, True), (70, 1, 256, False)])
def test_attn_over_a_long_cache(heads, H, D, latent):
    """One row tile split over many CTAs, and joined."""
    w = World(7, [9001, 20], H, D, 128, latent)
    check_attn(w, w.queries([1, 1], heads), [9001, 20], [1, 1], heads, 1)


@pytest.mark.parametrize("D,q_len", [(64, 1), (128, 1), (256, 1), (512, 1), (128, 70), (64, 70), (256, 70), (512, 70)])
def test_attn_with_scales_far_apart(D, q_len):
    """Blocks whose value scales differ by many powers of two, and scores that peak."""
    w = World(8, [400, 90], 1, D, 16, False, spread=9, k_spread=1)
    check_attn(w, w.queries([q_len, q_len], 4, 2.0), [400, 90], [q_len, q_len], 4, 1, torch.float32)


def test_attn_of_large_and_tiny_queries():
    w = World(9, [100, 100, 100], 1, 128, 16, False)
    q = w.queries([1, 1, 1], 2)
    q[0] *= 2.0 ** 100
    q[1] *= 2.0 ** -120
    q[2] = 0
    cache, plan, out, lse, st = run_attn(w, q, [100] * 3, [1] * 3, 2, 1, torch.float32)
    want, wl, _, _, _ = ref.attn(w.k, w.ks, w.v, w.vs, q.double().numpy(), w.rid, [100] * 3, [1] * 3, w.lens, w.table, 1,
                              1 / math.sqrt(128))
    got = out.cpu().numpy()
    # one entry takes all of the first query: its value, exactly; the others weigh all entries alike
    assert np.array_equal(got[0], want[0].astype(np.float32))
    assert np.abs(got[1:] - want[1:]).max() <= 2.0 ** -11 * 4
    assert np.abs(lse.cpu().numpy()[1:] - wl[1:]).max() <= 2.0 ** -18


def test_attn_of_equal_scores_is_the_mean():
    w = World(19, [333], 1, 128, 16, False)
    w.k[:] = np.where(w.k == 0x7F, 0x7F, 0)
    _, _, out, lse, st = run_attn(w, w.queries([1], 4), [333], [1], 4, 1, torch.float32)
    mean = ref.entries(w.v, w.vs, w.table[w.rid[0]], 333)[0].mean(0)
    assert np.abs(out.cpu().numpy()[0] - mean).max() <= 1e-5  # equal weights are powers of two times one number
    assert np.abs(lse.cpu().numpy() - math.log(333)).max() <= 2.0 ** -20


@pytest.mark.parametrize("heads,D,latent", [(4, 128, False), (4, 64, False), (4, 256, True), (4, 512, True), (32, 128, False),
                                            (16, 64, True), (16, 256, False), (8, 512, True), (8, 512, False)])
def test_nan_values_reach_only_queries_that_see_them(heads, D, latent):
    n, q_lens = 70, [9]
    w = World(11, [n], 1, D, 16, latent)
    at = n - 4  # hidden from the first five of nine queries
    blk = w.table[w.rid[0], at // 16]
    pool = w.k if latent else w.v
    pool[blk, 0, at % 16, 5] = 0xFF
    q = w.queries(q_lens, heads)
    _, _, out, lse, st = run_attn(w, q, [n], q_lens, heads, 1, torch.float32)
    assert st == 0
    got = np.isnan(out.cpu().numpy())
    sees = np.arange(9) + (n - 9) >= at
    want = np.zeros_like(got)
    want[sees, :, 5] = True
    if latent:
        want[sees] = True  # the key is NaN too: the whole row's weights are
    assert np.array_equal(got, want)


@pytest.mark.parametrize("heads,D", [(4, 64), (3, 128), (4, 256), (1, 512)])
@pytest.mark.parametrize("latent", [False, True])
def test_nan_values_of_few_rows(heads, D, latent):
    w = World(16, [70, 33], 1, D, 16, latent)
    for b, at in ((0, 69), (1, 20)):  # request 0's is hidden from the first of its two queries, request 1's from none
        (w.k if latent else w.v)[w.table[w.rid[b], at // 16], 0, at % 16, 7] = 0xFF
    q = w.queries([2, 2], heads)
    _, _, out, lse, st = run_attn(w, q, [70, 33], [2, 2], heads, 1, torch.float32)
    assert st == 0
    got = np.isnan(out.cpu().numpy())
    want = np.zeros_like(got)
    want[1:, :, slice(None) if latent else 7] = True
    assert np.array_equal(got, want)


@pytest.mark.parametrize("heads,D", [(8, 64), (12, 64), (4, 128), (16, 128), (2, 256), (12, 256), (8, 512), (16, 512)])
@pytest.mark.parametrize("latent", [False, True])
def test_nan_values_in_the_first_tile_of_items_that_follow_one_another(heads, D, latent):
    """A thousand requests of a few entries, several to a CTA, each with one NaN in its only tile: a warp marks it as
    soon as the copies are in, and the marks of the item before must be gone by then, and its own must stay."""
    B = 1000
    lens = 5 + np.arange(B) % 11
    w = World(18, lens, 1, D, 16, latent)
    chan = np.arange(B) * 37 % D
    for b in range(0, B, 2):  # every other request's
        (w.k if latent else w.v)[w.table[w.rid[b], 0], 0, b % lens[b], chan[b]] = 0xFF
    _, _, out, lse, st = run_attn(w, w.queries([1] * B, heads), lens, [1] * B, heads, 1, torch.float32)
    assert st == 0
    want = np.zeros((B, heads, D), bool)
    for b in range(0, B, 2):
        want[b, :, slice(None) if latent else chan[b]] = True
    assert np.array_equal(np.isnan(out.cpu().numpy()), want)
    assert np.array_equal(np.isnan(lse.cpu().numpy()), np.repeat((np.arange(B) % 2 == 0)[:, None] & latent, heads, 1))


@pytest.mark.parametrize("heads,D", [(48, 512), (40, 256), (96, 128), (80, 64), (300, 128)])
@pytest.mark.parametrize("n", [17, 128, 1000])
def test_nan_values_in_the_last_slot(heads, D, n):
    """A NaN in the very last channel of the newest entry's value, the last that a tile's values bring: seen by the last query alone,
    hidden from the one before."""
    B = 64
    H = -(-heads // 256)
    w = World(21, [n] * B, H, D, 16, False)
    for b in range(B):
        w.v[w.table[w.rid[b], (n - 1) // 16], H - 1, (n - 1) % 16, D - 1] = 0x7F
    _, _, out, lse, st = run_attn(w, w.queries([2] * B, heads), [n] * B, [2] * B, heads, 1, torch.float32)
    assert st == 0 and bool(torch.isfinite(lse).all())
    want = np.zeros(out.shape, bool)
    want[1::2, (H - 1) * (heads // H):, D - 1] = True
    assert np.array_equal(np.isnan(out.cpu().numpy()), want)


@pytest.mark.parametrize("heads,D,latent", [(64, 512, True), (48, 512, False), (64, 256, True), (40, 256, False), (96, 128, False),
                                             (80, 64, True)])
def test_nan_values_beside_shares_without_entries(heads, D, latent):
    """Tiles of about a hundred entries, cut so that some CTAs end with a tile's start and none of its entries, after a
    tile with a NaN: what the one marked must not show in the other's part."""
    B = 500
    lens = 80 + np.arange(B) % 40
    w = World(20, lens, 1, D, 16, latent)
    for b in range(0, B, 2):
        (w.k if latent else w.v)[w.table[w.rid[b], 4], 0, b % 16, 9] = 0xFF
    _, plan, out, lse, st = run_attn(w, w.queries([1] * B, heads), lens, [1] * B, heads, 1, torch.float32)
    assert st == 0
    raw = plan.buffer.cpu().numpy()
    head = raw[:64].view(np.uint32)
    off = (64 + 4 * (int(head[8]) + 1) + 63) // 64 * 64
    off = (off + 4 * int(head[8]) + 63) // 64 * 64
    it = raw[off:off + 48 * int(head[0])].view(np.uint32).reshape(-1, 12)
    assert (it[:, 4] == it[:, 5]).any()  # there are such shares
    want = np.zeros((B, heads, D), bool)
    for b in range(0, B, 2):
        want[b, :, slice(None) if latent else 9] = True
    assert np.array_equal(np.isnan(out.cpu().numpy()), want)


@pytest.mark.parametrize("heads,D", [(4, 64), (4, 128), (3, 256), (1, 512), (32, 64), (32, 128), (16, 256), (8, 512), (64, 512)])
@pytest.mark.parametrize("n", [70, 128, 131, 2500])
def test_lse_of_a_latent_row_that_sees_a_nan_is_nan(heads, D, n):
    """A NaN entry of a latent cache is a NaN score of the rows that see it: their lse is NaN as well, whichever kernel
    takes them and wherever in a tile the entry lies; the others' is that of a cache without it."""
    w = World(22, [n, 60], 1, D, 16, True)
    q, lens = w.queries([9, 9], heads), [n, 60]
    _, _, out0, lse0, st0 = run_attn(w, q, lens, [9, 9], heads, 1, torch.float32)
    at = n - 4  # hidden from the first five of nine queries
    w.k[w.table[w.rid[0], at // 16], 0, at % 16, 5] = 0xFF
    cache, _, out, lse, st = run_attn(w, q, lens, [9, 9], heads, 1, torch.float32)
    assert st == st0 == 0
    sees = np.zeros(18, bool)
    sees[:9] = np.arange(9) + (n - 9) >= at
    got = lse.cpu().numpy()
    assert np.array_equal(np.isnan(got), np.repeat(sees[:, None], heads, 1))
    assert np.array_equal(np.isnan(out.cpu().numpy()), np.broadcast_to(sees[:, None, None], out.shape))
    assert np.array_equal(got[~sees], lse0.cpu().numpy()[~sees])
    assert np.array_equal(out.cpu().numpy()[~sees], out0.cpu().numpy()[~sees])


@pytest.mark.parametrize("depth", [14.3, 18.3, 21.3, 24.3])
@pytest.mark.parametrize("D,latent,heads,n,first", [(512, True, 64, 3000, 0), (512, False, 32, 3000, 1700), (256, False, 48, 3000, 5),
                                                 (256, True, 64, 3000, 2900), (512, True, 64, 100001, 3), (128, True, 96, 3000, 0),
                                                 (128, False, 8, 3000, 40)])
def test_many_small_weights_behind_a_large_one(depth, D, latent, heads, n, first):
    """One entry with nearly all of a row's weight and none of the values, and many with 2^-depth of it: what the many
    give is there.  Every SM has whole requests, so a row's entries stand under one reference.

    A weight is off by 2^-9 of it (three e5m2 terms, each leaves 2^-3) and 2^-11 (fp16), and by e5m2's last 2^-17, where the
    row's largest is 2^12 or more.  The fp16 kernels keep to the same bounds."""
    B, T = 304, 128
    scale = depth * math.log(2) / (8 * 14)
    r = np.random.RandomState(23)
    blocks = -(-n // T)
    vals = ref.round8(r.uniform(0.5, 2.0, (n, D)))
    k = np.zeros((n, D), np.uint8)
    k[:, 0] = ref.round8(np.full(n, -6.0))
    k[first, 0] = ref.round8(8.0)
    if latent:
        k[:, 1:] = vals[:, 1:]
        k[first, 1:] = 0
    vals[first] = 0

    def pool(x):
        full = np.zeros((blocks * T, D), np.uint8)
        full[:n] = x
        t = torch.as_tensor(full.reshape(blocks, 1, T, D), device=DEV).view(torch.float8_e4m3fn)
        return t, torch.ones(blocks, 1, device=DEV)

    cache = ckv.Q8Cache(*pool(k), *((None, None) if latent else pool(vals)))
    table = i32(np.arange(blocks)[None])
    q = torch.zeros(B, heads, D, dtype=torch.bfloat16, device=DEV)
    q[:, :, 0] = 8.0
    st, one = status(), i64([1] * B)
    plan = ckv.plan_q8_attn(cache, heads, 1, i64([0] * B), i64([n] * B), one, i64([n] * B), B, status=st)
    out, lse = ckv.q8_attn(cache, q, plan, table, scale, out_dtype=torch.float32, status=st)
    torch.cuda.synchronize()
    assert int(st[0]) == 0
    s = np.full(n, -6.0 * 8 * scale)
    s[first] = 64 * scale
    p = np.exp(s - s[first])
    v = ref.E4M3[k if latent else vals]
    want = (p @ v) / p.sum()
    mag = (p @ np.abs(v)) / p.sum()
    eps = 64 * scale * (D + 8) * 2.0 ** -23 + 64 * 2.0 ** -22
    tol = mag * (2.0 ** -9 + 2.0 ** -11 + 2 * eps + (n + 32) * 2.0 ** -23) + n * 2.0 ** -29 * np.abs(np.delete(v, first, 0)).max(0) / p.sum()
    got = out.double().cpu().numpy()
    sl = slice(1, None) if latent else slice(None)  # a latent cache's channel 0 is the score's
    err = np.abs(got - want)[..., sl] - tol[sl]
    assert (err <= 0).all(), (err.max(), want[5], got[0, 0, 5], tol[5])
    assert np.abs(lse.cpu().numpy() - (s[first] + math.log(p.sum()))).max() <= 4 * eps


@pytest.mark.parametrize("heads,D,latent", [(4, 64, False), (4, 128, True), (3, 256, False), (1, 512, True), (40, 64, True), (40, 128, False),
                                             (40, 256, False), (40, 256, True), (20, 512, False), (64, 512, True)])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_queries_that_are_not_finite(heads, D, latent, bad):
    """inf * k is an infinity of either sign or NaN, so the softmax over such scores is NaN, in that row alone."""
    w = World(24, [300, 40], 1, D, 16, latent)
    q = w.queries([2, 2], heads)
    _, _, out0, lse0, st0 = run_attn(w, q, [300, 40], [2, 2], heads, 1, torch.float32)
    q[1, heads - 1, 7] = q[2, 0, D - 1] = bad
    _, _, out, lse, st = run_attn(w, q, [300, 40], [2, 2], heads, 1, torch.float32)
    assert st == st0 == 0
    nan = np.zeros((4, heads), bool)
    nan[1, heads - 1] = nan[2, 0] = True
    assert np.array_equal(np.isnan(lse.cpu().numpy()), nan)
    assert np.array_equal(np.isnan(out.cpu().numpy()), np.repeat(nan[..., None], D, 2))
    assert np.array_equal(lse.cpu().numpy()[~nan], lse0.cpu().numpy()[~nan])
    assert np.array_equal(out.cpu().numpy()[~nan], out0.cpu().numpy()[~nan])


def test_plan_covers_every_tile_once():
    """The items of a plan, read back: for each tile they tile its entries, and parts are numbered without gaps.  The last
    six seeds' lengths add up to more than 32 bits hold."""
    for seed in range(18):
        r = np.random.RandomState(seed)
        B, H, heads = int(r.randint(1, 40)), int(r.choice([1, 2, 8])), 8 * int(r.choice([1, 2]))
        D = int(r.choice([64, 128, 256, 512]))
        lens = r.randint(0, int(r.choice([20, 3000, 60000])), B)
        q_lens = r.randint(0, 5, B)
        q_lens[0] = max(q_lens[0], int(r.choice([1, 200])))
        ratio = int(r.choice([1, 4, 128]))
        if seed >= 12:
            lens, ratio = r.randint(1 << 29, 1 << 30, B), 1
        seq = _seq(lens, q_lens, ratio)
        pool = torch.zeros(1, H, 16, D, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
        cache = ckv.Q8Cache(pool, torch.ones(1, H, device=DEV))
        st = status()
        plan = ckv.plan_q8_attn(cache, heads, ratio, i64(range(B)), i64(seq), i64(q_lens), i64(lens), int(q_lens.sum()),
                                status=st)
        torch.cuda.synchronize()
        assert int(st[0]) == 0
        raw = plan.buffer.cpu().numpy()
        head = raw[:64].view(np.uint32)
        n_items, ctas, parts, splits, rows, group, _, _, cap = (int(x) for x in head[:9])
        first = raw[64:64 + 4 * (cap + 1)].view(np.uint32)[:ctas + 1].astype(int)
        off = (64 + 4 * (cap + 1) + 63) // 64 * 64
        split = raw[off:off + 4 * cap].view(np.uint32)[:splits].astype(int)
        off = (off + 4 * cap + 63) // 64 * 64
        it = raw[off:off + 48 * n_items].view(np.uint32).reshape(-1, 12).astype(np.int64)
        assert first[0] == 0 and first[-1] == n_items and (np.diff(first) >= 1).all()
        tiles, part = {}, 0
        for k, x in enumerate(it):
            tiles.setdefault((x[0], x[3]), []).append((k, x))
        want = [(b, row) for b in range(B) for row in range(0, int(q_lens[b]) * group, rows)]
        assert sorted(tiles) == want
        starts = np.concatenate([[0], np.cumsum(q_lens)])
        got_splits = []
        for (b, row0), xs in sorted(tiles.items(), key=lambda t: t[1][0][0]):
            last = min(int(q_lens[b]) - 1, (row0 + rows - 1) // group)
            see = ref.visible(int(lens[b]), int(seq[b]), int(q_lens[b]), last, ratio)
            at = 0
            for c, (k, x) in enumerate(xs):
                assert x[1] == starts[b] and x[2] == q_lens[b] and x[6] == lens[b] and x[9] == c and x[10] == len(xs)
                assert x[4] == at and x[4] % 16 == 0 and x[5] >= x[4]
                at = x[5]
                assert x[8] == (0xFFFFFFFF if len(xs) == 1 else part)
            assert at == see
            if len(xs) > 1:
                got_splits.append(xs[0][0])
                part += len(xs)
        assert got_splits == list(split) and part == parts <= 2 * cap


def test_attn_flags_bad_data():
    w = World(12, [40, 40, 40], 1, 128, 16, False)
    q = w.queries([1, 1, 1], 2)
    table = w.table.copy()
    table[w.rid[1], 1] = w.blocks + 5
    cache, st = w.cache(), status()
    sent = torch.full((3, 2, 128), 7.0, device=DEV)
    plan = ckv.plan_q8_attn(cache, 2, 1, i64(w.rid), i64([40, 40, 3]), i64([1, 1, 1]), i64([40, 40, -1]), 3, status=st)
    ckv.q8_attn(cache, q.to(DEV), plan, i32(table), 0.1, out=sent, status=st)
    torch.cuda.synchronize()
    assert int(st[0]) == ckv.STATUS_BAD_LENGTH | ckv.STATUS_BAD_INDEX
    good = ref.attn(w.k, w.ks, w.v, w.vs, q.float().numpy(), w.rid, [40] * 3, [1] * 3, w.lens, w.table, 1, 0.1)[0]
    got = sent.cpu().numpy()
    assert np.abs(got[0] - good[0]).max() <= 0.01   # an ordinary request
    assert (got[2] == 7.0).all()                    # a refused one is left as it was
    # the entries of the block that does not exist do not count: the others' attention
    z = np.einsum("hd,sd->hs", q[1].float().numpy().astype(np.float64), ref.entries(w.k, w.ks, w.table[w.rid[1]], 40)[0]) * 0.1
    z[:, 16:32] = -np.inf
    p = np.exp(z - z.max(1, keepdims=True))
    want = (p / p.sum(1, keepdims=True)) @ ref.entries(w.v, w.vs, w.table[w.rid[1]], 40)[0]
    assert np.abs(got[1] - want).max() <= 0.01


@pytest.mark.parametrize("D,latent", [(64, False), (128, True), (256, False), (512, True)])
def test_missing_blocks_do_not_count_on_the_tensor_cores(D, latent):
    """The first 128 entries and later ones in blocks that do not exist: the other entries' attention."""
    n, heads = 300, 64
    w = World(16, [n], 1, D, 16, latent)
    q = w.queries([1], heads)
    good = w.table.copy()
    for j in [0, 1, 2, 3, 4, 5, 6, 7, 12]:
        w.table[w.rid[0], j] = [-1, w.blocks, 1 << 30][j % 3]
    _, _, out, lse, st = run_attn(w, q, [n], [1], heads, 1, torch.float32, scale=0.1)
    assert st == ckv.STATUS_BAD_INDEX
    k = ref.entries(w.k, w.ks, good[w.rid[0]], n)[0]
    v = k if latent else ref.entries(w.v, w.vs, good[w.rid[0]], n)[0]
    z = q[0].double().numpy() @ k.T * 0.1
    z[:, :128] = z[:, 192:208] = -np.inf
    p = np.exp(z - z.max(1, keepdims=True))
    want = (p / p.sum(1, keepdims=True)) @ v
    assert np.abs(out.cpu().numpy()[0] - want).max() <= 0.02
    assert np.abs(lse.cpu().numpy()[0] - np.log(p.sum(1)) - z.max(1)).max() <= 0.002


def test_scores_far_under_zero_on_the_tensor_cores():
    """Every score near -400: the weights are relative to the row's own largest, wherever that is."""
    for D, latent in [(128, False), (512, True)]:
        w = World(17, [260], 1, D, 16, latent, spread=0)
        k = np.zeros((w.blocks, 1, 16, D))
        r = np.random.RandomState(3)
        k[:] = r.standard_normal(k.shape)
        k[..., 0] = -8.0
        codes_ = ref.round8(k / 0.0625)
        w.k = np.where(w.k == 0x7F, 0x7F, codes_).astype(np.uint8)
        w.ks[:] = 0.0625
        q = torch.zeros(1, 64, D)
        q[:, :, 0] = 50.0
        q[:, :, 1:] = torch.as_tensor(r.standard_normal((1, 64, D - 1)) * 0.1)
        q = q.bfloat16()
        _, _, out, lse, st = run_attn(w, q, [260], [1], 64, 1, torch.float32, scale=1.0)
        assert st == 0
        want, wl, mag, big, flat = ref.attn(w.k, w.ks, w.v, w.vs, q.double().numpy(), w.rid, [260], [1], w.lens, w.table, 1, 1.0)
        tol, ltol = attn_bounds(D, 260, want, wl, mag, big, flat, 40.0, False, D >= 256)
        assert (wl < -380).all() and (np.abs(lse.cpu().numpy() - wl) <= ltol).all()
        assert (np.abs(out.cpu().numpy() - want) <= tol).all()


def test_attn_refuses_a_plan_of_another_shape():
    w = World(13, [40], 1, 128, 16, False)
    cache, st = w.cache(), status()
    plan = ckv.plan_q8_attn(cache, 2, 1, i64(w.rid), i64([40]), i64([1]), i64([40]), 1)
    out = torch.full((1, 4, 128), 7.0, device=DEV)
    ckv.q8_attn(cache, w.queries([1], 4).to(DEV), plan._replace(n_heads=4), i32(w.table), 0.1, out=out, status=st)
    torch.cuda.synchronize()
    assert int(st[0]) == ckv.STATUS_BAD_INDEX and (out == 7.0).all()


def test_rows_after_the_last_request_are_left_alone():
    w = World(14, [40], 1, 128, 16, False)
    cache, st = w.cache(), status()
    q = w.queries([3], 2)
    out, lse = torch.full((3, 2, 128), 7.0, device=DEV), torch.full((3, 2), 7.0, device=DEV)
    plan = ckv.plan_q8_attn(cache, 2, 1, i64(w.rid), i64([40]), i64([2]), i64([40]), 3, status=st)
    ckv.q8_attn(cache, q.to(DEV), plan, i32(w.table), 0.1, out=out, lse=lse, status=st)
    torch.cuda.synchronize()
    assert int(st[0]) == ckv.STATUS_BAD_TOTAL
    assert (out[2] == 7.0).all() and (lse[2] == 7.0).all() and not (out[:2] == 7.0).any()


def test_requests_whose_queries_do_not_all_exist_are_dropped():
    w = World(15, [40, 30, 20], 1, 128, 16, False)
    cache, st = w.cache(), status()
    q = w.queries([5], 2)
    out, lse = torch.full((5, 2, 128), 7.0, device=DEV), torch.full((5, 2), 7.0, device=DEV)
    args = i64(w.rid), i64([40, 30, 20]), i64([2, 4, 1]), i64([40, 30, 20])
    plan = ckv.plan_q8_attn(cache, 2, 1, *args, 5, status=st)
    ckv.q8_attn(cache, q.to(DEV), plan, i32(w.table), 0.1, out=out, lse=lse, status=st)
    torch.cuda.synchronize()
    assert int(st[0]) == ckv.STATUS_BAD_TOTAL
    assert (out[2:] == 7.0).all() and (lse[2:] == 7.0).all() and not (out[:2] == 7.0).any()
    weights, st = torch.zeros(w.blocks, 16, device=DEV), status()
    ckv.q8_weigh(cache, q.to(DEV), lse, weights, 1, *args, i32(w.table), 0.1, status=st)
    torch.cuda.synchronize()
    assert int(st[0]) == ckv.STATUS_BAD_TOTAL
    got = weights.cpu().numpy()
    assert got[w.table[w.rid[0], :3]].sum() > 0 and got[w.table[w.rid[1], :2]].sum() == 0 == got[w.table[w.rid[2], :2]].sum()


def test_offsets_past_32_bits():
    """Blocks at the far end of a pool of more than 2^32 bytes."""
    T, H, D = 128, 8, 512
    blocks = (1 << 32) // (T * H * D) + 40
    k = torch.zeros(blocks, H, T, D, dtype=torch.uint8, device=DEV)
    ks = torch.ones(blocks, H, device=DEV)
    cache, st = ckv.Q8Cache(k.view(torch.float8_e4m3fn), ks), status()
    n = 300
    used = [blocks - 1, blocks - 17, blocks - 5, 3]
    table = i32([used])
    x = torch.as_tensor(np.random.RandomState(0).standard_normal((n, H, D))).bfloat16()
    p = ckv.plan_q8_store(cache, i64([0]), i64([n]), i64([n]), n, table, status=st)
    ckv.q8_store(cache, x.to(DEV), None, *p, status=st)
    q = torch.as_tensor(np.random.RandomState(1).standard_normal((1, 16, D))).bfloat16()
    plan = ckv.plan_q8_attn(cache, 16, 1, i64([0]), i64([n]), i64([1]), i64([n]), 1, status=st)
    out, lse = ckv.q8_attn(cache, q.to(DEV), plan, table, 0.05, out_dtype=torch.float32, status=st)
    weights = torch.zeros(blocks, T, device=DEV)
    ckv.q8_weigh(cache, q.to(DEV), lse, weights, 1, i64([0]), i64([n]), i64([1]), i64([n]), table, 0.05, status=st)
    dst = i32([[blocks - 2]])
    kept, nl = ckv.q8_evict(cache, weights, i64([0]), i64([n]), table, dst, 100, 1, 20, status=st)
    torch.cuda.synchronize()
    assert int(st[0]) == 0
    small = {b: i for i, b in enumerate(used + [blocks - 2])}
    sk = np.stack([codes(cache.k[b]) for b in small])
    ss = np.stack([ks[b].cpu().numpy() for b in small])
    tab = np.arange(4)[None]
    wk, ws = np.zeros_like(sk), np.ones_like(ss)
    ref.store(wk, ws, x.float().numpy(), ref.store_plan([0], [n], [n], tab, T))
    assert ref.same_codes(sk[:4], wk[:4]) and np.array_equal(ss[:4], ws[:4])
    want, _, mag, _, _ = ref.attn(wk, ws, None, None, q.float().numpy(), [0], [n], [1], [n], tab, 1, 0.05)
    assert (np.abs(out.cpu().numpy() - want) <= mag * 2.0 ** -10 + 1e-6).all()
    w4 = np.stack([weights[b].cpu().numpy() for b in small])
    assert abs(w4[:4].sum() - 16) < 1e-3
    keep = ref.evict([(wk, ws)], w4.copy(), [0], [n], tab, np.array([[4]]), 100, 1, 20)
    assert kept.cpu().numpy()[0].tolist() == keep[0]
    assert ref.same_codes(sk[4][:, :100], wk[4][:, :100])


# ---------------------------------------------------------------------------------------------------------- weights
@pytest.mark.parametrize("case", range(len(ATTN)))
@pytest.mark.parametrize("decay", [1.0, 0.5])
def test_weigh(case, decay):
    lens, q_lens, heads, H, D, T, latent, ratio = ATTN[case]
    w = World(200 + case, lens, H, D, T, latent)
    q, seq = w.queries(q_lens, heads), _seq(lens, q_lens, ratio)
    scale = 1 / math.sqrt(D)
    cache, _, _, lse, _ = run_attn(w, q, seq, q_lens, heads, ratio)
    start = w.r.random_sample((w.blocks, T)).astype(np.float32)
    weights, st = torch.as_tensor(start, device=DEV), status()
    ckv.q8_weigh(cache, q.to(DEV), lse, weights, ratio, i64(w.rid), i64(seq), i64(q_lens), i64(lens), i32(w.table),
                 scale, decay, status=st)
    torch.cuda.synchronize()
    assert int(st[0]) == 0
    qn = q.float().numpy()
    want = ref.weigh(w.k, w.ks, start, qn, lse.cpu().numpy(), w.rid, seq, q_lens, w.lens, w.table, ratio, scale, decay)
    big = ref.attn(w.k, w.ks, w.v, w.vs, qn, w.rid, seq, q_lens, w.lens, w.table, ratio, scale)[3].max()
    # a score's D products (2^-23 each), the exponent's argument (a few roundings of its size), one sum over the rows
    rel = big * (D + 8) * 2.0 ** -23 + (3 * big + 60) * 2.0 ** -23 + int(np.sum(q_lens)) * heads * 2.0 ** -24
    got = weights.cpu().numpy()
    assert (np.abs(got - want) <= rel * np.abs(want) + 2.0 ** -24).all()
    untouched = want == start
    assert np.array_equal(got[untouched], start[untouched])


def test_weights_sum_to_the_heads_and_overwrite():
    w = World(31, [500, 60, 0], 2, 128, 32, False)
    q_lens, heads = [3, 1, 1], 8
    q = w.queries(q_lens, heads)
    cache, _, _, lse, _ = run_attn(w, q, [500, 60, 1], q_lens, heads, 1)
    weights = torch.full((w.blocks, 32), float("nan"), device=DEV)
    args = (1, i64(w.rid), i64([500, 60, 1]), i64(q_lens), i64(w.lens), i32(w.table), 1 / math.sqrt(128))
    ckv.q8_weigh(cache, q.to(DEV), lse, weights, *args, decay=0.0)
    got = weights.cpu().numpy()
    for b, n in enumerate([500, 60]):
        x = np.array([got[w.table[w.rid[b], p // 32], p % 32] for p in range(n)])
        assert abs(x.sum() - q_lens[b] * heads) <= 1e-4 * q_lens[b] * heads
    assert np.isnan(got).sum() == w.blocks * 32 - 560
    again = torch.full((w.blocks, 32), float("nan"), device=DEV)
    ckv.q8_weigh(cache, q.to(DEV), lse, again, *args, decay=0.0)
    assert torch.equal(weights.nan_to_num(-1), again.nan_to_num(-1))  # bit for bit


def test_weights_of_slots_that_are_used_again():
    """A pool whose weights hold what earlier owners received (NaN among it): entries stored with the weights start at
    0, also behind the last entry that an eviction kept, and every other slot is left as it was."""
    H, D, T, heads, scale = 2, 64, 16, 4, 0.125
    r = np.random.RandomState(32)
    cache, st = ckv.new_q8_cache(16, H, T, D), status()
    old = r.random_sample((16, T)).astype(np.float32) * 100
    old[3, 2] = old[5] = np.nan
    weights = torch.as_tensor(old, device=DEV)
    table, dst = i32([[5, 0, 3], [9, 1, 12]]), i32([[2, 14], [7, 11]])
    rid = i64([0, 1])

    def rows(n):
        return [torch.as_tensor(r.standard_normal((n, H, D))).bfloat16().to(DEV) for _ in range(2)]

    def step(kv, new, tab):
        plan, counts = ckv.plan_q8_store(cache, rid, i64(kv), i64(new), int(np.sum(new)), tab, status=st)
        ckv.q8_store(cache, *rows(int(np.sum(new))), plan, counts, status=st, weights=weights)

    want = old.copy()
    step([35, 20], [35, 20], table)
    for blocks, n in (([5, 0, 3], 35), ([9, 1, 12], 20)):
        for p in range(n):
            want[blocks[p // T], p % T] = 0
    assert np.array_equal(weights.cpu().numpy(), want, equal_nan=True)
    q = torch.as_tensor(r.standard_normal((2, heads, D))).bfloat16().to(DEV)
    one = i64([1, 1])
    plan = ckv.plan_q8_attn(cache, heads, 1, rid, i64([35, 20]), one, i64([35, 20]), 2, status=st)
    _, lse = ckv.q8_attn(cache, q, plan, table, scale, status=st)
    ckv.q8_weigh(cache, q, lse, weights, 1, rid, i64([35, 20]), one, i64([35, 20]), table, scale, status=st)
    got = weights.cpu().numpy()
    for blocks, n in (([5, 0, 3], 35), ([9, 1, 12], 20)):
        assert abs(sum(got[blocks[p // T], p % T] for p in range(n)) - heads) <= 1e-4
    kept, lens = ckv.q8_evict(cache, weights, rid, i64([35, 20]), table, dst, 18, 1, 4, status=st)
    before = weights.cpu().numpy()
    step([21, 19], [3, 1], dst)
    want = before.copy()
    want[14, 2:5] = want[11, 2] = 0
    assert lens.tolist() == [18, 18] and np.array_equal(weights.cpu().numpy(), want, equal_nan=True)
    torch.cuda.synchronize()
    assert int(st[0]) == 0
    with pytest.raises(ValueError):
        ckv.q8_store(cache, *rows(1), torch.zeros(1, 16, dtype=torch.uint8, device=DEV), weights=weights[:, :8])


# ----------------------------------------------------------------------------------------------------------- evict
EVICT = [  # lens, budget, sinks, recent, H, D, T, latent
    ([100], 40, 4, 10, 1, 64, 16, True),
    ([1500, 512, 0, 1, 513], 512, 4, 128, 1, 512, 64, True),
    ([300, 77, 200], 77, 0, 0, 2, 128, 32, False),
    ([300, 90], 64, 30, 34, 2, 128, 128, False),   # nothing to choose: sinks and recent fill the budget
    ([64] * 5, 1, 0, 1, 3, 256, 16, False),
    ([64] * 5, 1, 1, 0, 8, 64, 16, False),
    ([2500, 2100], 2000, 0, 5, 1, 64, 16, True),
]


@pytest.mark.parametrize("case", range(len(EVICT)))
@pytest.mark.parametrize("kind", ["spread", "ties", "odd"])
def test_evict(case, kind):
    lens, budget, sinks, recent, H, D, T, latent = EVICT[case]
    out_per = [-(-min(n, budget) // T) for n in lens]
    w = World(300 + case, lens, H, D, T, latent, spread=2, extra=sum(out_per) + 2)
    dst = np.full((w.table.shape[0], max(1, max(out_per))), -1, np.int32)
    at = 0
    for b, n in enumerate(out_per):
        dst[w.rid[b], :n] = w.spare[at:at + n]
        at += n
    if kind == "spread":
        weights = np.exp(4 * w.r.standard_normal((w.blocks, T))).astype(np.float32)
    elif kind == "ties":
        weights = w.r.randint(0, 3, (w.blocks, T)).astype(np.float32) * np.where(w.r.rand(w.blocks, T) < 0.5, -1, 1).astype(np.float32)
    else:
        weights = w.r.choice(np.array([np.nan, np.inf, -np.inf, 0.0, -0.0, 1e-42, -3.0, 5.0], np.float32), (w.blocks, T))
    cache, st, dw = w.cache(), status(), torch.as_tensor(weights, device=DEV)
    kept, nl = ckv.q8_evict(cache, dw, i64(w.rid), i64(lens), i32(w.table), i32(dst), budget, sinks, recent, status=st)
    torch.cuda.synchronize()
    assert int(st[0]) == 0
    pools = [(w.k, w.ks)] + ([] if latent else [(w.v, w.vs)])
    want = ref.evict(pools, weights, w.rid, lens, w.table, dst, budget, sinks, recent)
    assert nl.cpu().tolist() == [len(x) for x in want]
    for b, x in enumerate(want):
        assert kept.cpu().numpy()[b].tolist() == x + [-1] * (budget - len(x))
    assert np.array_equal(dw.cpu().numpy(), weights, equal_nan=True)
    assert ref.same_codes(codes(cache.k), w.k) and np.array_equal(cache.k_scale.cpu().numpy(), w.ks, equal_nan=True)
    if not latent:
        assert ref.same_codes(codes(cache.v), w.v) and np.array_equal(cache.v_scale.cpu().numpy(), w.vs, equal_nan=True)


def test_evict_of_more_entries_than_shared_memory_holds():
    n, budget = 70001, 5000
    T, blocks, out = 128, -(-70001 // 128), -(-5000 // 128)
    r = np.random.RandomState(4)
    weights = r.randint(0, 4000, (blocks + out, T)).astype(np.float32)  # many ties
    cache = ckv.new_q8_cache(blocks + out, 1, T, 64, latent=True)
    dw, st = torch.as_tensor(weights, device=DEV), status()
    table, dst = np.arange(blocks)[None], blocks + np.arange(out)[None]
    kept, nl = ckv.q8_evict(cache, dw, i64([0]), i64([n]), i32(table), i32(dst), budget, 7, 100, status=st)
    want = ref.evict_choice(weights[:blocks].reshape(-1)[:n], budget, 7, 100)
    assert int(st[0]) == 0 and nl.item() == budget and kept.cpu().numpy()[0].tolist() == want
    assert np.array_equal(dw[blocks:].cpu().numpy().reshape(-1)[:budget], weights[:blocks].reshape(-1)[want])


def test_evict_flags_bad_data():
    w = World(15, [40, 40, 40], 1, 64, 16, True, extra=8)
    dst = np.full((w.table.shape[0], 2), -1, np.int32)
    dst[w.rid[0]] = w.spare[:2]
    dst[w.rid[1]] = w.spare[2:4]
    table = w.table.copy()
    table[w.rid[0], 1] = -3          # a source block that does not exist
    cache, st = w.cache(), status()
    weights = torch.rand(w.blocks, 16, device=DEV)
    kept, nl = ckv.q8_evict(cache, weights, i64(w.rid), i64([40, 40, 10 ** 6]), i32(table), i32(dst), 20, 2, 4, status=st)
    torch.cuda.synchronize()
    assert int(st[0]) == ckv.STATUS_BAD_LENGTH | ckv.STATUS_BAD_INDEX
    assert nl.cpu().tolist() == [20, 20, 0] and (kept[2] == -1).all()


def test_evict_with_entries_in_blocks_that_do_not_exist():
    """Such an entry weighs as NaN does (only the others are kept while there are enough); one that is kept all the same, here a
    first entry, leaves its new slot as it was."""
    w = World(25, [64], 1, 64, 16, True, extra=4)
    table = w.table.copy()
    table[w.rid[0], 0], table[w.rid[0], 2] = -1, w.blocks  # entries 0 .. 15 and 32 .. 47
    dst = np.full((w.table.shape[0], 2), -1, np.int32)
    dst[w.rid[0]] = w.spare[:2]
    cache, st = w.cache(), status()
    weights = torch.rand(w.blocks, 16, device=DEV) + 1
    before, wb = codes(cache.k).copy(), weights.cpu().numpy().copy()
    kept, nl = ckv.q8_evict(cache, weights, i64(w.rid), i64([64]), i32(table), i32(dst), 20, 1, 3, status=st)
    torch.cuda.synchronize()
    assert int(st[0]) == ckv.STATUS_BAD_INDEX and nl.tolist() == [20]
    keep = kept.cpu().numpy()[0]
    place = lambda p: (w.table[w.rid[0], p // 16], p % 16)
    free = [p for p in list(range(16, 32)) + list(range(48, 61))]
    best = sorted(sorted(free, key=lambda p: -wb[place(p)])[:16])
    assert keep.tolist() == [0] + best + [61, 62, 63]
    after, wa = codes(cache.k), weights.cpu().numpy()
    d0 = dst[w.rid[0], 0]
    assert np.array_equal(after[d0, 0, 0], before[d0, 0, 0]) and wa[d0, 0] == wb[d0, 0]
    for i, p in enumerate(keep):
        if i:
            assert wa[dst[w.rid[0], i // 16], i % 16] == wb[place(p)]


# -------------------------------------------------------------------------------------------------------- together
def test_a_request_s_life():
    """Compressed rows through norm + RoPE into the cache, attention, weights, eviction, and on with the next rows and
    attention over what was kept: every step against the oracle."""
    hd, heads, T, ratio = 128, 16, 16, 4
    r = np.random.RandomState(21)
    B, steps = 3, 12
    rid = np.array([2, 0, 1])
    cache, st = ckv.new_q8_cache(40, 1, T, hd, latent=True), status()
    st_c = status()  # the compressor's planner flags the last step's request without tokens; the cache's do not
    k, ks = np.zeros((40, 1, T, hd), np.uint8), np.ones((40, 1), np.float32)
    table, dst = np.arange(18).reshape(3, 6), 18 + np.arange(18).reshape(3, 6)
    weights, wref = torch.zeros(40, T, device=DEV), np.zeros((40, T))
    state = torch.zeros(3 * 8, 4 * hd, dtype=torch.bfloat16, device=DEV)
    ape = torch.as_tensor(r.standard_normal((8, hd)) * 0.1).bfloat16().to(DEV)
    norm_w = torch.ones(hd, device=DEV)
    ang = np.arange(400)[:, None] * 10000.0 ** (-np.arange(0, 64, 2) / 64)
    freqs = torch.as_tensor(np.stack([np.cos(ang), np.sin(ang)], -1).astype(np.float32), device=DEV)
    seq, kv = np.array([0, 0, 0]), np.array([0, 0, 0])
    scale = 1 / math.sqrt(hd)

    def step(ext, tab):
        nonlocal seq, kv
        ext = np.asarray(ext)
        seq = seq + ext
        n = int(ext.sum())
        x = torch.as_tensor(r.standard_normal((n, 4 * hd))).bfloat16().to(DEV)
        out, plan_c, _, counts = ckv.prefill_step(4, hd, state, x, ape, i64(rid), i64(seq), i64(ext), ckv.OUT_COMPACT,
                                                  torch.float32, status=st_c)
        new = seq // ratio - (seq - ext) // ratio
        m = int(new.sum())
        rows = torch.zeros(max(m, 1), hd, dtype=torch.bfloat16, device=DEV)
        loc = np.full(n, -1, np.int64)
        at = row = 0
        for b in range(B):
            for p in range(seq[b] - ext[b], seq[b]):
                if (p + 1) % ratio == 0:
                    loc[row] = at
                    at += 1
                row += 1
        if m:
            ckv.norm_rope_store_prefill(4, out, plan_c, counts, norm_w, 1e-6, freqs, i64(loc), rows, status=st)
        kv = kv + new
        rows3 = rows[:m].view(m, 1, hd)
        if m:
            p = ckv.plan_q8_store(cache, i64(rid), i64(kv), i64(new), m, i32(tab), status=st)
            ckv.q8_store(cache, rows3, None, *p, status=st)
            ref.store(k, ks, rows3.float().cpu().numpy(), ref.store_plan(rid, kv, new, tab, T))
        torch.cuda.synchronize()
        assert ref.same_codes(codes(cache.k), k)
        q = torch.as_tensor(r.standard_normal((n, heads, hd)) * 1.5).bfloat16()
        plan = ckv.plan_q8_attn(cache, heads, ratio, i64(rid), i64(seq), i64(ext), i64(kv), n, status=st)
        o, lse = ckv.q8_attn(cache, q.to(DEV), plan, i32(tab), scale, status=st)
        want, wl, mag, big, flat = ref.attn(k, ks, None, None, q.float().numpy(), rid, seq, ext, kv, tab, ratio, scale)
        tol, _ = attn_bounds(hd, 200, want, wl, mag, big, flat, 448 * ks.max(), True)
        assert (np.abs(o.float().cpu().numpy() - want) <= tol).all()
        ckv.q8_weigh(cache, q.to(DEV), lse, weights, ratio, i64(rid), i64(seq), i64(ext), i64(kv), i32(tab), scale,
                     status=st)
        wref[:] = ref.weigh(k, ks, wref, q.float().numpy(), lse.cpu().numpy(), rid, seq, ext, kv, tab, ratio, scale, 1.0)
        assert np.abs(weights.cpu().numpy() - wref).max() <= 1e-3

    step([130, 301, 77], table)
    for _ in range(steps):
        step([1, 1, 1], table)
    kept, nl = ckv.q8_evict(cache, weights, i64(rid), i64(kv), i32(table), i32(dst), 30, 2, 8, status=st)
    wref[:] = weights.cpu().numpy()
    want = ref.evict([(k, ks)], wref, rid, kv, table, dst, 30, 2, 8)
    # the kernel chose by its own weights, evict() above moved the oracle's by the same ones
    w0 = weights.cpu().numpy()
    assert [x for x in nl.cpu().tolist()] == [len(x) for x in want]
    for b in range(B):
        assert kept.cpu().numpy()[b, :len(want[b])].tolist() == want[b]
    assert np.array_equal(w0[18:], wref[18:].astype(np.float32))
    assert ref.same_codes(codes(cache.k), k)
    kv = nl.cpu().numpy()
    for _ in range(steps):
        step([1, 1, 1], dst)
    assert int(st_c[0]) == 0
    step([5, 0, 9], dst)
    assert int(st[0]) == 0 and int(st_c[0]) == ckv.STATUS_BAD_LENGTH


def test_captured_step_replays_with_new_lengths_and_beside_another():
    """Plan, store, attention and weights in one graph, replayed after the lengths and rows on the device changed;
    two graphs with workspaces of their own run at the same time on two streams."""
    H, D, T, heads = 2, 128, 16, 8
    scale = 0.1

    class Side:
        def __init__(self, seed):
            self.w = World(seed, [100, 37], H, D, T, False, more=40)
            self.cache = self.w.cache()
            self.rid, self.kv, self.one, self.seq = i64(self.w.rid), i64([101, 38]), i64([1, 1]), i64([101, 38])
            self.table = i32(self.w.table)
            self.k = torch.zeros(2, H, D, dtype=torch.bfloat16, device=DEV)
            self.v, self.q = torch.zeros_like(self.k), torch.zeros(2, heads, D, dtype=torch.bfloat16, device=DEV)
            self.weights = torch.zeros(self.w.blocks, T, device=DEV)
            self.st = status()
            self.ws = ckv.q8_attn_workspace(self.cache, heads, 2, 2)

        def run(self):
            p = ckv.plan_q8_store(self.cache, self.rid, self.kv, self.one, 2, self.table, status=self.st)
            ckv.q8_store(self.cache, self.k, self.v, *p, status=self.st)
            plan = ckv.plan_q8_attn(self.cache, heads, 1, self.rid, self.seq, self.one, self.kv, 2, status=self.st)
            self.out, self.lse = ckv.q8_attn(self.cache, self.q, plan, self.table, scale, workspace=self.ws, status=self.st)
            ckv.q8_weigh(self.cache, self.q, self.lse, self.weights, 1, self.rid, self.seq, self.one, self.kv, self.table,
                         scale, status=self.st)

        def capture(self):
            s = torch.cuda.Stream()
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                self.run()
            torch.cuda.current_stream().wait_stream(s)
            torch.cuda.synchronize()
            self.graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(self.graph):
                self.run()
            # back to the start
            for x, y in zip(self.cache, self.w.cache()):
                x.view(torch.uint8).copy_(y.view(torch.uint8))
            self.weights.zero_()

    a, b = Side(41), Side(42)
    for s in (a, b):
        s.capture()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for step in range(30):
        fed = []
        for s in (a, b):
            k, v = (torch.as_tensor(s.w.r.standard_normal((2, H, D))).bfloat16() for _ in range(2))
            q = torch.as_tensor(s.w.r.standard_normal((2, heads, D)) * 1.5).bfloat16()
            s.k.copy_(k), s.v.copy_(v), s.q.copy_(q)
            s.kv.copy_(i64([101 + step, 38 + step])), s.seq.copy_(s.kv)
            fed.append((k, v, q))
        torch.cuda.synchronize()
        for s, stream in zip((a, b), streams):
            with torch.cuda.stream(stream):
                s.graph.replay()
        torch.cuda.synchronize()
        for s, (k, v, q) in zip((a, b), fed):
            w, kv = s.w, [101 + step, 38 + step]
            recs = ref.store_plan(w.rid, kv, [1, 1], w.table, T)
            ref.store(w.k, w.ks, k.float().numpy(), recs)
            ref.store(w.v, w.vs, v.float().numpy(), recs)
            assert ref.same_codes(codes(s.cache.k), w.k) and ref.same_codes(codes(s.cache.v), w.v)
            want, wl, mag, big, flat = ref.attn(w.k, w.ks, w.v, w.vs, q.float().numpy(), w.rid, kv, [1, 1], kv, w.table, 1, scale)
            tol, ltol = attn_bounds(D, 200, want, wl, mag, big, flat, 32.0, True)
            assert (np.abs(s.out.float().cpu().numpy() - want) <= tol).all()
            assert (np.abs(s.lse.cpu().numpy() - wl) <= ltol).all()
    for s in (a, b):
        assert int(s.st[0]) == 0
        assert abs(float(s.weights.sum()) - 30 * 2 * heads) < 1e-2


def test_on_another_stream():
    w = World(51, [300], 1, 128, 16, False)
    q = w.queries([1], 4).to(DEV)
    _, _, want, _, _ = run_attn(w, q, [300], [1], 4, 1)
    cache = w.cache()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    args = i64(w.rid), i64([300]), i64([1]), i64([300])
    table = i32(w.table)
    torch.cuda.synchronize()
    plan = ckv.plan_q8_attn(cache, 4, 1, *args, 1, stream=s)
    out, _ = ckv.q8_attn(cache, q, plan, table, 1 / math.sqrt(128), stream=s)
    s.synchronize()
    assert torch.equal(out, want)


def test_what_a_call_makes_belongs_to_its_stream():
    """The current stream still has work to do on memory that it has given back: results on another are not in it."""
    w = World(52, [300], 1, 128, 16, False)
    q, cache, table = w.queries([64], 8).to(DEV), w.cache(), i32(w.table)
    args = i64(w.rid), i64([300]), i64([64]), i64([300])
    plan = ckv.plan_q8_attn(cache, 8, 1, *args, 64)
    want, want_lse = ckv.q8_attn(cache, q, plan, table, 0.05, out_dtype=torch.float32)
    other, weights = ckv.new_q8_cache(64, 1, 16, 128), torch.rand(64, 16, device=DEV)
    src, dst, zero = i32([list(range(30))]), i32([list(range(30, 60))]), i64([0])
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)  # some milliseconds
    junk = [torch.full_like(x, 7) for x in (plan.buffer, want, want_lse, ckv.q8_attn_workspace(cache, 8, 1, 64))]
    del junk
    plan2 = ckv.plan_q8_attn(cache, 8, 1, *args, 64, stream=s)
    out, lse = ckv.q8_attn(cache, q, plan2, table, 0.05, out_dtype=torch.float32, stream=s)
    kept, lens = ckv.q8_evict(other, weights, zero, args[3], src, dst, 400, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    assert kept[0, :300].tolist() == list(range(300)) and lens.tolist() == [300]


def test_shapes_that_the_binding_refuses():
    w = World(52, [20], 2, 128, 16, False)
    cache, q = w.cache(), w.queries([1], 4).to(DEV)
    one, table = i64([20]), i32(w.table)
    plan = ckv.plan_q8_attn(cache, 4, 1, i64(w.rid), one, i64([1]), one, 1)
    bad = [
        lambda: ckv.q8_attn(cache, q.float(), plan, table, 0.1),
        lambda: ckv.q8_attn(cache, q[:, :2], plan, table, 0.1),
        lambda: ckv.q8_attn(cache, q, plan, table.long(), 0.1),
        lambda: ckv.q8_attn(cache, q, plan, table[0], 0.1),
        lambda: ckv.q8_attn(cache, q, plan, table, 0.1, out_dtype=torch.float16),
        lambda: ckv.q8_attn(cache, q, plan, table, 0.1, lse=torch.zeros(1, 4, device=DEV).half()),
        lambda: ckv.q8_attn(cache, q, plan, table, -0.1),
        lambda: ckv.q8_attn(cache, q, plan, table, 0.1, workspace=torch.zeros(16, dtype=torch.uint8, device=DEV)),
        lambda: ckv.plan_q8_attn(cache, 5, 1, i64(w.rid), one, i64([1]), one, 1),
        lambda: ckv.plan_q8_attn(cache, 4, 0, i64(w.rid), one, i64([1]), one, 1),
        lambda: ckv.plan_q8_attn(cache, 4, 1, i64(w.rid).int(), one, i64([1]), one, 1),
        lambda: ckv.plan_q8_attn(cache._replace(v=None), 4, 1, i64(w.rid), one, i64([1]), one, 1),
        lambda: ckv.plan_q8_attn(cache._replace(k_scale=cache.k_scale[:1]), 4, 1, i64(w.rid), one, i64([1]), one, 1),
        lambda: ckv.plan_q8_attn(cache._replace(k=cache.k.transpose(1, 2)), 4, 1, i64(w.rid), one, i64([1]), one, 1),
        lambda: ckv.q8_store(cache, torch.zeros(1, 2, 128, device=DEV), None, torch.zeros(1, 16, dtype=torch.uint8, device=DEV)),
        lambda: ckv.q8_store(cache, torch.zeros(1, 2, 128, device=DEV).half(), torch.zeros(1, 2, 128, device=DEV).half(),
                             torch.zeros(1, 16, dtype=torch.uint8, device=DEV)),
        lambda: ckv.q8_weigh(cache, q, torch.zeros(1, 4, device=DEV), torch.zeros(w.blocks, 8, device=DEV), 1, i64(w.rid),
                             one, i64([1]), one, table, 0.1),
        lambda: ckv.q8_evict(cache, torch.zeros(w.blocks, 16, device=DEV), i64(w.rid), one, table, table[:1], 4),
        lambda: ckv.q8_evict(cache, torch.zeros(w.blocks, 16, device=DEV), i64(w.rid), one, table, table, 4, 3, 2),
        lambda: ckv.q8_evict(cache, torch.zeros(w.blocks, 16, device=DEV), i64(w.rid), one, table, table, -1),
    ]
    for k, f in enumerate(bad):
        with pytest.raises((ValueError, ckv.CkvError)):
            f()
            pytest.fail(f"case {k} was taken")


def test_counts_past_32_bits_are_refused():
    """2^32 and a little more, which modulo 2^32 would be ordinary counts."""
    w = World(53, [20], 2, 128, 16, False)
    cache, q, big = w.cache(), w.queries([1], 4).to(DEV), 1 << 32
    rid, one, table = i64(w.rid), i64([20]), i32(w.table)
    weights, lse = torch.zeros(w.blocks, 16, device=DEV), torch.zeros(1, 4, device=DEV)
    bad = [
        lambda: ckv.plan_q8_store(cache, rid, one, i64([1]), big + 1, table, capacity=1),
        lambda: ckv.plan_q8_attn(cache, big + 4, 1, rid, one, i64([1]), one, 1),
        lambda: ckv.plan_q8_attn(cache, 4, big + 1, rid, one, i64([1]), one, 1),
        lambda: ckv.plan_q8_attn(cache, 4, 1, rid, one, i64([1]), one, big + 1),
        lambda: ckv.q8_attn_workspace(cache, 4, 1, big + 1),
        lambda: ckv.q8_attn_workspace(cache, 4, -1, 1),
        lambda: ckv.q8_weigh(cache, q, lse, weights, big + 1, rid, one, i64([1]), one, table, 0.1),
        lambda: ckv.q8_weigh(cache, q, lse, weights, -1, rid, one, i64([1]), one, table, 0.1),
        lambda: ckv.q8_evict(cache, weights, rid, one, table, table, 8, big, 0),
        lambda: ckv.q8_evict(cache, weights, rid, one, table, table, 8, 0, big + 1),
        lambda: ckv.q8_evict(cache, weights, rid, one, table, table, big + 8),
    ]
    for k, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"case {k} was taken")


@pytest.mark.parametrize("D,latent", [(128, False), (64, True), (512, True), (256, False)])
def test_waits_that_run_out_are_reported_and_leave_the_context_usable(D, latent):
    """The kernels whose roles hand tiles to one another, with a wait limit of a nanosecond: they end, say so, and the
    next launch computes as ever."""
    n, heads = 1500, 64
    w = World(61, [n], 1, D, 64, latent)
    q = w.queries([3], heads)
    cache, _, want, lse, st = run_attn(w, q, [n], [3], heads, 1)
    assert st == 0
    old = ckv.set_wait_limit_ns(1)
    try:
        _, _, _, _, st = run_attn(w, q, [n], [3], heads, 1)
        assert st == ckv.STATUS_TIMEOUT
        weigh = status()
        ckv.q8_weigh(cache, q.to(DEV), lse, torch.zeros(w.blocks, 64, device=DEV), 1, i64(w.rid), i64([n]), i64([3]),
                     i64([n]), i32(w.table), 1 / math.sqrt(D), status=weigh)
        torch.cuda.synchronize()
        assert int(weigh[0]) == (ckv.STATUS_TIMEOUT if D <= 128 else 0)  # from 256 channels on it waits for nobody
    finally:
        ckv.set_wait_limit_ns(old)
    _, _, again, _, st = run_attn(w, q, [n], [3], heads, 1)
    assert st == 0
    assert torch.equal(again, want)


def test_results_repeat_bit_for_bit():
    for D, latent, heads, q_len in [(128, False, 4, 1), (512, True, 64, 1), (128, False, 16, 60)]:
        w = World(62, [3000, 700], 1, D, 64, latent)
        q = w.queries([q_len, q_len], heads)
        first = run_attn(w, q, [3000, 700], [q_len] * 2, heads, 1)
        for _ in range(3):
            more = run_attn(w, q, [3000, 700], [q_len] * 2, heads, 1)
            assert torch.equal(first[2], more[2]) and torch.equal(first[3], more[3])


def test_many_requests_and_a_full_batch():
    """A batch of 1024 (the most), each of one entry or two, in every operator."""
    B = 1024
    lens = np.arange(B) % 3
    w = World(63, lens, 1, 64, 16, False, extra=2200)
    heads = 2
    q = w.queries([1] * B, heads)
    cache, _, out, lse, st = run_attn(w, q, np.maximum(lens, 1), [1] * B, heads, 1, torch.float32)
    want, wl, mag, big, flat = ref.attn(w.k, w.ks, w.v, w.vs, q.float().numpy(), w.rid, np.maximum(lens, 1), [1] * B,
                                        w.lens, w.table, 1, 1 / 8)
    tol, _ = attn_bounds(64, 2, want, wl, mag, big, flat, 20.0, False)
    assert st == 0 and (np.abs(out.cpu().numpy() - want) <= tol).all()
    weights, st = torch.zeros(w.blocks, 16, device=DEV), status()
    ckv.q8_weigh(cache, q.to(DEV), lse, weights, 1, i64(w.rid), i64(np.maximum(lens, 1)), i64([1] * B), i64(lens),
                 i32(w.table), 1 / 8, status=st)
    dst = np.full((w.table.shape[0], 1), -1, np.int32)
    dst[w.rid, 0] = w.spare[:B]
    kept, nl = ckv.q8_evict(cache, weights, i64(w.rid), i64(lens), i32(w.table), i32(dst), 1, 0, 1, status=st)
    torch.cuda.synchronize()
    assert int(st[0]) == 0
    assert abs(float(weights.sum()) - heads * (lens > 0).sum()) > 0  # the moved ones count twice
    assert nl.cpu().tolist() == np.minimum(lens, 1).tolist()
    assert kept.cpu().numpy()[:, 0].tolist() == [n - 1 for n in lens]

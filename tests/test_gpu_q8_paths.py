"""The 8-bit cache's kernels on the paths that small cases do not take: batches of several scans, plans of several strips, CTAs
with several units, requests of few and of many rows in one batch, pools and queries past 32 bits, captured tensor-core steps.  The oracle is the
definition in 64 bits, a request at a time."""
import math

import numpy as np
import pytest
import torch

from compressed_kv_attention_compressplan_gb300 import ckv
from tests import q8_ref as ref
from tests.test_gpu_q8 import DEV, World, attn_bounds, codes, i32, i64, run_attn, status

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ckv.load_library()


class Big(World):
    """A World of many entries, made on the GPU: every slot past a request's end and every unused block holds NaN."""

    def _side(self, spread):
        g = torch.Generator(device=DEV).manual_seed(int(self.r.randint(1 << 30)))
        shape = self.blocks, self.H, self.T, self.D
        pool = (torch.randn(shape, device=DEV, generator=g) * 16).to(torch.float8_e4m3fn).view(torch.uint8)
        scale = torch.exp2(torch.randint(-5, -2, shape[:2], device=DEV, generator=g).float())
        live = torch.zeros(self.blocks, dtype=torch.int64, device=DEV)  # entries of each block
        for b, n in enumerate(self.lens):
            per = -(-int(n) // self.T)
            if per:
                blk = torch.as_tensor(self.table[self.rid[b], :per].astype(np.int64), device=DEV)
                live[blk] = (int(n) - torch.arange(per, device=DEV) * self.T).clamp(max=self.T)
        pool.masked_fill_(torch.arange(self.T, device=DEV)[None, None, :, None] >= live[:, None, None, None], 0x7F)
        scale.masked_fill_((live == 0)[:, None], math.nan)
        return pool, scale

    def cache(self):
        sides = [(p.view(torch.float8_e4m3fn), s) for p, s in ((self.k, self.ks), (self.v, self.vs)) if p is not None]
        return ckv.Q8Cache(*sides[0], *(sides[1] if len(sides) > 1 else (None, None)))


def held(pool, scale, table_row, n):
    """[H, n, D] fp64 values of a request's first n entries, from torch pools of codes [blocks, H, T, D]."""
    T = pool.shape[2]
    blk = torch.as_tensor(np.asarray(table_row[:-(-n // T)], np.int64), device=pool.device)
    x = pool.view(torch.uint8)[blk].view(torch.float8_e4m3fn).double() * scale[blk].double()[:, :, None, None]
    return x.permute(1, 0, 2, 3).reshape(pool.shape[1], -1, pool.shape[3])[:, :n]


def oracle(cache, q, rid, seq, q_lens, lens, table, ratio, scale, lse=None):
    """(out, lse, mag, big, flat, received): as tests.q8_ref.attn, and the weight that each request's entries received
    under the given lse (one array a request)."""
    H = cache.k.shape[1]
    out, mag = torch.zeros(q.shape, dtype=torch.float64, device=DEV), torch.zeros(q.shape, dtype=torch.float64, device=DEV)
    got_lse, big, flat = (torch.full(q.shape[:2], x, dtype=torch.float64, device=DEV) for x in (-math.inf, 0.0, 0.0))
    received, at = [], 0
    for b in range(len(rid)):
        n, ql, S = int(lens[b]), int(q_lens[b]), int(seq[b])
        received.append(np.zeros(n))
        if n and ql:
            k = held(cache.k, cache.k_scale, table[rid[b]], n)
            v = k if cache.v is None else held(cache.v, cache.v_scale, table[rid[b]], n)
            pos = S - ql + 1 + torch.arange(ql, device=DEV)
            see = (n - (S // ratio - pos // ratio)).clamp(min=0)
            hidden = torch.arange(n, device=DEV)[None, None, None] >= see[:, None, None, None]
            x = q[at:at + ql].double().view(ql, H, -1, q.shape[2])
            z = (torch.einsum("qhgd,hsd->qhgs", x, k) * scale).masked_fill(hidden, -math.inf)
            l = torch.logsumexp(z, -1)
            p = (z - l[..., None]).exp().nan_to_num(0.0)

            def put(to, y):
                to[at:at + ql] = y.reshape(to[at:at + ql].shape)
            put(got_lse, l)
            put(out, torch.einsum("qhgs,hsd->qhgd", p, v))
            put(mag, torch.einsum("qhgs,hsd->qhgd", p, v.abs()))
            put(big, (torch.einsum("qhgd,hsd->qhgs", x.abs(), k.abs()) * scale).masked_fill(hidden, 0.0).amax(-1))
            put(flat, x.abs().amax(-1) * scale * k.abs().sum(-1).amax(-1)[None, :, None])
            if lse is not None:
                y = lse[at:at + ql].double().view(l.shape)[..., None]
                received[b] = (z - y).exp().nan_to_num(0.0).sum((0, 1, 2)).cpu().numpy()
        at += ql
    return [t.cpu().numpy() for t in (out, got_lse, mag, big, flat)] + [received]


def is_eight_bit(D, q_lens, group):
    return D >= 256 and int(np.sum(q_lens)) * group > (32 if D == 256 else 16) * len(q_lens)


def check(w, q_lens, heads, ratio=1, seq=None, decay=None, lens=None, seed=0):
    """Attention and, with a decay, the weights of a batch against the oracle."""
    lens = w.lens if lens is None else np.asarray(lens)
    seq = np.maximum(lens * ratio, q_lens) if seq is None else np.asarray(seq)
    q = w.queries(q_lens, heads).to(DEV)
    scale = 1 / math.sqrt(w.D)
    cache, plan, out, lse, st = run_attn(w, q, seq, q_lens, heads, ratio, torch.float32, lens=lens)
    assert st == 0
    want, wl, mag, big, flat, received = oracle(cache, q, w.rid, seq, q_lens, lens, w.table, ratio, scale, lse)
    side = cache.k_scale if cache.v is None else cache.v_scale
    vmax = 448 * float(side.nan_to_num(0.0).max())
    tol, ltol = attn_bounds(w.D, max(1, int(lens.max())), want, wl, mag, big, flat, vmax, False,
                            is_eight_bit(w.D, q_lens, heads // w.H))
    got, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
    assert np.isfinite(got).all()
    worst = np.abs(got - want) - tol
    assert (worst <= 0).all(), (worst.max(), np.unravel_index(worst.argmax(), worst.shape))
    assert np.array_equal(np.isneginf(gl), np.isneginf(wl))
    fin = np.isfinite(wl)
    assert (np.abs(gl[fin] - wl[fin]) <= ltol[fin]).all()
    if decay is None:
        return cache, plan, out, lse, None
    start = np.random.RandomState(seed).random_sample((w.blocks, w.T)).astype(np.float32)
    if decay == 0:
        start[0] = np.nan
    weights, st = torch.as_tensor(start, device=DEV), status()
    ckv.q8_weigh(cache, q, lse, weights, ratio, i64(w.rid), i64(seq), i64(q_lens), i64(lens), i32(w.table), scale, decay, status=st)
    torch.cuda.synchronize()
    assert int(st[0]) == 0
    new, touched = start.astype(np.float64), np.zeros(start.shape, bool)
    for b in range(len(lens)):
        if q_lens[b] and lens[b]:
            p = np.arange(int(lens[b]))
            at = w.table[w.rid[b], p // w.T], p % w.T
            new[at] = received[b] + (0 if decay == 0 else decay * new[at])
            touched[at] = True
    # the bound of the small cases: a score's D products, the exponent's argument, one sum over the rows
    top = big.max()
    rel = top * (w.D + 8) * 2.0 ** -23 + (3 * top + 60) * 2.0 ** -23 + int(np.max(q_lens)) * heads * 2.0 ** -24
    gw = weights.double().cpu().numpy()
    assert np.array_equal(gw[~touched], start[~touched], equal_nan=True)
    assert (np.abs(gw[touched] - new[touched]) <= rel * np.abs(new[touched]) + 2.0 ** -24).all()
    return cache, plan, out, lse, weights


@pytest.mark.parametrize("heads,D,q_len", [(2, 64, 1), (70, 128, 1), (35, 256, 2), (2, 512, 1)])
def test_a_full_batch_through_attention_weights_and_eviction(heads, D, q_len):
    """1024 requests of up to twelve entries, some of none and some without queries, in each weights kernel: the lengths are scanned
    in more than one round, and the eviction goes by the weights."""
    B, T, budget = 1024, 16, 5
    r = np.random.RandomState(70)
    lens = r.randint(0, 13, B)
    q_lens = np.where(r.rand(B) < 0.05, 0, q_len)
    if heads * q_len > 64:
        q_lens[:60] = q_len + 1  # more than 64 rows a request on average all the same
    w = World(71, lens, 1, D, T, D != 128, extra=B + 5)
    cache, _, _, _, weights = check(w, q_lens, heads, decay=1.0)
    dst = np.full((w.table.shape[0], 1), -1, np.int32)
    dst[w.rid, 0] = w.spare[:B]
    wn = weights.cpu().numpy()
    st = status()
    kept, nl = ckv.q8_evict(cache, weights, i64(w.rid), i64(lens), i32(w.table), i32(dst), budget, 1, 2, status=st)
    torch.cuda.synchronize()
    assert int(st[0]) == 0
    pools = [(w.k, w.ks)] + ([] if w.v is None else [(w.v, w.vs)])
    want = ref.evict(pools, wn, w.rid, lens, w.table, dst, budget, 1, 2)
    assert nl.tolist() == [len(x) for x in want]
    assert kept.cpu().numpy().tolist() == [x + [-1] * (budget - len(x)) for x in want]
    assert np.array_equal(weights.cpu().numpy(), wn, equal_nan=True)
    assert ref.same_codes(codes(cache.k), w.k) and np.array_equal(cache.k_scale.cpu().numpy(), w.ks, equal_nan=True)
    if w.v is not None:
        assert ref.same_codes(codes(cache.v), w.v) and np.array_equal(cache.v_scale.cpu().numpy(), w.vs, equal_nan=True)


UNEVEN = [19000, 0, 13001, 130, 27777, 21500, 1, 16003]
MANY, FEW = [32, 5, 0, 40, 33, 9, 70, 17], [1, 1, 0, 2, 1, 3, 1, 1]


@pytest.mark.parametrize("D,H,heads,q_lens,decay", [
    (64, 1, 4, MANY, 0.0), (64, 1, 4, MANY, 0.5), (64, 2, 8, MANY, 1.0), (128, 1, 4, MANY, 0.0), (128, 1, 4, MANY, 0.5),
    (128, 2, 8, MANY, 1.0), (256, 1, 4, MANY, 0.5), (256, 2, 8, MANY, 0.0), (512, 1, 4, MANY, 1.0), (64, 2, 8, FEW, 0.5),
    (128, 2, 8, FEW, 1.0), (256, 1, 16, FEW, 0.0), (512, 1, 4, FEW, 0.5)])
def test_weights_of_long_uneven_requests(D, H, heads, q_lens, decay):
    """More than two units of 128 entries to a CTA, over requests of uneven lengths and queries, some without: what a kernel
    keeps from one unit to the next."""
    w = Big(72, UNEVEN, H, D, 64, D == 512)
    assert sum(-(-n // 128) for n, ql in zip(UNEVEN, q_lens) if ql) > 4 * 152
    check(w, q_lens, heads, decay=decay)


@pytest.mark.parametrize("B,q_len,heads,H,D,tiles", [(16, 2048, 4, 1, 64, 512), (16, 2048, 4, 1, 128, 512), (12, 1600, 8, 2, 256, 1200),
                                                (300, 20, 16, 1, 512, 1500), (200, 10, 4, 1, 128, 600), (1024, 2, 64, 2, 128, 4096)])
def test_plans_of_several_strips(B, q_len, heads, H, D, tiles):
    """More row tiles than the plan's CTA has threads: every tile's items cover its entries once, and the attention is right."""
    r = np.random.RandomState(73)
    lens = r.randint(0, 300, B)
    q_lens = np.full(B, q_len)
    if q_len > 100:
        q_lens -= np.arange(B) % 3
    w = Big(74, lens, H, D, 16, True)
    ratio = 8
    seq = np.maximum(lens * ratio + np.arange(B) % ratio, q_lens)
    _, plan, _, _, _ = check(w, q_lens, heads, ratio, seq)
    raw = plan.buffer.cpu().numpy()
    head = raw[:64].view(np.uint32)
    n_items, ctas, parts, splits, rows, group, _, _, cap = (int(x) for x in head[:9])
    first = raw[64:64 + 4 * (cap + 1)].view(np.uint32)[:ctas + 1].astype(int)
    off = (64 + 4 * (cap + 1) + 63) // 64 * 64
    split = raw[off:off + 4 * cap].view(np.uint32)[:splits].astype(int)
    off = (off + 4 * cap + 63) // 64 * 64
    it = raw[off:off + 48 * n_items].view(np.uint32).reshape(-1, 12).astype(np.int64)
    assert first[0] == 0 and first[-1] == n_items and (np.diff(first) >= 1).all()
    want = [(int(w.rid[b]), row) for b in range(B) for row in range(0, int(q_lens[b]) * group, rows)]
    assert len(want) >= tiles > 256
    order = list(dict.fromkeys((int(x[0]), int(x[3])) for x in it))
    assert order == want  # tiles in order, a tile's items together
    starts = dict(zip(w.rid.tolist(), np.concatenate([[0], np.cumsum(q_lens)])[:-1]))
    of = {int(w.rid[b]): b for b in range(B)}
    k = part = 0
    got_splits = []
    for rid, row0 in want:
        b, n = of[rid], int(it[k][10])
        see = ref.visible(int(lens[b]), int(seq[b]), int(q_lens[b]), min(int(q_lens[b]) - 1, (row0 + rows - 1) // group), ratio)
        at = 0
        for c in range(n):
            x = it[k + c]
            assert (x[0], x[3], x[1], x[2], x[6], x[9], x[10]) == (rid, row0, starts[rid], q_lens[b], lens[b], c, n)
            assert x[4] == at and x[5] >= x[4]
            assert x[8] == (0xFFFFFFFF if n == 1 else part)
            at = x[5]
        assert at == see
        if n > 1:
            got_splits.append(k)
            part += n
        k += n
    assert k == n_items and got_splits == split.tolist() and part == parts <= 2 * cap


@pytest.mark.parametrize("chunk,D,H,heads,latent", [(2048, 128, 1, 4, False), (512, 128, 1, 4, False), (2048, 64, 1, 4, True),
                                                    (700, 512, 1, 8, True), (190, 512, 1, 4, True), (900, 256, 2, 8, False)])
def test_a_chunk_beside_single_tokens(chunk, D, H, heads, latent):
    """One request with a prompt's chunk and 63 with one token: the whole batch goes to one kernel by its average, to that for many
    rows (2048, 700 and 900 queries) or to that for few (512, 190)."""
    r = np.random.RandomState(75)
    lens = r.randint(1, 1500, 64)
    lens[31] = 2200
    q_lens = np.ones(64, np.int64)
    q_lens[31] = chunk
    w = Big(76, lens, H, D, 64, latent)
    check(w, q_lens, heads, decay=1.0)


@pytest.mark.parametrize("D,q_len,heads,latent", [(128, 20, 32, True), (64, 20, 64, True), (256, 20, 32, True), (512, 2, 512, True),
                                                  (128, 20, 32, False)])
def test_pools_past_32_bits_on_the_tensor_cores(D, q_len, heads, latent):
    """Blocks at both ends of pools of more than 2^32 bytes, in the kernels for many rows."""
    T, H, n = 128, 8, 400
    blocks = (1 << 32) // (T * H * D) + 40
    used = [blocks - 1, blocks - 17, 3, blocks - 5]
    r = np.random.RandomState(77)

    def side():
        pool = torch.zeros(blocks, H, T, D, dtype=torch.uint8, device=DEV)
        for b in used:
            pool[b] = torch.as_tensor(ref.round8(r.standard_normal((H, T, D)) * 16), device=DEV)
        return pool.view(torch.float8_e4m3fn), torch.full((blocks, H), 0.0625, device=DEV)

    cache = ckv.Q8Cache(*side(), *((None, None) if latent else side()))
    table = np.asarray([used], np.int32)
    q = torch.as_tensor(r.standard_normal((q_len, heads, D))).bfloat16().to(DEV)
    st, scale = status(), 1 / math.sqrt(D)
    args = i64([0]), i64([n]), i64([q_len]), i64([n])
    plan = ckv.plan_q8_attn(cache, heads, 1, *args, q_len, status=st)
    out, lse = ckv.q8_attn(cache, q, plan, i32(table), scale, out_dtype=torch.float32, status=st)
    weights = torch.zeros(blocks, T, device=DEV)
    ckv.q8_weigh(cache, q, lse, weights, 1, *args, i32(table), scale, status=st)
    torch.cuda.synchronize()
    assert int(st[0]) == 0
    want, wl, mag, big, flat, received = oracle(cache, q, [0], [n], [q_len], [n], table, 1, scale, lse)
    tol, ltol = attn_bounds(D, n, want, wl, mag, big, flat, 28.0, False, D >= 256)
    assert (np.abs(out.double().cpu().numpy() - want) <= tol).all()
    assert (np.abs(lse.double().cpu().numpy() - wl) <= ltol).all()
    got = torch.cat([weights[b] for b in used]).double().cpu().numpy()
    assert np.abs(got[:n] - received[0]).max() <= 1e-4 and (got[n:] == 0).all()
    assert abs(float(weights.double().sum()) - received[0].sum()) <= 1e-2


@pytest.mark.parametrize("D,q_len", [(64, 1 << 17), (256, 1 << 15), (512, 1 << 14)])
def test_queries_and_outputs_past_32_bits(D, q_len):
    """More than 2^32 bytes of queries and of outputs: the first and the last queries, over few entries."""
    heads, n = 256, 40
    q_len += 3
    w = World(78, [n], 1, D, 16, True)
    q = torch.zeros(q_len, heads, D, dtype=torch.bfloat16, device=DEV)
    ends = [0, 1, q_len // 2, q_len - 2, q_len - 1]
    q[ends] = torch.as_tensor(w.r.standard_normal((len(ends), heads, D))).bfloat16().to(DEV)
    assert q.numel() * 2 > 1 << 32
    st, cache = status(), w.cache()
    # entries of q_len tokens each but for the newest: every query sees all but the last entry, or all
    args = i64(w.rid), i64([q_len]), i64([q_len]), i64([n])
    ratio = 65536 if q_len > 65536 else q_len
    plan = ckv.plan_q8_attn(cache, heads, ratio, *args, q_len, status=st)
    out, lse = ckv.q8_attn(cache, q, plan, i32(w.table), 1 / math.sqrt(D), status=st)
    torch.cuda.synchronize()
    assert int(st[0]) == 0
    k = held(cache.k, cache.k_scale, w.table[w.rid[0]], n)[0]
    for i in ends:
        see = ref.visible(n, q_len, q_len, i, ratio)
        z = q[i].double() @ k[:see].T / math.sqrt(D)
        want = torch.softmax(z, -1) @ k[:see]
        assert (out[i].double() - want).abs().max() <= 0.05
        assert (lse[i].double() - torch.logsumexp(z, -1)).abs().max() <= 1e-3


@pytest.mark.parametrize("D,heads,latent", [(512, 64, True), (128, 96, False), (256, 48, False), (64, 80, True)])
def test_captured_steps_of_the_tensor_core_kernels(D, heads, latent):
    """Plan, attention and weights captured once and replayed with other lengths, queries and tables."""
    B, T = 3, 16
    w = World(79, [700, 300, 0], 1, D, T, latent, more=600)
    w.lens = np.asarray([1300, 900, 600])
    for name in ("k", "v"):  # entries in every place that the tables have
        if getattr(w, name) is not None:
            setattr(w, name, ref.round8(w.r.standard_normal(getattr(w, name).shape) * 16))
            setattr(w, name + "s", np.full((w.blocks, 1), 0.0625, np.float32))
    cache, st, scale = w.cache(), status(), 1 / math.sqrt(D)
    rid, seq, ext, kv = i64(w.rid), i64([700, 300, 1]), i64([2, 1, 1]), i64([700, 300, 0])
    q, table = torch.zeros(4, heads, D, dtype=torch.bfloat16, device=DEV), i32(w.table)
    weights = torch.zeros(w.blocks, T, device=DEV)
    ws = ckv.q8_attn_workspace(cache, heads, B, 4)

    def run():
        plan = ckv.plan_q8_attn(cache, heads, 1, rid, seq, ext, kv, 4, status=st)
        out, lse = ckv.q8_attn(cache, q, plan, table, scale, out_dtype=torch.float32, workspace=ws, status=st)
        ckv.q8_weigh(cache, q, lse, weights, 1, rid, seq, ext, kv, table, scale, 0.0, status=st)
        return out, lse

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        run()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = run()
    for lens, q_lens in (([700, 300, 0], [2, 1, 1]), ([1300, 3, 600], [1, 1, 2]), ([64, 900, 129], [0, 3, 1])):
        x = torch.as_tensor(w.r.standard_normal((4, heads, D))).bfloat16()
        q.copy_(x), seq.copy_(i64(np.maximum(lens, q_lens))), ext.copy_(i64(q_lens)), kv.copy_(i64(lens))
        weights.fill_(-1.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert int(st[0]) == 0
        want, wl, mag, big, flat, received = oracle(cache, q, w.rid, np.maximum(lens, q_lens), q_lens, lens, w.table, 1, scale, lse)
        tol, _ = attn_bounds(D, 1300, want, wl, mag, big, flat, 28.0, False, D >= 256)
        assert (np.abs(out.double().cpu().numpy() - want) <= tol).all()
        got = weights.cpu().numpy()
        for b in range(B):
            p = np.arange(lens[b])
            mine = got[w.table[w.rid[b], p // T], p % T]
            assert np.abs(mine - received[b]).max(initial=0) <= 1e-4 if q_lens[b] else (mine == -1).all()

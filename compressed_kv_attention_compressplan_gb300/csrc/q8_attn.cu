// q8_attn.cu -- softmax attention over the 8-bit paged cache: the plan, the
// split kernel for few rows (mma.sync) and the kernel that joins the splits.
//
// Mathematics.  With scores s_j = scale * log2(e) * k_scale_j * <q, k8_j> and
// value scales c_j the output is
//     out = sum_j 2^(s_j) c_j v8_j / sum_j 2^(s_j).
// c_j is folded into the exponent: with t_j = s_j + log2(c_j) and any m,
//     O = sum_j w_j v8_j,  L = sum_j w_j / c_j,  w_j = 2^(t_j - m),  out = O / L,
// so scaling the values costs one addend of a multiply-add that is there
// anyway, and w_j, the matrix operand, stays in fp16's range whatever the
// blocks' scales are.  m follows the rows' maximum of t (not of s) lazily: it
// is raised to 6 under the maximum when a t passes m + 14, so a weight is at most
// 2^14 (fp16's largest is 2^16) and weights keep fp16's full precision down
// to 2^-20 and are dropped only under 2^-31 of the largest.  L keeps fp32
// weights: c_j >= 2^-48 and c_j <= 2^48 bound w_j / c_j, and a w_j that the
// exponent's range drops (2^-126) weighs under 2^-24 of the sum.
//
// Precision.  k8 and v8 are exact in fp16.  A query row is scaled by a power of
// two that puts its largest value in [2^14, 2^15), then rounded to fp16: exact for
// bf16 input down to 2^-28 of that value.  Products accumulate in fp32; the
// weights' rounding to fp16 (2^-11 relative) is the one rounding that costs
// anything, and is below the bf16 output's.
//
// Bound of the split kernel.  The entries' bytes: a warp streams its tiles of 16 entries through a ring of its own, with as many
// stages as the CTAs that fit an SM leave, so that nothing but the copies is waited for.  64 requests of up to 16384 entries, eight kv
// heads, 1081 MB: 168 us, 6.4 TB/s or 95 % of the measured copy rate; two requests of 140001 entries, 145 MB: 31 us, 4.7 TB/s, with
// the first copies and the join of the parts (7 us) no longer small.
#include <algorithm>

#include "async_copy.cuh"
#include "q8_plan.cuh"

namespace ckv {

// ------------------------------------------------------------------- plan
namespace {

struct AttnPlanArgs {
  const int64_t* rid;
  const int64_t* seq_lens;
  const int64_t* extend_lens;
  const int64_t* kv_lens;
  uint32_t batch;
  uint32_t num_q;
  uint32_t ratio;
  Q8Geom g;
  uint8_t* plan;
  uint32_t* d_status;
};

// One CTA: requests are scanned once, then tiles in strips of kPlanThreads.  Latency bounds it: the lengths' loads, three block-wide
// scans and the items' stores, 7.4 us for 200 requests with 256 threads and 7.9 with 1024.
template <int kPlanThreads>
__global__ __launch_bounds__(kPlanThreads) void plan_q8_attn_kernel(const AttnPlanArgs a) {
  __shared__ uint32_t s_rid[kPlanThreads], s_qs[kPlanThreads], s_ql[kPlanThreads], s_kv[kPlanThreads],
      s_ph[kPlanThreads], s_tile[kPlanThreads];
  __shared__ unsigned long long s_pos[kPlanThreads];
  __shared__ uint32_t s_item[kPlanThreads], s_part[kPlanThreads];
  __shared__ unsigned long long s_scan[2][kPlanThreads / 32 + 1];
  __shared__ uint32_t s_most;
  pdl_wait();
  pdl_release();
  const uint32_t t = threadIdx.x;
  if (t == 0) s_most = 0;  // the scans' barriers come before its use
  const uint32_t M = a.g.rows, G = a.g.group;
  Q8Header* head = reinterpret_cast<Q8Header*>(a.plan);
  uint32_t* first = reinterpret_cast<uint32_t*>(a.plan + a.g.off_first);
  uint32_t* split = reinterpret_cast<uint32_t*>(a.plan + a.g.off_split);
  Q8Item* items = reinterpret_cast<Q8Item*>(a.plan + a.g.off_items);

  // requests
  unsigned long long q_len = 0;
  uint32_t kv = 0, phase = 0, rid = 0;
  bool ok = false;
  if (t < a.batch) {
    const int64_t r = a.rid[t], sl = a.seq_lens[t], el = a.extend_lens[t], kl = a.kv_lens[t];
    const bool len_ok = el >= 0 && el <= a.num_q;
    q_len = len_ok ? static_cast<unsigned long long>(el) : 0;
    ok = len_ok && sl >= el && sl <= 0x7FFFFFFF && kl >= 0 && kl <= 0x7FFFFFF0 && r >= 0 && r <= 0x7FFFFFFF;
    if (!ok) status_or(a.d_status, CKV_STATUS_BAD_LENGTH);
    if (ok) {
      kv = static_cast<uint32_t>(kl);
      phase = a.ratio - 1 - static_cast<uint32_t>(sl) % a.ratio;
      rid = static_cast<uint32_t>(r);
    }
  }
  unsigned long long total_q, total_tiles, qs, tile0;
  unsigned long long tiles = ok ? (static_cast<uint32_t>(q_len) * G + M - 1) / M : 0;
  block_exclusive2<kPlanThreads>(q_len, tiles, &qs, &tile0, &total_q, &total_tiles, s_scan);
  if (total_q > a.num_q) {  // requests whose queries do not all exist are dropped, and the others' tiles counted again
    if (qs + q_len > a.num_q) tiles = 0;
    tile0 = block_exclusive<kPlanThreads>(tiles, &total_tiles, s_scan[0]);
  }
  if (t < a.batch) {
    s_rid[t] = rid;
    s_qs[t] = static_cast<uint32_t>(qs);
    s_ql[t] = static_cast<uint32_t>(q_len);
    s_kv[t] = kv;
    s_ph[t] = phase;
    s_tile[t] = static_cast<uint32_t>(tile0);
  }
  __syncthreads();

  const uint32_t nt = static_cast<uint32_t>(total_tiles);
  // a tile's entries: those its last query sees
  auto tile_of = [&](uint32_t tile, uint32_t* b) -> uint32_t {
    *b = last_not_above(s_tile, a.batch, tile);
    const uint32_t j = tile - s_tile[*b];
    const uint32_t last =
        min(s_ql[*b] - 1, static_cast<uint32_t>((static_cast<unsigned long long>(j + 1) * M - 1) / G));
    return static_cast<uint32_t>(q8_visible(s_kv[*b], s_ql[*b] - 1 - last, s_ph[*b], a.ratio));
  };
  const uint32_t start = a.g.start_cost, grain = a.g.grain;  // grain is a power of two
  auto cost_of = [&](uint32_t seen) -> unsigned long long {
    return start + ((static_cast<unsigned long long>(seen) + grain - 1) & ~static_cast<unsigned long long>(grain - 1));
  };
  unsigned long long mine = 0;
  for (uint32_t i = t; i < nt; i += kPlanThreads) {
    uint32_t b;
    mine += cost_of(tile_of(i, &b));
  }
  unsigned long long total;
  const unsigned long long before = block_exclusive<kPlanThreads>(mine, &total, s_scan[0]);
  // 32-bit divisions where they do: a 64-bit one is some forty instructions that wait for one another, and there were ten
  const bool narrow = total <= 0x7FFFFFFFull;
  unsigned long long quota = narrow ? (static_cast<uint32_t>(total) + a.g.ctas - 1) / a.g.ctas : (total + a.g.ctas - 1) / a.g.ctas;
  quota = max(static_cast<unsigned long long>(a.g.min_quota), quota);
  quota = (quota + grain - 1) & ~static_cast<unsigned long long>(grain - 1);
  auto shares = [&](unsigned long long x) -> unsigned long long {  // x / quota, x <= total + quota
    return narrow ? static_cast<uint32_t>(x) / static_cast<uint32_t>(quota) : x / quota;
  };

  unsigned long long pos0 = 0;
  uint32_t item0 = 0, part0 = 0, split0 = 0;
  for (uint32_t i0 = 0; i0 < nt; i0 += kPlanThreads) {
    const uint32_t i = i0 + t;
    uint32_t b, n = 0;
    const unsigned long long cost = nt <= kPlanThreads ? mine : i < nt ? cost_of(tile_of(i, &b)) : 0;
    unsigned long long cost_sum = total, packed_sum, p = before;  // a single strip's sums are known
    if (nt > kPlanThreads) p = pos0 + block_exclusive<kPlanThreads>(cost, &cost_sum, s_scan[0]);
    if (cost) n = static_cast<uint32_t>(shares(p + cost - 1) - shares(p)) + 1;
    // items (32 bits), parts (16) and splits (16) of the strip, in one scan: parts are at most twice the CTAs
    const unsigned long long pk = n | (static_cast<unsigned long long>(n > 1 ? n : 0) << 32) |
                                  (static_cast<unsigned long long>(n > 1) << 48);
    const unsigned long long ex = block_exclusive<kPlanThreads>(pk, &packed_sum, s_scan[0]);
    const uint32_t it = item0 + static_cast<uint32_t>(ex);
    s_pos[t] = p;
    s_item[t] = it;
    s_part[t] = n > 1 ? part0 + (static_cast<uint32_t>(ex >> 32) & 0xFFFFu) : kInvalidU32;
    if (n > 1) {
      split[split0 + static_cast<uint32_t>(ex >> 48)] = it;
      atomicMax(&s_most, n);
    }
    __syncthreads();
    const uint32_t strip = min(static_cast<uint32_t>(kPlanThreads), nt - i0);
    const uint32_t end = item0 + static_cast<uint32_t>(packed_sum);
    for (uint32_t k = item0 + t; k < end; k += kPlanThreads) {
      const uint32_t s = last_not_above(s_item, strip, k);
      uint32_t rb;
      const uint32_t seen = tile_of(i0 + s, &rb);
      const unsigned long long len = cost_of(seen);
      const unsigned long long P = s_pos[s], cut = shares(P);
      const uint32_t c = k - s_item[s];
      const unsigned long long lo = c == 0 ? P : (cut + c) * quota;
      const unsigned long long hi = min(P + len, (cut + c + 1) * quota);
      const unsigned long long o0 = lo - P, o1 = hi - P;
      Q8Item r;
      r.rid = s_rid[rb];
      r.q_start = s_qs[rb];
      r.q_len = s_ql[rb];
      r.row0 = (i0 + s - s_tile[rb]) * M;
      r.kv_begin = o0 > start ? static_cast<uint32_t>(o0 - start) : 0;
      r.kv_end = o1 > start ? min(seen, static_cast<uint32_t>(o1 - start)) : 0;
      r.kv_len = s_kv[rb];
      r.phase = s_ph[rb];
      r.part = static_cast<int32_t>(s_part[s]);
      r.chunk = c;
      r.chunks = static_cast<uint32_t>(shares(P + len - 1) - cut) + 1;
      r.reserved = 0;
      items[k] = r;
      const unsigned long long cta = shares(lo);
      if (cta * quota == lo) first[cta] = k;
    }
    pos0 += cost_sum;
    item0 = end;
    part0 += static_cast<uint32_t>(packed_sum >> 32) & 0xFFFFu;
    split0 += static_cast<uint32_t>(packed_sum >> 48);
    __syncthreads();
  }
  if (t == 0) {
    const uint32_t ctas = static_cast<uint32_t>(shares(total + quota - 1));
    first[ctas] = item0;
    head->items = item0;
    head->ctas = ctas;
    head->parts = part0;
    head->splits = split0;
    head->rows = M;
    head->group = G;
    head->num_q = a.num_q;
    head->ratio = a.ratio;
    head->cap_ctas = a.g.ctas;
    head->batch = a.batch;
    head->most = s_most;  // (the last strip ended with a barrier)
    if (total_q != a.num_q) status_or(a.d_status, CKV_STATUS_BAD_TOTAL);
  }
}

}  // namespace

// ------------------------------------------------------------- geometry
namespace {

constexpr int kAttnWarps = 4;
constexpr int kAttnThreads = 32 * kAttnWarps;
constexpr int kTile = 16;  // entries a warp takes at a time

// kDw channels of a warp's part of a row, kNp warps to a row (512 channels: 2); kRows query rows of a tile, 8 or 16.
template <int kDw, int kNp, bool kShared, int kRows>
struct Cfg {
  static constexpr int kD = kDw * kNp;
  static constexpr int kGroups = kAttnWarps / kNp;  // warp groups, each with tiles of its own
  static constexpr int kTileBytes = kTile * kDw * (kShared ? 1 : 2);
  static constexpr int kStageBytes = kTileBytes;
  // As many stages as let kPerSm CTAs share an SM's 227 KB.  Eight rows and 128 channels, 64 requests of 8000 entries (1.05 GB): 162 us with two
  // CTAs of six stages, 186 with three of four; before that by a few instructions a tile more 174, 182, 188 with four of three and 280
  // with one of twelve.
  static constexpr int kPerSm = kDw == 64 ? 4 : kDw == 128 ? (kRows == 8 ? 2 : 3) : 2;
  static constexpr int kStages = kDw == 64                ? (kShared ? 8 : 6)
                                 : kDw == 128 && kRows == 8 ? (kShared ? 9 : 6)
                                 : kDw == 128               ? (kShared ? 7 : 4)
                                                            : (kShared ? 5 : 3);
  static_assert(kStages <= 16, "");
  static constexpr int kRingBytes = kAttnWarps * kStages * kStageBytes;
  static constexpr int kMergeStride = kD + 4;  // floats
  static constexpr int kMergeBytes = kGroups * kRows * kMergeStride * 4;
  static constexpr int kSmem = kRingBytes > kMergeBytes ? kRingBytes : kMergeBytes;
};

int per_sm_of(uint32_t head_dim, uint32_t rows) { return head_dim == 64 ? 4 : head_dim == 128 && rows == 16 ? 3 : 2; }

}  // namespace

int q8_attn_geom(const Q8Cache& c, uint32_t batch, uint32_t num_q, uint32_t n_heads, Q8Geom* g) {
  if (batch > CKV_MAX_BATCH || num_q > CKV_MAX_TOKENS) return CKV_ERR_SIZE;
  if (n_heads == 0 || n_heads % c.heads != 0 || n_heads / c.heads > CKV_Q8_MAX_GROUP) return CKV_ERR_SIZE;
  g->group = n_heads / c.heads;
  if (static_cast<uint64_t>(num_q) * g->group > 0x7FFFFFFFull) return CKV_ERR_SIZE;  // row numbers are 32-bit
  // The split kernel's tiles are 8 or 16 rows, and it reads a request's entries once for each; the tensor-core kernels' are 256, or 64
  // from 256 channels on, at nearly the same cost for a few rows as for all.  Where they cross, by rows of a request and kv head (us,
  // split kernel / tensor cores, 32 to 64 requests of 4096 entries): 64 channels 98 / 113 at 64 and 122 / 112 at 80; 128 channels
  // 184 / 188 at 64 and 222 / 190 at 80; 256 channels 62 / 65 at 32 and 82 / 68 at 48; 512 channels 62 / 72 at 16 and 102 / 75 at 32.
  const uint64_t most = c.head_dim <= 128 ? 64 : c.head_dim == 256 ? 32 : 16;
  g->tc = static_cast<uint64_t>(num_q) * g->group > most * batch && batch > 0;
  if (g->tc) {
    g->rows = c.head_dim <= 128 ? 256 : 64;
    g->ctas = std::max<uint32_t>(1, static_cast<uint32_t>(sm_count()) / c.heads);
    g->grain = 128;
    // What starting a tile takes, in entries' time: an item takes 17 k cycles beside 4.5 k for 128 entries (27 k beside 5 k from 256
    // channels on).  A chunk of three requests, one of them short: 823 us at 384, 773 at 512, 771 at 768, 774 at 896.
    g->start_cost = c.head_dim >= 256 ? 384 : 768;
    g->min_quota = 128;  // one request of 2048 latent entries: 20.6 us with one tile a CTA, 29.9 with two, 36 with four
  } else {
    g->rows = static_cast<uint64_t>(num_q) * g->group <= 8ull * batch ? 8 : 16;
    g->ctas = std::max<uint32_t>(1, static_cast<uint32_t>(sm_count()) * per_sm_of(c.head_dim, g->rows) / c.heads);
    g->start_cost = 128;
    g->grain = 16;  // quotas in whole 64 entries: 17.1 us against 15.8 for 8 requests of 1000, 23.2 against 20.8 for 16 of 2000
    g->min_quota = 128;
  }
  const uint64_t tiles = static_cast<uint64_t>(num_q) * g->group / g->rows + batch;
  const uint64_t items = tiles + g->ctas;
  g->cap_items = static_cast<uint32_t>(items);
  g->cap_parts = 2 * g->ctas;
  auto up = [](uint64_t x) { return (x + 63) & ~63ull; };
  g->off_first = sizeof(Q8Header);
  g->off_split = up(g->off_first + 4ull * (g->ctas + 1));
  g->off_items = up(g->off_split + 4ull * g->ctas);
  g->bytes = g->off_items + sizeof(Q8Item) * items;
  g->workspace = static_cast<uint64_t>(g->cap_parts) * c.heads * g->rows * (c.head_dim + 2) * 4;
  return CKV_OK;
}

namespace {

// ----------------------------------------------------------------- attention
// Fragments.  A warp's 16 rows are the MMA's m, 16 entries its n (scores) and k
// (values).  Sums over k may run in any order, so lane (g, q) = (lane / 4, lane % 4)
// takes as the k of its score fragments 16 consecutive channels of entry g, i.e. the
// 16 bytes of one shared-memory load, and the query fragments are laid out
// alike; and columns n of the value product may be any channels, so lane (g, q)
// takes 16 consecutive channels, chunk 8 jj + g, of entries 2q, 2q+1, 2q+8, 2q+9 --
// the four entries whose weights it holds from the scores.  Nothing is
// transposed or exchanged: one permute pairs two entries' bytes, one conversion
// gives the fragment.
//
// Up to eight rows (decode with groups of as many heads) the products are transposed: 16 entries are m, and the eight
// rows n, of the scores; 16 channels are m, and the rows n again, of the values.  That is half the products, exponentials and
// accumulators; the weights cross from entries to rows with one 8 x 8 transposition for eight entries.  One request of 777 entries 8.7 us against
// 9.4 with sixteen rows, 32 of 300 14.8 against 18.2, 64 of 8000 174 against 179.  What a tile costs in instructions counts to the end: a copy for its scales, sizes on whole tiles'
// copies and a division were 8 % of the 64 requests' time.
template <int kDw, int kNp, bool kShared, int kRows>
__global__ __launch_bounds__(kAttnThreads, (Cfg<kDw, kNp, kShared, kRows>::kPerSm)) void q8_attn_kernel(const AttnArgs a) {
  using C = Cfg<kDw, kNp, kShared, kRows>;
  constexpr bool kFew = kRows == 8;
  constexpr int kChunks = kDw / 16;             // 16-byte chunks of a row part
  constexpr int kOt = kFew ? kDw / 16 : kDw / 8;  // output tiles
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float s_m[C::kGroups][kRows], s_l[C::kGroups][kRows];
  __shared__ __align__(16) float s_x[kNp == 2 ? C::kGroups : 1][2][2][kNp == 2 ? 256 : 1];  // partial scores of a row's two warps
  __shared__ int s_nan[C::kD];  // first entry with a NaN value, by channel
  __shared__ int s_any_nan;

  pdl_wait();
  pdl_release();
  const Q8Header* head = reinterpret_cast<const Q8Header*>(a.plan);
  const uint32_t h = blockIdx.y;
  if (!plan_fits(head, a)) {
    if (blockIdx.x == 0 && h == 0 && threadIdx.x == 0) status_or(a.d_status, CKV_STATUS_BAD_INDEX);
    return;
  }
  if (blockIdx.x >= head->ctas) return;
  const uint32_t* first = reinterpret_cast<const uint32_t*>(a.plan + a.g.off_first);
  const Q8Item* items = reinterpret_cast<const Q8Item*>(a.plan + a.g.off_items);
  const uint32_t item0 = first[blockIdx.x], item1 = min(first[blockIdx.x + 1], a.g.cap_items);

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, q = lane & 3;
  const int grp = warp / kNp, half = warp % kNp;
  const uint32_t G = a.g.group, H = a.c.heads, T = a.c.block_tokens, t_shift = __ffs(T) - 1;
  const uint32_t ring = smem_addr(smem) + warp * C::kStages * C::kStageBytes;

  for (uint32_t it = item0; it < item1; ++it) {
    const Q8Item item = items[it];
    if (!item_fits(item, a)) {
      if (tid == 0) status_or(a.d_status, CKV_STATUS_BAD_INDEX);
      continue;
    }
    const uint32_t rows = min(static_cast<uint32_t>(kRows), item.q_len * G - item.row0);
    const int32_t* table = a.table + static_cast<size_t>(item.rid) * a.stride;
    __syncthreads();  // the previous item's reads of shared memory are done
    for (int c = tid; c < C::kD; c += kAttnThreads) s_nan[c] = 0x7FFFFFFF;
    if (tid == 0) s_any_nan = 0;

    // ---- tiles of this warp: grp, grp + kGroups, ... ; block numbers 32 tiles at a time, one to a lane
    const uint32_t n_all = item.kv_end > item.kv_begin ? (item.kv_end - item.kv_begin + kTile - 1) / kTile : 0;
    const uint32_t n_mine = n_all > static_cast<uint32_t>(grp) ? (n_all - grp + C::kGroups - 1) / C::kGroups : 0;
    auto entry_of = [&](uint32_t i) { return item.kv_begin + (grp + i * C::kGroups) * kTile; };
    auto block_at = [&](uint32_t i) -> int32_t { return i < n_mine ? __ldg(table + (entry_of(i) >> t_shift)) : -1; };
    int32_t blocks_now = block_at(lane), blocks_next = block_at(32 + lane);
    bool bad_block = false;
    auto issue = [&](uint32_t i) {
      if (i < n_mine) {
        if (i != 0 && (i & 31) == 0) {
          blocks_now = blocks_next;
          blocks_next = block_at(i + 32 + lane);
        }
        const int32_t b = __shfl_sync(0xFFFFFFFFu, blocks_now, i & 31);
        const bool ok = b >= 0 && static_cast<uint32_t>(b) < a.c.num_blocks;
        bad_block |= !ok;
        const uint32_t e0 = entry_of(i);
        const size_t bh = static_cast<size_t>(ok ? b : 0) * H + h;
        const size_t base = ((bh << t_shift) + (e0 & (T - 1))) * C::kD + half * kDw;
        const uint32_t dst = ring + (i % C::kStages) * C::kStageBytes;
        // entries past the request's end, and blocks that do not exist, read as zeros
        const uint32_t here = ok ? min(static_cast<uint32_t>(kTile), item.kv_len - e0) : 0;
        const uint8_t* k = a.c.k + base;
        const uint8_t* v = kShared ? nullptr : a.c.v + base;
        if (here == kTile) {
#pragma unroll
          for (int x = 0; x < kTile * kChunks / 32; ++x) {
            const uint32_t c = x * 32 + lane, t = c / kChunks, cc = c % kChunks;
            cp_async16(dst + tile_off<kDw>(t, cc), k + t * C::kD + cc * 16);
            if (!kShared) cp_async16(dst + kTile * kDw + tile_off<kDw>(t, cc), v + t * C::kD + cc * 16);
          }
        } else {
#pragma unroll 1
          for (int x = 0; x < kTile * kChunks / 32; ++x) {
            const uint32_t c = x * 32 + lane, t = c / kChunks, cc = c % kChunks;
            const uint32_t n = t < here ? 16u : 0u;
            cp_async16(dst + tile_off<kDw>(t, cc), k + t * C::kD + cc * 16, n);
            if (!kShared) cp_async16(dst + kTile * kDw + tile_off<kDw>(t, cc), v + t * C::kD + cc * 16, n);
          }
        }
      }
      cp_async_commit();
    };
#pragma unroll
    for (int s = 0; s < C::kStages - 1; ++s) issue(s);
    // Their scales are kept as the block numbers are, a lane to a tile; the next 32 are asked for half way through.  A block that does
    // not exist gets a negative one.
    float ks_now, vs_now, ks_next = 1.0f, vs_next = -1.0f;
    auto ask_scales = [&](int32_t b, float& k, float& v) {
      const bool ok = b >= 0 && static_cast<uint32_t>(b) < a.c.num_blocks;
      const size_t at = static_cast<size_t>(ok ? b : 0) * H + h;
      k = ld_ahead(a.c.k_scale + at);
      v = kShared ? k : ld_ahead(a.c.v_scale + at);
      v = ok ? v : -1.0f;
    };
    ask_scales(blocks_now, ks_now, vs_now);
    __syncthreads();  // s_nan and s_any_nan are cleared before any warp marks them; the copies are on their way meanwhile

    // ---- query fragments of rows g and g + 8 (few rows: of row g, and what belongs to it handed to the lanes with columns 2q and 2q + 1)
    uint32_t qf[kDw / 16][4];
    float rf[2];     // undoes the row's scaling
    int64_t vis[2];  // entries the row sees
    const uint32_t vis_min =
        static_cast<uint32_t>(q8_visible(item.kv_len, item.q_len - 1 - item.row0 / G, item.phase, a.ratio));
#pragma unroll
    for (int r = 0; r < (kFew ? 1 : 2); ++r) {
      const uint32_t row = g + 8 * r;
      const bool in = row < rows;
      const uint32_t rho = item.row0 + (in ? row : 0);
      const uint32_t i = rho / G, hg = rho % G;
      vis[r] = in ? q8_visible(item.kv_len, item.q_len - 1 - i, item.phase, a.ratio) : 0x7FFFFFFF;
      const __nv_bfloat16* p =
          a.q + (static_cast<size_t>(item.q_start + i) * a.n_heads + h * G + hg) * C::kD + half * kDw;
      rf[r] = load_query<kDw>(p, in, q, r, qf);
    }
    if (kFew) {
      const float rf_g = rf[0];
      const int vis_g = static_cast<int>(vis[0]);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        rf[e] = __shfl_sync(0xFFFFFFFFu, rf_g, (2 * q + e) * 4);
        vis[e] = __shfl_sync(0xFFFFFFFFu, vis_g, (2 * q + e) * 4);
      }
    }
    // Score e of half n is that of row r = row_of(e) of this lane's two, and entry score_entry(n, e) of the tile
    constexpr int kHalves = kFew ? 1 : 2;
    auto row_of = [](int e) { return kFew ? e & 1 : e >> 1; };
    auto score_entry = [&](int n, int e) { return kFew ? (e >> 1) * 8 + g : n * 8 + 2 * q + (e & 1); };

    float o[kOt][4];
#pragma unroll
    for (int i = 0; i < kOt; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.0f;
    float m[2] = {-3.4e38f, -3.4e38f}, l[2] = {0.0f, 0.0f};

    for (uint32_t i = 0; i < n_mine; ++i) {
      cp_async_wait<C::kStages - 2>();
      __syncwarp();  // every lane's copies of this tile are in; every lane has read the tile before it
      issue(i + C::kStages - 1);  // into the stage that the previous tile left
      const uint32_t st = ring + (i % C::kStages) * C::kStageBytes;
      if ((i & 31) == 16) ask_scales(blocks_next, ks_next, vs_next);  // (the copies are less than 16 tiles ahead)
      if ((i & 31) == 0 && i != 0) {
        ks_now = ks_next;
        vs_now = vs_next;
      }
      const float k_scale = __shfl_sync(0xFFFFFFFFu, ks_now, i & 31), v_scale = __shfl_sync(0xFFFFFFFFu, vs_now, i & 31);
      const bool tile_ok = v_scale > 0.0f;
      // scores
      float s[kHalves][4];
      if constexpr (kFew)
        tile_scores_t<kDw>(st, g, q, qf, s[0]);
      else
        tile_scores<kDw>(st, g, q, qf, s);
      float f[2] = {rf[0] * a.scale_log2, rf[1] * a.scale_log2};
      if (kNp == 2) {  // the two warps of a row add their halves of the channels
        float* own = s_x[grp][i & 1][half];
        const float* other = s_x[grp][i & 1][half ^ 1];
#pragma unroll
        for (int n = 0; n < kHalves; ++n) {
#pragma unroll
          for (int e = 0; e < 4; ++e) s[n][e] *= rf[row_of(e)];
          *reinterpret_cast<float4*>(own + n * 128 + lane * 4) = make_float4(s[n][0], s[n][1], s[n][2], s[n][3]);
        }
        asm volatile("bar.sync %0, 64;" ::"r"(1 + grp) : "memory");
#pragma unroll
        for (int n = 0; n < kHalves; ++n) {
          const float4 x = *reinterpret_cast<const float4*>(other + n * 128 + lane * 4);
          s[n][0] += x.x;  // addition commutes: both warps get the same sums
          s[n][1] += x.y;
          s[n][2] += x.z;
          s[n][3] += x.w;
        }
        f[0] = f[1] = a.scale_log2;
      }
      f[0] *= k_scale;
      f[1] *= k_scale;
      const float lv = __log2f(v_scale), iv = rcp(v_scale);
      const uint32_t e0 = entry_of(i);
      const bool edge = e0 + kTile > min(vis_min, item.kv_end) || !tile_ok;
#pragma unroll
      for (int n = 0; n < kHalves; ++n) {
#pragma unroll
        for (int e = 0; e < 4; ++e) s[n][e] = fmaf(s[n][e], f[row_of(e)], lv);
      }
      if (edge) {
#pragma unroll
        for (int n = 0; n < kHalves; ++n) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int64_t at = e0 + score_entry(n, e);
            if (at >= vis[row_of(e)] || at >= item.kv_end || !tile_ok) s[n][e] = -INFINITY;
          }
        }
      }
      // raise the reference where a score passes it by 14
      float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int n = 0; n < kHalves; ++n) {
#pragma unroll
        for (int e = 0; e < 4; ++e) top[row_of(e)] = fmaxf(top[row_of(e)], s[n][e]);
      }
      if (__any_sync(0xFFFFFFFFu, top[0] > m[0] + 14.0f || top[1] > m[1] + 14.0f)) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
#pragma unroll
          for (int x = kFew ? 4 : 1; x < (kFew ? 32 : 4); x <<= 1) top[r] = fmaxf(top[r], __shfl_xor_sync(0xFFFFFFFFu, top[r], x));
          const float now = fmaxf(m[r], top[r] - 6.0f);
          const float c = ex2(m[r] - now);
          m[r] = now;
          l[r] *= c;
#pragma unroll
          for (int x = 0; x < kOt; ++x) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (row_of(e) == r) o[x][e] *= c;
          }
        }
      }
      uint32_t p[2 * kHalves];
#pragma unroll
      for (int n = 0; n < kHalves; ++n) {
        const float w0 = ex2(s[n][0] - m[row_of(0)]), w1 = ex2(s[n][1] - m[row_of(1)]);
        const float w2 = ex2(s[n][2] - m[row_of(2)]), w3 = ex2(s[n][3] - m[row_of(3)]);
        if (kFew) {
          l[0] = fmaf(w0 + w2, iv, l[0]);
          l[1] = fmaf(w1 + w3, iv, l[1]);
        } else {
          l[0] = fmaf(w0 + w1, iv, l[0]);
          l[1] = fmaf(w2 + w3, iv, l[1]);
        }
        p[2 * n] = pack_f16x2(w0, w1);
        p[2 * n + 1] = pack_f16x2(w2, w3);
      }
      if (kFew) {  // from (entry g, rows 2q and 2q + 1) to (row g, entries 2q and 2q + 1)
        p[0] = transpose8(p[0]);
        p[1] = transpose8(p[1]);
      }
      // values.  A NaN must not reach rows that do not see its entry (0 * NaN): where some entries are hidden,
      // NaNs are taken out, and put back at the end into the rows that see them (s_nan).
      const uint32_t vt = kShared ? st : st + kTile * kDw;
      auto two_words = [&](uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, float(*acc)[4]) {
#pragma unroll
        for (int z = 0; z < 2; ++z) {  // two channels of the word
          const uint32_t lo = __byte_perm(a0, a1, z ? 0x7362 : 0x5140), hi = __byte_perm(a2, a3, z ? 0x7362 : 0x5140);
          if constexpr (kFew) {
            const uint32_t vf[4] = {q8_lo_f16x2(lo), q8_hi_f16x2(lo), q8_lo_f16x2(hi), q8_hi_f16x2(hi)};
            mma_f16(acc[z], vf, p[0], p[1]);
          } else {
            mma_f16(acc[2 * z], p, q8_lo_f16x2(lo), q8_lo_f16x2(hi));
            mma_f16(acc[2 * z + 1], p, q8_hi_f16x2(lo), q8_hi_f16x2(hi));
          }
        }
      };
      constexpr int kPerWord = kFew ? 2 : 4;  // output tiles of a word
      if (kDw == 64) {
        uint2 w[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const uint32_t t = 2 * q + (x & 1) + (x >> 1) * 8;
          w[x] = lds8(vt + tile_off<kDw>(t, g >> 1) + (g & 1) * 8);
          if (edge) {
            w[x].x = without_nan(w[x].x, e0 + t, s_nan + g * 8, &s_any_nan);
            w[x].y = without_nan(w[x].y, e0 + t, s_nan + g * 8 + 4, &s_any_nan);
          }
        }
        two_words(w[0].x, w[1].x, w[2].x, w[3].x, o);
        two_words(w[0].y, w[1].y, w[2].y, w[3].y, o + kPerWord);
      } else {
#pragma unroll
        for (int jj = 0; jj < kDw / 128; ++jj) {
          uint4 w[4];
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const uint32_t t = 2 * q + (x & 1) + (x >> 1) * 8;
            w[x] = lds16(vt + tile_off<kDw>(t, 8 * jj + g));
            if (edge) {
              int* nan = s_nan + half * kDw + (8 * jj + g) * 16;
              w[x].x = without_nan(w[x].x, e0 + t, nan, &s_any_nan);
              w[x].y = without_nan(w[x].y, e0 + t, nan + 4, &s_any_nan);
              w[x].z = without_nan(w[x].z, e0 + t, nan + 8, &s_any_nan);
              w[x].w = without_nan(w[x].w, e0 + t, nan + 12, &s_any_nan);
            }
          }
          two_words(w[0].x, w[1].x, w[2].x, w[3].x, o + (jj * 4 + 0) * kPerWord);
          two_words(w[0].y, w[1].y, w[2].y, w[3].y, o + (jj * 4 + 1) * kPerWord);
          two_words(w[0].z, w[1].z, w[2].z, w[3].z, o + (jj * 4 + 2) * kPerWord);
          two_words(w[0].w, w[1].w, w[2].w, w[3].w, o + (jj * 4 + 3) * kPerWord);
        }
      }
    }
    cp_async_wait<0>();
    if (bad_block && lane == 0) status_or(a.d_status, CKV_STATUS_BAD_INDEX);
    __syncthreads();  // the rings are idle: they become the merge area

    // ---- join the warps
    constexpr int kRun = kDw == 64 ? 8 : 16;  // consecutive channels of a lane
    float* merge = reinterpret_cast<float*>(smem) + grp * kRows * C::kMergeStride;
    if constexpr (kFew) {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) l[r] += __shfl_xor_sync(0xFFFFFFFFu, l[r], x);
        if (g == 0 && half == 0) {
          s_m[grp][2 * q + r] = m[r];
          s_l[grp][2 * q + r] = l[r];
        }
      }
#pragma unroll
      for (int x = 0; x < kOt; x += 2) {
        const int ch = half * kDw + (8 * (x / (kRun / 2)) + g) * kRun + 2 * (x % (kRun / 2));
#pragma unroll
        for (int r = 0; r < 2; ++r)
          *reinterpret_cast<float4*>(merge + (2 * q + r) * C::kMergeStride + ch) =
              make_float4(o[x][r], o[x][2 + r], o[x + 1][r], o[x + 1][2 + r]);
      }
    } else {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        l[r] += __shfl_xor_sync(0xFFFFFFFFu, l[r], 1);
        l[r] += __shfl_xor_sync(0xFFFFFFFFu, l[r], 2);
        if (q == 0 && half == 0) {
          s_m[grp][g + 8 * r] = m[r];
          s_l[grp][g + 8 * r] = l[r];
        }
      }
#pragma unroll
      for (int x = 0; x < kOt; x += 4) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
#pragma unroll
          for (int n = 0; n < 2; ++n) {  // column 2q + n of tile x: channel (8 (x / run) + 2q + n) * run + x % run
            const int ch = half * kDw + (8 * (x / kRun) + 2 * q + n) * kRun + x % kRun;
            *reinterpret_cast<float4*>(merge + (g + 8 * r) * C::kMergeStride + ch) =
                make_float4(o[x][2 * r + n], o[x + 1][2 * r + n], o[x + 2][2 * r + n], o[x + 3][2 * r + n]);
          }
        }
      }
    }
    __syncthreads();
    constexpr int kPerRow = kAttnThreads / kRows;  // threads of a row
    const uint32_t row = tid / kPerRow;
    if (row < rows) {
      float top = s_m[0][row];
#pragma unroll
      for (int w = 1; w < C::kGroups; ++w) top = fmaxf(top, s_m[w][row]);
      float c[C::kGroups], sum = 0.0f;
#pragma unroll
      for (int w = 0; w < C::kGroups; ++w) {
        c[w] = ex2(s_m[w][row] - top);
        sum = fmaf(s_l[w][row], c[w], sum);
      }
      const uint32_t rho = item.row0 + row, i = rho / G, hg = rho % G;
      const int64_t see = q8_visible(item.kv_len, item.q_len - 1 - i, item.phase, a.ratio);
      const size_t out_row = static_cast<size_t>(item.q_start + i) * a.n_heads + h * G + hg;
      const size_t part_row = (static_cast<size_t>(item.part + static_cast<int>(item.chunk)) * H + h) * kRows + row;
      const float inv = sum == 0.0f ? 0.0f : __fdiv_rn(1.0f, sum);
      const int any_nan = s_any_nan;
      for (int ch = tid % kPerRow * 4; ch < C::kD; ch += kPerRow * 4) {
        float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int w = 0; w < C::kGroups; ++w) {
          const float4 x = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(smem) +
                                                            (w * kRows + row) * C::kMergeStride + ch);
          v[0] = fmaf(x.x, c[w], v[0]);
          v[1] = fmaf(x.y, c[w], v[1]);
          v[2] = fmaf(x.z, c[w], v[2]);
          v[3] = fmaf(x.w, c[w], v[3]);
        }
        if (any_nan) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (s_nan[ch + e] < see) v[e] = __int_as_float(0x7FFFFFFF);
        }
        if (item.part >= 0) {
          *reinterpret_cast<float4*>(a.part_o + part_row * C::kD + ch) = make_float4(v[0], v[1], v[2], v[3]);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] *= inv;
          if (a.out_f32)
            store_row_chunk<float, 4>(static_cast<float*>(a.out) + out_row * C::kD + ch, v);
          else
            store_row_chunk<__nv_bfloat16, 4>(static_cast<__nv_bfloat16*>(a.out) + out_row * C::kD + ch, v);
        }
      }
      if (tid % kPerRow == 0) {
        if (item.part >= 0)
          a.part_ml[part_row] = make_float2(top, sum);
        else if (a.lse != nullptr)
          a.lse[out_row] = sum == 0.0f ? -INFINITY : (top + __log2f(sum)) * 0.69314718055994530942f;
      }
    }
  }
}

// ------------------------------------------------------------------- combine
// Joins a split tile's parts, in their order.  Where the parts are few a warp takes a
// row, so that a row is two trips to memory and no barrier, and a CTA eight rows; else
// the whole CTA takes a row: work number y + x * (rows / 8) is row x of the eight y,
// and only tiles of many parts have work beyond x = 0.  Bound: the parts' bytes (128 KB a part of 64 rows and 512 channels, 40 MB in
// 12 us), or two trips to memory (8 us from launch to end).
constexpr int kCombineThreads = 256;
constexpr int kCombineRows = kCombineThreads / 32;
constexpr uint32_t kFewParts = 16;
constexpr int kMaxParts = 2048;

__device__ __forceinline__ void store_out(const AttnArgs& a, size_t out_row, int d, int ch, float4 v, float inv) {
  const float r[4] = {v.x * inv, v.y * inv, v.z * inv, v.w * inv};
  if (a.out_f32)
    store_row_chunk<float, 4>(static_cast<float*>(a.out) + out_row * d + ch, r);
  else
    store_row_chunk<__nv_bfloat16, 4>(static_cast<__nv_bfloat16*>(a.out) + out_row * d + ch, r);
}

__device__ __forceinline__ void add_scaled(float4& v, const float4 x, float w) {
  v.x = fmaf(x.x, w, v.x);
  v.y = fmaf(x.y, w, v.y);
  v.z = fmaf(x.z, w, v.z);
  v.w = fmaf(x.w, w, v.w);
}

template <int kD>
__global__ __launch_bounds__(kCombineThreads) void q8_combine_kernel(const AttnArgs a) {
  constexpr int kLanes = kD / 4, kSplit = kCombineThreads / kLanes;
  __shared__ float s_w[kMaxParts], s_l[kMaxParts];
  __shared__ float s_red[kCombineThreads / 32];
  __shared__ float4 s_o[kCombineThreads];
  pdl_wait();
  pdl_release();
  const Q8Header* head = reinterpret_cast<const Q8Header*>(a.plan);
  if (!plan_fits(head, a)) return;
  const uint32_t G = a.g.group, H = a.c.heads, M = a.g.rows;
  const uint32_t* splits = reinterpret_cast<const uint32_t*>(a.plan + a.g.off_split);
  const Q8Item* items = reinterpret_cast<const Q8Item*>(a.plan + a.g.off_items);
  const uint32_t eights = min(head->splits, a.g.ctas) * H * (M / kCombineRows);
  const uint32_t work = head->most > kFewParts ? eights * kCombineRows : eights;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (uint32_t x = blockIdx.x; x < work; x += gridDim.x) {
    const uint32_t y = x % eights, of = M / kCombineRows, sub = x / eights;
    const uint32_t row0 = y % of * kCombineRows + sub, h = y / of % H, first = splits[y / of / H];
    if (first >= a.g.cap_items) continue;
    const Q8Item item = items[first];
    const uint64_t rows_left = static_cast<uint64_t>(item.q_len) * G - item.row0;
    if (!item_fits(item, a) || item.part < 0 || item.chunks > kMaxParts || row0 >= rows_left) continue;
    const size_t step = static_cast<size_t>(H) * M;
    if (item.chunks <= kFewParts) {
      if (sub != 0 || row0 + warp >= rows_left) continue;
      const uint32_t row = row0 + warp;
      const size_t r0 = (static_cast<size_t>(item.part) * H + h) * M + row;
      const bool in = static_cast<uint32_t>(lane) < item.chunks;
      const float2 ml = in ? a.part_ml[r0 + lane * step] : make_float2(-3.4e38f, 0.0f);
      float top = ml.x;
#pragma unroll
      for (int s = 16; s > 0; s >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, s));
      const float w = in ? ex2(ml.x - top) : 0.0f;
      float sum = ml.y * w;
#pragma unroll
      for (int s = 16; s > 0; s >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, s);
      const float inv = sum == 0.0f ? 0.0f : __fdiv_rn(1.0f, sum);
      constexpr int kVecs = kD < 128 ? 1 : kD / 128;
      const bool own = kD >= 128 || lane < kLanes;
      float4 v[kVecs];
#pragma unroll
      for (int z = 0; z < kVecs; ++z) v[z] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      const float* o = a.part_o + r0 * kD + lane * 4;
#pragma unroll 4
      for (uint32_t p = 0; p < item.chunks; ++p) {
        const float wp = __shfl_sync(0xFFFFFFFFu, w, p);
#pragma unroll
        for (int z = 0; z < kVecs; ++z)
          if (own) add_scaled(v[z], *reinterpret_cast<const float4*>(o + p * step * kD + z * 128), wp);
      }
      const uint32_t rho = item.row0 + row, i = rho / G, hg = rho % G;
      const size_t out_row = static_cast<size_t>(item.q_start + i) * a.n_heads + h * G + hg;
#pragma unroll
      for (int z = 0; z < kVecs; ++z)
        if (own) store_out(a, out_row, kD, lane * 4 + z * 128, v[z], inv);
      if (lane == 0 && a.lse != nullptr)
        a.lse[out_row] = sum == 0.0f ? -INFINITY : (top + __log2f(sum)) * 0.69314718055994530942f;
      continue;
    }
    const size_t r0 = (static_cast<size_t>(item.part) * H + h) * M + row0;
    __syncthreads();  // the previous row's reads of shared memory are done
    float top = -3.4e38f;
    for (uint32_t p = tid; p < item.chunks; p += kCombineThreads) {
      const float2 ml = a.part_ml[r0 + p * step];
      s_w[p] = ml.x;
      s_l[p] = ml.y;
      top = fmaxf(top, ml.x);
    }
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, s));
    if (lane == 0) s_red[warp] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kCombineThreads / 32; ++w) top = fmaxf(top, s_red[w]);
    __syncthreads();
    float sum = 0.0f;
    for (uint32_t p = tid; p < item.chunks; p += kCombineThreads) {
      const float w = ex2(s_w[p] - top);
      s_w[p] = w;
      sum = fmaf(s_l[p], w, sum);
    }
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, s);
    if (lane == 0) s_red[warp] = sum;
    __syncthreads();
    sum = 0.0f;
#pragma unroll
    for (int w = 0; w < kCombineThreads / 32; ++w) sum += s_red[w];
    const int ch = (tid % kLanes) * 4;
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
    for (uint32_t p = tid / kLanes; p < item.chunks; p += kSplit)
      add_scaled(v, *reinterpret_cast<const float4*>(a.part_o + (r0 + p * step) * kD + ch), s_w[p]);
    s_o[tid] = v;
    __syncthreads();
    if (tid < kLanes) {
      for (int k = 1; k < kSplit; ++k) add_scaled(v, s_o[tid + k * kLanes], 1.0f);
      const uint32_t rho = item.row0 + row0, i = rho / G, hg = rho % G;
      const size_t out_row = static_cast<size_t>(item.q_start + i) * a.n_heads + h * G + hg;
      store_out(a, out_row, kD, ch, v, sum == 0.0f ? 0.0f : __fdiv_rn(1.0f, sum));
      if (tid == 0 && a.lse != nullptr)
        a.lse[out_row] = sum == 0.0f ? -INFINITY : (top + __log2f(sum)) * 0.69314718055994530942f;
    }
  }
}

template <int kDw, int kNp, bool kShared, int kRows>
int launch_attn(const AttnArgs& a, cudaStream_t s) {
  using C = Cfg<kDw, kNp, kShared, kRows>;
  auto* kernel = q8_attn_kernel<kDw, kNp, kShared, kRows>;
  static std::atomic<uint64_t> done;
  const int rc = allow_smem(reinterpret_cast<const void*>(kernel), C::kSmem, done);
  if (rc) return rc;
  return launch_pdl(kernel, dim3(a.g.ctas, a.c.heads), dim3(kAttnThreads), C::kSmem, s, a);
}

template <int kRows>
int launch_split(const AttnArgs& a, cudaStream_t s) {
  const bool shared = a.c.v == nullptr;
  switch (a.c.head_dim) {
    case 64: return shared ? launch_attn<64, 1, true, kRows>(a, s) : launch_attn<64, 1, false, kRows>(a, s);
    case 128: return shared ? launch_attn<128, 1, true, kRows>(a, s) : launch_attn<128, 1, false, kRows>(a, s);
    case 256: return shared ? launch_attn<256, 1, true, kRows>(a, s) : launch_attn<256, 1, false, kRows>(a, s);
    default: return shared ? launch_attn<256, 2, true, kRows>(a, s) : launch_attn<256, 2, false, kRows>(a, s);
  }
}

int launch_combine(const AttnArgs& a, cudaStream_t s) {
  // at most four CTAs to an SM; they walk the rows
  const uint64_t rows = static_cast<uint64_t>(a.g.ctas) * a.c.heads * a.g.rows;
  const dim3 grid(static_cast<uint32_t>(std::min<uint64_t>(rows, 4ull * sm_count())));
  switch (a.c.head_dim) {
    case 64: return launch_pdl(q8_combine_kernel<64>, grid, dim3(kCombineThreads), 0, s, a);
    case 128: return launch_pdl(q8_combine_kernel<128>, grid, dim3(kCombineThreads), 0, s, a);
    case 256: return launch_pdl(q8_combine_kernel<256>, grid, dim3(kCombineThreads), 0, s, a);
    default: return launch_pdl(q8_combine_kernel<512>, grid, dim3(kCombineThreads), 0, s, a);
  }
}

}  // namespace
}  // namespace ckv

using namespace ckv;

extern "C" {

uint64_t ckv_q8_attn_plan_bytes(const ckv_q8_cache_t* cache, uint32_t n_heads, uint32_t batch, uint32_t num_q) {
  Q8Cache c;
  Q8Geom g;
  if (q8_cache_of(cache, &c) || q8_attn_geom(c, batch, num_q, n_heads, &g)) return 0;
  return g.bytes;
}

uint64_t ckv_q8_attn_workspace_bytes(const ckv_q8_cache_t* cache, uint32_t n_heads, uint32_t batch, uint32_t num_q) {
  Q8Cache c;
  Q8Geom g;
  if (q8_cache_of(cache, &c) || q8_attn_geom(c, batch, num_q, n_heads, &g)) return 0;
  return g.workspace;
}

int ckv_plan_q8_attn(const ckv_q8_cache_t* cache, uint32_t n_heads, uint32_t ratio, const int64_t* rid,
                     const int64_t* seq_lens, const int64_t* extend_lens, const int64_t* kv_lens, uint32_t batch,
                     uint32_t num_q, void* plan, uint64_t plan_bytes, uint32_t* d_status, ckv_stream_t stream) {
  Q8Cache c;
  AttnPlanArgs a{};
  int rc = q8_cache_of(cache, &c);
  if (rc) return rc;
  if (ratio == 0 || ratio > 65536) return CKV_ERR_RATIO;
  rc = q8_attn_geom(c, batch, num_q, n_heads, &a.g);
  if (rc) return rc;
  if (plan_bytes < a.g.bytes) return CKV_ERR_SIZE;
  if (!aligned16(plan)) return CKV_ERR_POINTER;
  if (batch > 0 &&
      (!aligned_to(rid, 8) || !aligned_to(seq_lens, 8) || !aligned_to(extend_lens, 8) || !aligned_to(kv_lens, 8)))
    return CKV_ERR_POINTER;
  a.rid = rid;
  a.seq_lens = seq_lens;
  a.extend_lens = extend_lens;
  a.kv_lens = kv_lens;
  a.batch = batch;
  a.num_q = num_q;
  a.ratio = ratio;
  a.plan = static_cast<uint8_t*>(plan);
  a.d_status = d_status;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return batch <= 256 ? launch_pdl(plan_q8_attn_kernel<256>, dim3(1), dim3(256), 0, s, a)
                      : launch_pdl(plan_q8_attn_kernel<1024>, dim3(1), dim3(1024), 0, s, a);
}

int ckv_q8_attn(const ckv_q8_cache_t* cache, uint32_t n_heads, uint32_t ratio, float scale, const void* q,
                uint32_t batch, uint32_t num_q, const int32_t* block_table, uint64_t table_stride, uint32_t num_reqs,
                const void* plan, uint64_t plan_bytes, int out_dtype, void* out, float* lse, void* workspace,
                uint64_t workspace_bytes, uint32_t* d_status, ckv_stream_t stream) {
  AttnArgs a{};
  int rc = q8_cache_of(cache, &a.c);
  if (rc) return rc;
  if (ratio == 0 || ratio > 65536) return CKV_ERR_RATIO;
  if (out_dtype != CKV_F32 && out_dtype != CKV_BF16) return CKV_ERR_DTYPE;
  if (!(scale > 0.0f) || !(scale < 1e30f)) return CKV_ERR_SIZE;
  rc = q8_attn_geom(a.c, batch, num_q, n_heads, &a.g);
  if (rc) return rc;
  if (num_q == 0 || batch == 0) return CKV_OK;
  rc = check_table(block_table, table_stride, num_reqs);
  if (rc) return rc;
  if (plan_bytes < a.g.bytes || workspace_bytes < a.g.workspace) return CKV_ERR_SIZE;
  if (!aligned16(q) || !aligned16(plan) || !aligned16(out) || !aligned16(workspace) ||
      (lse != nullptr && !aligned_to(lse, 4)))
    return CKV_ERR_POINTER;
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.batch = batch;
  a.num_q = num_q;
  a.n_heads = n_heads;
  a.ratio = ratio;
  a.scale_log2 = scale * kLog2e;
  a.table = block_table;
  a.stride = static_cast<uint32_t>(table_stride);
  a.num_reqs = num_reqs;
  a.plan = static_cast<const uint8_t*>(plan);
  a.out_f32 = out_dtype == CKV_F32;
  a.out = out;
  a.lse = lse;
  a.part_o = static_cast<float*>(workspace);
  a.part_ml = reinterpret_cast<float2*>(a.part_o + static_cast<size_t>(a.g.cap_parts) * a.c.heads * a.g.rows * a.c.head_dim);
  a.d_status = d_status;
  a.wait_ns = wait_limit_ns();
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  rc = !a.g.tc ? (a.g.rows == 8 ? launch_split<8>(a, s) : launch_split<16>(a, s)) : a.c.head_dim <= 128 ? launch_q8_attn_rows(a, s) : launch_q8_attn_tc(a, s);
  return rc ? rc : launch_combine(a, s);
}

}  // extern "C"

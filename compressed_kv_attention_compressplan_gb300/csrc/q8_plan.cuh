// q8_plan.cuh -- the attention plan over the 8-bit paged cache: how a step's
// (request, row tile) work is cut into equal shares, and where it lies.
//
// Work.  The rows of a request for one kv head are its q_len * group (query,
// head) pairs; a tile is `rows` consecutive ones, and its cost is the entries
// its last row sees, in units of entries, plus a fixed start-up.
// The tiles' costs are laid end to end and cut at multiples of one quota, so
// every CTA of a kv head gets the same number of entries whatever the lengths
// are (one wave, no tail); a tile that a cut crosses leaves partial results,
// which the combine kernel joins.  One plan serves every layer of a step.
//
// Buffer: header | first item of each CTA | first item of each split tile | items.
#pragma once

#include "q8.cuh"

namespace ckv {

struct alignas(16) Q8Item {  // 48 bytes, read and written 16 at a time
  uint32_t rid;
  uint32_t q_start;   // ragged query of the request's first row
  uint32_t q_len;
  uint32_t row0;      // the tile's first row
  uint32_t kv_begin;  // entries of this item
  uint32_t kv_end;
  uint32_t kv_len;    // of the request
  uint32_t phase;     // see q8_visible
  int32_t part;       // first partial slot of the tile; -1: this item is the whole tile
  uint32_t chunk;     // this item's number among the tile's
  uint32_t chunks;
  uint32_t reserved;
};
static_assert(sizeof(Q8Item) == 48, "");

struct Q8Header {  // 64 bytes
  uint32_t items;
  uint32_t ctas;
  uint32_t parts;
  uint32_t splits;
  uint32_t rows;  // the geometry the plan was made for; the attention checks it
  uint32_t group;
  uint32_t num_q;
  uint32_t ratio;
  uint32_t cap_ctas;
  uint32_t batch;
  uint32_t most;  // parts of the tile that has most
  uint32_t reserved[5];
};
static_assert(sizeof(Q8Header) == 64, "");

struct Q8Geom {
  bool tc;             // the tensor-core kernel takes it, not the split kernel
  uint32_t start_cost; // entries that starting a tile costs; a multiple of 16
  uint32_t rows;       // rows of a tile
  uint32_t group;      // query heads of a kv head
  uint32_t ctas;       // CTAs of a kv head
  uint32_t min_quota;  // entries
  uint32_t grain;      // entries are counted in these, and the quota is a multiple: 16, or the tensor-core kernels' tile
  uint32_t cap_items;
  uint32_t cap_parts;
  uint64_t off_first, off_split, off_items, bytes;
  uint64_t workspace;
};

// From sizes alone (and the device's SM count), the same for the plan and the
// attention call.  CKV_OK or CKV_ERR_SIZE.
int q8_attn_geom(const Q8Cache& c, uint32_t batch, uint32_t num_q, uint32_t n_heads, Q8Geom* g);
// Any batch.  many: lists of several queries a request: the split kernel hides its items' starts with more CTAs an SM instead of
// memory's latency with deeper rings (ckv_q8_attn_blocks has the rule).
int q8_attn_geom_of(const Q8Cache& c, uint32_t batch, uint32_t num_q, uint32_t n_heads, bool many, Q8Geom* g);

// Arguments of the attention kernels.
struct AttnArgs {
  Q8Cache c;
  Q8Geom g;
  const __nv_bfloat16* q;
  uint32_t batch;
  uint32_t num_q;
  uint32_t n_heads;
  uint32_t ratio;
  float scale_log2;
  const int32_t* table;
  uint32_t stride;
  uint32_t num_reqs;
  const uint32_t* lens;  // NULL; or a table for each (request, kv head), and its entries here
  bool many;             // see q8_attn_geom_of
  const uint8_t* plan;
  int out_f32;
  void* out;
  float* lse;
  float* part_o;    // [part][kv head][row][head_dim]
  float2* part_ml;  // [part][kv head][row]
  uint64_t wait_ns;
  uint32_t* d_status;
};

__device__ __forceinline__ bool item_fits(const Q8Item& item, const AttnArgs& a) {
  return item.rid < a.num_reqs && static_cast<uint64_t>(item.q_start) + item.q_len <= a.num_q &&
         item.row0 < static_cast<uint64_t>(item.q_len) * a.g.group &&
         item.kv_len <= static_cast<uint64_t>(a.stride) * a.c.block_tokens && item.kv_end <= item.kv_len &&
         (item.part < 0 || (static_cast<uint64_t>(item.part) + item.chunks <= a.g.cap_parts && item.chunk < item.chunks));
}

__device__ __forceinline__ bool plan_fits(const Q8Header* h, const AttnArgs& a) {
  return h->rows == a.g.rows && h->group == a.g.group && h->num_q == a.num_q && h->ratio == a.ratio &&
         h->cap_ctas == a.g.ctas && h->batch == a.batch;
}

// An item, and its block table, for kv head h.  Where the heads have tables of their own (kLists), the item, which was planned
// for the longest, is cut down to the head's entries.  A template: the same test at run time cost a prefill chunk 1.8 %.
// kWords: read by words, where registers in fours would spill (the 8-bit kernel).
template <bool kLists, bool kWords = false>
__device__ __forceinline__ Q8Item item_for(const Q8Item* at, const AttnArgs& a, uint32_t h) {
  Q8Item r;
  if constexpr (kWords) {
    const uint32_t* from = reinterpret_cast<const uint32_t*>(at);
    uint32_t* to = reinterpret_cast<uint32_t*>(&r);
#pragma unroll
    for (int w = 0; w < static_cast<int>(sizeof(Q8Item) / 4); ++w) to[w] = from[w];
  } else {
    r = *at;
  }
  if (kLists) {  // as they were planned
    r.q_start = r.rid;
    r.q_len = 1;
    r.phase = 0;
  }
  if (kLists && r.rid < a.num_reqs) {
    r.kv_len = min(r.kv_len, a.lens[static_cast<size_t>(r.rid) * a.c.heads + h]);
    r.kv_end = min(r.kv_end, r.kv_len);
    r.kv_begin = min(r.kv_begin, r.kv_end);
  }
  return r;
}
template <bool kLists>
__device__ __forceinline__ const int32_t* table_for(const AttnArgs& a, const Q8Item& item, uint32_t h) {
  return a.table + (kLists ? static_cast<size_t>(item.rid) * a.c.heads + h : static_cast<size_t>(item.rid)) * a.stride;
}

// Takes the NaNs out of a word of four channels of entry e, noting the first entry with one for each channel.
__device__ __forceinline__ uint32_t without_nan(uint32_t w, int e, int* s_nan, int* s_any_nan) {
  const uint32_t bad = q8_nan_bytes(w);
  if (bad) {
    for (int z = 0; z < 4; ++z)
      if (bad >> (8 * z) & 1) atomicMin(s_nan + z, e);
    *s_any_nan = 1;
  }
  return w & ~bad;
}

// ---------------------------------------------------------------- cutting
template <int kThreads>
struct CutShared {
  unsigned long long pos[kThreads];
  uint32_t item[kThreads], part[kThreads];
  unsigned long long scan[2][kThreads / 32 + 1];
  uint32_t most, longest;
};

// Lays nt tiles' costs end to end, cuts them at multiples of one quota and writes the plan: header, first items, split tiles and items.
// Fewer tiles than CTAs may be cut evenly instead (kEven), each into pieces of one length and a CTA to a piece: no CTA then starts
// two tiles, which is most of a piece's time where tiles are short (64 lists of 32 blocks, latent: 59 us instead of 67).
// By one CTA, whose threads all call it.  tiles(tile, item) gives a tile's entries (kInvalidU32: the tile
// is left out) and, where item is not NULL, its rid, q_start, q_len, row0, kv_len and phase.
template <int kThreads, bool kEven, typename Tiles>
__device__ __forceinline__ void cut_tiles(const Q8Geom& g, uint8_t* plan, uint32_t nt, uint32_t num_q, uint32_t ratio, uint32_t batch,
                                          const Tiles& tiles, CutShared<kThreads>& sh) {
  const uint32_t t = threadIdx.x;
  if (t == 0) sh.most = sh.longest = 0;  // the scans' barriers come before their use
  Q8Header* head = reinterpret_cast<Q8Header*>(plan);
  uint32_t* first = reinterpret_cast<uint32_t*>(plan + g.off_first);
  uint32_t* split = reinterpret_cast<uint32_t*>(plan + g.off_split);
  Q8Item* items = reinterpret_cast<Q8Item*>(plan + g.off_items);
  const uint32_t start = g.start_cost, grain = g.grain;  // grain is a power of two
  auto cost_of = [&](uint32_t seen) -> unsigned long long {
    if (seen == kInvalidU32) return 0;
    return start + ((static_cast<unsigned long long>(seen) + grain - 1) & ~static_cast<unsigned long long>(grain - 1));
  };
  unsigned long long mine = 0;
  for (uint32_t i = t; i < nt; i += kThreads) mine += cost_of(tiles(i, nullptr));
  unsigned long long total;
  const unsigned long long before = block_exclusive<kThreads>(mine, &total, sh.scan[0]);
  // 32-bit divisions where they do: a 64-bit one is some forty instructions that wait for one another, and there were ten
  const bool narrow = total <= 0x7FFFFFFFull;
  unsigned long long quota = narrow ? (static_cast<uint32_t>(total) + g.ctas - 1) / g.ctas : (total + g.ctas - 1) / g.ctas;
  quota = max(static_cast<unsigned long long>(g.min_quota), quota);
  quota = (quota + grain - 1) & ~static_cast<unsigned long long>(grain - 1);
  auto shares = [&](unsigned long long x) -> unsigned long long {  // x / quota, x <= total + quota
    return narrow ? static_cast<uint32_t>(x) / static_cast<uint32_t>(quota) : x / quota;
  };

  uint32_t piece = 0;  // entries of an even piece
  if (kEven && nt <= kThreads) {
    const uint32_t seen = t < nt ? tiles(t, nullptr) : kInvalidU32;
    if (seen != kInvalidU32) atomicMax(&sh.longest, seen);
    const uint32_t valid = __syncthreads_count(seen != kInvalidU32), pieces = valid ? g.ctas / valid : 0;
    if (pieces > 0) {
      const uint32_t len = max(g.min_quota, ((sh.longest + pieces - 1) / pieces + grain - 1) & ~(grain - 1));
      if (len <= quota) piece = len;
    }
  }

  unsigned long long pos0 = 0;
  uint32_t item0 = 0, part0 = 0, split0 = 0;
  for (uint32_t i0 = 0; i0 < nt; i0 += kThreads) {
    const uint32_t i = i0 + t;
    uint32_t n = 0;
    const unsigned long long cost = nt <= kThreads ? mine : i < nt ? cost_of(tiles(i, nullptr)) : 0;
    unsigned long long cost_sum = total, packed_sum, p = before;  // a single strip's sums are known
    if (nt > kThreads) p = pos0 + block_exclusive<kThreads>(cost, &cost_sum, sh.scan[0]);
    if (cost) n = static_cast<uint32_t>(shares(p + cost - 1) - shares(p)) + 1;
    if (kEven && piece && cost) n = max(1u, (tiles(i, nullptr) + piece - 1) / piece);
    // items (32 bits), parts (16) and splits (16) of the strip, in one scan: parts are at most twice the CTAs
    const unsigned long long pk = n | (static_cast<unsigned long long>(n > 1 ? n : 0) << 32) |
                                  (static_cast<unsigned long long>(n > 1) << 48);
    const unsigned long long ex = block_exclusive<kThreads>(pk, &packed_sum, sh.scan[0]);
    const uint32_t it = item0 + static_cast<uint32_t>(ex);
    sh.pos[t] = p;
    sh.item[t] = it;
    sh.part[t] = n > 1 ? part0 + (static_cast<uint32_t>(ex >> 32) & 0xFFFFu) : kInvalidU32;
    if (n > 1) {
      split[split0 + static_cast<uint32_t>(ex >> 48)] = it;
      atomicMax(&sh.most, n);
    }
    __syncthreads();
    const uint32_t strip = min(static_cast<uint32_t>(kThreads), nt - i0);
    const uint32_t end = item0 + static_cast<uint32_t>(packed_sum);
    for (uint32_t k = item0 + t; k < end; k += kThreads) {
      const uint32_t s = last_not_above(sh.item, strip, k);
      Q8Item r;
      const uint32_t seen = tiles(i0 + s, &r);
      if (kEven && piece) {
        r.chunk = k - sh.item[s];
        r.chunks = max(1u, (seen + piece - 1) / piece);
        r.kv_begin = r.chunk * piece;
        r.kv_end = min(seen, r.kv_begin + piece);
        r.part = static_cast<int32_t>(sh.part[s]);
        r.reserved = 0;
        items[k] = r;
        first[k] = k;
        continue;
      }
      const unsigned long long len = cost_of(seen);
      const unsigned long long P = sh.pos[s], cut = shares(P);
      const uint32_t c = k - sh.item[s];
      const unsigned long long lo = c == 0 ? P : (cut + c) * quota;
      const unsigned long long hi = min(P + len, (cut + c + 1) * quota);
      const unsigned long long o0 = lo - P, o1 = hi - P;
      r.kv_begin = o0 > start ? static_cast<uint32_t>(o0 - start) : 0;
      r.kv_end = o1 > start ? min(seen, static_cast<uint32_t>(o1 - start)) : 0;
      r.part = static_cast<int32_t>(sh.part[s]);
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
    const uint32_t ctas = kEven && piece ? item0 : static_cast<uint32_t>(shares(total + quota - 1));
    first[ctas] = item0;
    head->items = item0;
    head->ctas = ctas;
    head->parts = part0;
    head->splits = split0;
    head->rows = g.rows;
    head->group = g.group;
    head->num_q = num_q;
    head->ratio = ratio;
    head->cap_ctas = g.ctas;
    head->batch = batch;
    head->most = sh.most;  // (the last strip ended with a barrier)
  }
}

// All of an attention call but its plan.
int launch_q8_attn(const AttnArgs& a, cudaStream_t s);
// The tensor-core kernels, for tiles of many rows (g.tc); the parts that they leave are joined by the caller.
int launch_q8_attn_tc(const AttnArgs& a, cudaStream_t s);    // 256 channels and more
int launch_q8_attn_rows(const AttnArgs& a, cudaStream_t s);  // up to 128 channels

}  // namespace ckv

// q8_blocks.cu -- sparse attention over the 8-bit paged cache: which blocks each
// query reads, and the attention over them.
//
// Choosing.  A row is the scores of one (query, kv head).  Scores become order-preserving 32-bit keys; the key at the
// border is found, and the blocks above it, and as many at it as are missing, are listed in order with ballots.  No
// sum of rounded numbers is involved, so the choice is exact: equal scores go to the lower block.
//
// Attention.  A query's list for one kv head, looked up in its request's block table, is the block table of a request of
// its own with one query, which sees all of it: the listed blocks ascend, so that the one block of which a query
// sees a part is the last.  So the attention kernels take lists as they take requests; what is added is a
// table for each (query, kv head), the entries that it holds, and a plan over the queries, all made on the card.
#include <algorithm>

#include "q8_blocks.cuh"
#include "q8_plan.cuh"

namespace ckv {
namespace {

// ------------------------------------------------------------------- select
constexpr int kSelThreads = 256;

struct SelectArgs {
  const float* scores;
  BlockReqs r;
  uint32_t heads, width, block_tokens;
  uint32_t budget, sinks, recent;
  int32_t* blocks;
};

// Larger keys for larger scores; NaN below everything, the two zeros alike.
__device__ __forceinline__ uint32_t score_key(float w) {
  if (w != w) return 0;
  const uint32_t u = __float_as_uint(w + 0.0f);
  return u ^ (u >> 31 ? 0xFFFFFFFFu : 0x80000000u);
}

// Rows of up to 32 kKeys blocks: a warp takes a row, its keys in registers, block j in lane j % 32.  The border is found a bit at a
// time: of the keys' common prefix and a one, how many are not under it?  One vote-free sum over the warp (redux) a bit, and an
// end as soon as the count is right.  Instructions (two thirds of the issue slots) and that chain bound it: 25 MB of scores, rows of up to 512 blocks, in 32 us;
// 512 rows of up to 1024 in 10.1, a launch and a row's chain; the rows of the first with up to 1024 blocks 81.  With 32-bit comparisons for every bit
// 36, 10.9 and 100; and then with the bits that all keys share looked for first 39, or the keys near the border gathered 36, 13 and 193.
template <int kKeys>
__global__ __launch_bounds__(kSelThreads, kKeys == 32 ? 3 : kKeys == 16 ? 5 : 6) void q8_select_warp_kernel(const SelectArgs a) {
  __shared__ uint32_t s_q[CKV_MAX_BATCH];
  __shared__ BlockReq s_req[CKV_MAX_BATCH];
  __shared__ unsigned long long s_scan64[kSelThreads / 32 + 1];
  pdl_wait();
  pdl_release();
  scan_queries<kSelThreads>(a.r, s_q, s_req, s_scan64);
  const uint32_t lane = threadIdx.x & 31, T = a.block_tokens;
  const uint64_t rows = static_cast<uint64_t>(a.r.num_q) * a.heads;
  for (uint64_t row = blockIdx.x * static_cast<uint64_t>(kSelThreads / 32) + (threadIdx.x >> 5); row < rows;
       row += gridDim.x * static_cast<uint64_t>(kSelThreads / 32)) {
    BlockReq req;
    uint32_t i;
    if (!request_of(static_cast<uint32_t>(row / a.heads), s_q, s_req, a.r.batch, &req, &i)) continue;
    const uint32_t n = (seen_by(req, i, a.r.ratio) + T - 1) / T;
    int32_t* out = a.blocks + row * a.budget;
    if (n <= a.budget) {
      for (uint32_t j = lane; j < a.budget; j += 32) out[j] = j < n ? static_cast<int32_t>(j) : -1;
      continue;
    }
    const float* scores = a.scores + row * a.width;
    const uint32_t hi = n - a.recent;
    uint32_t key[kKeys];
#pragma unroll
    for (int x = 0; x < kKeys; ++x) {
      const uint32_t j = x * 32 + lane;
      key[x] = j < n ? __float_as_uint(__ldg(scores + j)) : 0x7FFFFFFFu;
    }
    // the first and the last ones count as the largest there are, what is not there as nothing, as NaN does
#pragma unroll
    for (int x = 0; x < kKeys; ++x) {
      const uint32_t j = x * 32 + lane;
      key[x] = j < a.sinks || (j >= hi && j < n) ? 0xFFFFFFFFu : score_key(__uint_as_float(key[x]));
    }
    // the largest border that `budget` keys are not under: its upper 15 bits from two keys a register, min(key - c + 1, 1) or 0 for each
    uint32_t pairs[kKeys / 2];
#pragma unroll
    for (int x = 0; x < kKeys / 2; ++x) pairs[x] = __byte_perm(key[2 * x] >> 1, key[2 * x + 1] >> 1, 0x7632);
    uint32_t border = 0, count = 0;
    for (uint32_t bit = 0x4000u; bit != 0 && count != a.budget; bit >>= 1) {
      const uint32_t c = border | bit, add = ((1 - c) & 0xFFFFu) * 0x10001u;
      uint32_t sum = 0;
#pragma unroll
      for (int x = 0; x < kKeys / 4; ++x) sum += __viaddmin_s16x2_relu(pairs[x], add, 0x10001u);
      if (n > kKeys * 16) {  // the other half of the keys
#pragma unroll
        for (int x = kKeys / 4; x < kKeys / 2; ++x) sum += __viaddmin_s16x2_relu(pairs[x], add, 0x10001u);
      }
      sum = __reduce_add_sync(0xFFFFFFFFu, sum);
      count = (sum & 0xFFFFu) + (sum >> 16);
      if (count >= a.budget) border = c;
    }
    border <<= 17;
    for (uint32_t bit = 0x10000u; bit != 0 && count != a.budget; bit >>= 1) {
      const uint32_t c = border | bit;
      count = 0;
#pragma unroll
      for (int x = 0; x < kKeys; ++x) count += key[x] >= c;
      count = __reduce_add_sync(0xFFFFFFFFu, count);
      if (count >= a.budget) border = c;
    }
    const uint32_t below = (1u << lane) - 1;
    uint32_t taken = 0;
    if (count == a.budget) {
#pragma unroll
      for (int x = 0; x < kKeys; ++x) {
        const bool take = key[x] >= border;
        const uint32_t votes = __ballot_sync(0xFFFFFFFFu, take);
        if (take) out[taken + __popc(votes & below)] = static_cast<int32_t>(x * 32 + lane);
        taken += __popc(votes);
      }
      continue;
    }
    // those above the border, and the first of those at it
    uint32_t above = 0;
#pragma unroll
    for (int x = 0; x < kKeys; ++x) above += key[x] > border;
    uint32_t left = a.budget - __reduce_add_sync(0xFFFFFFFFu, above);
#pragma unroll
    for (int x = 0; x < kKeys; ++x) {
      const uint32_t j = x * 32 + lane;
      const uint32_t ties = __ballot_sync(0xFFFFFFFFu, key[x] == border && j < n);
      const bool take = key[x] > border || (key[x] == border && j < n && __popc(ties & below) < left);
      const uint32_t votes = __ballot_sync(0xFFFFFFFFu, take);
      if (take) out[taken + __popc(votes & below)] = static_cast<int32_t>(j);
      taken += __popc(votes);
      left -= min(left, static_cast<uint32_t>(__popc(ties)));
    }
  }
}

// Longer rows than a warp's registers hold: a CTA takes a row, and reads it five times, from L2 after the first.  Each of them ends in a barrier and
// a scan, which bound it: 512 rows of 2048 blocks 18.0 us, of 8192 62; 18144 rows of 2048 382 us, of 8192 1220.  At 1024 blocks, which the warps still take, 512
// rows 11.3 here and 10.1 there, 18144 rows 222 and 69; at 256 512 rows 6.8 and 5.2.
__global__ __launch_bounds__(kSelThreads) void q8_select_kernel(const SelectArgs a) {
  constexpr uint32_t kBins = 256;
  __shared__ uint32_t s_q[CKV_MAX_BATCH];
  __shared__ BlockReq s_req[CKV_MAX_BATCH];
  __shared__ unsigned long long s_scan64[kSelThreads / 32 + 1];
  __shared__ uint32_t s_scan[kSelThreads / 32 + 1];
  __shared__ uint32_t s_bin[kBins];
  __shared__ uint32_t s_pick, s_left;
  pdl_wait();
  pdl_release();
  scan_queries<kSelThreads>(a.r, s_q, s_req, s_scan64);
  const uint32_t t = threadIdx.x, T = a.block_tokens;
  const uint64_t rows = static_cast<uint64_t>(a.r.num_q) * a.heads;
  for (uint64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    BlockReq req;
    uint32_t i;
    if (!request_of(static_cast<uint32_t>(row / a.heads), s_q, s_req, a.r.batch, &req, &i)) continue;
    const uint32_t n = (seen_by(req, i, a.r.ratio) + T - 1) / T;
    int32_t* out = a.blocks + row * a.budget;
    if (n <= a.budget) {
      for (uint32_t j = t; j < a.budget; j += kSelThreads) out[j] = j < n ? static_cast<int32_t>(j) : -1;
      continue;
    }
    const float* scores = a.scores + row * a.width;
    const uint32_t lo = a.sinks, hi = n - a.recent, want = a.budget - a.sinks - a.recent;  // candidates lo .. hi - 1: more than wanted
    // the key at rank `want` from the top, eight bits at a time
    uint32_t prefix = 0, mask = 0, left = want;
    if (want > 0) {
      for (int shift = 24; shift >= 0; shift -= 8) {
        __syncthreads();
        s_bin[t] = 0;
        __syncthreads();
        for (uint32_t j = lo + t; j < hi; j += kSelThreads) {
          const uint32_t k = score_key(scores[j]);
          if ((k & mask) == prefix) atomicAdd(&s_bin[k >> shift & 255], 1u);
        }
        __syncthreads();
        // bin 255 - t: how many are in bins above it
        const uint32_t c = s_bin[kBins - 1 - t];
        uint32_t sum;
        const uint32_t above = block_exclusive<kSelThreads>(c, &sum, s_scan);
        if (above < left && above + c >= left) {
          s_pick = kBins - 1 - t;
          s_left = left - above;
        }
        __syncthreads();
        prefix |= s_pick << shift;
        mask |= 255u << shift;
        left = s_left;
      }
    }
    // those above the border, and the first `left` at it, between the first and the last ones
    for (uint32_t j = t; j < a.sinks; j += kSelThreads) out[j] = static_cast<int32_t>(j);
    for (uint32_t j = t; j < a.recent; j += kSelThreads) out[a.sinks + want + j] = static_cast<int32_t>(hi + j);
    if (want > 0) {
      uint32_t taken = 0, ties = 0;  // so far
      for (uint32_t j0 = lo; j0 < hi; j0 += kSelThreads) {
        const uint32_t j = j0 + t;
        const uint32_t k = j < hi ? score_key(scores[j]) : 0;
        const bool tie = j < hi && k == prefix, over = j < hi && k > prefix;
        uint32_t tie_sum, sum;
        const uint32_t tie_rank = ties + block_exclusive<kSelThreads>(static_cast<uint32_t>(tie), &tie_sum, s_scan);
        const bool take = over || (tie && tie_rank < left);
        const uint32_t at = taken + block_exclusive<kSelThreads>(static_cast<uint32_t>(take), &sum, s_scan);
        if (take) out[a.sinks + at] = static_cast<int32_t>(j);
        taken += sum;
        ties += tie_sum;
      }
    }
    __syncthreads();  // s_pick, s_left and s_bin are read
  }
}

// ------------------------------------------------------------------- lists
constexpr int kListThreads = 256;

struct ListArgs {
  BlockReqs r;
  uint32_t heads, block_tokens;
  const int32_t* blocks;
  uint32_t budget;
  const int32_t* table;
  uint32_t stride;
  int32_t* tables;   // [num_q, heads, budget]: block numbers
  uint32_t* lens;    // [num_q, heads]: entries in them; kInvalidU32: no request's query
};

// A warp takes lists first, first + step, ..., 32 numbers at a time; three dependent reads and a scan over the lanes, 5 us a launch.
__device__ __forceinline__ void make_lists(const ListArgs& a, const uint32_t* s_q, const BlockReq* s_req, uint64_t first,
                                           uint64_t step) {
  const uint32_t lane = threadIdx.x & 31, T = a.block_tokens;
  const uint64_t lists = static_cast<uint64_t>(a.r.num_q) * a.heads;
  for (uint64_t at = first; at < lists; at += step) {
    BlockReq req;
    uint32_t i;
    if (!request_of(static_cast<uint32_t>(at / a.heads), s_q, s_req, a.r.batch, &req, &i)) {
      if (lane == 0) a.lens[at] = kInvalidU32;
      continue;
    }
    const uint32_t seen = seen_by(req, i, a.r.ratio), visible = (seen + T - 1) / T;
    const int32_t* table = a.table + static_cast<size_t>(req.rid) * a.stride;
    const int32_t* list = a.blocks + at * a.budget;
    int32_t* out = a.tables + at * a.budget;
    int32_t before = -1;  // the largest number so far
    uint32_t kept = 0;
    bool part = false, bad = false;
    for (uint32_t j0 = 0; j0 < a.budget; j0 += 32) {
      const int32_t v = j0 + lane < a.budget ? __ldg(list + j0 + lane) : -1;
      int32_t top = v;  // the largest up to this lane
#pragma unroll
      for (int s = 1; s < 32; s <<= 1) {
        const int32_t x = __shfl_up_sync(0xFFFFFFFFu, top, s);
        if (static_cast<int>(lane) >= s) top = max(top, x);
      }
      const int32_t up = __shfl_up_sync(0xFFFFFFFFu, top, 1);
      const int32_t prior = max(before, lane == 0 ? -1 : up);
      before = max(before, __shfl_sync(0xFFFFFFFFu, top, 31));
      bad |= v >= 0 && v <= prior;
      const bool take = v > prior && static_cast<uint32_t>(v) < visible;
      const uint32_t votes = __ballot_sync(0xFFFFFFFFu, take);
      if (take) out[kept + __popc(votes & ((1u << lane) - 1))] = __ldg(table + v);
      part |= take && static_cast<uint32_t>(v) == visible - 1;
      kept += __popc(votes);
    }
    if (__any_sync(0xFFFFFFFFu, bad) && lane == 0) status_or(a.r.d_status, CKV_STATUS_BAD_INDEX);
    const bool last = __any_sync(0xFFFFFFFFu, part);  // the last block that the query sees, maybe in part, is listed
    if (lane == 0) a.lens[at] = kept * T - (last ? visible * T - seen : 0);
  }
}

__global__ __launch_bounds__(kListThreads) void q8_lists_kernel(const ListArgs a) {
  __shared__ uint32_t s_q[CKV_MAX_BATCH];
  __shared__ BlockReq s_req[CKV_MAX_BATCH];
  __shared__ unsigned long long s_scan[kListThreads / 32 + 1];
  pdl_wait();
  pdl_release();
  scan_queries<kListThreads>(a.r, s_q, s_req, s_scan);
  make_lists(a, s_q, s_req, blockIdx.x * static_cast<uint64_t>(kListThreads / 32) + (threadIdx.x >> 5),
             gridDim.x * static_cast<uint64_t>(kListThreads / 32));
}

constexpr int kPlanThreads = 1024;

// The plan, by one CTA; and the lists before it where every warp of it has one at most, which saves a launch: a call for one
// query takes the host 29 us instead of 33, the card 15.3 instead of 15.7.  With two lists to a warp the card takes longer
// (64 lists of 32 blocks 62 us instead of 59).
constexpr uint64_t kFewLists = kPlanThreads / 32;

template <bool kFew>
__global__ __launch_bounds__(kPlanThreads) void plan_q8_lists_kernel(const ListArgs a, const Q8Geom g, uint8_t* plan) {
  __shared__ CutShared<kPlanThreads> s_cut;
  __shared__ uint32_t s_q[kFew ? CKV_MAX_BATCH : 1];
  __shared__ BlockReq s_req[kFew ? CKV_MAX_BATCH : 1];
  pdl_wait();
  pdl_release();
  if (kFew) {
    scan_queries<kPlanThreads>(a.r, s_q, s_req, s_cut.scan[0]);
    make_lists(a, s_q, s_req, threadIdx.x >> 5, kPlanThreads / 32);
    __syncthreads();
  }
  const uint32_t M = g.rows, per = (g.group + M - 1) / M, H = a.heads;  // tiles of a query
  auto tiles = [&](uint32_t tile, Q8Item* r) -> uint32_t {
    const uint32_t n = tile / per;
    const uint32_t* lens = a.lens + static_cast<size_t>(n) * H;
    uint32_t most = lens[0];  // of the heads' lists, the longest
    for (uint32_t h = 1; h < H; ++h) most = max(most, lens[h]);
    if (r != nullptr) {
      r->rid = n;
      r->q_start = n;
      r->q_len = 1;
      r->row0 = (tile - n * per) * M;
      r->kv_len = most;
      r->phase = 0;
    }
    return most;
  };
  cut_tiles<kPlanThreads, true>(g, plan, a.r.num_q * per, a.r.num_q, 1, a.r.num_q, tiles, s_cut);
}

// Where the workspace's pieces lie.
struct ListSpace {
  uint64_t plan, tables, lens, parts, bytes;
};

int list_space(const Q8Cache& c, uint32_t n_heads, uint32_t num_q, uint32_t budget, bool many, Q8Geom* g, ListSpace* w) {
  // entries of a list are counted in 32 bits
  if (budget == 0 || static_cast<uint64_t>(budget) * c.block_tokens > 0x7FFFFFF0ull) return CKV_ERR_SIZE;
  // one size for both: the caller asks for it without naming the batch, which decides between them
  uint64_t plan = 0, parts = 0;
  for (int i = 0; i < 2; ++i) {
    const int rc = q8_attn_geom_of(c, num_q, num_q, n_heads, i == 0 ? !many : many, g);
    if (rc) return rc;
    plan = std::max(plan, g->bytes);
    parts = std::max(parts, g->workspace);
  }
  auto up = [](uint64_t x) { return (x + 255) & ~255ull; };
  const uint64_t lists = static_cast<uint64_t>(num_q) * c.heads;
  w->plan = 0;
  w->tables = up(plan);
  w->lens = up(w->tables + lists * budget * 4);
  w->parts = up(w->lens + lists * 4);
  w->bytes = w->parts + parts;
  return CKV_OK;
}

}  // namespace
}  // namespace ckv

using namespace ckv;

extern "C" {

int ckv_q8_block_select(const float* scores, uint32_t n_kv_heads, uint32_t width, uint32_t block_tokens, uint32_t ratio,
                        uint32_t num_q, const int64_t* seq_lens, const int64_t* extend_lens, const int64_t* kv_lens,
                        uint32_t batch, uint32_t budget, uint32_t sinks, uint32_t recent, int32_t* blocks,
                        uint32_t* d_status, ckv_stream_t stream) {
  SelectArgs a{};
  if (block_tokens != 16 && block_tokens != 32 && block_tokens != 64 && block_tokens != 128) return CKV_ERR_SIZE;
  if (n_kv_heads == 0 || n_kv_heads > CKV_Q8_MAX_KV_HEADS || num_q > CKV_MAX_TOKENS) return CKV_ERR_SIZE;
  if (width == 0 || width > 0x7FFFFFFFu || budget == 0 || budget > 0x7FFFFFFFu) return CKV_ERR_SIZE;
  if (sinks > budget || recent > budget - sinks) return CKV_ERR_SIZE;
  const int rc = check_lens(batch, ratio, seq_lens, extend_lens, kv_lens);
  if (rc) return rc;
  if (num_q == 0 || batch == 0) return CKV_OK;
  if (!aligned_to(scores, 4) || !aligned_to(blocks, 4)) return CKV_ERR_POINTER;
  a.scores = scores;
  a.r = {nullptr, seq_lens, extend_lens, kv_lens, batch, num_q, ratio, 1, static_cast<int64_t>(width) * block_tokens, d_status};
  a.heads = n_kv_heads;
  a.width = width;
  a.block_tokens = block_tokens;
  a.budget = budget;
  a.sinks = sinks;
  a.recent = recent;
  a.blocks = blocks;
  const uint64_t rows = static_cast<uint64_t>(num_q) * n_kv_heads;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (width <= 1024) {
    const uint64_t ctas = (rows + kSelThreads / 32 - 1) / (kSelThreads / 32);
    const uint32_t per_sm = width <= 256 ? 6 : width <= 512 ? 5 : 3;  // that fit it
    const dim3 grid(static_cast<uint32_t>(std::min<uint64_t>(ctas, static_cast<uint64_t>(per_sm) * sm_count())));
    auto* kernel = width <= 128 ? q8_select_warp_kernel<4> : width <= 256 ? q8_select_warp_kernel<8>
                   : width <= 512 ? q8_select_warp_kernel<16> : q8_select_warp_kernel<32>;
    return launch_pdl(kernel, grid, dim3(kSelThreads), 0, s, a);
  }
  const dim3 grid(static_cast<uint32_t>(std::min<uint64_t>(rows, 8ull * sm_count())));
  return launch_pdl(q8_select_kernel, grid, dim3(kSelThreads), 0, s, a);
}

uint64_t ckv_q8_attn_blocks_workspace_bytes(const ckv_q8_cache_t* cache, uint32_t n_heads, uint32_t num_q,
                                            uint32_t budget) {
  Q8Cache c;
  Q8Geom g;
  ListSpace w;
  if (q8_cache_of(cache, &c) || list_space(c, n_heads, num_q, budget, false, &g, &w)) return 0;
  return w.bytes;
}

int ckv_q8_attn_blocks(const ckv_q8_cache_t* cache, uint32_t n_heads, uint32_t ratio, float scale, const void* q,
                       uint32_t num_q, const int32_t* blocks, uint32_t budget, const int64_t* rid,
                       const int64_t* seq_lens, const int64_t* extend_lens, const int64_t* kv_lens, uint32_t batch,
                       const int32_t* block_table, uint64_t table_stride, uint32_t num_reqs, int out_dtype, void* out,
                       float* lse, void* workspace, uint64_t workspace_bytes, uint32_t* d_status, ckv_stream_t stream) {
  AttnArgs a{};
  ListSpace w;
  int rc = q8_cache_of(cache, &a.c);
  if (rc) return rc;
  if (out_dtype != CKV_F32 && out_dtype != CKV_BF16) return CKV_ERR_DTYPE;
  if (!(scale > 0.0f) || !(scale < 1e30f)) return CKV_ERR_SIZE;
  rc = check_lens(batch, ratio, seq_lens, extend_lens, kv_lens);
  if (rc) return rc;
  // Three queries a request and more take four CTAs an SM with shorter rings instead of two (128 channels, up to eight heads to a kv head), us there
  // instead of: lists of 32 blocks of 64, eight kv heads, 64 requests of three queries 137 / 152, of four 175 / 195 (161 / 194 where a request's lists are alike),
  // of eight 326 / 367, eight requests of four 36.7 / 42.7, one of four 20.5 / 19.0; chunks of 430 queries 180 / 232.  Of one query it depends on how many
  // there are: one to six requests 18.7 to 21.4 / 17.7 to 21.1, eight 23.6 / 23.6, sixteen 30.4 / 31.9, 64 60 / 66, and with lists of 128 blocks 173 / 166.
  a.many = num_q > 2 * batch;
  rc = list_space(a.c, n_heads, num_q, budget, a.many, &a.g, &w);
  if (rc) return rc;
  if (num_q == 0 || batch == 0) return CKV_OK;
  rc = check_table(block_table, table_stride, num_reqs);
  if (rc) return rc;
  if (workspace_bytes < w.bytes) return CKV_ERR_SIZE;
  if (!aligned16(q) || !aligned16(out) || !aligned16(workspace) || (lse != nullptr && !aligned_to(lse, 4)) ||
      !aligned_to(blocks, 4) || !aligned_to(rid, 8))
    return CKV_ERR_POINTER;
  uint8_t* space = static_cast<uint8_t*>(workspace);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);

  ListArgs l{};
  const int64_t most = static_cast<int64_t>(table_stride) * a.c.block_tokens;
  l.r = {rid, seq_lens, extend_lens, kv_lens, batch, num_q, ratio, num_reqs, most, d_status};
  l.heads = a.c.heads;
  l.block_tokens = a.c.block_tokens;
  l.blocks = blocks;
  l.budget = budget;
  l.table = block_table;
  l.stride = static_cast<uint32_t>(table_stride);
  l.tables = reinterpret_cast<int32_t*>(space + w.tables);
  l.lens = reinterpret_cast<uint32_t*>(space + w.lens);
  const uint64_t lists = static_cast<uint64_t>(num_q) * a.c.heads;
  uint8_t* plan = space + w.plan;
  if (lists <= kFewLists) {
    rc = launch_pdl(plan_q8_lists_kernel<true>, dim3(1), dim3(kPlanThreads), 0, s, l, a.g, plan);
  } else {
    const uint64_t ctas = (lists + kListThreads / 32 - 1) / (kListThreads / 32);
    const uint32_t grid = static_cast<uint32_t>(std::min<uint64_t>(ctas, 4ull * sm_count()));
    rc = launch_pdl(q8_lists_kernel, dim3(grid), dim3(kListThreads), 0, s, l);
    if (rc) return rc;
    rc = launch_pdl(plan_q8_lists_kernel<false>, dim3(1), dim3(kPlanThreads), 0, s, l, a.g, plan);
  }
  if (rc) return rc;

  a.q = static_cast<const __nv_bfloat16*>(q);
  a.batch = num_q;
  a.num_q = num_q;
  a.n_heads = n_heads;
  a.ratio = 1;
  a.scale_log2 = scale * kLog2e;
  a.table = l.tables;
  a.stride = budget;
  a.num_reqs = num_q;
  a.lens = l.lens;
  a.plan = plan;
  a.out_f32 = out_dtype == CKV_F32;
  a.out = out;
  a.lse = lse;
  a.part_o = reinterpret_cast<float*>(space + w.parts);
  a.part_ml = reinterpret_cast<float2*>(a.part_o + static_cast<size_t>(a.g.cap_parts) * a.c.heads * a.g.rows * a.c.head_dim);
  a.d_status = d_status;
  a.wait_ns = wait_limit_ns();
  return launch_q8_attn(a, s);
}

}  // extern "C"

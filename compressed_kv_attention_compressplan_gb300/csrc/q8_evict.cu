// q8_evict.cu -- eviction from the 8-bit paged cache by accumulated attention
// weight: of a request with more than `budget` entries the first `sinks` and
// the newest `recent` stay, and of the others those of largest weight (equal
// weights: the lower position), in their order; they move into blocks that the
// caller names, so blocks that requests share are never written.
//
// Two launches.  Choosing: a CTA per request finds the weight at the border
// by a radix selection (11 + 11 + 10 bits of an order-preserving key) and
// lists the kept positions with ballots; only the weights are read.  Moving: a
// CTA per new block gathers its entries; a (block, head)'s scale is the
// largest of its sources', so entries only ever divide by a power of two.
//
// Bound.  Moving: the kept entries' bytes, read and written once: 32 requests cut down to 4096 entries of eight heads, 393 MB in
// 68 us, 5.8 TB/s or 85 % of the measured copy rate.  Choosing: latency, 18 us for 16384 weights (three passes over
// keys in shared memory, then one that lists) and 9.5 us for 1500: with a CTA to a request most of the card is idle, but a request's
// passes depend on one another.
#include <algorithm>

#include "q8.cuh"

namespace ckv {
namespace {

constexpr int kSelThreads = 1024;
constexpr int kBins = 2048;
constexpr uint32_t kMaxKeys = 49152;  // keys kept in shared memory; later ones are read again

struct EvictArgs {
  Q8Cache c;
  const int64_t* rid;
  const int64_t* kv_lens;
  uint32_t batch;
  const int32_t* table;
  uint32_t stride;
  const int32_t* dst_table;
  uint32_t dst_stride;
  uint32_t num_reqs;
  uint32_t budget, sinks, recent;
  float* weights;
  int32_t* kept;
  int64_t* new_lens;
  uint32_t keys_cap;
  uint32_t* d_status;
};

// Larger keys for larger weights; NaN below everything, the two zeros alike.
__device__ __forceinline__ uint32_t key_of(float w) {
  if (w != w) return 0;
  const uint32_t u = __float_as_uint(w + 0.0f);
  return u ^ (u >> 31 ? 0xFFFFFFFFu : 0x80000000u);
}

__global__ __launch_bounds__(kSelThreads) void q8_evict_select_kernel(const EvictArgs a) {
  extern __shared__ uint32_t s_key[];
  __shared__ uint32_t s_bin[kBins];
  __shared__ uint32_t s_scan[kSelThreads / 32 + 1];
  __shared__ uint32_t s_above[32], s_equal[32];
  __shared__ uint32_t s_pick, s_left;
  pdl_wait();
  pdl_release();
  const uint32_t t = threadIdx.x, lane = t & 31, warp = t >> 5, T = a.c.block_tokens;
  const uint32_t b = blockIdx.x;
  const int64_t r = a.rid[b], kl = a.kv_lens[b];
  int32_t* kept = a.kept + static_cast<size_t>(b) * a.budget;
  const bool ok = r >= 0 && r < a.num_reqs && kl >= 0 && kl <= static_cast<int64_t>(a.stride) * T && kl <= 0x7FFFFFF0;
  const uint32_t len = ok ? static_cast<uint32_t>(kl) : 0;
  if (t == 0) {
    if (!ok) status_or(a.d_status, CKV_STATUS_BAD_LENGTH);
    a.new_lens[b] = min(len, a.budget);
  }
  if (len <= a.budget) {
    for (uint32_t i = t; i < a.budget; i += kSelThreads) kept[i] = i < len ? static_cast<int32_t>(i) : -1;
    return;
  }
  const int32_t* table = a.table + static_cast<size_t>(r) * a.stride;
  const uint32_t n = len - a.sinks - a.recent;  // candidates: positions sinks .. sinks + n - 1
  const uint32_t want = a.budget - a.sinks - a.recent;
  const uint32_t t_shift = __ffs(T) - 1;
  bool bad = false;
  // nothing here branches, so that a thread's reads overlap: a block that does not exist reads block 0's weight and drops it
  auto read_key = [&](uint32_t i) -> uint32_t {
    const uint32_t p = a.sinks + i;
    const int32_t blk = __ldg(table + (p >> t_shift));
    const bool ok = static_cast<uint32_t>(blk) < a.c.num_blocks;
    bad |= !ok;
    const uint32_t k = key_of(a.weights[(static_cast<size_t>(ok ? blk : 0) << t_shift) + (p & (T - 1))]);
    return ok ? k : 0u;
  };
  const uint32_t cached = min(n, a.keys_cap);
#pragma unroll 1
  for (uint32_t i0 = t; i0 < cached; i0 += 8 * kSelThreads) {
    uint32_t k[8];
#pragma unroll
    for (int x = 0; x < 8; ++x) k[x] = read_key(min(i0 + x * kSelThreads, n - 1));
#pragma unroll
    for (int x = 0; x < 8; ++x)
      if (i0 + x * kSelThreads < cached) s_key[i0 + x * kSelThreads] = k[x];
  }
  auto key_at = [&](uint32_t i) { return i < cached ? s_key[i] : read_key(i); };
  __syncthreads();

  // the key at rank `want` from the top, 11, 11 and 10 bits at a time
  uint32_t prefix = 0, mask = 0, left = want;
  if (want > 0) {
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
      const uint32_t bins = pass == 2 ? 1024 : 2048;
      __syncthreads();
      for (uint32_t i = t; i < kBins; i += kSelThreads) s_bin[i] = 0;
      __syncthreads();
      for (uint32_t i = t; i < n; i += kSelThreads) {
        const uint32_t k = key_at(i);
        if ((k & mask) == prefix) atomicAdd(&s_bin[(k >> shift) & (bins - 1)], 1u);
      }
      __syncthreads();
      // counts from the top: thread t owns bins 2t and 2t + 1 counted from the highest
      const bool mine = 2 * t + 1 < bins;
      const uint32_t hi = mine ? bins - 1 - 2 * t : 1, lo = hi - 1;
      const uint32_t c_hi = mine ? s_bin[hi] : 0, c_lo = mine ? s_bin[lo] : 0;
      uint32_t total;
      const uint32_t above = block_exclusive<kSelThreads>(c_hi + c_lo, &total, s_scan);
      if (mine && above < left && above + c_hi + c_lo >= left) {
        const bool first = above + c_hi >= left;
        s_pick = first ? hi : lo;
        s_left = left - above - (first ? 0 : c_hi);
      }
      __syncthreads();
      prefix |= s_pick << shift;
      mask |= (bins - 1) << shift;
      left = s_left;
    }
  }
  // `left` of the entries with key == prefix stay: the lowest positions.  Every warp lists its run of candidates.
  const uint32_t run = ((n + 31) / 32 + 31) & ~31u;
  const uint32_t lo = min(n, warp * run), hi = min(n, lo + run);
  uint32_t above = 0, equal = 0;
  for (uint32_t i = lo + lane; i < hi; i += 32) {
    const uint32_t k = key_at(i);
    above += want > 0 && k > prefix;
    equal += want > 0 && k == prefix;
  }
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) {
    above += __shfl_xor_sync(0xFFFFFFFFu, above, s);
    equal += __shfl_xor_sync(0xFFFFFFFFu, equal, s);
  }
  if (lane == 0) {
    s_above[warp] = above;
    s_equal[warp] = equal;
  }
  __syncthreads();
  uint32_t at = a.sinks, eq = 0;
  for (uint32_t w = 0; w < warp; ++w) {
    at += s_above[w];
    eq += s_equal[w];
  }
  at += min(eq, left);
  const uint32_t below = (1u << lane) - 1;
  for (uint32_t i0 = lo; i0 < hi; i0 += 32) {
    const uint32_t i = i0 + lane;
    const uint32_t k = i < hi ? key_at(i) : 0;
    const uint32_t m_eq = __ballot_sync(0xFFFFFFFFu, i < hi && want > 0 && k == prefix);
    const bool keep = i < hi && want > 0 && (k > prefix || (k == prefix && eq + __popc(m_eq & below) < left));
    const uint32_t m = __ballot_sync(0xFFFFFFFFu, keep);
    if (keep) kept[at + __popc(m & below)] = static_cast<int32_t>(a.sinks + i);
    at += __popc(m);
    eq += __popc(m_eq);
  }
  for (uint32_t i = t; i < a.sinks; i += kSelThreads) kept[i] = static_cast<int32_t>(i);
  for (uint32_t i = t; i < a.recent; i += kSelThreads)
    kept[a.budget - a.recent + i] = static_cast<int32_t>(len - a.recent + i);
  if (bad) status_or(a.d_status, CKV_STATUS_BAD_INDEX);
}

constexpr int kMoveWarps = 8;

// One CTA per (new block, request); a warp per (head, side), or several where
// there are fewer of those than warps.
__global__ __launch_bounds__(32 * kMoveWarps, 4) void q8_evict_move_kernel(const EvictArgs a) {
  __shared__ int32_t s_blk[128];
  __shared__ uint32_t s_slot[128];
  pdl_wait();
  pdl_release();
  const uint32_t T = a.c.block_tokens, D = a.c.head_dim, H = a.c.heads;
  const uint32_t t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const uint32_t b = blockIdx.y, j = blockIdx.x;
  const uint32_t count = static_cast<uint32_t>(a.new_lens[b]);
  if (j * T >= count) return;
  const uint32_t n = min(T, count - j * T);
  const int64_t r = a.rid[b];
  const int32_t dst = j < a.dst_stride ? a.dst_table[static_cast<size_t>(r) * a.dst_stride + j] : -1;
  if (dst < 0 || static_cast<uint32_t>(dst) >= a.c.num_blocks) {
    if (t == 0 && blockIdx.z == 0) status_or(a.d_status, CKV_STATUS_BAD_INDEX);
    return;
  }
  if (t < 128) {
    int32_t blk = -1;
    uint32_t slot = 0;
    if (t < n) {
      const uint32_t p = static_cast<uint32_t>(a.kept[static_cast<size_t>(b) * a.budget + j * T + t]);
      slot = p % T;
      blk = p / T < a.stride ? __ldg(a.table + static_cast<size_t>(r) * a.stride + p / T) : -1;
      if (blk < 0 || static_cast<uint32_t>(blk) >= a.c.num_blocks) {
        blk = -1;
        status_or(a.d_status, CKV_STATUS_BAD_INDEX);
      } else if (blockIdx.z == 0) {
        a.weights[static_cast<size_t>(dst) * T + t] = a.weights[static_cast<size_t>(blk) * T + slot];
      }
    }
    s_blk[t] = blk;
    s_slot[t] = slot;
  }
  __syncthreads();
  const uint32_t units = H * (a.c.v != nullptr ? 2 : 1);
  const uint32_t wpu = units >= kMoveWarps ? 1 : kMoveWarps / units;  // warps of a unit
  const uint32_t lanes = D / 16, per = 32 / lanes;                    // lanes of an entry, entries a warp moves at once
  const uint32_t sub = warp % wpu;
  for (uint32_t u = blockIdx.z * (kMoveWarps / wpu) + warp / wpu; u < units; u += gridDim.z * (kMoveWarps / wpu)) {
    const uint32_t h = u % H;
    uint8_t* pool = u >= H ? a.c.v : a.c.k;
    float* scales = u >= H ? a.c.v_scale : a.c.k_scale;
    float s[4], top = 0.0f;
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const uint32_t e = x * 32 + lane;
      const int32_t blk = e < n ? s_blk[e] : -1;
      s[x] = blk >= 0 ? __ldcg(scales + static_cast<size_t>(blk) * H + h) : 0.0f;
      top = fmaxf(top, s[x]);
    }
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, x));
    const float inv = top > 0.0f ? 1.0f / top : 0.0f;
    uint8_t* out = pool + (static_cast<size_t>(dst) * H + h) * T * D;
    const uint32_t step = per * wpu;
    constexpr int kBatch = 4;  // entries of a lane whose loads are in flight together
#pragma unroll 1
    for (uint32_t e0 = sub * per; e0 < n; e0 += kBatch * step) {
      const uint32_t c = lane % lanes;
      uint4 v[kBatch];
#pragma unroll
      for (int x = 0; x < kBatch; ++x) {
        const uint32_t e = e0 + x * step + lane / lanes, el = min(e, 127u);
        const int32_t blk = s_blk[el];
        v[x] = ld_stream16_if(pool + ((static_cast<size_t>(max(blk, 0)) * H + h) * T + s_slot[el]) * D + c * 16,
                              e < n && blk >= 0);
      }
#pragma unroll
      for (int x = 0; x < kBatch; ++x) {
        const uint32_t e = e0 + x * step + lane / lanes, el = min(e, 127u);
        // the factor of entry e sits in lane e % 32, register e / 32
        const float s0 = __shfl_sync(0xFFFFFFFFu, s[0], el & 31), s1 = __shfl_sync(0xFFFFFFFFu, s[1], el & 31);
        const float s2 = __shfl_sync(0xFFFFFFFFu, s[2], el & 31), s3 = __shfl_sync(0xFFFFFFFFu, s[3], el & 31);
        const float f = (el < 32 ? s0 : el < 64 ? s1 : el < 96 ? s2 : s3) * inv;
        if (e < n && s_blk[el] >= 0) {
          if (f != 1.0f) {
            v[x].x = q8_rescale4(v[x].x, f);
            v[x].y = q8_rescale4(v[x].y, f);
            v[x].z = q8_rescale4(v[x].z, f);
            v[x].w = q8_rescale4(v[x].w, f);
          }
          st16(out + static_cast<size_t>(e) * D + c * 16, v[x]);
        }
      }
    }
    if (sub == 0 && lane == 0 && top > 0.0f) scales[static_cast<size_t>(dst) * H + h] = top;
  }
}

}  // namespace
}  // namespace ckv

using namespace ckv;

extern "C" int ckv_q8_evict(const ckv_q8_cache_t* cache, float* weights, const int64_t* rid, const int64_t* kv_lens,
                            uint32_t batch, const int32_t* block_table, uint64_t table_stride,
                            const int32_t* dst_table, uint64_t dst_stride, uint32_t num_reqs, uint32_t budget,
                            uint32_t sinks, uint32_t recent, int32_t* kept, int64_t* new_lens, uint32_t* d_status,
                            ckv_stream_t stream) {
  EvictArgs a{};
  int rc = q8_cache_of(cache, &a.c);
  if (rc) return rc;
  if (batch > CKV_MAX_BATCH || budget == 0 || budget > CKV_MAX_TOKENS) return CKV_ERR_SIZE;
  if (static_cast<uint64_t>(sinks) + recent > budget) return CKV_ERR_SIZE;
  if (batch == 0) return CKV_OK;
  rc = check_table(block_table, table_stride, num_reqs);
  if (rc) return rc;
  rc = check_table(dst_table, dst_stride, num_reqs);
  if (rc) return rc;
  if (!aligned_to(weights, 4) || !aligned_to(rid, 8) || !aligned_to(kv_lens, 8) || !aligned_to(kept, 4) ||
      !aligned_to(new_lens, 8))
    return CKV_ERR_POINTER;
  a.rid = rid;
  a.kv_lens = kv_lens;
  a.batch = batch;
  a.table = block_table;
  a.stride = static_cast<uint32_t>(table_stride);
  a.dst_table = dst_table;
  a.dst_stride = static_cast<uint32_t>(dst_stride);
  a.num_reqs = num_reqs;
  a.budget = budget;
  a.sinks = sinks;
  a.recent = recent;
  a.weights = weights;
  a.kept = kept;
  a.new_lens = new_lens;
  a.d_status = d_status;
  const uint64_t longest = static_cast<uint64_t>(table_stride) * a.c.block_tokens;
  a.keys_cap = longest <= budget ? 0 : static_cast<uint32_t>(std::min<uint64_t>(longest, kMaxKeys));
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  static std::atomic<uint64_t> done;
  rc = allow_smem(reinterpret_cast<const void*>(q8_evict_select_kernel), kMaxKeys * 4, done);
  if (rc) return rc;
  rc = launch_pdl(q8_evict_select_kernel, dim3(batch), dim3(kSelThreads), a.keys_cap * 4, s, a);
  if (rc) return rc;
  const uint64_t most = std::min<uint64_t>(budget, longest);
  const uint32_t blocks = static_cast<uint32_t>((most + a.c.block_tokens - 1) / a.c.block_tokens);
  const uint32_t units = a.c.heads * (a.c.v != nullptr ? 2 : 1);
  const uint32_t z = std::max<uint32_t>(1, std::min<uint32_t>(units / kMoveWarps, 8));
  return launch_pdl(q8_evict_move_kernel, dim3(blocks, batch, z), dim3(32 * kMoveWarps), 0, s, a);
}

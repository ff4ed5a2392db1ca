// q8_store.cu -- appending rows to the 8-bit paged cache: the plan (which
// blocks a step's new rows touch) and the quantising store.
//
// A block's scale is the smallest power of two with which its largest finite
// value fits e4m3.  A request's rows arrive in order, so a touched block is
// either fresh (its first new slot is slot 0: the scale comes from the new rows
// alone) or was begun by earlier rows, whose scale can only grow: then the
// earlier entries are divided by the growth, exactly but for subnormals.
//
// Bound.  Many rows: the rows' bytes, read from memory for the scale and once more, from L1 or L2, for the codes.  16 requests of eight heads,
// 255 MB: the store takes 43 us, 5.9 TB/s or 88 % of the measured copy rate (2 us more with each value's magnitude taken in fp32); with the plan 47.  A decode step (a row for some of 256
// requests) is two launches, 4.7 and 4.2 us, which the host's two calls (26 us) hide.  A CTA takes one (block, head, side), since its
// scale needs all its rows before any is stored.
#include <algorithm>

#include "q8.cuh"

namespace ckv {
namespace {

constexpr int kPlanThreads = 1024;

struct StorePlanArgs {
  const int64_t* rid;
  const int64_t* kv_lens;
  const int64_t* new_lens;
  uint32_t batch;
  uint32_t num_rows;
  const int32_t* table;
  uint32_t stride;
  uint32_t num_reqs;
  uint32_t block_tokens;
  uint32_t num_blocks;
  uint32_t capacity;
  int pad_invalid;
  ckv_q8_store_plan_t* plan;
  uint32_t* d_counts;
  uint32_t* d_status;
};

// Every CTA scans the (at most 1024) lengths itself and emits its share of
// the records, so the records' order is a closed form of the lengths.
__global__ __launch_bounds__(kPlanThreads) void plan_q8_store_kernel(const StorePlanArgs a) {
  __shared__ uint32_t s_rec[CKV_MAX_BATCH];    // first record of each request
  __shared__ uint32_t s_row[CKV_MAX_BATCH];    // first ragged row
  __shared__ uint32_t s_start[CKV_MAX_BATCH];  // first new entry's position
  __shared__ uint32_t s_len[CKV_MAX_BATCH];    // new entries
  __shared__ uint32_t s_rid[CKV_MAX_BATCH];
  __shared__ unsigned long long s_scan[kPlanThreads / 32 + 1];
  pdl_wait();
  pdl_release();
  const uint32_t t = threadIdx.x, T = a.block_tokens;
  uint32_t n = 0, start = 0, rid = 0, touched = 0;
  unsigned long long rows = 0;
  if (t < a.batch) {
    const int64_t r = a.rid[t], kv = a.kv_lens[t], nw = a.new_lens[t];
    bool bad = nw < 0 || nw > a.num_rows;
    rows = bad ? 0 : static_cast<unsigned long long>(nw);
    bad |= kv < nw || kv > static_cast<int64_t>(a.stride) * T || kv > 0x7FFFFFF0 || r < 0 || r >= a.num_reqs;
    if (!bad && nw > 0) {
      n = static_cast<uint32_t>(nw);
      start = static_cast<uint32_t>(kv - nw);
      rid = static_cast<uint32_t>(r);
      touched = (start + n - 1) / T - start / T + 1;
    }
    if (bad && blockIdx.x == 0) status_or(a.d_status, CKV_STATUS_BAD_LENGTH);
  }
  unsigned long long total_rows, total_recs;
  const unsigned long long row = block_exclusive<kPlanThreads>(rows, &total_rows, s_scan);
  const unsigned long long rec =
      block_exclusive<kPlanThreads>(static_cast<unsigned long long>(touched), &total_recs, s_scan);
  // a request whose rows do not all lie in the input stores nothing: its records are invalid
  if (t < a.batch) {
    s_rec[t] = static_cast<uint32_t>(rec);
    s_row[t] = row + rows <= a.num_rows ? static_cast<uint32_t>(row) : kInvalidU32;
    s_start[t] = start;
    s_len[t] = n;
    s_rid[t] = rid;
  }
  __syncthreads();
  const uint32_t recs = static_cast<uint32_t>(min(total_recs, 0xFFFFFFFFull));
  if (blockIdx.x == 0 && t == 0) {
    a.d_counts[0] = recs;
    a.d_counts[1] = static_cast<uint32_t>(min(total_rows, 0xFFFFFFFFull));
    a.d_counts[2] = a.d_counts[3] = 0;
    if (total_rows != a.num_rows) status_or(a.d_status, CKV_STATUS_BAD_TOTAL);
    if (recs > a.capacity) status_or(a.d_status, CKV_STATUS_CAPACITY);
  }
  const uint32_t end = a.pad_invalid ? a.capacity : min(recs, a.capacity);
  for (uint32_t i = blockIdx.x * kPlanThreads + t; i < end; i += gridDim.x * kPlanThreads) {
    uint4 out = make_uint4(kInvalidU32, kInvalidU32, kInvalidU32, kInvalidU32);
    if (i < recs) {
      // requests without rows share their successor's first record: the last of them owns it
      const uint32_t b = last_not_above(s_rec, a.batch, i);
      const uint32_t first = s_start[b] / T, j = i - s_rec[b];
      const uint32_t lo = max(s_start[b], (first + j) * T);
      const uint32_t hi = min(s_start[b] + s_len[b], (first + j + 1) * T);
      const int32_t block = a.table[static_cast<size_t>(s_rid[b]) * a.stride + first + j];
      if (block < 0 || static_cast<uint32_t>(block) >= a.num_blocks) {
        status_or(a.d_status, CKV_STATUS_BAD_INDEX);
      } else if (s_row[b] != kInvalidU32) {
        out = make_uint4(static_cast<uint32_t>(block), s_row[b] + (lo - s_start[b]), (lo % T) | ((hi - lo) << 16), 0);
      }
    }
    *reinterpret_cast<uint4*>(a.plan + i) = out;
  }
}

struct StoreArgs {
  Q8Cache c;
  const void* k_rows;
  const void* v_rows;
  uint32_t num_rows;
  const ckv_q8_store_plan_t* plan;
  const uint32_t* d_counts;
  uint32_t capacity;
  uint32_t sides;
  float* weights;  // NULL: left alone
  uint32_t* d_status;
};

constexpr int kStoreThreads = 128;  // at least the slots of a block

// 16 channels of a row as fp32.
__device__ __forceinline__ void load16(const float* p, float (&x)[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint4 v = ld_cached16(p + 4 * i);
#pragma unroll
    for (int j = 0; j < 4; ++j) x[4 * i + j] = unpack<float>(v, j);
  }
}
__device__ __forceinline__ void load16(const __nv_bfloat16* p, float (&x)[16]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint4 v = ld_cached16(p + 8 * i);
#pragma unroll
    for (int j = 0; j < 8; ++j) x[8 * i + j] = unpack<__nv_bfloat16>(v, j);
  }
}

// The largest magnitude of 16 channels, NaNs passed over.
__device__ __forceinline__ float largest16(const float* p) {
  float x[16], m = 0.0f;
  load16(p, x);
#pragma unroll
  for (int j = 0; j < 16; ++j) m = fmaxf(m, fabsf(x[j]));
  return m;
}
__device__ __forceinline__ float largest16(const __nv_bfloat16* p) {  // two at a time, as they are
  const uint4 a = ld_cached16(p), b = ld_cached16(p + 8);
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  __nv_bfloat162 m = __float2bfloat162_rn(0.0f);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t x = w[j] & 0x7FFF7FFFu;
    m = __hmax2(m, *reinterpret_cast<const __nv_bfloat162*>(&x));
  }
  return fmaxf(__low2float(m), __high2float(m));
}

// One CTA per (touched block, head, side).
template <typename TIn>
__global__ __launch_bounds__(kStoreThreads) void q8_store_kernel(const StoreArgs a) {
  __shared__ float s_max[kStoreThreads / 32];
  pdl_wait();
  pdl_release();
  const uint32_t n = count_or_capacity(a.d_counts, 0, a.capacity);
  const uint32_t H = a.c.heads, D = a.c.head_dim, T = a.c.block_tokens;
  const uint32_t units = H * a.sides;
  const uint32_t vecs = D / 16;
  for (uint32_t i = blockIdx.x; i < n; i += gridDim.x) {
    const uint4 rec = __ldg(reinterpret_cast<const uint4*>(a.plan + i));
    if (rec.x == kInvalidU32) continue;
    const uint32_t block = rec.x, row0 = rec.y, off = rec.z & 0xFFFFu, cnt = rec.z >> 16;
    if (block >= a.c.num_blocks || cnt == 0 || off + cnt > T || static_cast<uint64_t>(row0) + cnt > a.num_rows) {
      if (threadIdx.x == 0) status_or(a.d_status, CKV_STATUS_BAD_INDEX);
      continue;
    }
    // new entries have had no attention yet, whatever the slots' last owners had
    if (a.weights != nullptr && blockIdx.y == 0 && threadIdx.x < cnt)
      a.weights[static_cast<size_t>(block) * T + off + threadIdx.x] = 0.0f;
    for (uint32_t u = blockIdx.y; u < units; u += gridDim.y) {
      const bool second = u >= H;
      const uint32_t h = second ? u - H : u;
      const TIn* rows = static_cast<const TIn*>(second ? a.v_rows : a.k_rows) + (static_cast<size_t>(row0) * H + h) * D;
      uint8_t* pool = (second ? a.c.v : a.c.k) + (static_cast<size_t>(block) * H + h) * T * D;
      float* scale = (second ? a.c.v_scale : a.c.k_scale) + static_cast<size_t>(block) * H + h;
      const float old = off ? *scale : 0.0f;
      auto vec = [&](uint32_t w) { return rows + static_cast<size_t>(w / vecs) * H * D + (w % vecs) * 16; };
      float m = 0.0f;
      for (uint32_t w = threadIdx.x; w < cnt * vecs; w += kStoreThreads) m = fmaxf(m, largest16(vec(w)));
      if (m == INFINITY) {  // NaN and infinities do not count
        m = 0.0f;
        for (uint32_t w = threadIdx.x; w < cnt * vecs; w += kStoreThreads) {
          float x[16];
          load16(vec(w), x);
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const float ax = fabsf(x[j]);
            m = ax < INFINITY ? fmaxf(m, ax) : m;
          }
        }
      }
#pragma unroll
      for (int s = 16; s > 0; s >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, s));
      if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = m;
      __syncthreads();
      m = s_max[0];
#pragma unroll
      for (int w = 1; w < kStoreThreads / 32; ++w) m = fmaxf(m, s_max[w]);
      const float now = fmaxf(pow2f(q8_need_exp(m)), old);
      const float inv = 1.0f / now;
      for (uint32_t w = threadIdx.x; w < cnt * vecs; w += kStoreThreads) {
        float x[16];
        load16(vec(w), x);
        uint4 o;
        o.x = q8_pack4(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv);
        o.y = q8_pack4(x[4] * inv, x[5] * inv, x[6] * inv, x[7] * inv);
        o.z = q8_pack4(x[8] * inv, x[9] * inv, x[10] * inv, x[11] * inv);
        o.w = q8_pack4(x[12] * inv, x[13] * inv, x[14] * inv, x[15] * inv);
        st16(pool + static_cast<size_t>(off) * D + w * 16, o);
      }
      if (off && now > old) {  // the entries that were there follow the scale
        const float f = old * inv;
        for (uint32_t w = threadIdx.x; w < off * vecs; w += kStoreThreads) {
          uint4 v = *reinterpret_cast<const uint4*>(pool + w * 16);
          v.x = q8_rescale4(v.x, f);
          v.y = q8_rescale4(v.y, f);
          v.z = q8_rescale4(v.z, f);
          v.w = q8_rescale4(v.w, f);
          st16(pool + w * 16, v);
        }
      }
      __syncthreads();  // every thread has read the old scale and s_max
      if (threadIdx.x == 0) *scale = now;
    }
  }
}

int store_rows(const ckv_q8_cache_t* cache, int in_dtype, const void* k_rows, const void* v_rows, uint32_t num_rows,
               const ckv_q8_store_plan_t* plan, const uint32_t* d_counts, uint32_t capacity, float* weights,
               uint32_t* d_status, ckv_stream_t stream) {
  StoreArgs a{};
  const int rc = q8_cache_of(cache, &a.c);
  if (rc) return rc;
  if (in_dtype != CKV_F32 && in_dtype != CKV_BF16) return CKV_ERR_DTYPE;
  if (num_rows > CKV_MAX_TOKENS || capacity > CKV_MAX_TOKENS) return CKV_ERR_SIZE;
  if (num_rows == 0 || capacity == 0) return CKV_OK;
  if (!aligned16(k_rows) || (a.c.v != nullptr) != (v_rows != nullptr) || (v_rows != nullptr && !aligned16(v_rows)))
    return CKV_ERR_POINTER;
  if (!aligned16(plan) || (d_counts != nullptr && !aligned_to(d_counts, 4))) return CKV_ERR_POINTER;
  a.k_rows = k_rows;
  a.v_rows = v_rows;
  a.num_rows = num_rows;
  a.plan = plan;
  a.d_counts = d_counts;
  a.capacity = capacity;
  a.sides = v_rows != nullptr ? 2 : 1;
  a.weights = weights;
  a.d_status = d_status;
  const dim3 grid(std::min<uint32_t>(capacity, 65536u), a.c.heads * a.sides);
  return launch_pdl(in_dtype == CKV_BF16 ? q8_store_kernel<__nv_bfloat16> : q8_store_kernel<float>, grid,
                    dim3(kStoreThreads), 0, reinterpret_cast<cudaStream_t>(stream), a);
}

}  // namespace
}  // namespace ckv

using namespace ckv;

extern "C" {

uint32_t ckv_capacity_q8_store(uint32_t batch, uint32_t num_rows, uint32_t block_tokens) {
  if (block_tokens == 0) return 0;
  // a request with n rows touches at most (n - 2) / T + 2 blocks, and never more than n
  const uint64_t most = static_cast<uint64_t>(num_rows) / block_tokens + 2ull * std::min(batch, num_rows);
  return static_cast<uint32_t>(std::min<uint64_t>(num_rows, most));
}

int ckv_plan_q8_store(const ckv_q8_cache_t* cache, const int64_t* rid, const int64_t* kv_lens,
                      const int64_t* new_lens, uint32_t batch, uint32_t num_rows, const int32_t* block_table,
                      uint64_t table_stride, uint32_t num_reqs, uint32_t capacity, int pad_invalid,
                      ckv_q8_store_plan_t* plan, uint32_t* d_counts, uint32_t* d_status, ckv_stream_t stream) {
  StorePlanArgs a{};
  Q8Cache c;
  int rc = q8_cache_of(cache, &c);
  if (rc) return rc;
  if (batch > CKV_MAX_BATCH || num_rows > CKV_MAX_TOKENS || capacity > CKV_MAX_TOKENS) return CKV_ERR_SIZE;
  rc = check_table(block_table, table_stride, num_reqs);
  if (rc) return rc;
  if (!aligned_to(d_counts, 16) || (capacity > 0 && !aligned16(plan))) return CKV_ERR_POINTER;
  if (batch > 0 && (!aligned_to(rid, 8) || !aligned_to(kv_lens, 8) || !aligned_to(new_lens, 8))) return CKV_ERR_POINTER;
  a.rid = rid;
  a.kv_lens = kv_lens;
  a.new_lens = new_lens;
  a.batch = batch;
  a.num_rows = num_rows;
  a.table = block_table;
  a.stride = static_cast<uint32_t>(table_stride);
  a.num_reqs = num_reqs;
  a.block_tokens = c.block_tokens;
  a.num_blocks = c.num_blocks;
  a.capacity = capacity;
  a.pad_invalid = pad_invalid;
  a.plan = plan;
  a.d_counts = d_counts;
  a.d_status = d_status;
  const uint32_t grid = std::min<uint32_t>(32, std::max<uint32_t>(1, (capacity + kPlanThreads - 1) / kPlanThreads));
  return launch_pdl(plan_q8_store_kernel, dim3(grid), dim3(kPlanThreads), 0, reinterpret_cast<cudaStream_t>(stream), a);
}

int ckv_q8_store(const ckv_q8_cache_t* cache, int in_dtype, const void* k_rows, const void* v_rows, uint32_t num_rows,
                 const ckv_q8_store_plan_t* plan, const uint32_t* d_counts, uint32_t capacity, uint32_t* d_status,
                 ckv_stream_t stream) {
  return store_rows(cache, in_dtype, k_rows, v_rows, num_rows, plan, d_counts, capacity, nullptr, d_status, stream);
}

int ckv_q8_store_reset(const ckv_q8_cache_t* cache, int in_dtype, const void* k_rows, const void* v_rows,
                       uint32_t num_rows, const ckv_q8_store_plan_t* plan, const uint32_t* d_counts, uint32_t capacity,
                       float* weights, uint32_t* d_status, ckv_stream_t stream) {
  if (!aligned_to(weights, 4)) return CKV_ERR_POINTER;
  return store_rows(cache, in_dtype, k_rows, v_rows, num_rows, plan, d_counts, capacity, weights, d_status, stream);
}

}  // extern "C"

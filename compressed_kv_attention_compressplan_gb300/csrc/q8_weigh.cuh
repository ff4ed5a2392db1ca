// q8_weigh.cuh -- what the kernels for the cached entries' attention weights share.
#pragma once

#include "q8.cuh"

namespace ckv {

struct WeighArgs {
  Q8Cache c;
  const __nv_bfloat16* q;
  const float* lse;
  uint32_t num_q;
  uint32_t n_heads;
  uint32_t group;
  uint32_t ratio;
  float scale_log2;
  float decay;
  float* weights;
  const int64_t* rid;
  const int64_t* seq_lens;
  const int64_t* extend_lens;
  const int64_t* kv_lens;
  uint32_t batch;
  const int32_t* table;
  uint32_t stride;
  uint32_t num_reqs;
  uint32_t head_warps;  // warps that share a tile's heads: a power of two
  uint64_t wait_ns;
  uint32_t* d_status;
};

// two e4m3 values (as an fp16 pair) -> a bf16 pair, exact
__device__ __forceinline__ uint32_t f16x2_to_bf16x2(uint32_t h) {
  const float2 f = f16x2_to_f32(h);
  return pack_bf16x2(f.x, f.y);
}

__device__ __forceinline__ void put_weight(const WeighArgs& a, int32_t block, uint32_t slot, float w) {
  float* dst = a.weights + static_cast<size_t>(block) * a.c.block_tokens + slot;
  *dst = a.decay == 0.0f ? w : fmaf(a.decay, *dst, w);
}

// Units (runs of unit_entries entries) before every request that has queries, and its first ragged query; by a block of
// kThreads.  s_meta, where it is wanted: {entries, queries, phase, rid} of those requests.
template <int kThreads>
__device__ __forceinline__ uint32_t scan_requests(const WeighArgs& a, uint32_t unit_entries, uint32_t* s_unit, uint32_t* s_q,
                                                  uint32_t* s_scan, unsigned long long* s_scan64,
                                                  uint4* s_meta = nullptr) {
  uint32_t units = 0;
  unsigned long long queries = 0;
  for (uint32_t b0 = 0; b0 < a.batch; b0 += kThreads) {
    const uint32_t b = b0 + threadIdx.x;
    uint32_t n = 0;
    unsigned long long ql = 0;
    if (b < a.batch) {
      const int64_t el = a.extend_lens[b], kl = a.kv_lens[b], sl = a.seq_lens[b], r = a.rid[b];
      const bool len_ok = el >= 0 && el <= a.num_q;
      ql = len_ok ? static_cast<unsigned long long>(el) : 0;
      const bool ok = len_ok && sl >= el && sl <= 0x7FFFFFFF && kl >= 0 && kl <= 0x7FFFFFF0 &&
                      kl <= static_cast<int64_t>(a.stride) * a.c.block_tokens && r >= 0 && r < a.num_reqs;
      if (!ok && blockIdx.x == 0) status_or(a.d_status, CKV_STATUS_BAD_LENGTH);
      if (ok && s_meta != nullptr)
        s_meta[b] = make_uint4(static_cast<uint32_t>(kl), static_cast<uint32_t>(el), a.ratio - 1 - static_cast<uint32_t>(sl) % a.ratio,
                               static_cast<uint32_t>(r));
      n = ok && el > 0 ? static_cast<uint32_t>((kl + unit_entries - 1) / unit_entries) : 0;
    }
    unsigned long long ql_sum;
    const unsigned long long q0 = queries + block_exclusive<kThreads>(ql, &ql_sum, s_scan64);
    if (q0 + ql > a.num_q) n = 0;
    uint32_t n_sum;
    const uint32_t u0 = units + block_exclusive<kThreads>(n, &n_sum, s_scan);
    if (b < a.batch) {
      s_unit[b] = u0;
      s_q[b] = static_cast<uint32_t>(q0);
    }
    units += n_sum;
    queries += ql_sum;
  }
  if (blockIdx.x == 0 && threadIdx.x == 0 && queries != a.num_q) status_or(a.d_status, CKV_STATUS_BAD_TOTAL);
  __syncthreads();
  return units;
}

// The tensor-core kernel, for many rows; up to 128 channels.
int launch_q8_weigh_tc(const WeighArgs& a, cudaStream_t s);

}  // namespace ckv

// q8_blocks.cuh -- what the kernels of the sparse attention share: the requests
// of a step, and which of them a ragged query belongs to.
#pragma once

#include "q8.cuh"

namespace ckv {

struct BlockReqs {
  const int64_t* rid;  // NULL: not wanted
  const int64_t* seq_lens;
  const int64_t* extend_lens;
  const int64_t* kv_lens;
  uint32_t batch;
  uint32_t num_q;
  uint32_t ratio;
  uint32_t num_reqs;
  int64_t most;  // entries that a request has at most
  uint32_t* d_status;
};

struct BlockReq {
  uint32_t kv_len, q_len, phase, rid;  // q_len 0: none of its queries counts
};

// The requests and the first ragged query of each, by a block of kThreads; every thread calls it.
template <int kThreads>
__device__ __forceinline__ void scan_queries(const BlockReqs& a, uint32_t* s_q, BlockReq* s_req, unsigned long long* s_scan) {
  unsigned long long queries = 0;
  for (uint32_t b0 = 0; b0 < a.batch; b0 += kThreads) {
    const uint32_t b = b0 + threadIdx.x;
    unsigned long long ql = 0;
    BlockReq r = {0, 0, 0, 0};
    if (b < a.batch) {
      const int64_t el = a.extend_lens[b], kl = a.kv_lens[b], sl = a.seq_lens[b], id = a.rid != nullptr ? a.rid[b] : 0;
      const bool len_ok = el >= 0 && el <= a.num_q;
      ql = len_ok ? static_cast<unsigned long long>(el) : 0;
      const bool ok = len_ok && sl >= el && sl <= 0x7FFFFFFF && kl >= 0 && kl <= 0x7FFFFFF0 && kl <= a.most && id >= 0 &&
                      id < a.num_reqs;
      if (!ok && blockIdx.x == 0) status_or(a.d_status, CKV_STATUS_BAD_LENGTH);
      if (ok) r = {static_cast<uint32_t>(kl), static_cast<uint32_t>(el), a.ratio - 1 - static_cast<uint32_t>(sl) % a.ratio, static_cast<uint32_t>(id)};
    }
    unsigned long long sum;
    const unsigned long long q0 = queries + block_exclusive<kThreads>(ql, &sum, s_scan);
    if (b < a.batch) {
      if (q0 + ql > a.num_q) r.q_len = 0;
      s_q[b] = static_cast<uint32_t>(min(q0, 0xFFFFFFFFull));
      s_req[b] = r;
    }
    queries += sum;
  }
  if (blockIdx.x == 0 && threadIdx.x == 0 && queries != a.num_q) status_or(a.d_status, CKV_STATUS_BAD_TOTAL);
  __syncthreads();
}

// The request of ragged query n, and the query's number in it; false if it has none.  Requests without queries share their
// successor's first one: the last of them owns it.
__device__ __forceinline__ bool request_of(uint32_t n, const uint32_t* s_q, const BlockReq* s_req, uint32_t batch, BlockReq* r, uint32_t* i) {
  if (batch == 0) return false;
  const uint32_t b = last_not_above(s_q, batch, n);
  *r = s_req[b];
  *i = n - s_q[b];
  return *i < r->q_len;
}

// Entries that query i of a request sees.
__device__ __forceinline__ uint32_t seen_by(const BlockReq& r, uint32_t i, uint32_t ratio) {
  const uint32_t after = r.q_len - 1 - i;
  if (ratio == 1) return r.kv_len - min(r.kv_len, after);  // without the division
  return static_cast<uint32_t>(q8_visible(r.kv_len, after, r.phase, ratio));
}

// Host checks of the lengths' arrays.
inline int check_lens(uint32_t batch, uint32_t ratio, const int64_t* seq_lens, const int64_t* extend_lens, const int64_t* kv_lens) {
  if (ratio == 0 || ratio > 65536) return CKV_ERR_RATIO;
  if (batch > CKV_MAX_BATCH) return CKV_ERR_SIZE;
  if (batch > 0 && (!aligned_to(seq_lens, 8) || !aligned_to(extend_lens, 8) || !aligned_to(kv_lens, 8))) return CKV_ERR_POINTER;
  return CKV_OK;
}

}  // namespace ckv

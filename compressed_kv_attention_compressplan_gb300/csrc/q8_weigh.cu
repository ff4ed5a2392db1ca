// q8_weigh.cu -- how much attention each cached entry received: for every
// entry of the batch's requests,
//     weights[slot] = decay * weights[slot] + sum over queries and heads of p,
//     p = 2^(scale log2(e) k_scale <q, k8> - lse log2(e)),
// with lse the attention's log-sum-exp, so p is the softmax weight itself and
// one pass over the keys does: the values are not read and no maximum is kept.
//
// Bound: the keys' bytes when a request has few rows; the exponentials and
// products when it has many.  An entry belongs to one CTA, which walks all
// rows and heads in a fixed order: no atomics, and results that repeat bit for
// bit.  A warp holds 16 entries of one kv head as bf16 fragments (exact, and
// queries are bf16 already, so a row tile costs loads and products only) and streams
// the request's rows past them; the CTA's warps share out kv heads, then
// entries, and the heads are summed through shared memory in head order.
#include <algorithm>

#include "q8.cuh"

namespace ckv {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kTile = 16;

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
  uint32_t* d_status;
};

__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// two e4m3 values (as an fp16 pair) -> a bf16 pair, exact
__device__ __forceinline__ uint32_t f16x2_to_bf16x2(uint32_t h) {
  const float2 f = f16x2_to_f32(h);
  return pack_bf16x2(f.x, f.y);
}

template <int kD>
__global__ __launch_bounds__(kThreads) void q8_weigh_kernel(const WeighArgs a) {
  constexpr int kKj = kD / 64;
  __shared__ uint32_t s_unit[CKV_MAX_BATCH];
  __shared__ uint32_t s_q[CKV_MAX_BATCH];
  __shared__ uint32_t s_scan[kWarps + 1];
  __shared__ unsigned long long s_scan64[kWarps + 1];
  __shared__ float s_sum[kWarps][kTile];
  pdl_wait();
  pdl_release();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, q = lane & 3;
  const uint32_t T = a.c.block_tokens, H = a.c.heads, G = a.group;
  const uint32_t unit_entries = kWarps / a.head_warps * kTile;

  // units (runs of unit_entries entries) of every request, and its first ragged query
  uint32_t units = 0;
  unsigned long long queries = 0;
  for (uint32_t b0 = 0; b0 < a.batch; b0 += kThreads) {
    const uint32_t b = b0 + tid;
    uint32_t n = 0;
    unsigned long long ql = 0;
    if (b < a.batch) {
      const int64_t el = a.extend_lens[b], kl = a.kv_lens[b], sl = a.seq_lens[b], r = a.rid[b];
      const bool len_ok = el >= 0 && el <= a.num_q;
      ql = len_ok ? static_cast<unsigned long long>(el) : 0;
      const bool ok = len_ok && sl >= el && sl <= 0x7FFFFFFF && kl >= 0 && kl <= 0x7FFFFFF0 &&
                      kl <= static_cast<int64_t>(a.stride) * T && r >= 0 && r < a.num_reqs;
      if (!ok && blockIdx.x == 0) status_or(a.d_status, CKV_STATUS_BAD_LENGTH);
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
  if (blockIdx.x == 0 && tid == 0 && queries != a.num_q) status_or(a.d_status, CKV_STATUS_BAD_TOTAL);
  __syncthreads();

  for (uint32_t u = blockIdx.x; u < units; u += gridDim.x) {
    const uint32_t b = last_not_above(s_unit, a.batch, u);
    const uint32_t kv_len = static_cast<uint32_t>(a.kv_lens[b]);
    const uint32_t q_len = static_cast<uint32_t>(a.extend_lens[b]);
    const uint32_t phase = a.ratio - 1 - static_cast<uint32_t>(a.seq_lens[b]) % a.ratio;
    const uint32_t rows = q_len * G;
    const uint32_t e0 = (u - s_unit[b]) * unit_entries + warp / a.head_warps * kTile;
    float sum[2][2] = {};  // entries 8 n + 2q + {0, 1}
    int32_t block = -1;
    if (e0 < kv_len) {
      block = __ldg(a.table + static_cast<size_t>(a.rid[b]) * a.stride + e0 / T);
      if (block < 0 || static_cast<uint32_t>(block) >= a.c.num_blocks) {
        if (lane == 0) status_or(a.d_status, CKV_STATUS_BAD_INDEX);
        block = -1;
      }
    }
    if (block >= 0) {
      for (uint32_t h = warp % a.head_warps; h < H; h += a.head_warps) {
        const size_t bh = static_cast<size_t>(block) * H + h;
        const uint8_t* k = a.c.k + (bh * T + e0 % T) * kD;
        const float f = a.scale_log2 * __ldg(a.c.k_scale + bh);
        uint32_t kf[2][kKj * 4][2];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
#pragma unroll
          for (int j = 0; j < kKj; ++j) {
            const uint4 w = ld_stream16(k + static_cast<size_t>(n * 8 + g) * kD + (j * 4 + q) * 16);
            const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int s = 0; s < 4; ++s) {
              kf[n][j * 4 + s][0] = f16x2_to_bf16x2(q8_lo_f16x2(x[s]));
              kf[n][j * 4 + s][1] = f16x2_to_bf16x2(q8_hi_f16x2(x[s]));
            }
          }
        }
        for (uint32_t r0 = 0; r0 < rows; r0 += 16) {
          float s[2][4] = {};
          float off[2];
          int64_t vis[2];
          const __nv_bfloat16* p[2];
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const uint32_t rho = min(r0 + g + 8 * r, rows - 1);
            const uint32_t i = rho / G, hg = rho % G;
            const size_t row = static_cast<size_t>(s_q[b] + i) * a.n_heads + h * G + hg;
            vis[r] = r0 + g + 8 * r < rows ? q8_visible(kv_len, q_len - 1 - i, phase, a.ratio) : 0;
            const float lse = __ldg(a.lse + row);
            off[r] = lse == -INFINITY ? -INFINITY : lse * -kLog2e;  // a row that saw nothing weighs nothing
            p[r] = a.q + row * kD;
          }
#pragma unroll
          for (int j = 0; j < kKj; ++j) {
            uint4 v[2][2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              v[r][0] = ld_cached16(p[r] + (j * 4 + q) * 16);
              v[r][1] = ld_cached16(p[r] + (j * 4 + q) * 16 + 8);
            }
#pragma unroll
            for (int st = 0; st < 4; ++st) {
              const uint4 x0 = v[0][st >> 1], x1 = v[1][st >> 1];
              uint32_t af[4];
              af[0] = st & 1 ? x0.z : x0.x;
              af[1] = st & 1 ? x1.z : x1.x;
              af[2] = st & 1 ? x0.w : x0.y;
              af[3] = st & 1 ? x1.w : x1.y;
              mma_bf16(s[0], af, kf[0][j * 4 + st][0], kf[0][j * 4 + st][1]);
              mma_bf16(s[1], af, kf[1][j * 4 + st][0], kf[1][j * 4 + st][1]);
            }
          }
#pragma unroll
          for (int n = 0; n < 2; ++n) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int64_t at = e0 + n * 8 + 2 * q + (e & 1);
              const float w = ex2(fmaf(s[n][e], f, off[e >> 1]));
              sum[n][e & 1] += at < vis[e >> 1] ? w : 0.0f;
            }
          }
        }
      }
    }
    // rows of the fragment (the lanes of one column), then the heads' warps in order
#pragma unroll
    for (int n = 0; n < 2; ++n) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) sum[n][e] += __shfl_xor_sync(0xFFFFFFFFu, sum[n][e], x);
        if (g == 0) s_sum[warp][n * 8 + 2 * q + e] = sum[n][e];
      }
    }
    __syncthreads();
    if (warp % a.head_warps == 0 && lane < kTile && block >= 0 && e0 + lane < kv_len) {
      float w = 0.0f;
      for (uint32_t x = 0; x < a.head_warps; ++x) w += s_sum[warp + x][lane];
      float* dst = a.weights + static_cast<size_t>(block) * T + e0 % T + lane;
      *dst = a.decay == 0.0f ? w : fmaf(a.decay, *dst, w);
    }
    __syncthreads();
  }
}

template <int kD>
int launch_weigh(const WeighArgs& a, cudaStream_t s) {
  const uint32_t grid = 2u * static_cast<uint32_t>(sm_count());
  return launch_pdl(q8_weigh_kernel<kD>, dim3(grid), dim3(kThreads), 0, s, a);
}

}  // namespace
}  // namespace ckv

using namespace ckv;

extern "C" int ckv_q8_weigh(const ckv_q8_cache_t* cache, uint32_t n_heads, uint32_t ratio, float scale, float decay,
                            const void* q, const float* lse, uint32_t num_q, const int64_t* rid,
                            const int64_t* seq_lens, const int64_t* extend_lens, const int64_t* kv_lens,
                            uint32_t batch, const int32_t* block_table, uint64_t table_stride, uint32_t num_reqs,
                            float* weights, uint32_t* d_status, ckv_stream_t stream) {
  WeighArgs a{};
  int rc = q8_cache_of(cache, &a.c);
  if (rc) return rc;
  if (ratio == 0 || ratio > 65536) return CKV_ERR_RATIO;
  if (!(scale > 0.0f) || !(scale < 1e30f) || !(decay >= 0.0f) || !(decay <= 1.0f)) return CKV_ERR_SIZE;
  if (batch > CKV_MAX_BATCH || num_q > CKV_MAX_TOKENS) return CKV_ERR_SIZE;
  if (n_heads == 0 || n_heads % a.c.heads != 0 || n_heads / a.c.heads > CKV_Q8_MAX_GROUP) return CKV_ERR_SIZE;
  a.group = n_heads / a.c.heads;
  if (static_cast<uint64_t>(num_q) * a.group > 0x7FFFFFFFull) return CKV_ERR_SIZE;  // row numbers are 32-bit
  if (batch == 0 || num_q == 0) return CKV_OK;
  rc = check_table(block_table, table_stride, num_reqs);
  if (rc) return rc;
  if (!aligned16(q) || !aligned_to(lse, 4) || !aligned_to(weights, 4) || !aligned_to(rid, 8) ||
      !aligned_to(seq_lens, 8) || !aligned_to(extend_lens, 8) || !aligned_to(kv_lens, 8))
    return CKV_ERR_POINTER;
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.lse = lse;
  a.num_q = num_q;
  a.n_heads = n_heads;
  a.ratio = ratio;
  a.scale_log2 = scale * kLog2e;
  a.decay = decay;
  a.weights = weights;
  a.rid = rid;
  a.seq_lens = seq_lens;
  a.extend_lens = extend_lens;
  a.kv_lens = kv_lens;
  a.batch = batch;
  a.table = block_table;
  a.stride = static_cast<uint32_t>(table_stride);
  a.num_reqs = num_reqs;
  a.head_warps = 1;
  while (a.head_warps * 2 <= std::min<uint32_t>(a.c.heads, kWarps)) a.head_warps *= 2;
  a.d_status = d_status;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  switch (a.c.head_dim) {
    case 64: return launch_weigh<64>(a, s);
    case 128: return launch_weigh<128>(a, s);
    case 256: return launch_weigh<256>(a, s);
    default: return launch_weigh<512>(a, s);
  }
}

// q8_rope_store.cu -- appending rows to the 8-bit paged cache with their norm
// and their positions' rotation on the way (see q8_store.cu for the blocks'
// scales and the plan).
//
// A key row is y = x * w / sqrt(mean(x^2) + eps), then pairs of channels turn by
// the angle of the row's position, (a, b) -> (a cos - b sin, a sin + b cos).  Eight
// pairs are a thread's: channels 16 j .. 16 j + 15 where pairs are neighbours, or
// two runs of eight channels half the rotated width apart, so that no value crosses
// threads in either style.  Products are rounded by themselves (no fused multiply-add), so a rotated value
// does not depend on how a compiler would contract it.
#include <algorithm>

#include "q8.cuh"

namespace ckv {
namespace {

constexpr int kThreads = 128;

struct RopeStoreArgs {
  Q8Cache c;
  const void* k_rows;
  const void* v_rows;
  uint64_t k_stride, v_stride;
  uint32_t num_rows;
  const int64_t* positions;
  const float* weight;  // NULL: no norm
  float eps;
  const float* freqs;
  uint32_t max_pos, begin, dim;
  int halves;
  const ckv_q8_store_plan_t* plan;
  const uint32_t* d_counts;
  uint32_t capacity;
  uint32_t sides;
  float* weights;
  uint32_t* d_status;
};

__device__ __forceinline__ void load8(const float* p, float* x) {
  const uint4 a = ld_cached16(p), b = ld_cached16(p + 4);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    x[j] = unpack<float>(a, j);
    x[4 + j] = unpack<float>(b, j);
  }
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float* x) {
  const uint4 a = ld_cached16(p);
#pragma unroll
  for (int j = 0; j < 8; ++j) x[j] = unpack<__nv_bfloat16>(a, j);
}

// One CTA per (touched block, head, side).
template <typename TIn, int kD>
__global__ __launch_bounds__(kThreads) void q8_rope_store_kernel(const RopeStoreArgs a) {
  constexpr uint32_t kLanes = kD / 16;  // threads of a row
  constexpr uint32_t kStep = kThreads / kLanes;
  __shared__ float s_max[kThreads / 32];
  pdl_wait();
  pdl_release();
  const uint32_t n = count_or_capacity(a.d_counts, 0, a.capacity);
  const uint32_t H = a.c.heads, T = a.c.block_tokens;
  const uint32_t j = threadIdx.x % kLanes, r0 = threadIdx.x / kLanes;
  // this thread's two runs of eight channels, and the pairs that they hold
  uint32_t c0 = 16 * j, c1 = 16 * j + 8, pair = (c0 - a.begin) / 2;
  bool turns = c0 >= a.begin && c0 < a.begin + a.dim;
  if (a.halves && a.dim) {
    turns = j < a.dim / 16;
    pair = 8 * j;
    const uint32_t rest = 16 * (j - a.dim / 16);  // the channels that do not turn, two runs to a thread
    c0 = turns ? a.begin + 8 * j : rest < a.begin ? rest : rest + a.dim;
    c1 = turns ? c0 + a.dim / 2 : c0 + 8;
  }
  for (uint32_t i = blockIdx.x; i < n; i += gridDim.x) {
    const uint4 rec = __ldg(reinterpret_cast<const uint4*>(a.plan + i));
    if (rec.x == kInvalidU32) continue;
    const uint32_t block = rec.x, row0 = rec.y, off = rec.z & 0xFFFFu, cnt = rec.z >> 16;
    if (block >= a.c.num_blocks || cnt == 0 || off + cnt > T || static_cast<uint64_t>(row0) + cnt > a.num_rows) {
      if (threadIdx.x == 0) status_or(a.d_status, CKV_STATUS_BAD_INDEX);
      continue;
    }
    for (uint32_t u = blockIdx.y; u < H * a.sides; u += gridDim.y) {
      const bool second = u >= H;
      const uint32_t h = second ? u - H : u;
      const TIn* rows = second ? static_cast<const TIn*>(a.v_rows) + row0 * a.v_stride
                               : static_cast<const TIn*>(a.k_rows) + row0 * a.k_stride;
      rows += static_cast<size_t>(h) * kD;
      const uint64_t stride = second ? a.v_stride : a.k_stride;
      uint8_t* pool = (second ? a.c.v : a.c.k) + (static_cast<size_t>(block) * H + h) * T * kD;
      float* scale = (second ? a.c.v_scale : a.c.k_scale) + static_cast<size_t>(block) * H + h;
      const float old = off ? *scale : 0.0f;
      // Row r's values; false where it is not stored.  All threads of a warp call it.
      auto row_of = [&](uint32_t r, float (&x)[16]) -> bool {
        bool in = r < cnt;
        int64_t pos = 0;
        if (in && a.dim) {
          pos = __ldg(a.positions + row0 + r);
          in = pos >= 0 && pos < a.max_pos;
        }
#pragma unroll
        for (int z = 0; z < 16; ++z) x[z] = 0.0f;
        if (in) {
          load8(rows + r * stride + c0, x);
          load8(rows + r * stride + c1, x + 8);
        }
        if (second) return in;
        if (a.weight != nullptr) {
          float s = 0.0f;
#pragma unroll
          for (int z = 0; z < 16; ++z) s = fmaf(x[z], x[z], s);
#pragma unroll
          for (uint32_t z = 1; z < kLanes; z <<= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, z);
          const float inv = __fdiv_rn(1.0f, __fsqrt_rn(fmaf(s, 1.0f / kD, a.eps)));
          float w[16];
          load8(a.weight + c0, w);
          load8(a.weight + c1, w + 8);
#pragma unroll
          for (int z = 0; z < 16; ++z) x[z] = __fmul_rn(__fmul_rn(x[z], w[z]), inv);
        }
        if (turns && in) {
          const float* f = a.freqs + (static_cast<size_t>(pos) * (a.dim / 2) + pair) * 2;
          float cs[16];
          load8(f, cs);
          load8(f + 8, cs + 8);
          auto turn = [&](float& p, float& q, int z) {
            const float c = cs[2 * z], s = cs[2 * z + 1], x0 = p, x1 = q;
            p = __fsub_rn(__fmul_rn(x0, c), __fmul_rn(x1, s));
            q = __fadd_rn(__fmul_rn(x0, s), __fmul_rn(x1, c));
          };
          if (a.halves) {
#pragma unroll
            for (int z = 0; z < 8; ++z) turn(x[z], x[8 + z], z);
          } else {
#pragma unroll
            for (int z = 0; z < 8; ++z) turn(x[2 * z], x[2 * z + 1], z);
          }
        }
        return in;
      };
      float m = 0.0f;
      bool all = true;
      for (uint32_t r = r0; r - r0 < cnt; r += kStep) {
        float x[16];
        all &= row_of(r, x) || r >= cnt;
#pragma unroll
        for (int z = 0; z < 16; ++z) {  // NaN and infinities do not count
          const float ax = fabsf(x[z]);
          m = ax < INFINITY ? fmaxf(m, ax) : m;
        }
      }
      if (!all && j == 0) status_or(a.d_status, CKV_STATUS_BAD_INDEX);
#pragma unroll
      for (int s = 16; s > 0; s >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, s));
      if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = m;
      __syncthreads();
      m = s_max[0];
#pragma unroll
      for (int w = 1; w < kThreads / 32; ++w) m = fmaxf(m, s_max[w]);
      const float now = fmaxf(pow2f(q8_need_exp(m)), old);
      const float inv = 1.0f / now;
      for (uint32_t r = r0; r - r0 < cnt; r += kStep) {
        float x[16];
        if (row_of(r, x)) {
          uint8_t* to = pool + static_cast<size_t>(off + r) * kD;
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            uint2 o;
            o.x = q8_pack4(x[8 * z] * inv, x[8 * z + 1] * inv, x[8 * z + 2] * inv, x[8 * z + 3] * inv);
            o.y = q8_pack4(x[8 * z + 4] * inv, x[8 * z + 5] * inv, x[8 * z + 6] * inv, x[8 * z + 7] * inv);
            *reinterpret_cast<uint2*>(to + (z ? c1 : c0)) = o;
          }
          // a new entry has had no attention yet, whatever the slot's last owner had
          if (a.weights != nullptr && u == 0 && j == 0) a.weights[static_cast<size_t>(block) * T + off + r] = 0.0f;
        }
      }
      if (off && now > old) {  // the entries that were there follow the scale
        const float f = old * inv;
        for (uint32_t w = threadIdx.x; w < off * kLanes; w += kThreads) {
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

template <typename TIn>
int launch(const RopeStoreArgs& a, cudaStream_t s) {
  const dim3 grid(std::min<uint32_t>(a.capacity, 65536u), a.c.heads * a.sides);
  switch (a.c.head_dim) {
    case 64: return launch_pdl(q8_rope_store_kernel<TIn, 64>, grid, dim3(kThreads), 0, s, a);
    case 128: return launch_pdl(q8_rope_store_kernel<TIn, 128>, grid, dim3(kThreads), 0, s, a);
    case 256: return launch_pdl(q8_rope_store_kernel<TIn, 256>, grid, dim3(kThreads), 0, s, a);
    default: return launch_pdl(q8_rope_store_kernel<TIn, 512>, grid, dim3(kThreads), 0, s, a);
  }
}

}  // namespace
}  // namespace ckv

using namespace ckv;

extern "C" int ckv_q8_rope_store(const ckv_q8_cache_t* cache, int in_dtype, const void* k_rows, uint64_t k_stride,
                                 const void* v_rows, uint64_t v_stride, uint32_t num_rows, const int64_t* positions,
                                 const float* norm_weight, float eps, const float* freqs, uint32_t max_pos,
                                 uint32_t rope_begin, uint32_t rope_dim, int halves, const ckv_q8_store_plan_t* plan,
                                 const uint32_t* d_counts, uint32_t capacity, float* weights, uint32_t* d_status,
                                 ckv_stream_t stream) {
  RopeStoreArgs a{};
  const int rc = q8_cache_of(cache, &a.c);
  if (rc) return rc;
  if (in_dtype != CKV_F32 && in_dtype != CKV_BF16) return CKV_ERR_DTYPE;
  if (rope_dim % 32 != 0 || rope_begin % 16 != 0 || rope_dim > a.c.head_dim || rope_begin > a.c.head_dim - rope_dim)
    return CKV_ERR_HEAD_DIM;
  if (num_rows > CKV_MAX_TOKENS || capacity > CKV_MAX_TOKENS) return CKV_ERR_SIZE;
  if (norm_weight != nullptr && (!(eps > 0.0f) || !(eps < 1e30f))) return CKV_ERR_SIZE;
  if (num_rows == 0 || capacity == 0) return CKV_OK;
  const uint64_t least = static_cast<uint64_t>(a.c.heads) * a.c.head_dim, whole = in_dtype == CKV_BF16 ? 8 : 4;
  auto stride_ok = [&](uint64_t s) { return s >= least && s % whole == 0 && s < 1ull << 32; };
  if (!stride_ok(k_stride) || (v_rows != nullptr && !stride_ok(v_stride))) return CKV_ERR_SIZE;
  if (!aligned16(k_rows) || (a.c.v != nullptr) != (v_rows != nullptr) || (v_rows != nullptr && !aligned16(v_rows)))
    return CKV_ERR_POINTER;
  if (rope_dim != 0 && (!aligned_to(positions, 8) || !aligned16(freqs))) return CKV_ERR_POINTER;
  if (norm_weight != nullptr && !aligned16(norm_weight)) return CKV_ERR_POINTER;
  if (!aligned16(plan) || (d_counts != nullptr && !aligned_to(d_counts, 4))) return CKV_ERR_POINTER;
  if (weights != nullptr && !aligned_to(weights, 4)) return CKV_ERR_POINTER;
  a.k_rows = k_rows;
  a.v_rows = v_rows;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.num_rows = num_rows;
  a.positions = positions;
  a.weight = norm_weight;
  a.eps = eps;
  a.freqs = freqs;
  a.max_pos = max_pos;
  a.begin = rope_begin;
  a.dim = rope_dim;
  a.halves = halves != 0;
  a.plan = plan;
  a.d_counts = d_counts;
  a.capacity = capacity;
  a.sides = v_rows != nullptr ? 2 : 1;
  a.weights = weights;
  a.d_status = d_status;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return in_dtype == CKV_BF16 ? launch<__nv_bfloat16>(a, s) : launch<float>(a, s);
}

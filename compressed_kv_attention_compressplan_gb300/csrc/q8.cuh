// q8.cuh -- what the kernels of the 8-bit paged cache share: its layout, the
// e4m3 conversions, block scans and the per-request lengths.
//
// Layout.  k (and v) is [num_blocks, n_kv_heads, T, head_dim] bytes, one e4m3
// value each; k_scale (v_scale) is [num_blocks, n_kv_heads] fp32.  The value
// held is e4m3 * scale.  The T entries of one (block, head) are one run of
// T * head_dim bytes, so any 16 of them (T is a multiple of 16) are one run
// too and share one scale: the attention kernels take 16 entries at a time.
//
// Scales are powers of two, 2^kQ8ExpMin .. 2^kQ8ExpMax.  e4m3 is a floating
// type, so dividing by a power of two costs no precision down to its
// subnormals, and a block whose scale has to grow (a larger row arrives, or
// entries of several blocks come together) is rewritten exactly, apart from
// entries that fall into the subnormals, 2^-15 and less of the block's largest.
// The exponents' range keeps every product of two scales and a weight inside
// fp32's range (see the attention kernel's weights).
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "common.cuh"
#include "launch.h"

namespace ckv {

constexpr int kQ8ExpMin = -48;
constexpr int kQ8ExpMax = 48;

struct Q8Cache {
  uint8_t* k;
  float* k_scale;
  uint8_t* v;        // NULL: the values are k
  float* v_scale;
  uint32_t num_blocks;
  uint32_t block_tokens;
  uint32_t heads;
  uint32_t head_dim;
};

// Copies and checks the caller's cache description.
inline int q8_cache_of(const ckv_q8_cache_t* c, Q8Cache* out) {
  if (c == nullptr) return CKV_ERR_POINTER;
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256 && c->head_dim != 512) return CKV_ERR_HEAD_DIM;
  if (c->block_tokens != 16 && c->block_tokens != 32 && c->block_tokens != 64 && c->block_tokens != 128)
    return CKV_ERR_SIZE;
  if (c->n_kv_heads == 0 || c->n_kv_heads > CKV_Q8_MAX_KV_HEADS || c->num_blocks == 0 || c->num_blocks > 0x7FFFFFFFu)
    return CKV_ERR_SIZE;
  if (!aligned16(c->k) || !aligned16(c->k_scale)) return CKV_ERR_POINTER;
  if ((c->v == nullptr) != (c->v_scale == nullptr)) return CKV_ERR_POINTER;
  if (c->v != nullptr && (!aligned16(c->v) || !aligned16(c->v_scale))) return CKV_ERR_POINTER;
  out->k = static_cast<uint8_t*>(c->k);
  out->k_scale = c->k_scale;
  out->v = static_cast<uint8_t*>(c->v);
  out->v_scale = c->v_scale;
  out->num_blocks = c->num_blocks;
  out->block_tokens = c->block_tokens;
  out->heads = c->n_kv_heads;
  out->head_dim = c->head_dim;
  return CKV_OK;
}

inline bool aligned_to(const void* p, uintptr_t n) {
  return p != nullptr && (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0;
}

// Block table argument: int32 [num_reqs, stride], row rid of a request.
inline int check_table(const int32_t* table, uint64_t stride, uint32_t num_reqs) {
  if (stride == 0 || stride > 0x7FFFFFFFull || num_reqs == 0) return CKV_ERR_SIZE;
  return aligned_to(table, 4) ? CKV_OK : CKV_ERR_POINTER;
}

// ---------------------------------------------------------------- e4m3
// The smallest e with a <= 448 * 2^e (448 = 0.875 * 2^9 is e4m3's largest
// value), from a's own bits and so exact; a is finite and not negative.
__device__ __forceinline__ int q8_need_exp(float a) {
  const uint32_t u = __float_as_uint(a);
  // a = 1.f * 2^(x - 127): 1.f <= 1.75 asks for x - 127 - 8, a larger one for one more
  const int e = static_cast<int>(u >> 23) - 127 - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return min(max(e, kQ8ExpMin), kQ8ExpMax);
}

__device__ __forceinline__ float pow2f(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

// Two fp32 -> two e4m3, round to nearest even, values past 448 to 448, NaN to NaN.
__device__ __forceinline__ uint32_t q8_pack2(float lo, float hi) {
  return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ uint32_t q8_pack4(float a, float b, float c, float d) {
  return q8_pack2(a, b) | (q8_pack2(c, d) << 16);
}

// The two e4m3 values in the low / high half of w as an fp16 pair (exact).
__device__ __forceinline__ uint32_t q8_lo_f16x2(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(r) : "r"(w));
  return r;
}
__device__ __forceinline__ uint32_t q8_hi_f16x2(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(r) : "r"(w));
  return r;
}

__device__ __forceinline__ float2 f16x2_to_f32(uint32_t h) {
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// Four e4m3 values times a power of two f <= 1, rounded back to e4m3.
__device__ __forceinline__ uint32_t q8_rescale4(uint32_t w, float f) {
  const float2 a = f16x2_to_f32(q8_lo_f16x2(w));
  const float2 b = f16x2_to_f32(q8_hi_f16x2(w));
  return q8_pack4(a.x * f, a.y * f, b.x * f, b.y * f);
}

// 0xFF in every byte of w that is an e4m3 NaN (0x7F or 0xFF).
__device__ __forceinline__ uint32_t q8_nan_bytes(uint32_t w) { return __vcmpeq4(w & 0x7F7F7F7Fu, 0x7F7F7F7Fu); }

// Two fp32 products at once (see f2_add and f2_fma).
__device__ __forceinline__ F2 f2_mul(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}

// ---------------------------------------------------------------- scans
// Exclusive scan of v over a block of kThreads threads, and the total.
// s_warp: kThreads / 32 + 1 words of shared memory; all threads call it.
template <int kThreads, typename T>
__device__ __forceinline__ T block_exclusive(T v, T* total, T* s_warp) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  T incl = v;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const T n = __shfl_up_sync(0xFFFFFFFFu, incl, off);
    if (lane >= off) incl += n;
  }
  __syncthreads();  // an earlier scan's reads of s_warp are done
  if (lane == 31) s_warp[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    T w = lane < kThreads / 32 ? s_warp[lane] : T(0);
    const T own = w;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const T n = __shfl_up_sync(0xFFFFFFFFu, w, off);
      if (lane >= off) w += n;
    }
    if (lane < kThreads / 32) s_warp[lane] = w - own;
    if (lane == 31) s_warp[kThreads / 32] = w;
  }
  __syncthreads();
  *total = s_warp[kThreads / 32];
  return s_warp[warp] + incl - v;
}

// The last index i with s[i] <= x, for ascending s[0 .. n) with s[0] <= x.
template <typename T>
__device__ __forceinline__ uint32_t last_not_above(const T* s, uint32_t n, T x) {
  uint32_t lo = 0, hi = n;  // s[lo] <= x, s[hi] > x (or hi == n)
  while (hi - lo > 1) {
    const uint32_t mid = (lo + hi) >> 1;
    if (s[mid] <= x)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// ---------------------------------------------------------------- visibility
// Query i of a request's q_len queries sees its first
//     kv_len - (floor(S / R) - floor((S - q_len + i + 1) / R))
// entries (S tokens so far, R tokens to a cached entry): the entries whose
// group ends after the query are hidden, counted back from the newest, so the
// count stays right when older entries were evicted.  With d = q_len - 1 - i
// tokens after the query and phase = R - 1 - S % R the bracket is
// floor((d + phase) / R).
__device__ __forceinline__ int64_t q8_visible(int64_t kv_len, uint32_t after, uint32_t phase, uint32_t ratio) {
  const int64_t v = kv_len - static_cast<int64_t>((after + phase) / ratio);
  return v < 0 ? 0 : v;
}

// ---------------------------------------------------------------- copies
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
  // bytes 16, or 0 to write zeros (src is not read then)
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A streamed 16-byte load, or zeros where `in` is false: predicated, so that nothing waits for it
// before its first use (a branch around the load would, where the paths join).
__device__ __forceinline__ uint4 ld_stream16_if(const void* p, bool in) {
  uint4 v;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.u32 p, %5, 0;\n\t"
      "mov.u32 %0, 0;\n\tmov.u32 %1, 0;\n\tmov.u32 %2, 0;\n\tmov.u32 %3, 0;\n\t"
      "@p ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];\n\t}"
      : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w)
      : "l"(p), "r"(in ? 1u : 0u));
  return v;
}

__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint2 lds8(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ float lds_f32(uint32_t a) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds_u32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void sts_u32(uint32_t a, uint32_t v) {
  asm volatile("st.shared.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}

}  // namespace ckv

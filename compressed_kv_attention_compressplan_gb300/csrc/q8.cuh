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

#include <atomic>

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

// Lets `kernel` use `bytes` of shared memory; asked of the driver once a device (`done`: a bit for each).
inline int allow_smem(const void* kernel, uint32_t bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return CKV_ERR_LAUNCH;
  const uint64_t bit = dev >= 0 && dev < 64 ? 1ull << dev : 0;
  if (done.load(std::memory_order_relaxed) & bit) return CKV_OK;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes)) != cudaSuccess) {
    cudaGetLastError();
    return CKV_ERR_LAUNCH;
  }
  done.fetch_or(bit, std::memory_order_relaxed);
  return CKV_OK;
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

// 1 / x to a unit in the last place, x normal: one instruction where a division takes ten and a branch.
__device__ __forceinline__ float rcp(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

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

// Two such scans between the same barriers.
template <int kThreads, typename T>
__device__ __forceinline__ void block_exclusive2(T v0, T v1, T* out0, T* out1, T* total0, T* total1, T (*s_warp)[kThreads / 32 + 1]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  T a = v0, b = v1;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const T x = __shfl_up_sync(0xFFFFFFFFu, a, off), y = __shfl_up_sync(0xFFFFFFFFu, b, off);
    if (lane >= off) {
      a += x;
      b += y;
    }
  }
  __syncthreads();  // an earlier scan's reads of s_warp are done
  if (lane == 31) {
    s_warp[0][warp] = a;
    s_warp[1][warp] = b;
  }
  __syncthreads();
  // every warp adds the warps' sums up for itself: one barrier less
  const T x = lane < kThreads / 32 ? s_warp[0][lane] : T(0), y = lane < kThreads / 32 ? s_warp[1][lane] : T(0);
  T p = x, q = y;
#pragma unroll
  for (int off = 1; off < kThreads / 32; off <<= 1) {
    const T u = __shfl_up_sync(0xFFFFFFFFu, p, off), v = __shfl_up_sync(0xFFFFFFFFu, q, off);
    if (lane >= off) {
      p += u;
      q += v;
    }
  }
  const T base0 = __shfl_sync(0xFFFFFFFFu, p - x, warp), base1 = __shfl_sync(0xFFFFFFFFu, q - y, warp);
  *out0 = base0 + a - v0;
  *out1 = base1 + b - v1;
  *total0 = __shfl_sync(0xFFFFFFFFu, p, kThreads / 32 - 1);
  *total1 = __shfl_sync(0xFFFFFFFFu, q, kThreads / 32 - 1);
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

// ---------------------------------------------------------------- fragments
// fp16 x fp16 -> fp32, 16 x 8 x 16
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Byte offset of 16-byte chunk cc of token t in a tile of 16 kDw-byte rows.  The
// chunks of a 128-byte line are permuted by the token (or line), so that both
// the K fragments' reads (2 tokens, 4 chunks of each) and the V fragments'
// (4 tokens, 2 chunks) take every bank once.
template <int kDw>
__device__ __forceinline__ uint32_t tile_off(uint32_t t, uint32_t cc) {
  if (kDw == 64) {
    const uint32_t line = t >> 1, pos = (t & 1) * 4 + cc;
    return line * 128 + ((pos ^ (line & 7)) << 4);
  }
  const uint32_t line = t * (kDw / 128) + (cc >> 3);
  return line * 128 + (((cc & 7) ^ (t & 7)) << 4);
}

// Chunk j of the kDw / 64 that lane (g, q) = (lane / 4, lane % 4) multiplies per entry.
template <int kDw>
__device__ __forceinline__ int lane_chunk(int j, int q) {
  return kDw == 64 ? q : 8 * (j >> 1) + 2 * q + (j & 1);
}

// A query row's part of the fragments (r: 0 for the lane's row g, 1 for g + 8): scaled by a power of two that puts
// the row's largest value in [2^14, 2^15) and rounded to fp16; returns what undoes the scaling.
template <int kDw>
__device__ __forceinline__ float load_query(const __nv_bfloat16* p, bool in, int q, int r, uint32_t (&qf)[kDw / 16][4]) {
  uint4 v[kDw / 64][2];
  float m = 0.0f;
#pragma unroll
  for (int j = 0; j < kDw / 64; ++j) {
    const int cc = lane_chunk<kDw>(j, q);
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      v[j][w] = in ? ld_cached16(p + cc * 16 + w * 8) : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(unpack<__nv_bfloat16>(v[j][w], e)));
    }
  }
  m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
  m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
  const int ex = min(126, 14 - (static_cast<int>(__float_as_uint(m) >> 23) - 127));
  const float up = pow2f(ex);
#pragma unroll
  for (int j = 0; j < kDw / 64; ++j) {
#pragma unroll
    for (int s = 0; s < 4; ++s) {  // k step 4 j + s: channels 4 s .. 4 s + 3 of the chunk
      const uint4 x = v[j][s >> 1];
      const int e = (s & 1) * 4;
      qf[j * 4 + s][r] = pack_f16x2(unpack<__nv_bfloat16>(x, e) * up, unpack<__nv_bfloat16>(x, e + 1) * up);
      qf[j * 4 + s][2 + r] = pack_f16x2(unpack<__nv_bfloat16>(x, e + 2) * up, unpack<__nv_bfloat16>(x, e + 3) * up);
    }
  }
  return pow2f(-ex);
}

// ---------------------------------------------------------------- copies
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
  // bytes 16, or 0 to write zeros (src is not read then)
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Arrives on an mbarrier (as one of its count) when this thread's copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" ::"r"(bar) : "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A load made well before its use, and issued where it stands: a plain __ldg may be moved down to its first use to save
// a register, and its latency with it.
__device__ __forceinline__ int32_t ld_ahead(const int32_t* p) {
  int32_t v;
  asm volatile("ld.global.nc.s32 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}
__device__ __forceinline__ float ld_ahead(const float* p) {
  float v;
  asm volatile("ld.global.nc.f32 %0, [%1];" : "=f"(v) : "l"(p));
  return v;
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

// Scores of 16 query rows against the 16 entries of a tile at shared address st: s[n] are entries 8 n .. 8 n + 7.
template <int kDw>
__device__ __forceinline__ void tile_scores(uint32_t st, int g, int q, const uint32_t (&qf)[kDw / 16][4], float (&s)[2][4]) {
#pragma unroll
  for (int n = 0; n < 2; ++n) {
    s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.0f;
#pragma unroll
    for (int j = 0; j < kDw / 64; ++j) {
      const uint4 w = lds16(st + tile_off<kDw>(n * 8 + g, lane_chunk<kDw>(j, q)));
      mma_f16(s[n], qf[j * 4 + 0], q8_lo_f16x2(w.x), q8_hi_f16x2(w.x));
      mma_f16(s[n], qf[j * 4 + 1], q8_lo_f16x2(w.y), q8_hi_f16x2(w.y));
      mma_f16(s[n], qf[j * 4 + 2], q8_lo_f16x2(w.z), q8_hi_f16x2(w.z));
      mma_f16(s[n], qf[j * 4 + 3], q8_lo_f16x2(w.w), q8_hi_f16x2(w.w));
    }
  }
}

// The same with the entries as the product's rows: score e is that of entry (e >> 1) * 8 + g and column 2q + (e & 1).
template <int kDw>
__device__ __forceinline__ void tile_scores_t(uint32_t st, int g, int q, const uint32_t (&qf)[kDw / 16][4], float (&s)[4]) {
  s[0] = s[1] = s[2] = s[3] = 0.0f;
#pragma unroll
  for (int j = 0; j < kDw / 64; ++j) {
    const int cc = lane_chunk<kDw>(j, q);
    const uint4 lo = lds16(st + tile_off<kDw>(g, cc)), hi = lds16(st + tile_off<kDw>(8 + g, cc));
    const uint32_t x[4] = {lo.x, lo.y, lo.z, lo.w}, y[4] = {hi.x, hi.y, hi.z, hi.w};
#pragma unroll
    for (int z = 0; z < 4; ++z) {
      const uint32_t kf[4] = {q8_lo_f16x2(x[z]), q8_lo_f16x2(y[z]), q8_hi_f16x2(x[z]), q8_hi_f16x2(y[z])};
      mma_f16(s, kf, qf[j * 4 + z][0], qf[j * 4 + z][2]);
    }
  }
}

// 8 x 8 values of 16 bits, two to a lane, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

}  // namespace ckv

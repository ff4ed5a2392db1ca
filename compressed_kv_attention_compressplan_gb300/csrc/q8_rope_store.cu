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
//
// Bound.  The rows' bytes, and a thread's work for sixteen channels: 276 MB of bf16 rows and codes (16 requests of up to 4096 new rows, eight kv
// heads of 128 channels, K and V) take 55 us, 5.0 TB/s or 75 % of the copy rate, with the registers (96) leaving 20 warps to an SM.  With angles
// in registers (128, so 16 warps) 66 us; and then a first pass for the scale and a second for the codes 93, one unit to a CTA 90, rows ahead by
// asynchronous copies 73.
#include <algorithm>

#include "async_copy.cuh"
#include "q8.cuh"

namespace ckv {
namespace {

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

// What a thread has of a row: two runs of eight channels, and the pairs that they hold.
struct Lane {
  uint32_t c0, c1, pair;
  bool turns;
};

__device__ __forceinline__ Lane lane_of(const RopeStoreArgs& a, uint32_t j) {
  Lane l = {16 * j, 16 * j + 8, (16 * j - a.begin) / 2, 16 * j >= a.begin && 16 * j < a.begin + a.dim};
  if (a.halves && a.dim) {
    l.turns = j < a.dim / 16;
    l.pair = 8 * j;
    const uint32_t rest = 16 * (j - a.dim / 16);  // the channels that do not turn, two runs to a thread
    l.c0 = l.turns ? a.begin + 8 * j : rest < a.begin ? rest : rest + a.dim;
    l.c1 = l.turns ? l.c0 + a.dim / 2 : l.c0 + 8;
  }
  return l;
}

// A key row's norm (all threads of a warp call it) and its rotation, where this thread's channels turn.
template <int kD>
__device__ __forceinline__ float norm_of(const RopeStoreArgs& a, float s) {  // s: this thread's sum of squares
#pragma unroll
  for (uint32_t z = 1; z < kD / 16; z <<= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, z);
  return __fdiv_rn(1.0f, __fsqrt_rn(fmaf(s, 1.0f / kD, a.eps)));
}

template <int kD>
__device__ __forceinline__ void normalise(const RopeStoreArgs& a, const float (&w)[16], float (&x)[16]) {
  float s = 0.0f;
#pragma unroll
  for (int z = 0; z < 16; ++z) s = fmaf(x[z], x[z], s);
  const float inv = norm_of<kD>(a, s);
#pragma unroll
  for (int z = 0; z < 16; ++z) x[z] = __fmul_rn(__fmul_rn(x[z], w[z]), inv);
}

// The cosines and sines of a thread's eight pairs, and its channels turned by them.
__device__ __forceinline__ void angles(const RopeStoreArgs& a, const Lane& l, uint32_t pos, float (&cs)[16]) {
  const float* f = a.freqs + (static_cast<size_t>(pos) * (a.dim / 2) + l.pair) * 2;
  load8(f, cs);
  load8(f + 8, cs + 8);
}

__device__ __forceinline__ void rotate(const RopeStoreArgs& a, const float (&cs)[16], float (&x)[16]) {
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

// The largest magnitude, NaN passed over.
__device__ __forceinline__ float largest(float m, const float (&x)[16]) {
#pragma unroll
  for (int z = 0; z < 16; ++z) m = fmaxf(m, fabsf(x[z]));
  return m;
}
// The same of a thread's rows in `in`, infinities passed over too: done where there is one.
template <int kVecs>
__device__ __forceinline__ float largest_finite(const float (&x)[kVecs][16], uint32_t in) {
  float m = 0.0f;
#pragma unroll
  for (int v = 0; v < kVecs; ++v) {
#pragma unroll
    for (int z = 0; z < 16; ++z)
      if (in >> v & 1) m = fabsf(x[v][z]) < INFINITY ? fmaxf(m, fabsf(x[v][z])) : m;
  }
  return m;
}
template <typename TIn>
__device__ __forceinline__ float largest_raw(float m, const uint4 (&raw)[sizeof(TIn)]) {
#pragma unroll
  for (int c = 0; c < static_cast<int>(sizeof(TIn)); ++c) {
    if constexpr (sizeof(TIn) == 2) {  // two at a time, as they are
      const uint32_t w[4] = {raw[c].x, raw[c].y, raw[c].z, raw[c].w};
      __nv_bfloat162 t = __float2bfloat162_rn(0.0f);
#pragma unroll
      for (int z = 0; z < 4; ++z) {
        const uint32_t x = w[z] & 0x7FFF7FFFu;
        t = __hmax2(t, *reinterpret_cast<const __nv_bfloat162*>(&x));
      }
      m = fmaxf(m, fmaxf(__low2float(t), __high2float(t)));
    } else {
#pragma unroll
      for (int z = 0; z < 4; ++z) m = fmaxf(m, fabsf(unpack<float>(raw[c], z)));
    }
  }
  return m;
}

__device__ __forceinline__ void put16(uint8_t* to, const Lane& l, const float (&x)[16], float inv) {
  uint2 o[2];
#pragma unroll
  for (int z = 0; z < 2; ++z) {
    o[z].x = q8_pack4(x[8 * z] * inv, x[8 * z + 1] * inv, x[8 * z + 2] * inv, x[8 * z + 3] * inv);
    o[z].y = q8_pack4(x[8 * z + 4] * inv, x[8 * z + 5] * inv, x[8 * z + 6] * inv, x[8 * z + 7] * inv);
  }
  if (l.c1 == l.c0 + 8) {
    st16(to + l.c0, make_uint4(o[0].x, o[0].y, o[1].x, o[1].y));
  } else {
    *reinterpret_cast<uint2*>(to + l.c0) = o[0];
    *reinterpret_cast<uint2*>(to + l.c1) = o[1];
  }
}

// The largest over a CTA: one barrier, and s_max is free again after the next.
__device__ __forceinline__ float cta_max(float m, float* s_max) {
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, s));
  if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = m;
  __syncthreads();
  m = s_max[0];
  for (uint32_t w = 1; w < blockDim.x / 32; ++w) m = fmaxf(m, s_max[w]);
  return m;
}

// The first `off` entries of a block follow its scale, which grew by 1 / f.
template <int kD>
__device__ __forceinline__ void follow(uint8_t* pool, uint32_t off, float f, uint32_t t, uint32_t threads) {
  for (uint32_t w = t; w < off * (kD / 16); w += threads) {
    uint4 v = *reinterpret_cast<const uint4*>(pool + w * 16);
    v.x = q8_rescale4(v.x, f);
    v.y = q8_rescale4(v.y, f);
    v.z = q8_rescale4(v.z, f);
    v.w = q8_rescale4(v.w, f);
    st16(pool + w * 16, v);
  }
}

// A record's unit: a (head, side) of its block.
template <typename TIn, int kD>
struct Unit {
  uint32_t block, row0, off, cnt, u, h;
  bool ok, second;
  __device__ __forceinline__ Unit(const RopeStoreArgs& a, const uint4& rec, uint32_t unit) {
    block = rec.x, row0 = rec.y, off = rec.z & 0xFFFFu, cnt = rec.z >> 16, u = unit;
    ok = rec.x != kInvalidU32 && block < a.c.num_blocks && cnt != 0 && off + cnt <= a.c.block_tokens &&
         static_cast<uint64_t>(row0) + cnt <= a.num_rows;
    if (rec.x != kInvalidU32 && !ok && threadIdx.x == 0) status_or(a.d_status, CKV_STATUS_BAD_INDEX);
    second = u >= a.c.heads;
    h = second ? u - a.c.heads : u;
  }
  __device__ __forceinline__ const TIn* row(const RopeStoreArgs& a, uint32_t r) const {
    const uint64_t at = static_cast<uint64_t>(row0) + r;
    return static_cast<const TIn*>(second ? a.v_rows : a.k_rows) + at * (second ? a.v_stride : a.k_stride) + static_cast<size_t>(h) * kD;
  }
  __device__ __forceinline__ uint8_t* entries(const RopeStoreArgs& a) const {
    return (second ? a.c.v : a.c.k) + (static_cast<size_t>(block) * a.c.heads + h) * a.c.block_tokens * kD;
  }
  __device__ __forceinline__ float* scale(const RopeStoreArgs& a) const {
    return (second ? a.c.v_scale : a.c.k_scale) + static_cast<size_t>(block) * a.c.heads + h;
  }
  __device__ __forceinline__ void reset(const RopeStoreArgs& a, uint32_t r) const {
    if (a.weights != nullptr && u == 0) a.weights[static_cast<size_t>(block) * a.c.block_tokens + off + r] = 0.0f;
  }
};

// A CTA takes a record and some of its units, one after the other.  A thread keeps its places in the block, kVecs rows and
// sixteen channels of each: positions, angles and the norm's weights are read once for all heads and stay in shared memory, where nobody else
// touches them, and a unit's values in registers from the search for the scale to the codes, while the next unit's rows are on their way.
template <typename TIn, int kD, int kVecs, int kThreads, int kPerSm>
__global__ __launch_bounds__(kThreads, kPerSm) void q8_rope_store_kernel(const RopeStoreArgs a, uint32_t units_of_cta, uint32_t parts) {
  constexpr uint32_t kLanes = kD / 16;      // threads of a row
  constexpr uint32_t kLoads = sizeof(TIn);  // 16-byte loads of sixteen channels
  constexpr uint32_t kElems = 16 / sizeof(TIn);
  __shared__ float s_max[2][32];
  __shared__ float4 s_cs[kVecs][4][kThreads], s_w[4][kThreads];  // angles, weights: a thread reads back what itself has put
  pdl_wait();
  pdl_release();
  const uint32_t n = count_or_capacity(a.d_counts, 0, a.capacity), H = a.c.heads, T = a.c.block_tokens, step = blockDim.x / kLanes;
  const uint32_t j = threadIdx.x % kLanes, r0 = threadIdx.x / kLanes;
  const Lane l = lane_of(a, j);
  const uint32_t u0 = blockIdx.x % parts * units_of_cta, u1 = min(H * a.sides, u0 + units_of_cta);
  uint32_t flip = 0;
  if (a.weight != nullptr && u0 < H) {
    float w[16];
    load8(a.weight + l.c0, w);
    load8(a.weight + l.c1, w + 8);
#pragma unroll
    for (int z = 0; z < 4; ++z) s_w[z][threadIdx.x] = make_float4(w[4 * z], w[4 * z + 1], w[4 * z + 2], w[4 * z + 3]);
  }
  for (uint32_t i = blockIdx.x / parts; i < n; i += gridDim.x / parts) {
    const uint4 rec = __ldg(reinterpret_cast<const uint4*>(a.plan + i));
    const Unit<TIn, kD> first(a, rec, u0);
    if (!first.ok) continue;
    const uint32_t off = first.off, cnt = first.cnt;
    // places that are stored, and their angles
    uint32_t in = 0;
    int64_t pos[kVecs];
#pragma unroll
    for (int v = 0; v < kVecs; ++v) pos[v] = a.dim && r0 + v * step < cnt ? __ldg(a.positions + first.row0 + r0 + v * step) : 0;
    uint4 raw[kVecs][kLoads];
    float old_next;
    auto load = [&](const TIn* src, uint64_t stride, const float* scale) {
      old_next = off ? *scale : 0.0f;
#pragma unroll
      for (int v = 0; v < kVecs; ++v) {
        const bool here = r0 + v * step < cnt;
#pragma unroll
        for (uint32_t c = 0; c < kLoads; ++c)
          raw[v][c] = ld_stream16_if(src + v * step * stride + (c < kLoads / 2 ? l.c0 : l.c1) + c % (kLoads / 2) * kElems, here);
      }
    };
    const size_t block0 = static_cast<size_t>(first.block) * H;  // (block, head) of head 0
    const uint64_t row = static_cast<uint64_t>(first.row0) + r0;
    const TIn* k_src = static_cast<const TIn*>(a.k_rows) + row * a.k_stride;
    const TIn* v_src = a.sides == 2 ? static_cast<const TIn*>(a.v_rows) + row * a.v_stride : nullptr;
    auto load_unit = [&](uint32_t u) {
      if (u < H)
        load(k_src + u * kD, a.k_stride, a.c.k_scale + block0 + u);
      else
        load(v_src + (u - H) * kD, a.v_stride, a.c.v_scale + block0 + u - H);
    };
    load_unit(u0);
    bool bad = false;
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
      const bool here = r0 + v * step < cnt, at = a.dim == 0 || (pos[v] >= 0 && pos[v] < a.max_pos);
      bad |= here && !at;
      in |= (here && at ? 1u : 0u) << v;
      if (l.turns && here && at && u0 < H) {
        float cs[16];
        angles(a, l, static_cast<uint32_t>(pos[v]), cs);
#pragma unroll
        for (int z = 0; z < 4; ++z) s_cs[v][z][threadIdx.x] = make_float4(cs[4 * z], cs[4 * z + 1], cs[4 * z + 2], cs[4 * z + 3]);
      }
    }
    if (bad && j == 0) status_or(a.d_status, CKV_STATUS_BAD_INDEX);
    // a new entry has had no attention yet, whatever the slot's last owner had
    if (a.weights != nullptr && u0 == 0 && j == 0) {
#pragma unroll
      for (int v = 0; v < kVecs; ++v)
        if (in >> v & 1) a.weights[static_cast<size_t>(first.block) * T + off + r0 + v * step] = 0.0f;
    }
    const uint32_t to = (off + r0) * kD;  // this thread's first entry
    auto finish = [&](const float (&x)[kVecs][16], float m, float old, uint8_t* entries, float* scale) {
      if (m == INFINITY) m = largest_finite(x, in);
      const float now = fmaxf(pow2f(q8_need_exp(cta_max(m, s_max[flip]))), old), inv = 1.0f / now;
      flip ^= 1;
#pragma unroll
      for (int v = 0; v < kVecs; ++v)
        if (in >> v & 1) put16(entries + to + v * step * kD, l, x[v], inv);
      if (off && now > old) follow<kD>(entries, off, old * inv, threadIdx.x, blockDim.x);
      if (threadIdx.x == 0) *scale = now;  // every thread has read the old one before the barrier
    };
    uint32_t u = u0;
#pragma unroll 1
    for (; u < min(u1, H); ++u) {  // keys
      const float old = old_next;
      float x[kVecs][16], m = 0.0f;
#pragma unroll
      for (int v = 0; v < kVecs; ++v) {
#pragma unroll
        for (uint32_t c = 0; c < kLoads; ++c) {
#pragma unroll
          for (int z = 0; z < static_cast<int>(kElems); ++z) x[v][c * kElems + z] = unpack<TIn>(raw[v][c], z);
        }
      }
      if (u + 1 < u1) load_unit(u + 1);
#pragma unroll
      for (int v = 0; v < kVecs; ++v) {
        auto back = [&](const float4 (&from)[4][kThreads], float (&y)[16]) {
#pragma unroll
          for (int z = 0; z < 4; ++z) {
            const float4 c = from[z][threadIdx.x];
            y[4 * z] = c.x, y[4 * z + 1] = c.y, y[4 * z + 2] = c.z, y[4 * z + 3] = c.w;
          }
        };
        float y[16];
        if (a.weight != nullptr) {
          back(s_w, y);
          normalise<kD>(a, y, x[v]);
        }
        if (l.turns) {
          back(s_cs[v], y);
          rotate(a, y, x[v]);
        }
        if (in >> v & 1) m = largest(m, x[v]);
      }
      finish(x, m, old, a.c.k + (block0 + u) * T * kD, a.c.k_scale + block0 + u);
    }
#pragma unroll 1
    for (; u < u1; ++u) {  // values
      const float old = old_next;
      float x[kVecs][16], m = 0.0f;
#pragma unroll
      for (int v = 0; v < kVecs; ++v) {
        if (in >> v & 1) m = largest_raw<TIn>(m, raw[v]);
#pragma unroll
        for (uint32_t c = 0; c < kLoads; ++c) {
#pragma unroll
          for (int z = 0; z < static_cast<int>(kElems); ++z) x[v][c * kElems + z] = unpack<TIn>(raw[v][c], z);
        }
      }
      if (u + 1 < u1) load_unit(u + 1);
      finish(x, m, old, a.c.v + (block0 + u - H) * T * kD, a.c.v_scale + block0 + u - H);
    }
  }
}

// Larger blocks (1024 and 2048 vectors of sixteen channels): a CTA takes one unit, four rows to a thread, which stay in registers
// from the search for the scale to the codes.  Such units are few, and what hides a unit's chain of reads is the others on the
// SM: with the next unit's rows ahead, and so half as many units on an SM, 64 entries of 512 channels took 45 us instead of 40.
template <typename TIn, int kD>
__global__ __launch_bounds__(512, 1) void q8_rope_store_hold_kernel(const RopeStoreArgs a) {
  constexpr uint32_t kLanes = kD / 16;
  constexpr int kVecs = 4;
  __shared__ float s_max[16];
  pdl_wait();
  pdl_release();
  const uint32_t n = count_or_capacity(a.d_counts, 0, a.capacity), units = a.c.heads * a.sides, step = blockDim.x / kLanes;
  const uint32_t j = threadIdx.x % kLanes, r0 = threadIdx.x / kLanes;
  const Lane l = lane_of(a, j);
  for (uint32_t i = blockIdx.x; i < n; i += gridDim.x) {
    const uint4 rec = __ldg(reinterpret_cast<const uint4*>(a.plan + i));
    for (uint32_t u = blockIdx.y; u < units; u += gridDim.y) {
      const Unit<TIn, kD> unit(a, rec, u);
      if (!unit.ok) break;
      const float old = unit.off ? *unit.scale(a) : 0.0f;
      float x[kVecs][16], m = 0.0f;
      int64_t pos[kVecs];
      uint32_t in = 0;  // bit v: row v is stored
      bool bad = false;
#pragma unroll
      for (int v = 0; v < kVecs; ++v) pos[v] = a.dim && r0 + v * step < unit.cnt ? __ldg(a.positions + unit.row0 + r0 + v * step) : 0;
#pragma unroll
      for (int v = 0; v < kVecs; ++v) {
#pragma unroll
        for (int z = 0; z < 16; ++z) x[v][z] = 0.0f;
        if (r0 + v * step < unit.cnt) {
          load8(unit.row(a, r0 + v * step) + l.c0, x[v]);
          load8(unit.row(a, r0 + v * step) + l.c1, x[v] + 8);
        }
      }
#pragma unroll
      for (int v = 0; v < kVecs; ++v) {
        const bool here = r0 + v * step < unit.cnt, at = a.dim == 0 || (pos[v] >= 0 && pos[v] < a.max_pos);
        bad |= here && !at;
        in |= (here && at ? 1u : 0u) << v;
      }
      if (bad && j == 0) status_or(a.d_status, CKV_STATUS_BAD_INDEX);
      if (!unit.second) {
        if (a.weight != nullptr) {
          float w[16];
          load8(a.weight + l.c0, w);
          load8(a.weight + l.c1, w + 8);
#pragma unroll
          for (int v = 0; v < kVecs; ++v) normalise<kD>(a, w, x[v]);
        }
        if (l.turns) {
#pragma unroll
          for (int v = 0; v < kVecs; ++v) {
            if (!(in >> v & 1)) continue;
            float cs[16];
            angles(a, l, static_cast<uint32_t>(pos[v]), cs);
            rotate(a, cs, x[v]);
          }
        }
      }
#pragma unroll
      for (int v = 0; v < kVecs; ++v)
        if (in >> v & 1) m = largest(m, x[v]);
      if (m == INFINITY) m = largest_finite(x, in);
      const float now = fmaxf(pow2f(q8_need_exp(cta_max(m, s_max))), old), inv = 1.0f / now;
      uint8_t* entries = unit.entries(a);
#pragma unroll
      for (int v = 0; v < kVecs; ++v) {
        if (!(in >> v & 1)) continue;
        put16(entries + static_cast<size_t>(unit.off + r0 + v * step) * kD, l, x[v], inv);
        if (j == 0) unit.reset(a, r0 + v * step);
      }
      if (unit.off && now > old) follow<kD>(entries, unit.off, old * inv, threadIdx.x, blockDim.x);
      __syncthreads();  // every thread has read s_max
      if (threadIdx.x == 0) *unit.scale(a) = now;
    }
  }
}

// Units whose rows do not fit the registers (128 entries of 512 channels): a row is read again for its codes, which comes from L2.
// 37545 latent rows with a norm, 67 MB, take 45 us here, 36 in blocks of 64 entries (the kernel above), 35 in blocks of 32 and 33 in blocks of 16.
constexpr int kWideThreads = 512;

template <typename TIn, int kD>
__global__ __launch_bounds__(kWideThreads, 2) void q8_rope_store_wide_kernel(const RopeStoreArgs a) {
  constexpr uint32_t kLanes = kD / 16, kStep = kWideThreads / kLanes;
  __shared__ float s_max[16];
  pdl_wait();
  pdl_release();
  const uint32_t n = count_or_capacity(a.d_counts, 0, a.capacity), units = a.c.heads * a.sides;
  const uint32_t j = threadIdx.x % kLanes, r0 = threadIdx.x / kLanes;
  const Lane l = lane_of(a, j);
  for (uint32_t i = blockIdx.x; i < n; i += gridDim.x) {
    const uint4 rec = __ldg(reinterpret_cast<const uint4*>(a.plan + i));
    for (uint32_t u = blockIdx.y; u < units; u += gridDim.y) {
      const Unit<TIn, kD> unit(a, rec, u);
      if (!unit.ok) break;
      const float old = unit.off ? *unit.scale(a) : 0.0f;
      // row r's values; false where it is not stored (all threads of a warp call it)
      auto values = [&](uint32_t r, float (&x)[16]) -> bool {
        const bool here = r < unit.cnt;
        const int64_t pos = here && a.dim ? __ldg(a.positions + unit.row0 + r) : 0;
        const bool in = here && (a.dim == 0 || (pos >= 0 && pos < a.max_pos));
        if (in) {
          const TIn* src = unit.row(a, r);
          load8(src + l.c0, x);
          load8(src + l.c1, x + 8);
        } else {
#pragma unroll
          for (int z = 0; z < 16; ++z) x[z] = 0.0f;
        }
        if (!unit.second) {
          if (a.weight != nullptr) {
            float w[16];
            load8(a.weight + l.c0, w);
            load8(a.weight + l.c1, w + 8);
            normalise<kD>(a, w, x);
          }
          if (l.turns && in) {
            float cs[16];
            angles(a, l, static_cast<uint32_t>(pos), cs);
            rotate(a, cs, x);
          }
        }
        return in;
      };
      float m = 0.0f;
      bool bad = false;
#pragma unroll 2
      for (uint32_t r = r0; r - r0 < unit.cnt; r += kStep) {
        float x[16];
        bad |= !values(r, x) && r < unit.cnt;
#pragma unroll
        for (int z = 0; z < 16; ++z) m = fabsf(x[z]) < INFINITY ? fmaxf(m, fabsf(x[z])) : m;
      }
      if (bad && j == 0) status_or(a.d_status, CKV_STATUS_BAD_INDEX);
      const float now = fmaxf(pow2f(q8_need_exp(cta_max(m, s_max))), old), inv = 1.0f / now;
      uint8_t* entries = unit.entries(a);
#pragma unroll 2
      for (uint32_t r = r0; r - r0 < unit.cnt; r += kStep) {
        float x[16];
        if (!values(r, x)) continue;
        put16(entries + static_cast<size_t>(unit.off + r) * kD, l, x, inv);
        if (j == 0) unit.reset(a, r);
      }
      if (unit.off && now > old) follow<kD>(entries, unit.off, old * inv, threadIdx.x, kWideThreads);
      __syncthreads();  // every thread has read s_max
      if (threadIdx.x == 0) *unit.scale(a) = now;
    }
  }
}

template <typename TIn, int kD>
int launch(const RopeStoreArgs& a, cudaStream_t s) {
  const uint32_t vecs = a.c.block_tokens * (kD / 16), units = a.c.heads * a.sides;
  const uint32_t records = std::min<uint32_t>(a.capacity, 65536u);
  // As many of a record's units to a CTA as leave every SM two dozen
  const uint64_t most = std::max<uint64_t>(1, static_cast<uint64_t>(a.capacity) * units / (24ull * sm_count()));
  uint32_t parts = static_cast<uint32_t>((units + most - 1) / most);
  const uint32_t per = (units + parts - 1) / parts;
  parts = (units + per - 1) / per;
  const dim3 grid(records * parts);
  // Threads that a barrier joins, against registers: 16 requests of up to 4096 new rows, eight kv heads, K and V, us (whole call; each size of
  // blocks with lengths of its own, so that only figures of one size compare): blocks of 32
  // entries of 128 channels 60 with two vectors a thread and five CTAs of 128 an SM, 61 with four vectors and 64 threads, 68 with one and 256; 64
  // entries 77 with four vectors and three CTAs of 128, 85 to 89 with two vectors and two or three CTAs of 256, 101 with one and 512; 16 entries
  // of 64 channels 27.6 with 16 CTAs of 32 an SM and 31 with 20.  In fp32 five CTAs spill: 32 entries 81 with four and 90 with five.
  if (vecs <= 64) return launch_pdl(q8_rope_store_kernel<TIn, kD, 2, 32, 16>, grid, dim3(32), 0, s, a, per, parts);
  if (vecs <= 128) return launch_pdl(q8_rope_store_kernel<TIn, kD, 2, 64, 8>, grid, dim3(64), 0, s, a, per, parts);
  if (vecs <= 256) return launch_pdl(q8_rope_store_kernel<TIn, kD, 2, 128, sizeof(TIn) == 2 ? 5 : 4>, grid, dim3(128), 0, s, a, per, parts);
  if (vecs <= 512) return launch_pdl(q8_rope_store_kernel<TIn, kD, 4, 128, 3>, grid, dim3(128), 0, s, a, per, parts);
  if (vecs <= 2048) return launch_pdl(q8_rope_store_hold_kernel<TIn, kD>, dim3(records, units), dim3(vecs / 4), 0, s, a);
  if constexpr (kD == 512) return launch_pdl(q8_rope_store_wide_kernel<TIn, kD>, dim3(records, units), dim3(kWideThreads), 0, s, a);
  return CKV_ERR_SIZE;  // not reached
}

template <typename TIn>
int launch_for(const RopeStoreArgs& a, cudaStream_t s) {
  switch (a.c.head_dim) {
    case 64: return launch<TIn, 64>(a, s);
    case 128: return launch<TIn, 128>(a, s);
    case 256: return launch<TIn, 256>(a, s);
    default: return launch<TIn, 512>(a, s);
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
  return in_dtype == CKV_BF16 ? launch_for<__nv_bfloat16>(a, s) : launch_for<float>(a, s);
}

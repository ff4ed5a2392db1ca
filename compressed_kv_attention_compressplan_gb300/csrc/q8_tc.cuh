// q8_tc.cuh -- what the tensor-core attention kernels over the 8-bit cache
// share: bounded waits between their roles, and the warps that turn e4m3
// entries into fp16 operands.
#pragma once

#include "async_copy.cuh"
#include "q8_plan.cuh"
#include "tcgen05.cuh"

namespace ckv {

constexpr int kEntries = 128;                // entries of a tile
constexpr uint32_t kSlice = kEntries * 128;  // bytes of 64 channels of a tile in fp16

// A wait that, once it has run out, lets the rest of the loop run without waiting: every barrier is
// still reached, the kernel ends, and the status says so.  The limit is counted in SM clocks, two to a
// nanosecond (about the highest rate, so a slower clock only waits longer).  A wait that is over before it
// starts still takes some 130 cycles, and one that hands over between two warps as many (262 for a round trip), so a tile's
// waits are few.
struct Waiter {
  long long limit;
  bool live;
  // one thread's wait
  template <bool kShort>
  __device__ __forceinline__ bool passed(uint64_t* barrier, uint32_t parity) {
    const uint32_t bar = smem_addr(barrier);
    bool done = kShort ? mbar_test_wait(bar, parity) : mbar_try_wait(bar, parity);
    if (!done) {
      const long long t0 = clock64();
      do {
        done = kShort ? mbar_test_wait(bar, parity) : mbar_try_wait(bar, parity);
      } while (!done && clock64() - t0 <= limit);
    }
    return done;
  }
  // a warp's: its lanes decide together
  template <bool kShort>
  __device__ __forceinline__ void wait(uint64_t* barrier, uint32_t parity) {
    if (live) live = __all_sync(0xFFFFFFFFu, passed<kShort>(barrier, parity));
  }
  // one thread's that acts alone
  template <bool kShort>
  __device__ __forceinline__ void wait_alone(uint64_t* barrier, uint32_t parity) {
    if (live) live = passed<kShort>(barrier, parity);
  }
};

// Takes the NaNs out of 16 channels of entry e: see the split kernel.  Out of line: it runs for next to no tile.
static __device__ __noinline__ uint4 without_nans(uint4 x, int e, int* nan, int step, int* any) {
  uint32_t* y = reinterpret_cast<uint32_t*>(&x);
  for (int z = 0; z < 4; ++z) {
    const uint32_t bad = q8_nan_bytes(y[z]);
    if (bad) {
      for (int b = 0; b < 4; ++b)
        if (bad >> (8 * b) & 1) atomicMin(nan + step * (4 * z + b), e);
      *any = 1;
      y[z] &= ~bad;
    }
  }
  return x;
}

// The scales of a tile's eight runs of 16 entries (a run lies in one block), for kernels whose threads see all
// entries of a tile, by a warp of its own: {scale log2(e) k_scale, log2(v_scale), 1 / v_scale} where the softmax reads
// them.  Lane r % 8 has run r, its block number two tiles ahead and its scales one ahead.  A run that does not
// exist gets log2 = -infinity, i.e. no weight.  The warp goes with the converting ones, so it is never three tiles ahead of the
// softmax, and four tiles' worth are kept.
template <typename C, bool kShort, typename Sh>
__device__ __forceinline__ void scale_tiles(const AttnArgs& a, const Q8Item& item, Sh& sh, Waiter& w, uint32_t h,
                                            const int32_t* table, uint32_t n_tiles, uint32_t tiles_before) {
  const int lane = threadIdx.x & 31, run = lane & 7;
  const uint32_t t_shift = __ffs(a.c.block_tokens) - 1, last = item.kv_end > 0 ? item.kv_end - 1 : 0;
  const float* v_scale = a.c.v != nullptr ? a.c.v_scale : a.c.k_scale;
  int32_t blk;
  float ks, vs;
  bool ok;
  auto ask = [&](uint32_t tile) { blk = ld_ahead(table + (min(item.kv_begin + tile * kEntries + run * 16, last) >> t_shift)); };
  auto load = [&]() {
    ok = static_cast<uint32_t>(blk) < a.c.num_blocks;
    const size_t at = static_cast<size_t>(ok ? blk : 0) * a.c.heads + h;
    ks = ld_ahead(a.c.k_scale + at);
    vs = ld_ahead(v_scale + at);
  };
  ask(0);
  load();
  ask(1);
  for (uint32_t j = 0; j < n_tiles; ++j) {
    const uint32_t g = tiles_before + j, st = g % C::kStages, use = g / C::kStages, slot = g & 3;
    const float f = ok ? ks * a.scale_log2 : 1.0f, lv = ok ? __log2f(vs) : -INFINITY, iv = ok ? __fdiv_rn(1.0f, vs) : 0.0f;
    load();
    ask(j + 2);
    w.template wait<kShort>(&sh.k_free[st], (use & 1) ^ 1);
    if (lane < 8) {
      sh.f[slot][run] = f;
      sh.lv[slot][run] = lv;
      sh.iv[slot][run] = iv;
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_addr(&sh.k_full[st]));
  }
}

// The converting warps' work for one item.  C: kSlices slices of 64 channels, kStages stages, kLoads 16-byte loads of
// a thread per slice, kUnits slices of a tile (K's, then V's).
template <typename C, bool kShort, typename Sh>
__device__ __forceinline__ void convert_tiles(const AttnArgs& a, const Q8Item& item, Sh& sh, Waiter& w, int cw, uint32_t h,
                                              const int32_t* table, uint32_t n_tiles, uint32_t tiles_before,
                                              uint32_t vis_min, uint32_t k_at, uint32_t v_at) {
  // ---- e4m3 -> fp16 operands.  Lane l takes 16 channels, chunk l % 4 of a slice, of entries l / 4 + 8 * ...: the
  // eight lanes of a store's phase take two entries, whose chunks the swizzle puts in different banks.
  const int lane = threadIdx.x & 31, q = lane & 3;
  const uint32_t H = a.c.heads, T = a.c.block_tokens, t_shift = __ffs(T) - 1;
  const uint32_t last = item.kv_end > 0 ? item.kv_end - 1 : 0;
  constexpr bool kShared = C::kLatent;
  constexpr int kD = 64 * C::kSlices;
  const uint32_t tok = cw * 8 + (lane >> 2);  // load i: entry tok + i * (8 * kConvWarps)
  const uint32_t st0 = tok * 128 + (((2 * q) ^ (tok & 7)) << 4), st1 = tok * 128 + (((2 * q + 1) ^ (tok & 7)) << 4);
  const uint8_t* src[C::kLoads];  // the K addresses of a tile's entries
  uint32_t here = 0;              // bit i: load i's entry exists
  bool bad = false;
  // Block numbers are asked for a tile before the addresses are made from them, at places that always exist, so
  // that no load here waits for another.
  int32_t blk[C::kLoads];
  auto ask = [&](uint32_t tile) {
#pragma unroll
    for (int i = 0; i < C::kLoads; ++i) {
      const uint32_t e = item.kv_begin + tile * kEntries + tok + i * (8 * C::kConvWarps);
      blk[i] = ld_ahead(table + (min(e, last) >> t_shift));
    }
  };
  auto locate = [&](uint32_t tile, const uint8_t*(&o)[C::kLoads]) -> uint32_t {
    uint32_t mask = 0;
#pragma unroll
    for (int i = 0; i < C::kLoads; ++i) {
      const uint32_t e = item.kv_begin + tile * kEntries + tok + i * (8 * C::kConvWarps);
      const bool in = tile < n_tiles && e < item.kv_end;
      const bool ok = static_cast<uint32_t>(blk[i]) < a.c.num_blocks;  // negative ones are large
      o[i] = a.c.k + (((static_cast<size_t>(ok ? blk[i] : 0) * H + h) << t_shift) + (e & (T - 1))) * kD + q * 16;
      mask |= (in && ok ? 1u : 0u) << i;
      bad |= in && !ok;
    }
    return mask;
  };
  const ptrdiff_t v_off = kShared ? 0 : a.c.v - a.c.k;
  uint4 buf[C::kUnits][C::kLoads];  // a tile ahead of what is stored
  auto load = [&](uint4(&d)[C::kLoads], int unit, const uint8_t* const(&o)[C::kLoads], uint32_t mask) {
    const ptrdiff_t at = unit < C::kSlices ? unit * 64 : v_off + (unit - C::kSlices) * 64;
#pragma unroll
    for (int i = 0; i < C::kLoads; ++i) d[i] = ld_stream16_if(o[i] + at, mask >> i & 1);
  };
  ask(0);
  here = locate(0, src);
  ask(1);
#pragma unroll
  for (int u = 0; u < C::kUnits; ++u) load(buf[u], u, src, here);
  for (uint32_t j = 0; j < n_tiles; ++j) {
    const uint32_t g = tiles_before + j, st = g % C::kStages, use = g / C::kStages;
    const uint32_t e0 = item.kv_begin + j * kEntries;
    const bool edge = e0 + kEntries > vis_min;
#pragma unroll
    for (int u = 0; u < C::kUnits; ++u) {
      const bool is_v = u >= C::kSlices;
      const int s = is_v ? u - C::kSlices : u;
      if (s == 0) w.template wait<kShort>(is_v ? &sh.v_free[st] : &sh.k_free[st], (use & 1) ^ 1);
      if ((is_v || kShared) && edge) {
#pragma unroll
        for (int i = 0; i < C::kLoads; ++i)
          buf[u][i] = without_nans(buf[u][i], e0 + tok + i * (8 * C::kConvWarps),
                                   kShared ? sh.nan : sh.nan + s * 64 + q * 16, kShared ? 0 : 1, &sh.any_nan);
      }
      const uint32_t dst = (is_v ? v_at : k_at) + (st * C::kSlices + s) * kSlice;
#pragma unroll
      for (int i = 0; i < C::kLoads; ++i) {
        const uint4 y = buf[u][i];
        asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(dst + st0 + i * (8 * C::kConvWarps) * 128),
                     "r"(q8_lo_f16x2(y.x)), "r"(q8_hi_f16x2(y.x)), "r"(q8_lo_f16x2(y.y)), "r"(q8_hi_f16x2(y.y))
                     : "memory");
        asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(dst + st1 + i * (8 * C::kConvWarps) * 128),
                     "r"(q8_lo_f16x2(y.z)), "r"(q8_hi_f16x2(y.z)), "r"(q8_lo_f16x2(y.w)), "r"(q8_hi_f16x2(y.w))
                     : "memory");
      }
      if (u == 0) {
        // the next tile's addresses, from block numbers that were asked for before the entries just stored
        here = locate(j + 1, src);
        ask(j + 2);
      }
      if (s == C::kSlices - 1) {
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(is_v ? &sh.v_full[st] : &sh.k_full[st]));
      }
      load(buf[u], u, src, here);  // the next tile's
    }
  }
  if (bad) status_or(a.d_status, CKV_STATUS_BAD_INDEX);
}

}  // namespace ckv

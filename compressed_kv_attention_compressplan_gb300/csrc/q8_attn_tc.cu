// q8_attn_tc.cu -- attention over the 8-bit paged cache on the 5th-generation
// tensor cores from 256 channels on: decode where many heads share one latent
// cache, and prefill chunks.  The mathematics is the split kernel's.
//
// Transposed 8-bit products.  A tile is 128 entries, the M of both products, and its
// e4m3 values are the operands as they lie in the cache -- nothing is converted:
//     S^T [128 entries x 64 rows] = K8 Q^T,   O^T [128 channels x 64 rows] += V8^T W^T.
// What is wider than 8 bits is a sum of 8-bit terms.  A query row is scaled by a power of
// two that puts its largest value in [2^7, 2^8) and is e4m3 + e4m3: bf16's 8 bits are 4
// and 4, so the two are exact down to 2^-9 of that value, and under it the error is
// at most 2^-17 of it; both are columns of one product (N = 128), whose halves are added.
// A weight (at most 2^15, see kTop) is e5m2 + e5m2 + e5m2, each the nearest
// to what the ones before leave: off by 2^-9 of it in all, or, where a weight is so small that
// the terms reach e5m2's last place, by 2^-17, 2^-29 of the row's largest.
//
// The accumulators of 512 channels by 64 rows take 256 columns of tensor memory, so the
// whole width of a latent entry fits beside two buffers of scores, and its entries are read
// once.  With entries on the lanes a thread owns one entry: the entry's scales are two
// registers of its own, row sums stay in registers until the end, and no score crosses
// lanes but in the rare step that raises a row's reference (one vote a tile asks for it).
// The weights go through shared memory as they stand: an entry's row of 64 of them is the
// swizzled row that the second product reads.
//
// Roles.  Four warps copy entries into the operands' swizzled layout, 128 channels at a time, as
// the second product hands them back; one thread issues the products; groups of four warps
// take 16 rows each through the softmax.
//
// Bound.  512 channels: a tile is 64 KB from memory, 2.8 k cycles of an SM's share of it;
// shared memory feeds the products 128 KB and 288 KB, 3.3 k cycles.  Measured: 5.0 k a tile and 27 k an item (its 64
// rows of queries split into terms, the first entries, the last product and 128 KB of partial results); the latent case, 140 MB and
// 33.6 GF, takes 67 us here (the plan 6.5 before it, the join 11 after it) and 81 in all.  A tile's chain with two stages of entries -- copied 3.5 k, scores, weights 3 k, second
// product 2.3 k -- is what bounds it; a third stage does not fit.  Entries turned into fp16 for fp16 products took 126 us instead of
// 109 at that point: twice the shared-memory traffic.
#include <algorithm>

#include "q8_tc.cuh"

namespace ckv {
namespace {

constexpr uint32_t kSlice8 = kEntries * 128;  // bytes of 128 channels of a tile
constexpr uint32_t kTerm = kEntries * 64;     // bytes of one term of a tile's weights
// A row's reference is raised to kRest under its maximum when an exponent passes it by kTop.  e5m2 ends at 57344 above and at 2^-16
// below, so a row's largest weight stands close under the top: what is left of a weight under 2^-16 is lost, and that is
// 2^-17, 2^-29 of a largest weight of 2^12.  Latent decode and chunks of 512 queries over 8192 entries of 512 and of 256 channels: 79, 315 and
// 286 us at 14 and 6, where a weight lost up to 2^-23 of the largest; 81, 320 and 286 at 15 and 12; 82, 327 and 287 at 15.5 and 13.
constexpr float kTop = 15.0f, kRest = 12.0f;

template <int kD, bool kShared>
struct TcCfg {
  static_assert(kD == 256 || kD == 512, "");
  static constexpr int kRows = 64;
  static constexpr int kSlices = kD / 128;  // also the accumulators, of 128 channels each
  static constexpr int kStages = kD == 512 && !kShared ? 1 : 2;
  static constexpr int kFree = kShared ? kSlices : 1;  // barriers that hand a K stage back
  static constexpr int kGroups = kRows / 16;  // softmax groups of four warps
  static constexpr int kSoftWarps = 4 * kGroups;
  static constexpr int kCopyWarps = 4;  // four more leave a thread 72 registers, which spill into memory that has next to no L1
  static constexpr int kWarps = kSoftWarps + kCopyWarps + 1;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr uint32_t kTile = kSlices * kSlice8;
  static constexpr uint32_t kQBytes = kSlices * kSlice8;  // 64 rows, two terms
  static constexpr uint32_t kKBytes = kStages * kTile;
  static constexpr uint32_t kVBytes = kShared ? 0 : kKBytes;
  static constexpr uint32_t kPBytes = 3 * kTerm;
  static constexpr uint32_t kBytes = kQBytes + kKBytes + kVBytes + kPBytes + 1024;  // and the alignment
  // one CTA to an SM: a second would wait for the first one's tensor memory
  static constexpr uint32_t kSmem = kBytes < 120 * 1024 ? 120 * 1024 : kBytes;
  static constexpr uint32_t kSCol = 2 * kRows;   // columns of a buffer of scores: both terms'
  static constexpr uint32_t kOCol = 2 * kSCol;   // the accumulators
  static constexpr uint32_t kCols = 512;
  static_assert(kOCol + kSlices * kRows <= 512, "");
};

template <int kD, bool kShared>
struct alignas(16) TcShared {
  using C = TcCfg<kD, kShared>;
  uint64_t k_full[C::kStages][C::kSlices], k_free[C::kStages][C::kFree];
  uint64_t v_full[C::kStages][C::kSlices], v_free[C::kStages];
  uint64_t s_full[2], s_free[2], q_full, p_full, pv_done, idle;
  alignas(16) float rf[C::kRows];  // read four at a time
  alignas(16) float neg_m[C::kRows];
  float fac[C::kRows], up[C::kRows];
  int vis[C::kRows];
  int set[C::kRows];  // the row's reference has been set
  size_t out_row[C::kRows];
  float red[4][C::kRows];
  int nan[kShared ? 1 : kD];  // first entry with a NaN (a latent cache: in any channel, else by channel)
  int any_nan;
  uint32_t tmem;
};

// Two fp16 values as the sum of three e5m2 pairs (16 bits each), each the nearest to what is left.
__device__ __forceinline__ void three_terms(uint32_t h, uint32_t (&t)[3]) {
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    uint16_t b;
    asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(b) : "r"(h));
    t[i] = b;
    if (i < 2) {
      const uint32_t back = __byte_perm(b, 0, 0x1404);  // e5m2 is fp16's upper byte
      const __half2 left = __hsub2(*reinterpret_cast<const __half2*>(&h), *reinterpret_cast<const __half2*>(&back));
      h = *reinterpret_cast<const uint32_t*>(&left);
    }
  }
}

__device__ __forceinline__ bool group_any(int id, bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %2, 0;\n\t"
      "bar.red.or.pred q, %1, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(x ? 1u : 0u)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void group_sync(int id) { asm volatile("bar.sync %0, 128;" ::"r"(id) : "memory"); }

template <int kD, bool kShared, bool kShort, bool kLists>
__global__ __launch_bounds__((TcCfg<kD, kShared>::kThreads), 1) void q8_attn_tc_kernel(const AttnArgs a) {
  using C = TcCfg<kD, kShared>;
  constexpr int kN = C::kRows;
  extern __shared__ uint8_t raw[];
  __shared__ TcShared<kD, kShared> sh;
  pdl_wait();
  pdl_release();
  const Q8Header* head = reinterpret_cast<const Q8Header*>(a.plan);
  const uint32_t h = blockIdx.y;
  if (!plan_fits(head, a)) {
    if (blockIdx.x == 0 && h == 0 && threadIdx.x == 0) status_or(a.d_status, CKV_STATUS_BAD_INDEX);
    return;
  }
  if (blockIdx.x >= head->ctas) return;
  const uint32_t* first = reinterpret_cast<const uint32_t*>(a.plan + a.g.off_first);
  const Q8Item* items = reinterpret_cast<const Q8Item*>(a.plan + a.g.off_items);
  const uint32_t item0 = first[blockIdx.x], item1 = min(first[blockIdx.x + 1], a.g.cap_items);

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t G = a.g.group, H = a.c.heads, T = a.c.block_tokens, t_shift = __ffs(T) - 1;
  const uint32_t base = (smem_addr(raw) + 1023) & ~1023u;
  const uint32_t q_at = base, k_at = q_at + C::kQBytes, v_at = kShared ? k_at : k_at + C::kKBytes;
  const uint32_t p_at = k_at + C::kKBytes + C::kVBytes;
  const bool copy = warp >= C::kSoftWarps && warp < C::kSoftWarps + C::kCopyWarps;
  const bool soft = warp < C::kSoftWarps;

  if (warp == C::kWarps - 1) tmem_alloc(smem_addr(&sh.tmem), C::kCols);
  if (tid == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      for (int x = 0; x < C::kSlices; ++x) {
        mbar_init(smem_addr(&sh.k_full[s][x]), 32 * C::kCopyWarps);
        mbar_init(smem_addr(&sh.v_full[s][x]), 32 * C::kCopyWarps);
      }
      for (int x = 0; x < C::kFree; ++x) mbar_init(smem_addr(&sh.k_free[s][x]), 1);
      mbar_init(smem_addr(&sh.v_free[s]), 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(smem_addr(&sh.s_full[s]), 1);
      mbar_init(smem_addr(&sh.s_free[s]), C::kSoftWarps);
    }
    mbar_init(smem_addr(&sh.q_full), C::kSoftWarps);
    mbar_init(smem_addr(&sh.p_full), C::kSoftWarps);
    mbar_init(smem_addr(&sh.pv_done), 1);
    mbar_init(smem_addr(&sh.idle), 1);
    fence_mbar_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  Waiter w{static_cast<long long>(a.wait_ns) * 2, true};
  uint32_t tiles_before = 0;  // tiles of earlier items: the barriers' phases go on
  uint32_t items_before = 0;

  for (uint32_t it = item0; it < item1; ++it) {
    const Q8Item item = item_for<kLists, true>(items + it, a, h);
    if (!item_fits(item, a)) {
      if (tid == 0) status_or(a.d_status, CKV_STATUS_BAD_INDEX);
      continue;
    }
    const uint32_t rows = min(static_cast<uint32_t>(kN), item.q_len * G - item.row0);
    const int32_t* table = table_for<kLists>(a, item, h);
    const uint32_t n_tiles =
        item.kv_end > item.kv_begin ? (item.kv_end - item.kv_begin + kEntries - 1) / kEntries : 0;
    const uint32_t last = item.kv_end > 0 ? item.kv_end - 1 : 0;
    const uint32_t vis_min = min(item.kv_end, static_cast<uint32_t>(q8_visible(item.kv_len, item.q_len - 1 - item.row0 / G,
                                                                             item.phase, a.ratio)));
    if (copy) {
      // ---- entries into the operands, 128 channels (a slice) at a time: lane l takes 16-byte chunk l % 8 of four entries
      // at once.  A chunk arrives at its barrier when it has landed.
      constexpr int kStride = C::kCopyWarps * 4, kSteps = kEntries / kStride;
      const int cw = warp - C::kSoftWarps, cc = lane & 7;
      const uint32_t entry0 = cw * 4 + (lane >> 3);  // entry of step i: entry0 + kStride i
      bool bad = false;
      for (int c = tid - 32 * C::kSoftWarps; c < (kShared ? 1 : kD); c += 32 * C::kCopyWarps) sh.nan[c] = 0x7FFFFFFF;
      if (cw == 0 && lane == 0) sh.any_nan = 0;
      asm volatile("bar.sync 15, %0;" ::"n"(32 * C::kCopyWarps) : "memory");
      // lane r < 8 keeps the block number of run r (16 entries), asked for a tile ahead
      auto ask = [&](uint32_t tile) {
        return __ldg(table + (min(item.kv_begin + tile * kEntries + (lane & 7) * 16, last) >> t_shift));
      };
      int32_t runs = ask(0), runs_next = ask(1), runs_after = ask(2);
      // a tile's runs, each one piece of memory, are asked into L2 two tiles before they are copied
      auto prefetch = [&](uint32_t tile, int32_t b) {
        const uint32_t e = item.kv_begin + tile * kEntries + lane * 16;
        if (cw == 0 && lane < 8 && tile < n_tiles && e < item.kv_end && static_cast<uint32_t>(b) < a.c.num_blocks) {
          const size_t at = (((static_cast<size_t>(b) * H + h) << t_shift) + (e & (T - 1))) * kD;
          bulk_prefetch_l2(a.c.k + at, 16 * kD);
          if (!kShared) bulk_prefetch_l2(a.c.v + at, 16 * kD);
        }
      };
      prefetch(0, runs);
      prefetch(1, runs_next);
      for (uint32_t j = 0; j < n_tiles; ++j) {
        const uint32_t g = tiles_before + j, st = g % C::kStages, use = g / C::kStages;
        const uint32_t e0 = item.kv_begin + j * kEntries;
        const bool edge = e0 + kEntries > vis_min;
        const int32_t now = runs;
        prefetch(j + 2, runs_after);
        runs = runs_next;
        runs_next = runs_after;
        runs_after = ask(j + 3);
        size_t off[kSteps];
        uint32_t in = 0;  // bit i: step i's entry exists
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
          const uint32_t t = entry0 + kStride * i, e = e0 + t;
          const int32_t b = __shfl_sync(0xFFFFFFFFu, now, t >> 4);
          const bool valid = static_cast<uint32_t>(b) < a.c.num_blocks;
          off[i] = (((static_cast<size_t>(valid ? b : 0) * H + h) << t_shift) + (e & (T - 1))) * kD + cc * 16;
          in |= (valid && e < item.kv_end ? 1u : 0u) << i;
          bad |= !valid && e < item.kv_end;
        }
        const uint32_t put = entry0 * 128 + ((cc ^ (entry0 & 7)) << 4);  // kStride entries on, the swizzle is the same
#pragma unroll 1
        for (int u = 0; u < C::kSlices * (kShared ? 1 : 2); ++u) {
          const bool side = u >= C::kSlices;
          const int s = side ? u - C::kSlices : u;
          const uint8_t* pool = (side ? a.c.v : a.c.k) + s * 128;
          const uint32_t to = (side ? v_at : k_at) + st * C::kTile + s * kSlice8 + put;
          uint64_t* full = side ? &sh.v_full[st][s] : &sh.k_full[st][s];
          if (side) {
            if (s == 0) w.wait<kShort>(&sh.v_free[st], (use & 1) ^ 1);
          } else if (kShared || s == 0) {
            w.wait<kShort>(&sh.k_free[st][kShared ? s : 0], (use & 1) ^ 1);
          }
#pragma unroll
          for (int i = 0; i < kSteps; ++i) cp_async16(to + i * (kStride * 128), pool + off[i], in >> i & 1 ? 16u : 0u);  // others: zeros
          if ((side || kShared) && edge) {
            // some rows do not see some of these entries: their values' NaNs are taken out (see the split kernel)
            cp_async_commit();
            cp_async_wait<0>();
#pragma unroll 1
            for (int i = 0; i < kSteps; ++i) {
              const uint32_t at = to + i * (kStride * 128);
              const uint4 x = lds16(at);
              if (q8_nan_bytes(x.x) | q8_nan_bytes(x.y) | q8_nan_bytes(x.z) | q8_nan_bytes(x.w)) {
                const uint4 y = without_nans(x, e0 + entry0 + kStride * i, kShared ? sh.nan : sh.nan + s * 128 + cc * 16,
                                             kShared ? 0 : 1, &sh.any_nan);
                asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(y.x), "r"(y.y), "r"(y.z), "r"(y.w)
                             : "memory");
              }
            }
            mbar_arrive(smem_addr(full));
          } else {
            cp_async_arrive(smem_addr(full));
          }
        }
      }
      // none of these copies may land after the CTA is gone
      cp_async_commit();
      cp_async_wait<0>();
      if (bad) status_or(a.d_status, CKV_STATUS_BAD_INDEX);
    } else if (soft) {
      // ---- the rows: query operand, scaling, visibility; a warp takes four rows, and loads two at a time
      constexpr int kPer = kD / 32;  // consecutive channels of a lane
#pragma unroll 1
      for (int n0 = warp; n0 < kN; n0 += 2 * C::kSoftWarps) {
        uint4 x[2][kPer / 8];
        size_t row[2];
        uint32_t query[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const uint32_t n = n0 + r * C::kSoftWarps;
          const bool in = n < rows;
          const uint32_t rho = item.row0 + (in ? n : 0), hg = rho % G;
          query[r] = rho / G;
          row[r] = static_cast<size_t>(item.q_start + query[r]) * a.n_heads + h * G + hg;
#pragma unroll
          for (int e = 0; e < kPer / 8; ++e)
            x[r][e] = in ? ld_cached16(a.q + row[r] * kD + lane * kPer + 8 * e) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int n = n0 + r * C::kSoftWarps;
          float m = 0.0f;
#pragma unroll
          for (int e = 0; e < kPer / 8; ++e) {
#pragma unroll
            for (int z = 0; z < 8; ++z) m = fmaxf(m, fabsf(unpack<__nv_bfloat16>(x[r][e], z)));
          }
#pragma unroll
          for (int s = 16; s > 0; s >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, s));
          const int ex = min(126, 7 - (static_cast<int>(__float_as_uint(m) >> 23) - 127));
          // e4m3 has no infinity: a row with one is NaN, as its scores' softmax is
          const float up = m == INFINITY ? __int_as_float(0x7FFFFFFF) : pow2f(ex);
          // eight channels at a time; term t of the row is row n + 64 t of the operand
#pragma unroll
          for (int e = 0; e < kPer / 8; ++e) {
            float v[8];
#pragma unroll
            for (int z = 0; z < 8; ++z) v[z] = unpack<__nv_bfloat16>(x[r][e], z) * up;
            const uint32_t c = lane * kPer + 8 * e;
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              const uint32_t y[2] = {q8_pack4(v[0], v[1], v[2], v[3]), q8_pack4(v[4], v[5], v[6], v[7])};
              const uint32_t to = n + 64 * t;
              asm volatile("st.shared.v2.u32 [%0], {%1,%2};" ::"r"(q_at + (c >> 7) * kSlice8 + to * 128 +
                                                                   ((((c & 127) >> 4) ^ (to & 7)) << 4) + (c & 15)),
                           "r"(y[0]), "r"(y[1])
                           : "memory");
              if (t == 0) {
#pragma unroll
                for (int z = 0; z < 2; ++z) {
                  const float2 lo = f16x2_to_f32(q8_lo_f16x2(y[z])), hi = f16x2_to_f32(q8_hi_f16x2(y[z]));
                  v[4 * z] -= lo.x;
                  v[4 * z + 1] -= lo.y;
                  v[4 * z + 2] -= hi.x;
                  v[4 * z + 3] -= hi.y;
                }
              }
            }
          }
          if (lane == 0) {
            sh.rf[n] = pow2f(-ex) * a.scale_log2;
            sh.neg_m[n] = 0.0f;
            sh.set[n] = 0;
            sh.vis[n] = static_cast<uint32_t>(n) < rows
                            ? static_cast<int>(q8_visible(item.kv_len, item.q_len - 1 - query[r], item.phase, a.ratio))
                            : 0x7FFFFFFF;
            sh.out_row[n] = row[r];
          }
        }
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&sh.q_full));
      asm volatile("bar.sync 14, 512;" ::: "memory");  // every group reads rows that other warps prepared

      // ---- softmax of 16 rows (columns of S^T); this thread's entry is its lane
      const int group = warp >> 2, quarter = warp & 3, bar = 1 + group;
      const int c0 = group * 16, entry = quarter * 32 + lane;
      const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
      float l[16];
#pragma unroll
      for (int c = 0; c < 16; ++c) l[c] = 0.0f;
      // the entry's block is asked for a tile ahead of its scales, and those a tile ahead of their use
      auto block_of = [&](uint32_t tile) { return __ldg(table + (min(item.kv_begin + tile * kEntries + entry, last) >> t_shift)); };
      auto valid = [&](int32_t b) { return static_cast<uint32_t>(b) < a.c.num_blocks; };
      auto scale_of = [&](const float* s, int32_t b) { return __ldg(s + static_cast<size_t>(valid(b) ? b : 0) * H + h); };
      const float* vs = kShared ? a.c.k_scale : a.c.v_scale;
      bool missed = false;
      int32_t b_now = block_of(0), b_next = block_of(1);
      float ks_now = scale_of(a.c.k_scale, b_now), vs_now = scale_of(vs, b_now);
      for (uint32_t j = 0; j < n_tiles; ++j) {
        const uint32_t g = tiles_before + j, sb = g & 1;
        const float kf = ks_now, lv = __log2f(vs_now), iv = __fdiv_rn(1.0f, vs_now);
        const bool exists = valid(b_now) && item.kv_begin + j * kEntries + entry < item.kv_end;
        b_now = b_next;
        ks_now = scale_of(a.c.k_scale, b_now);
        vs_now = scale_of(vs, b_now);
        b_next = block_of(j + 2);
        const uint32_t e0 = item.kv_begin + j * kEntries;

        w.wait<kShort>(&sh.s_full[sb], (g >> 1) & 1);
        tc_fence_after();
        const bool edge = e0 + kEntries > vis_min || !exists;
        // Rows see their entries from the first on, so the first tile sets every reference that will be used, unless
        // entries were missing there.
        const bool unset = j == 0 || missed;
        missed = !exists && e0 + entry < item.kv_end;
        const F2 kf2 = f2_pack(kf, kf), lv2 = f2_pack(lv, lv), iv2 = f2_pack(iv, iv);
        float x[16];  // the exponents t - m
        {
          float y[16];
          tmem_load16(tmem + lanes + sb * C::kSCol + c0, x);
          tmem_load16(tmem + lanes + sb * C::kSCol + kN + c0, y);
#pragma unroll
          for (int c = 0; c < 16; ++c) x[c] += y[c];
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&sh.s_free[sb]));
        float most = -INFINITY;
#pragma unroll
        for (int c = 0; c < 16; c += 4) {
          const float4 rf = *reinterpret_cast<const float4*>(sh.rf + c0 + c);
          const float4 nm = *reinterpret_cast<const float4*>(sh.neg_m + c0 + c);
          const F2 y0 = f2_fma(f2_pack(x[c], x[c + 1]), f2_mul(kf2, f2_pack(rf.x, rf.y)), f2_add(lv2, f2_pack(nm.x, nm.y)));
          const F2 y1 =
              f2_fma(f2_pack(x[c + 2], x[c + 3]), f2_mul(kf2, f2_pack(rf.z, rf.w)), f2_add(lv2, f2_pack(nm.z, nm.w)));
          f2_unpack(y0, x[c], x[c + 1]);
          f2_unpack(y1, x[c + 2], x[c + 3]);
        }
        if (edge) {
          const int e = exists ? static_cast<int>(e0 + entry) : 0x7FFFFFFF;
#pragma unroll
          for (int c = 0; c < 16; ++c)
            if (e >= sh.vis[c0 + c]) x[c] = -INFINITY;
        }
#pragma unroll
        for (int c = 0; c < 16; ++c) most = fmaxf(most, x[c]);
        if (group_any(bar, most > kTop || unset)) {  // raise the rows' references
          float top = -INFINITY;
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            float y = x[c];
#pragma unroll
            for (int s = 16; s > 0; s >>= 1) y = fmaxf(y, __shfl_xor_sync(0xFFFFFFFFu, y, s));
            if (lane == c) top = y;
          }
          if (lane < 16) sh.red[quarter][c0 + lane] = top;
          group_sync(bar);
          if (quarter == 0 && lane < 16) {
            const int c = c0 + lane;
            top = fmaxf(fmaxf(sh.red[0][c], sh.red[1][c]), fmaxf(sh.red[2][c], sh.red[3][c]));
            // a row's first entry sets its reference, wherever that is; later ones only raise it
            const bool fresh = sh.set[c] == 0 && top > -INFINITY;
            const float up = fresh ? top - kRest : fmaxf(0.0f, top - kRest);
            sh.neg_m[c] -= up;
            sh.up[c] = up;
            sh.fac[c] = fresh ? 1.0f : ex2(-up);
            if (fresh) sh.set[c] = 1;
          }
          group_sync(bar);
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            x[c] -= sh.up[c0 + c];
            l[c] *= sh.fac[c0 + c];
          }
          if (j > 0) {
            w.wait<kShort>(&sh.pv_done, (g & 1) ^ 1);
            tc_fence_after();
#pragma unroll 1
            for (int b = 0; b < C::kSlices; ++b) {
              float o[16];
              const uint32_t at = tmem + lanes + C::kOCol + b * kN + c0;
              tmem_load16(at, o);
#pragma unroll
              for (int c = 0; c < 16; ++c) o[c] *= sh.fac[c0 + c];
              tmem_store16(at, o);
            }
            tc_fence_before();
          }
        }
        uint32_t p[3][4];
#pragma unroll
        for (int c = 0; c < 16; c += 4) {
          uint32_t t[2][3];
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const int z = c + 2 * y;
            const float w0 = ex2(x[z]), w1 = ex2(x[z + 1]);
            const F2 sum = f2_fma(f2_pack(w0, w1), iv2, f2_pack(l[z], l[z + 1]));
            f2_unpack(sum, l[z], l[z + 1]);
            three_terms(pack_f16x2(w0, w1), t[y]);
          }
#pragma unroll
          for (int i = 0; i < 3; ++i) p[i][c / 4] = __byte_perm(t[0][i], t[1][i], 0x5410);
        }
        w.wait<kShort>(&sh.pv_done, (g & 1) ^ 1);  // the second product is done with the tile before
        // rows of 64 bytes: 16-byte chunk c of row r sits at chunk c ^ (r / 2 % 4)
#pragma unroll
        for (int i = 0; i < 3; ++i)
          asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(p_at + i * kTerm + entry * 64 +
                                                                     ((group ^ ((entry >> 1) & 3)) << 4)),
                       "r"(p[i][0]), "r"(p[i][1]), "r"(p[i][2]), "r"(p[i][3])
                       : "memory");
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&sh.p_full));
      }
      // ---- the rows' sums, then the output
      {
        float mine = 0.0f;
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          float x = l[c];
#pragma unroll
          for (int s = 16; s > 0; s >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, s);
          if (lane == c) mine = x;
        }
        if (lane < 16) sh.red[quarter][c0 + lane] = mine;
        group_sync(bar);
        if (quarter == 0 && lane < 16) {
          const int c = c0 + lane;
          float sum = (sh.red[0][c] + sh.red[1][c]) + (sh.red[2][c] + sh.red[3][c]);
          // A latent cache's NaN is a NaN score of the rows that see it.  The last tile's scores are in, so its keys' marks are;
          // without tiles nothing orders the read after the clearing.
          if (kShared && n_tiles > 0 && sh.any_nan != 0 && sh.nan[0] < sh.vis[c]) sum = __int_as_float(0x7FFFFFFF);
          sh.fac[c] = sum == 0.0f ? 0.0f : __fdiv_rn(1.0f, sum);
          if (static_cast<uint32_t>(c) < rows) {
            if (item.part >= 0)
              a.part_ml[(static_cast<size_t>(item.part + static_cast<int>(item.chunk)) * H + h) * kN + c] =
                  make_float2(sum == 0.0f ? -3.4e38f : -sh.neg_m[c], sum);
            else if (a.lse != nullptr)
              a.lse[sh.out_row[c]] = sum == 0.0f ? -INFINITY : (__log2f(sum) - sh.neg_m[c]) * 0.69314718055994530942f;
          }
        }
        group_sync(bar);
      }
      if (n_tiles > 0) w.wait<kShort>(&sh.pv_done, (tiles_before + n_tiles - 1) & 1);
      tc_fence_after();
      const bool any_nan = !kShared && n_tiles > 0 && sh.any_nan != 0;  // values may be marked up to their product
#pragma unroll 1
      for (int b = 0; b < C::kSlices; ++b) {
        const int d = b * 128 + entry;  // this lane's channel
        const int nan_at = any_nan ? sh.nan[d] : 0x7FFFFFFF;
        float o[16];
        if (n_tiles > 0) {
          tmem_load16(tmem + lanes + C::kOCol + b * kN + c0, o);
        } else {
#pragma unroll
          for (int c = 0; c < 16; ++c) o[c] = 0.0f;
        }
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          const int n = c0 + c;
          if (static_cast<uint32_t>(n) < rows) {
            float v = nan_at < sh.vis[n] ? __int_as_float(0x7FFFFFFF) : o[c];
            if (item.part >= 0) {
              a.part_o[((static_cast<size_t>(item.part + static_cast<int>(item.chunk)) * H + h) * kN + n) * kD + d] = v;
            } else {
              v *= sh.fac[n];
              if (a.out_f32)
                static_cast<float*>(a.out)[sh.out_row[n] * kD + d] = v;
              else
                static_cast<__nv_bfloat16*>(a.out)[sh.out_row[n] * kD + d] = __float2bfloat16_rn(v);
            }
          }
        }
      }
      tc_fence_before();
    } else if (elect_one()) {
      // ---- the products, by one thread, which also waits for what they need.  The entries were copied by other threads without
      // a fence of theirs, so the fence between their stores and the tensor core's reads stands here.
      auto scores = [&](uint32_t g) {
        const uint32_t st = g % C::kStages, use = g / C::kStages, sb = g & 1;
        w.wait_alone<kShort>(&sh.s_free[sb], ((g >> 1) & 1) ^ 1);
#pragma unroll 1
        for (int s = 0; s < C::kSlices; ++s) {
          w.wait_alone<kShort>(&sh.k_full[st][s], use & 1);
          fence_async_smem();
          tc_fence_after();
          if (w.live) {
            const uint64_t ka = smem_operand(k_at + st * C::kTile + s * kSlice8, 0);
            const uint64_t qb = smem_operand(q_at + s * kSlice8, 0);
#pragma unroll
            for (int x = 0; x < 4; ++x)  // 32 channels, 32 bytes of a row
              tc_mma_8(tmem + sb * C::kSCol, ka + 2 * x, qb + 2 * x, mma_shape(128, 2 * kN, false, false), s > 0 || x > 0);
          }
        }
        if (!kShared) tc_commit(smem_addr(&sh.k_free[st][0]));
        tc_commit(smem_addr(&sh.s_full[sb]));
      };
      auto values = [&](uint32_t g, bool fresh) {
        const uint32_t st = g % C::kStages, use = g / C::kStages;
        w.wait_alone<kShort>(&sh.p_full, g & 1);
        if (!kShared) {
          for (int s = 0; s < C::kSlices; ++s) w.wait_alone<kShort>(&sh.v_full[st][s], use & 1);
        }
        fence_async_smem();
        tc_fence_after();
#pragma unroll
        for (int b = 0; b < C::kSlices; ++b) {
          if (w.live) {
            const uint64_t va = smem_operand(v_at + st * C::kTile + b * kSlice8, 0);
#pragma unroll
            for (int i = 0; i < 3; ++i) {
              const uint64_t pb = smem_operand64(p_at + i * kTerm);
#pragma unroll
              for (int x = 0; x < 4; ++x)  // 32 entries: 32 rows of 128 and of 64 bytes
                tc_mma_8(tmem + C::kOCol + b * kN, va + 256 * x, pb + 128 * x,
                         mma_shape(128, kN, true, true) | kBIsE5m2, !fresh || i > 0 || x > 0);
            }
          }
          if (kShared) tc_commit(smem_addr(&sh.k_free[st][b]));
        }
        if (!kShared) tc_commit(smem_addr(&sh.v_free[st]));
        tc_commit(smem_addr(&sh.pv_done));
      };
      w.wait_alone<kShort>(&sh.q_full, items_before & 1);
      // the second product runs a tile behind the first
      for (uint32_t j = 0; j < n_tiles; ++j) {
        scores(tiles_before + j);
        if (j > 0) values(tiles_before + j - 1, j == 1);
      }
      if (n_tiles > 0) values(tiles_before + n_tiles - 1, n_tiles == 1);
    }
    __syncwarp();
    tiles_before += n_tiles;
    ++items_before;
    __syncthreads();  // the next item's rows take the place of this one's
    tc_fence_after();
  }
  if (warp == C::kWarps - 1) {
    // every product is done before its memory is given back
    if (elect_one()) tc_commit(smem_addr(&sh.idle));
    __syncwarp();
    const bool done = warp_wait_for<false>(smem_addr(&sh.idle), 0, kWaitLimitNs);
    if (!done) w.live = false;
    tmem_free(tmem, C::kCols);
  }
  if (!w.live) status_or(a.d_status, CKV_STATUS_TIMEOUT);
}

template <int kD, bool kShared, bool kLists>
int launch_for(const AttnArgs& a, cudaStream_t s) {
  using C = TcCfg<kD, kShared>;
  auto* kernel = a.wait_ns < kShortWaitNs ? q8_attn_tc_kernel<kD, kShared, true, kLists>
                                          : q8_attn_tc_kernel<kD, kShared, false, kLists>;
  static std::atomic<uint64_t> done[2];
  const int rc = allow_smem(reinterpret_cast<const void*>(kernel), C::kSmem, done[a.wait_ns < kShortWaitNs ? 1 : 0]);
  if (rc) return rc;
  return launch_pdl(kernel, dim3(a.g.ctas, a.c.heads), dim3(C::kThreads), C::kSmem, s, a);
}

template <int kD, bool kShared>
int launch(const AttnArgs& a, cudaStream_t s) {
  return a.lens != nullptr ? launch_for<kD, kShared, true>(a, s) : launch_for<kD, kShared, false>(a, s);
}

}  // namespace

int launch_q8_attn_tc(const AttnArgs& a, cudaStream_t s) {
  const bool shared = a.c.v == nullptr;
  switch (a.c.head_dim) {
    case 256: return shared ? launch<256, true>(a, s) : launch<256, false>(a, s);
    default: return shared ? launch<512, true>(a, s) : launch<512, false>(a, s);
  }
}

}  // namespace ckv

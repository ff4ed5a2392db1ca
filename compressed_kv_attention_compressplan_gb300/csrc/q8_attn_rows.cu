// q8_attn_rows.cu -- attention over the 8-bit paged cache on the 5th-generation
// tensor cores, up to 128 channels: prefill chunks and batches whose requests bring
// many rows.  The mathematics is the split kernel's.
//
// A CTA takes 256 rows as two tiles of 128, M of both products:
//     S [128 rows x 128 entries] = Q K8^T,   O [128 rows x channels] += W V8.
// Two threads own a row, one for each half of a tile's entries, so a row's reference,
// sum and scaling are registers, a tile's entries come in eight runs of 16 that share
// their scales, and all that crosses threads is one vote a tile between two warps (and
// the two maxima when a reference has to rise).  W takes the place of S in tensor memory,
// as the A operand of the second product.  The two row tiles take turns: while one's softmax runs, the
// other's products do.  K and V are turned into fp16 once for both.
//
// Weights are made in one pass under the reference as it stands and held in registers; only when an exponent turns out to
// pass it by 14 is it raised and the pass repeated.
//
// Roles.  Sixteen softmax warps, eight that convert entries, one for the scales, one thread that issues all products and waits for what
// they need.  An item's entries are on their way while its rows are prepared.
//
// Bound.  Per tile of 128 entries and 256 rows at 128 channels: products 2.0 k cycles (64 for each of
// 32, measured alone and beside busy warps), exponentials 1.0 k (32 a cycle), shared memory 256 KB or 2.0 k.  Measured: 3.6 to 4.5 k a
// tile and 17 k an item, 762 GF in 0.77 ms (53 % of the measured bf16 rate): what a tile waits for is the chain of its
// row tile -- weights 2 k, the second product and the next scores 1.3 k, handing over four times -- which the
// other row tile only half covers, since tensor memory has no room for a second buffer of scores.
#include <algorithm>

#include "q8_tc.cuh"

namespace ckv {
namespace {

template <int kD, bool kShared>
struct RowsCfg {
  static constexpr bool kLatent = kShared;
  static constexpr int kRows = 256;
  static constexpr int kSlices = kD / 64;
  static constexpr int kStages = 2;
  static constexpr int kSoftWarps = 16;  // of each row tile: four for the first 64 entries, four for the others
  static constexpr int kConvWarps = 8;
  static constexpr int kWarps = kSoftWarps + kConvWarps + 2;  // the scales' and the products'
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kLoads = kEntries / (8 * kConvWarps);
  static constexpr int kUnits = kSlices * (kShared ? 1 : 2);
  static constexpr uint32_t kQBytes = kSlices * 2 * kSlice;
  static constexpr uint32_t kKBytes = kStages * kSlices * kSlice;
  static constexpr uint32_t kVBytes = kShared ? 0 : kKBytes;
  static constexpr uint32_t kBytes = kQBytes + kKBytes + kVBytes + 1024;  // and the alignment
  // one CTA to an SM: a second would wait for the first one's tensor memory
  static constexpr uint32_t kSmem = kBytes < 120 * 1024 ? 120 * 1024 : kBytes;
  static constexpr uint32_t kOCol = 256;  // scores of the two row tiles, then their outputs
  static constexpr uint32_t kCols = 512;
  static_assert(kOCol + 2 * kD <= 512, "");
};

template <int kD, bool kShared>
struct alignas(16) RowsShared {
  using C = RowsCfg<kD, kShared>;
  uint64_t k_full[C::kStages], k_free[C::kStages], v_full[C::kStages], v_free[C::kStages];
  uint64_t q_full, s_full[2], p_full[2], o_done, idle;
  alignas(16) float f[4][8];  // see scale_tiles
  alignas(16) float lv[4][8];
  alignas(16) float iv[4][8];
  float rf[C::kRows];
  float both[2][C::kRows];  // what the two owners of a row tell each other
  int nan[kShared ? 1 : kD];
  int any_nan;
  uint32_t tmem;
};

// A vote and a barrier of the two warps that share 32 rows.
__device__ __forceinline__ bool pair_any(int id, bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %2, 0;\n\t"
      "bar.red.or.pred q, %1, 64, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(x ? 1u : 0u)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void pair_sync(int id) { asm volatile("bar.sync %0, 64;" ::"r"(id) : "memory"); }

template <int kD, bool kShared, bool kShort, bool kLists>
__global__ __launch_bounds__((RowsCfg<kD, kShared>::kThreads), 1) void q8_attn_rows_kernel(const AttnArgs a) {
  using C = RowsCfg<kD, kShared>;
  extern __shared__ uint8_t raw[];
  __shared__ RowsShared<kD, kShared> sh;
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
  const uint32_t G = a.g.group, H = a.c.heads;
  const uint32_t base = (smem_addr(raw) + 1023) & ~1023u;
  const uint32_t q_at = base, k_at = q_at + C::kQBytes, v_at = kShared ? k_at : k_at + C::kKBytes;
  const bool soft = warp < C::kSoftWarps;
  const bool conv = !soft && warp < C::kSoftWarps + C::kConvWarps;

  if (warp == C::kWarps - 1) tmem_alloc(smem_addr(&sh.tmem), C::kCols);
  if (tid == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(smem_addr(&sh.k_full[s]), C::kConvWarps + 1);
      mbar_init(smem_addr(&sh.v_full[s]), C::kConvWarps);
      mbar_init(smem_addr(&sh.k_free[s]), 1);
      mbar_init(smem_addr(&sh.v_free[s]), 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(smem_addr(&sh.s_full[t]), 1);
      mbar_init(smem_addr(&sh.p_full[t]), C::kSoftWarps / 2);
    }
    mbar_init(smem_addr(&sh.q_full), C::kSoftWarps);
    mbar_init(smem_addr(&sh.o_done), 1);
    mbar_init(smem_addr(&sh.idle), 1);
    fence_mbar_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  Waiter w{static_cast<long long>(a.wait_ns) * 2, true};
  uint32_t tiles_before = 0;  // tiles of earlier items: the barriers' phases go on
  uint32_t items_before = 0;  // earlier items

  for (uint32_t it = item0; it < item1; ++it) {
    const Q8Item item = item_for<kLists>(items + it, a, h);
    __syncthreads();  // the item before is done with what this one's takes the place of
    tc_fence_after();
    if (!item_fits(item, a)) {
      if (tid == 0) status_or(a.d_status, CKV_STATUS_BAD_INDEX);
      continue;
    }
    const uint32_t rows = min(static_cast<uint32_t>(C::kRows), item.q_len * G - item.row0);
    const int32_t* table = table_for<kLists>(a, item, h);
    const uint32_t n_tiles =
        item.kv_end > item.kv_begin ? (item.kv_end - item.kv_begin + kEntries - 1) / kEntries : 0;
    const int tiles = rows > 128 ? 2 : 1;  // row tiles with rows
    const uint32_t vis_min = min(item.kv_end, static_cast<uint32_t>(q8_visible(item.kv_len, item.q_len - 1 - item.row0 / G,
                                                                             item.phase, a.ratio)));
    if (conv) {
      for (int c = tid - 32 * C::kSoftWarps; c < (kShared ? 1 : kD); c += 32 * C::kConvWarps) sh.nan[c] = 0x7FFFFFFF;
      if (tid == 32 * C::kSoftWarps) sh.any_nan = 0;
      asm volatile("bar.sync 9, %0;" ::"n"(32 * C::kConvWarps) : "memory");
      convert_tiles<C, kShort>(a, item, sh, w, warp - C::kSoftWarps, h, table, n_tiles, tiles_before, vis_min, k_at, v_at);
    } else if (soft) {
      const int rt = warp >> 3, half = warp >> 2 & 1, quarter = warp & 3, pair = 1 + rt * 4 + quarter;
      // ---- the rows' query operand and scaling: eight channels of a row to a lane, the loads of several rows in flight together
      {
        constexpr int kLanes = kD / 8, kPer = 32 / kLanes;             // lanes of a row, rows of a warp at a time
        constexpr int kTimes = C::kRows / (kPer * C::kSoftWarps), kBatch = kTimes < 4 ? kTimes : 4;
        const int sub = lane / kLanes, cl = lane % kLanes;
#pragma unroll 1
        for (int t0 = 0; t0 < kTimes; t0 += kBatch) {
          uint4 x[kBatch];
#pragma unroll
          for (int b = 0; b < kBatch; ++b) {
            const uint32_t n = ((t0 + b) * C::kSoftWarps + warp) * kPer + sub;
            const bool in = n < rows;
            const uint32_t rho = item.row0 + (in ? n : 0), i = rho / G, hg = rho % G;
            const size_t row = static_cast<size_t>(item.q_start + i) * a.n_heads + h * G + hg;
            x[b] = ld_stream16_if(a.q + row * kD + cl * 8, in);
          }
#pragma unroll
          for (int b = 0; b < kBatch; ++b) {
            const uint32_t n = ((t0 + b) * C::kSoftWarps + warp) * kPer + sub, r = n & 127;
            const uint32_t y[4] = {x[b].x, x[b].y, x[b].z, x[b].w};
            float m = 0.0f;
#pragma unroll
            for (int e = 0; e < 4; ++e) m = fmaxf(m, fmaxf(fabsf(bf16lo(y[e])), fabsf(bf16hi(y[e]))));
#pragma unroll
            for (int s = kLanes / 2; s > 0; s >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, s));
            const int ex = min(126, 14 - (static_cast<int>(__float_as_uint(m) >> 23) - 127));
            const float up = pow2f(ex);
            uint32_t z[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) z[e] = pack_f16x2(bf16lo(y[e]) * up, bf16hi(y[e]) * up);
            asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(q_at + ((n >> 7) * C::kSlices + (cl >> 3)) * kSlice + r * 128 +
                                                                        (((cl & 7) ^ (r & 7)) << 4)),
                         "r"(z[0]), "r"(z[1]), "r"(z[2]), "r"(z[3])
                         : "memory");
            if (cl == 0) sh.rf[n] = pow2f(-ex);
          }
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&sh.q_full));
        asm volatile("bar.sync 10, %0;" ::"n"(32 * C::kSoftWarps) : "memory");
      }
      if (rt < tiles) {
        const uint32_t n = rt * 128 + quarter * 32 + lane;  // row of the item
        const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
        // this half's scores; its weights take the first 32 of these columns
        const uint32_t s_at = tmem + lanes + rt * 128 + half * 64, o_at = tmem + lanes + C::kOCol + rt * kD;
        const bool in = n < rows;
        const int see = static_cast<int>(q8_visible(item.kv_len, item.q_len - 1 - (item.row0 + (in ? n : 0)) / G, item.phase, a.ratio));
        const uint32_t vis = in ? min(item.kv_end, static_cast<uint32_t>(see)) : item.kv_end;
        const float rf = sh.rf[n];
        // never 0, which would make NaN of a hidden score's -infinity; a factor this small makes 0 of any other
        auto factor = [&](float f) { return fmaxf(f * rf, 1.2e-38f); };
        // 16 scores' weights, and their sum over the value scale
        auto weights = [&](const float(&x)[16], float f, float b, float iv, uint32_t(&p)[8], float& sum_to) {
          const F2 f2 = f2_pack(f, f), b2 = f2_pack(b, b);
          F2 sum = f2_pack(0.0f, 0.0f);
#pragma unroll
          for (int y = 0; y < 16; y += 2) {
            float t0, t1;
            f2_unpack(f2_fma(f2_pack(x[y], x[y + 1]), f2, b2), t0, t1);
            const float w0 = ex2(t0), w1 = ex2(t1);
            sum = f2_add(sum, f2_pack(w0, w1));
            p[y >> 1] = pack_f16x2(w0, w1);
          }
          float s0, s1;
          f2_unpack(sum, s0, s1);
          sum_to = fmaf(s0 + s1, iv, sum_to);
        };
        float m = 0.0f, l = 0.0f;
        bool set = false;  // the row's reference has been set: by its first entry, wherever that is; later ones raise it
        for (uint32_t j = 0; j < n_tiles; ++j) {
          const uint32_t g = tiles_before + j, slot = g & 3;
          const uint32_t e0 = item.kv_begin + j * kEntries;
          const bool edge = e0 + kEntries > vis_min;
          const int hidden = static_cast<int>(vis) - static_cast<int>(e0 + half * 64);  // this half's entries from here on
          const float* f_at = sh.f[slot] + half * 4;
          const float* lv_at = sh.lv[slot] + half * 4;
          const float* iv_at = sh.iv[slot] + half * 4;
          w.wait<kShort>(&sh.s_full[rt], g & 1);
          tc_fence_after();
          // The weights under the reference as it stands, kept in registers, and the largest exponent: a run's scores share
          // their positive factor, so the largest of each run will do.
          float top = -INFINITY, more = l;
          uint32_t p[4][8];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            float x[16];
            tmem_load16(s_at + 16 * c, x);
            const float f = factor(f_at[c]), lv = lv_at[c];
            float y = -INFINITY;
            if (edge) {
#pragma unroll
              for (int z = 0; z < 16; ++z) x[z] = 16 * c + z < hidden ? x[z] : -INFINITY;
            }
#pragma unroll
            for (int z = 0; z < 16; ++z) y = fmaxf(y, x[z]);
            top = fmaxf(top, y == -INFINITY ? -INFINITY : fmaf(y, f, lv));
            weights(x, f, lv - m, iv_at[c], p[c], more);
          }
          if (pair_any(pair, set ? top > m + 14.0f : top > -INFINITY)) {
            // a reference rises (the first entry that a row sees sets it): once a row and now and then
            sh.both[half][n] = top;
            pair_sync(pair);
            top = fmaxf(top, sh.both[half ^ 1][n]);
            const bool raise = set ? top > m + 14.0f : top > -INFINITY;
            const float now = raise ? top - 6.0f : m;
            const float fac = set ? ex2(m - now) : 1.0f;
            m = now;
            l *= fac;
            set |= raise;
            if (j > 0) {  // the scores are in, so the products before them are done; each owner takes half the channels
#pragma unroll 1
              for (int c = half * (kD / 2); c < (half + 1) * (kD / 2); c += 16) {
                float o[16];
                tmem_load16(o_at + c, o);
#pragma unroll
                for (int y = 0; y < 16; ++y) o[y] *= fac;
                tmem_store16(o_at + c, o);
              }
            }
            more = l;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              float x[16];
              tmem_load16(s_at + 16 * c, x);
              if (edge) {
#pragma unroll
                for (int z = 0; z < 16; ++z) x[z] = 16 * c + z < hidden ? x[z] : -INFINITY;
              }
              weights(x, factor(f_at[c]), lv_at[c] - m, iv_at[c], p[c], more);
            }
            pair_sync(pair);  // both have read what the other told
          }
          l = more;
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_put8(s_at + 8 * c, p[c]);  // over scores that are done with
          tmem_store_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_addr(&sh.p_full[rt]));
        }
        // ---- the output: each owner writes half the channels
        sh.both[half][n] = l;
        pair_sync(pair);
        l = sh.both[0][n] + sh.both[1][n];
        // A latent cache's NaN is a NaN score of the rows that see it.  The last tile's scores are in, so its keys' marks are.
        if (kShared && n_tiles > 0 && sh.any_nan != 0 && sh.nan[0] < see) l = __int_as_float(0x7FFFFFFF);
        uint32_t again = n;  // (the place is worked out here and not kept over the tiles)
        asm volatile("" : "+r"(again));
        const uint32_t rho = item.row0 + (in ? again : 0), i = rho / G, hg = rho % G;
        const unsigned long long out_row = static_cast<unsigned long long>(item.q_start + i) * a.n_heads + h * G + hg;
        const size_t part_row = (static_cast<size_t>(item.part + static_cast<int>(item.chunk)) * H + h) * C::kRows + n;
        const float inv = l == 0.0f ? 0.0f : __fdiv_rn(1.0f, l);
        if (in && half == 0) {
          if (item.part >= 0)
            a.part_ml[part_row] = make_float2(l == 0.0f ? -3.4e38f : m, l);
          else if (a.lse != nullptr)
            a.lse[out_row] = l == 0.0f ? -INFINITY : (m + __log2f(l)) * 0.69314718055994530942f;
        }
        w.wait<kShort>(&sh.o_done, items_before & 1);
        tc_fence_after();
        const bool any_nan = !kShared && n_tiles > 0 && sh.any_nan != 0;  // values may be marked up to their product
        // 32 channels at a time through shared memory (the operands are done with), so that a store takes whole lines: 16 bytes a
        // lane of 32 rows took 8 k cycles of an item
        const uint32_t stage = base + warp * 4096, row_sw = lane & 7;
#pragma unroll 1
        for (int c0 = half * (kD / 2); c0 < (half + 1) * (kD / 2); c0 += 32) {
#pragma unroll 1
          for (int c = 0; c < 32; c += 16) {
            float o[16];
            if (n_tiles > 0) {
              tmem_load16(o_at + c0 + c, o);
            } else {
#pragma unroll
              for (int y = 0; y < 16; ++y) o[y] = 0.0f;
            }
            if (any_nan) {
#pragma unroll
              for (int y = 0; y < 16; ++y)
                if (sh.nan[c0 + c + y] < see) o[y] = __int_as_float(0x7FFFFFFF);
            }
            const float by = item.part >= 0 ? 1.0f : inv;
#pragma unroll
            for (int y = 0; y < 16; y += 4)
              asm volatile("st.shared.v4.f32 [%0], {%1,%2,%3,%4};" ::"r"(stage + lane * 128 + ((((c + y) >> 2) ^ row_sw) << 4)),
                           "f"(o[y] * by), "f"(o[y + 1] * by), "f"(o[y + 2] * by), "f"(o[y + 3] * by)
                           : "memory");
          }
          __syncwarp();
#pragma unroll 2
          for (int r0 = 0; r0 < 32; r0 += 4) {
            const int r = r0 + (lane >> 3);
            const uint4 v = lds16(stage + r * 128 + (((lane & 7) ^ (r & 7)) << 4));
            const size_t to = (item.part >= 0 ? part_row - lane + r : __shfl_sync(0xFFFFFFFFu, out_row, r)) * kD + c0 + (lane & 7) * 4;
            if (n - lane + r >= rows) continue;
            if (item.part >= 0)
              *reinterpret_cast<uint4*>(a.part_o + to) = v;
            else if (a.out_f32)
              *reinterpret_cast<uint4*>(static_cast<float*>(a.out) + to) = v;
            else
              *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + to) =
                  make_uint2(pack_bf16x2(__uint_as_float(v.x), __uint_as_float(v.y)), pack_bf16x2(__uint_as_float(v.z), __uint_as_float(v.w)));
          }
          __syncwarp();
        }
        tc_fence_before();
      }
    } else if (warp == C::kSoftWarps + C::kConvWarps) {
      scale_tiles<C, kShort>(a, item, sh, w, h, table, n_tiles, tiles_before);
    } else if (elect_one()) {
      // ---- the products, by one thread, which also waits for what they need.  Products run in the order of issue, so a tile's scores
      // overwrite the weights that the product before them has read.
      // A wait that is over at once still takes some 130 cycles, so there are few: K and V are waited for once for both row
      // tiles, and before the weights, so that nothing but the products stands between those and the next scores.
      auto scores = [&](int rt, uint32_t st) {
        if (w.live) {
          const uint64_t qa = smem_operand(q_at + rt * C::kSlices * kSlice, 0);
          const uint64_t kb = smem_operand(k_at + st * C::kSlices * kSlice, 0);
#pragma unroll
          for (int s = 0; s < C::kSlices; ++s) {
#pragma unroll
            for (int x = 0; x < 4; ++x)  // 16 channels, 32 bytes of a row
              tc_mma(tmem + rt * 128, qa + s * (kSlice >> 4) + 2 * x, kb + s * (kSlice >> 4) + 2 * x,
                     mma_shape(128, 128, false, false), s > 0 || x > 0);
          }
        }
        tc_commit(smem_addr(&sh.s_full[rt]));
      };
      if (n_tiles > 0) {
        uint32_t st = tiles_before % C::kStages;
        w.wait_alone<kShort>(&sh.q_full, items_before & 1);
        w.wait_alone<kShort>(&sh.k_full[st], (tiles_before / C::kStages) & 1);
        tc_fence_after();
        for (int rt = 0; rt < tiles; ++rt) scores(rt, st);
        if (!kShared) tc_commit(smem_addr(&sh.k_free[st]));
#pragma unroll 1
        for (uint32_t j = 0; j < n_tiles; ++j) {
          const uint32_t g = tiles_before + j, next = (g + 1) % C::kStages;
          const bool more = j + 1 < n_tiles;
          if (!kShared) w.wait_alone<kShort>(&sh.v_full[st], (g / C::kStages) & 1);
          if (more) w.wait_alone<kShort>(&sh.k_full[next], ((g + 1) / C::kStages) & 1);
#pragma unroll 1
          for (int rt = 0; rt < tiles; ++rt) {
            w.wait_alone<kShort>(&sh.p_full[rt], g & 1);
            tc_fence_after();
            if (w.live) {
              const uint64_t vb = smem_operand(v_at + st * C::kSlices * kSlice, kSlice);
#pragma unroll
              for (int x = 0; x < 8; ++x)  // 16 entries: 8 columns of weights (each half's from its own 64 on), 16 rows
                tc_mma_ts(tmem + C::kOCol + rt * kD, tmem + rt * 128 + (x >> 2) * 64 + 8 * (x & 3), vb + 128 * x,
                          mma_shape(128, kD, false, true), j > 0 || x > 0);
            }
            if (rt == tiles - 1) tc_commit(smem_addr(kShared ? &sh.k_free[st] : &sh.v_free[st]));
            if (more) scores(rt, next);
          }
          if (more && !kShared) tc_commit(smem_addr(&sh.k_free[next]));
          st = next;
        }
      }
      tc_commit(smem_addr(&sh.o_done));
    }
    __syncwarp();
    // A row tile that was skipped has no phases of its own: both tiles' barriers go on together
    if (tiles == 1 && n_tiles & 1) {
      if (tid == 0) mbar_arrive(smem_addr(&sh.s_full[1]));
      if (soft && warp >= C::kSoftWarps / 2 && lane == 0) mbar_arrive(smem_addr(&sh.p_full[1]));
    }
    tiles_before += n_tiles;
    ++items_before;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
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
  using C = RowsCfg<kD, kShared>;
  auto* kernel = a.wait_ns < kShortWaitNs ? q8_attn_rows_kernel<kD, kShared, true, kLists>
                                          : q8_attn_rows_kernel<kD, kShared, false, kLists>;
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

int launch_q8_attn_rows(const AttnArgs& a, cudaStream_t s) {
  const bool shared = a.c.v == nullptr;
  if (a.c.head_dim == 64) return shared ? launch<64, true>(a, s) : launch<64, false>(a, s);
  return shared ? launch<128, true>(a, s) : launch<128, false>(a, s);
}

}  // namespace ckv

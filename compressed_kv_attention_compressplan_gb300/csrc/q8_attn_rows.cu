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
// Bound.  Per tile of 128 entries and 256 rows at 128 channels: products 2.0 k
// cycles, exponentials 1.0 k (32 a cycle), shared memory 256 KB or 2.0 k, and about
// 3.5 instructions for each of the 32 k scores.
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
  static constexpr int kWarps = kSoftWarps + kConvWarps + 1;
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
  uint64_t s_full[2], p_full[2], o_done, idle;
  alignas(16) float f[4][8];  // see GroupScales
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

template <int kD, bool kShared, bool kShort>
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
      mbar_init(smem_addr(&sh.k_full[s]), C::kConvWarps);
      mbar_init(smem_addr(&sh.v_full[s]), C::kConvWarps);
      mbar_init(smem_addr(&sh.k_free[s]), 1);
      mbar_init(smem_addr(&sh.v_free[s]), 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(smem_addr(&sh.s_full[t]), 1);
      mbar_init(smem_addr(&sh.p_full[t]), C::kSoftWarps / 2);
    }
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
  uint32_t items_before = 0;  // earlier items that had tiles

  for (uint32_t it = item0; it < item1; ++it) {
    const Q8Item item = items[it];
    if (!item_fits(item, a)) {
      if (tid == 0) status_or(a.d_status, CKV_STATUS_BAD_INDEX);
      continue;
    }
    const uint32_t rows = min(static_cast<uint32_t>(C::kRows), item.q_len * G - item.row0);
    const int32_t* table = a.table + static_cast<size_t>(item.rid) * a.stride;
    const uint32_t n_tiles =
        item.kv_end > item.kv_begin ? (item.kv_end - item.kv_begin + kEntries - 1) / kEntries : 0;
    const int tiles = rows > 128 ? 2 : 1;  // row tiles with rows
    const uint32_t vis_min = min(item.kv_end, static_cast<uint32_t>(q8_visible(item.kv_len, item.q_len - 1 - item.row0 / G,
                                                                             item.phase, a.ratio)));
    // ---- the rows' query operand and scaling
    constexpr int kPer = kD / 32, kBatch = 4;  // consecutive channels of a lane; rows whose loads are in flight together
    for (int n0 = warp; n0 < tiles * 128; n0 += kBatch * C::kWarps) {
      uint32_t x[kBatch][kPer / 2];
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const uint32_t n = n0 + b * C::kWarps;
        const bool in = n < rows;
        const uint32_t rho = item.row0 + (in ? n : 0), i = rho / G, hg = rho % G;
        const size_t row = static_cast<size_t>(item.q_start + i) * a.n_heads + h * G + hg;
        const uint32_t* p = reinterpret_cast<const uint32_t*>(a.q + row * kD + lane * kPer);
#pragma unroll
        for (int e = 0; e < kPer / 2; ++e) x[b][e] = in ? __ldg(p + e) : 0u;
      }
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int n = n0 + b * C::kWarps;
        if (n >= tiles * 128) break;
        float m = 0.0f;
#pragma unroll
        for (int e = 0; e < kPer / 2; ++e) m = fmaxf(m, fmaxf(fabsf(bf16lo(x[b][e])), fabsf(bf16hi(x[b][e]))));
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, s));
        const int ex = min(126, 14 - (static_cast<int>(__float_as_uint(m) >> 23) - 127));
        const float up = pow2f(ex);
        const int r = n & 127;
#pragma unroll
        for (int e = 0; e < kPer / 2; ++e) {
          const uint32_t c = lane * kPer + 2 * e;
          sts_u32(q_at + ((n >> 7) * C::kSlices + (c >> 6)) * kSlice + r * 128 + ((((c & 63) >> 3) ^ (r & 7)) << 4) + (c & 7) * 2,
                  pack_f16x2(bf16lo(x[b][e]) * up, bf16hi(x[b][e]) * up));
        }
        if (lane == 0) sh.rf[n] = pow2f(-ex);
      }
    }
    for (int c = tid; c < (kShared ? 1 : kD); c += C::kThreads) sh.nan[c] = 0x7FFFFFFF;
    if (tid == 0) sh.any_nan = 0;
    fence_async_smem();
    __syncthreads();

    if (conv) {
      convert_tiles<C, kShort>(a, item, sh, w, warp - C::kSoftWarps, h, table, n_tiles, tiles_before, vis_min, k_at, v_at);
    } else if (soft) {
      const int rt = warp >> 3, half = warp >> 2 & 1, quarter = warp & 3, pair = 1 + rt * 4 + quarter;
      if (rt < tiles) {
        const uint32_t n = rt * 128 + quarter * 32 + lane;  // row of the item
        const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
        // this half's scores; its weights take the first 32 of these columns
        const uint32_t s_at = tmem + lanes + rt * 128 + half * 64, o_at = tmem + lanes + C::kOCol + rt * kD;
        const bool in = n < rows;
        const uint32_t rho = item.row0 + (in ? n : 0), i = rho / G, hg = rho % G;
        const int64_t see = q8_visible(item.kv_len, item.q_len - 1 - i, item.phase, a.ratio);
        const uint32_t vis = in ? static_cast<uint32_t>(min(static_cast<int64_t>(item.kv_end), see)) : item.kv_end;
        const float rf = sh.rf[n];
        // never 0, which would make NaN of a hidden score's -infinity; a factor this small makes 0 of any other
        auto factor = [&](float f) { return fmaxf(f * rf, 1.2e-38f); };
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
          // the largest exponent: a run's scores share their positive factor, so the largest of each run will do
          float top = -INFINITY;
#pragma unroll
          for (int c = 0; c < 64; c += 32) {
            float x[32];
            tmem_load32(s_at + c, x);
            if (edge) {
#pragma unroll
              for (int y = 0; y < 32; ++y) x[y] = c + y < hidden ? x[y] : -INFINITY;
            }
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              float y = x[16 * r];
#pragma unroll
              for (int z = 1; z < 16; ++z) y = fmaxf(y, x[16 * r + z]);
              top = fmaxf(top, y == -INFINITY ? -INFINITY : fmaf(y, factor(f_at[(c >> 4) + r]), lv_at[(c >> 4) + r]));
            }
          }
          if (pair_any(pair, set ? top > m + 14.0f : top > -INFINITY)) {
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
            pair_sync(pair);  // both have read what the other told
          }
#pragma unroll
          for (int c = 0; c < 64; c += 16) {
            float x[16];
            tmem_load16(s_at + c, x);
            if (edge) {
#pragma unroll
              for (int y = 0; y < 16; ++y) x[y] = c + y < hidden ? x[y] : -INFINITY;
            }
            uint32_t p[8];
            const float f = factor(f_at[c >> 4]), b = lv_at[c >> 4] - m;
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
            l = fmaf(s0 + s1, iv_at[c >> 4], l);
            tmem_put8(s_at + (c >> 1), p);  // over scores that are in registers or done with
          }
          tmem_store_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_addr(&sh.p_full[rt]));
        }
        // ---- the output: each owner writes half the channels
        sh.both[half][n] = l;
        pair_sync(pair);
        l = sh.both[0][n] + sh.both[1][n];
        const size_t out_row = static_cast<size_t>(item.q_start + i) * a.n_heads + h * G + hg;
        const size_t part_row = (static_cast<size_t>(item.part + static_cast<int>(item.chunk)) * H + h) * C::kRows + n;
        const float inv = l == 0.0f ? 0.0f : __fdiv_rn(1.0f, l);
        if (in && half == 0) {
          if (item.part >= 0)
            a.part_ml[part_row] = make_float2(l == 0.0f ? -3.4e38f : m, l);
          else if (a.lse != nullptr)
            a.lse[out_row] = l == 0.0f ? -INFINITY : (m + __log2f(l)) * 0.69314718055994530942f;
        }
        if (n_tiles > 0) w.wait<kShort>(&sh.o_done, items_before & 1);
        tc_fence_after();
        const int any_nan = sh.any_nan;
#pragma unroll 1
        for (int c = half * (kD / 2); c < (half + 1) * (kD / 2); c += 16) {
          float o[16];
          if (n_tiles > 0) {
            tmem_load16(o_at + c, o);
          } else {
#pragma unroll
            for (int y = 0; y < 16; ++y) o[y] = 0.0f;
          }
          if (!in) continue;
          if (any_nan) {
#pragma unroll
            for (int y = 0; y < 16; ++y)
              if (sh.nan[kShared ? 0 : c + y] < see) o[y] = __int_as_float(0x7FFFFFFF);
          }
#pragma unroll
          for (int y = 0; y < 16; y += 8) {
            float v[8];
#pragma unroll
            for (int z = 0; z < 8; ++z) v[z] = item.part >= 0 ? o[y + z] : o[y + z] * inv;
            if (item.part >= 0)
              store_row_chunk<float, 8>(a.part_o + part_row * kD + c + y, v);
            else if (a.out_f32)
              store_row_chunk<float, 8>(static_cast<float*>(a.out) + out_row * kD + c + y, v);
            else
              store_row_chunk<__nv_bfloat16, 8>(static_cast<__nv_bfloat16*>(a.out) + out_row * kD + c + y, v);
          }
        }
        tc_fence_before();
      }
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
        tc_commit(smem_addr(&sh.o_done));
      }
    }
    __syncwarp();
    // A row tile that was skipped has no phases of its own: both tiles' barriers go on together
    if (tiles == 1 && n_tiles & 1) {
      if (tid == 0) mbar_arrive(smem_addr(&sh.s_full[1]));
      if (soft && warp >= C::kSoftWarps / 2 && lane == 0) mbar_arrive(smem_addr(&sh.p_full[1]));
    }
    tiles_before += n_tiles;
    items_before += n_tiles > 0;
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

template <int kD, bool kShared>
int launch(const AttnArgs& a, cudaStream_t s) {
  using C = RowsCfg<kD, kShared>;
  auto* kernel = a.wait_ns < kShortWaitNs ? q8_attn_rows_kernel<kD, kShared, true> : q8_attn_rows_kernel<kD, kShared, false>;
  static std::atomic<uint64_t> done[2];
  const int rc = allow_smem(reinterpret_cast<const void*>(kernel), C::kSmem, done[a.wait_ns < kShortWaitNs ? 1 : 0]);
  if (rc) return rc;
  return launch_pdl(kernel, dim3(a.g.ctas, a.c.heads), dim3(C::kThreads), C::kSmem, s, a);
}

}  // namespace

int launch_q8_attn_rows(const AttnArgs& a, cudaStream_t s) {
  const bool shared = a.c.v == nullptr;
  if (a.c.head_dim == 64) return shared ? launch<64, true>(a, s) : launch<64, false>(a, s);
  return shared ? launch<128, true>(a, s) : launch<128, false>(a, s);
}

}  // namespace ckv

// q8_score_tc.cu -- the blocks' scores for many query rows (chunked prefill) on the 5th-generation
// tensor cores, up to 128 channels.  The mathematics is q8_score.cu's:
//     S [128 blocks x 128 query rows] = [hi, lo] [max(q, 0), min(q, 0)]^T.
// With blocks as the product's rows a thread of the epilogue owns a block: the maximum over a query's heads is one over its own
// registers, and a warp's scores of a query are 128 consecutive bytes.
//
// A segment is 128 blocks of a (request, kv head) and all row tiles of the request; segments are laid end to end, and every CTA takes as many of
// their tiles, so that it loads bounds as seldom as possible.  A unit is a CTA's part of a segment.  Roles: sixteen warps make the
// operands (fp16, exact from e4m3; query rows scaled by a power of two), the next tile's loads on their way while one
// is stored; one thread issues the products; eight warps finish the scores.  Rows of heads that do not exist repeat the
// group's last head, so that no maximum has to leave them out.
//
// Bound.  The roles' sequence itself: 3 requests of up to 512 blocks, 500 to 1024 queries each, 32 heads over eight kv heads of 128 channels, eleven tiles a
// CTA, take 37.5 us, and 20.9 are left without loads, conversions, products and the scores' way out: the launch, the requests' scan and a unit's place
// (9 us is a call of one tile a CTA), the barriers between the roles and the operands' stores of 64 KB a tile.  Without the conversions
// 34.9, without the scores' way out 32.5, without both 26.7; then without the products too 23.9, without the rows' loads too 23.5, without the bounds' 26.6.
// Tried: units of four for each SM, dealt out one by one, 40;
// rows kept and bounds streamed past them 43 (a unit's start, three dependent reads, then comes every four tiles); eight warps making operands
// 74, with spilled registers for the loads on their way, or 46 beside kept rows; sixteen warps for the scores there 51; the places behind
// the last tile filled first 39.
#include <algorithm>

#include "q8_score.cuh"
#include "q8_tc.cuh"

namespace ckv {
namespace {

constexpr uint32_t kTile = 128;  // blocks, and query rows, of a product

template <int kD>
struct StCfg {
  static constexpr int kLoadWarps = 16, kOutWarps = 8;
  static constexpr int kWarps = kLoadWarps + kOutWarps + 1;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kSlices = 2 * kD / 64;  // of 64 values of the depth
  static constexpr uint32_t kOperand = kSlices * kSlice;
  static constexpr int kLanes = kD / 8;          // threads of a query row, and of a block's bounds, 16 bytes each
  static constexpr int kRows = 32 / kLanes;      // rows of a warp at a time
  static constexpr int kTimes = kTile / kLoadWarps / kRows;  // for its share of a tile
  static constexpr uint32_t kBytes = 3 * kOperand + 1024;  // bounds, two stages of queries, the alignment
  static constexpr uint32_t kSmem = kBytes < 120 * 1024 ? 120 * 1024 : kBytes;  // one CTA to an SM: see the attention
  static constexpr uint32_t kCols = 256;
};

struct alignas(16) StShared {
  uint64_t a_full, a_free, q_full[2], q_free[2], s_full[2], s_free[2], rows_full[4], idle;
  alignas(16) float rf[4][kTile];  // of four row tiles: what undoes a row's scaling
  uint32_t lim[4][kTile];          // and the blocks that its query sees; kInvalidU32: there is none
  float ks[3][kTile];              // of three units: the blocks' scales; negative: a block that does not exist
  uint32_t first_q[CKV_MAX_BATCH];
  BlockReq req[CKV_MAX_BATCH];
  unsigned long long first_tile[CKV_MAX_BATCH];
  unsigned long long begin;  // of this CTA's tiles
  uint32_t tiles;
  uint32_t tmem;
};

struct StUnit {
  uint32_t b, h, block0, tile0, tiles;  // request, kv head, first block, row tiles
};

template <int kD, bool kShort>
__global__ __launch_bounds__(StCfg<kD>::kThreads, 1) void q8_score_tc_kernel(const ScoreArgs a, uint32_t span_shift) {
  using C = StCfg<kD>;
  extern __shared__ uint8_t raw[];
  __shared__ StShared sh;
  pdl_wait();
  pdl_release();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t T = a.c.block_tokens, t_shift = __ffs(T) - 1, H = a.c.heads, G = a.group;
  unsigned long long* scan = reinterpret_cast<unsigned long long*>(sh.lim);  // before the roles begin
  scan_queries<C::kThreads>(a.r, sh.first_q, sh.req, scan);
  auto row_tiles = [&](const BlockReq& r) { return ((r.q_len << span_shift) + kTile - 1) / kTile; };
  unsigned long long total = 0;  // tiles
  for (uint32_t b0 = 0; b0 < a.r.batch; b0 += C::kThreads) {
    const uint32_t b = b0 + tid;
    unsigned long long n = 0;
    if (b < a.r.batch)
      n = static_cast<unsigned long long>(row_tiles(sh.req[b])) * H * score_tiles<kTile>(sh.req[b], a.r.ratio, t_shift);
    unsigned long long sum;
    const unsigned long long at = total + block_exclusive<C::kThreads>(n, &sum, scan);
    if (b < a.r.batch) sh.first_tile[b] = at;
    total += sum;
  }
  const unsigned long long share = (total + gridDim.x - 1) / gridDim.x, begin = blockIdx.x * share;
  const bool idle = begin >= total;
  if (tid == 0) {
    sh.begin = begin;
    sh.tiles = idle ? 0 : static_cast<uint32_t>(min(share, total - begin));
  }
  const uint32_t base = (smem_addr(raw) + 1023) & ~1023u;
  const uint32_t a_at = base, q_at = base + C::kOperand;
  if (warp == C::kWarps - 1 && !idle) tmem_alloc(smem_addr(&sh.tmem), C::kCols);
  if (tid == 0) {
    mbar_init(smem_addr(&sh.a_full), C::kLoadWarps);
    mbar_init(smem_addr(&sh.a_free), 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(smem_addr(&sh.q_full[s]), C::kLoadWarps);
      mbar_init(smem_addr(&sh.q_free[s]), 1);
      mbar_init(smem_addr(&sh.s_full[s]), 1);
      mbar_init(smem_addr(&sh.s_free[s]), C::kOutWarps);
    }
    for (int s = 0; s < 4; ++s) mbar_init(smem_addr(&sh.rows_full[s]), C::kLoadWarps);
    mbar_init(smem_addr(&sh.idle), 1);
    fence_mbar_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  Waiter w{static_cast<long long>(a.wait_ns) * 2, true};

  auto unit_of = [&](uint32_t done) -> StUnit {
    StUnit x;
    const unsigned long long at = sh.begin + done;
    x.b = last_not_above(sh.first_tile, a.r.batch, at);
    const BlockReq r = sh.req[x.b];
    const uint32_t tiles = row_tiles(r), block_tiles = score_tiles<kTile>(r, a.r.ratio, t_shift);
    const unsigned long long rel = at - sh.first_tile[x.b], y = rel / tiles;
    x.tile0 = static_cast<uint32_t>(rel - y * tiles);
    x.tiles = min(sh.tiles - done, tiles - x.tile0);
    x.h = static_cast<uint32_t>(y / block_tiles);
    x.block0 = static_cast<uint32_t>(y % block_tiles) * kTile;
    return x;
  };
  // every role walks the same (unit, row tile) sequence; uc and qc count units and row tiles
  uint32_t uc = 0, qc = 0;
  if (warp < C::kLoadWarps) {
    // ---- operands.  A warp makes its share of the rows of each; lane l has 16 bytes, chunk l % kLanes, of a row
    const uint32_t chunk = lane % C::kLanes, row0 = warp * (kTile / C::kLoadWarps) + lane / C::kLanes;
    const __half2 zero = __float2half2_rn(0.0f);
    int32_t blk[C::kTimes];
    auto ask = [&](uint32_t done) {
      if (done >= sh.tiles) return;
      const StUnit x = unit_of(done);
      const BlockReq r = sh.req[x.b];
      const uint32_t blocks = (seen_by(r, r.q_len - 1, a.r.ratio) + T - 1) >> t_shift;
#pragma unroll
      for (int i = 0; i < C::kTimes; ++i) {
        const uint32_t j = x.block0 + row0 + i * C::kRows;
        blk[i] = j < blocks ? ld_ahead(a.table + static_cast<size_t>(r.rid) * a.stride + j) : -1;
      }
    };
    uint4 rows[C::kTimes];
    auto load_row = [&](const StUnit& x, uint32_t t, int i) {
      const uint32_t rho = (x.tile0 + t) * kTile + row0 + i * C::kRows, n = rho >> span_shift;
      const uint32_t head = min(rho & ((1u << span_shift) - 1), G - 1);
      rows[i] = ld_stream16_if(a.q + (static_cast<size_t>(sh.first_q[x.b] + n) * a.n_heads + x.h * G + head) * kD + chunk * 8, n < sh.req[x.b].q_len);
    };
    ask(0);
    for (; qc < sh.tiles; ++uc) {
      const StUnit x = unit_of(qc);
      const BlockReq r = sh.req[x.b];
      // A unit's bounds are not kept in registers beside its rows: what does not fit them comes back from L2, as its shared memory
      // leaves next to no L1 (74 us so, with both a unit ahead).
      uint4 bounds[C::kTimes];
      float scale[C::kTimes];
      const uint32_t blocks = (seen_by(r, r.q_len - 1, a.r.ratio) + T - 1) >> t_shift;
#pragma unroll
      for (int i = 0; i < C::kTimes; ++i) {
        const bool ok = static_cast<uint32_t>(blk[i]) < a.c.num_blocks;
        if (!ok && chunk == 0 && x.block0 + row0 + i * C::kRows < blocks) status_or(a.r.d_status, CKV_STATUS_BAD_INDEX);
        const size_t bh = static_cast<size_t>(ok ? blk[i] : 0) * H + x.h;
        bounds[i] = ld_stream16_if(a.bounds + bh * 2 * kD + chunk * 16, ok);
        scale[i] = ok ? ld_ahead(a.c.k_scale + bh) : -1.0f;
      }
      ask(qc + x.tiles);
      w.wait<kShort>(&sh.a_free, (uc & 1) ^ 1);
#pragma unroll
      for (int i = 0; i < C::kTimes; ++i) {
        const uint32_t n = row0 + i * C::kRows, side = chunk / (kD / 16), c = chunk % (kD / 16);  // 16 channels of a side
        const uint32_t to = a_at + (side * (kD / 64) + (c >> 2)) * kSlice + n * 128;
        const uint32_t y[4] = {bounds[i].x, bounds[i].y, bounds[i].z, bounds[i].w};
#pragma unroll
        for (int z = 0; z < 2; ++z)
          asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(to + ((((c & 3) * 2 + z) ^ (n & 7)) << 4)), "r"(q8_lo_f16x2(y[2 * z])),
                       "r"(q8_hi_f16x2(y[2 * z])), "r"(q8_lo_f16x2(y[2 * z + 1])), "r"(q8_hi_f16x2(y[2 * z + 1]))
                       : "memory");
        if (chunk == 0) sh.ks[uc % 3][n] = scale[i];
      }
#pragma unroll
      for (int i = 0; i < C::kTimes; ++i) load_row(x, 0, i);
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&sh.a_full));
      for (uint32_t t = 0; t < x.tiles; ++t, ++qc) {
        const uint32_t qs = qc & 1;
        w.wait<kShort>(&sh.q_free[qs], ((qc >> 1) & 1) ^ 1);
#pragma unroll
        for (int i = 0; i < C::kTimes; ++i) {
          const uint32_t n = row0 + i * C::kRows, y[4] = {rows[i].x, rows[i].y, rows[i].z, rows[i].w};
          float m = 0.0f;
#pragma unroll
          for (int z = 0; z < 4; ++z) m = fmaxf(m, fmaxf(fabsf(bf16lo(y[z])), fabsf(bf16hi(y[z]))));
#pragma unroll
          for (int s = C::kLanes / 2; s > 0; s >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, s));
          const int ex = min(126, 14 - (static_cast<int>(__float_as_uint(m) >> 23) - 127));
          const float up = pow2f(ex);
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int z = 0; z < 4; ++z) {
            const __half2 v = as_half2(pack_f16x2(bf16lo(y[z]) * up, bf16hi(y[z]) * up));
            hi[z] = as_u32(__hmax2_nan(v, zero));
            lo[z] = as_u32(__hmin2_nan(v, zero));
          }
          if (t + 1 < x.tiles) load_row(x, t + 1, i);  // its place is free
          const uint32_t to = q_at + qs * C::kOperand + (chunk >> 3) * kSlice + n * 128 + (((chunk & 7) ^ (n & 7)) << 4);
          asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(to), "r"(hi[0]), "r"(hi[1]), "r"(hi[2]), "r"(hi[3]) : "memory");
          asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(to + (kD / 64) * kSlice), "r"(lo[0]), "r"(lo[1]), "r"(lo[2]), "r"(lo[3]) : "memory");
          if (chunk == 0) {
            const uint32_t q = ((x.tile0 + t) * kTile + n) >> span_shift;
            sh.rf[qc & 3][n] = row_factor(a, ex);
            sh.lim[qc & 3][n] = q < r.q_len ? (seen_by(r, q, a.r.ratio) + T - 1) >> t_shift : kInvalidU32;
          }
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(smem_addr(&sh.q_full[qs]));
          mbar_arrive(smem_addr(&sh.rows_full[qc & 3]));
        }
      }
    }
  } else if (warp < C::kLoadWarps + C::kOutWarps) {
    // ---- scores: a thread owns a block (its lane of tensor memory) and 64 of a tile's query rows
    const int group = (warp - C::kLoadWarps) >> 2, quarter = warp & 3, entry = quarter * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    for (; qc < sh.tiles; ++uc) {
      const StUnit x = unit_of(qc);
      const uint32_t j = x.block0 + entry, q0 = sh.first_q[x.b];
      float ks = 0.0f;
      for (uint32_t t = 0; t < x.tiles; ++t, ++qc) {
        const uint32_t sb = qc & 1;
        // the rows' factors and limits, and the blocks' scales, which are in before them.  Their places are taken again by the fourth
        // tile (third unit) after this one, which is stored after the product of the second tile after it, and that comes after these reads.
        w.wait<kShort>(&sh.rows_full[qc & 3], (qc >> 2) & 1);
        w.wait<kShort>(&sh.s_full[sb], (qc >> 1) & 1);
        tc_fence_after();
        if (t == 0) ks = sh.ks[uc % 3][entry];
        const float k = ks * a.scale;
        const uint32_t n0 = ((x.tile0 + t) * kTile + group * 64) >> span_shift;  // the first row's query
        float* out = a.scores + (static_cast<size_t>(q0 + n0) * H + x.h) * a.width + j;
        const size_t step = static_cast<size_t>(H) * a.width;
        const uint32_t* lim = sh.lim[qc & 3] + group * 64;
        auto put = [&](uint32_t row, float v) {
          const uint32_t limit = lim[row];
          if (limit == kInvalidU32 || j >= a.width) return;
          out[(row >> span_shift) * step] = j < limit && ks > 0.0f ? v * k : -INFINITY;
        };
        float top = -INFINITY;  // of 64 heads, over the first half
#pragma unroll 1
        for (int half = 0; half < 64; half += 32) {
          float s[32];
          tmem_load32(tmem + lanes + sb * kTile + group * 64 + half, s);
          const float* rf = sh.rf[qc & 3] + group * 64 + half;
#pragma unroll
          for (int c = 0; c < 32; c += 4) {
            const float4 f = *reinterpret_cast<const float4*>(rf + c);
            s[c] *= f.x;
            s[c + 1] *= f.y;
            s[c + 2] *= f.z;
            s[c + 3] *= f.w;
          }
          // a pairwise maximum over a query's rows, in place: after round r every 2^r-th register holds one
          auto reduce = [&](auto shift) {
            constexpr int kShift = decltype(shift)::value;
#pragma unroll
            for (int d = 1; d < (1 << kShift); d <<= 1) {
#pragma unroll
              for (int c = 0; c < 32; c += 2 * d) s[c] = max_nan(s[c], s[c + d]);
            }
          };
          auto finish = [&](auto shift) {
            constexpr int kShift = decltype(shift)::value;
            reduce(shift);
#pragma unroll
            for (int c = 0; c < 32; c += 1 << kShift) put(half + c, s[c]);
          };
          switch (span_shift) {
            case 0: finish(std::integral_constant<int, 0>()); break;
            case 1: finish(std::integral_constant<int, 1>()); break;
            case 2: finish(std::integral_constant<int, 2>()); break;
            case 3: finish(std::integral_constant<int, 3>()); break;
            case 4: finish(std::integral_constant<int, 4>()); break;
            case 5: finish(std::integral_constant<int, 5>()); break;
            default:
              reduce(std::integral_constant<int, 5>());
              top = max_nan(top, s[0]);
              if (half != 0) put(0, top);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&sh.s_free[sb]));  // and its rows' factors and limits
      }
    }
  } else {
    for (; qc < sh.tiles; ++uc) {
      const StUnit x = unit_of(qc);
      w.wait<kShort>(&sh.a_full, uc & 1);
      for (uint32_t t = 0; t < x.tiles; ++t, ++qc) {
        const uint32_t sb = qc & 1;
        w.wait<kShort>(&sh.q_full[sb], (qc >> 1) & 1);
        w.wait<kShort>(&sh.s_free[sb], ((qc >> 1) & 1) ^ 1);
        tc_fence_after();
        if (elect_one()) {
          if (w.live) {
#pragma unroll
            for (int s = 0; s < C::kSlices; ++s) {
              const uint64_t ma = smem_operand(a_at + s * kSlice, 0), mb = smem_operand(q_at + sb * C::kOperand + s * kSlice, 0);
#pragma unroll
              for (int y = 0; y < 4; ++y)
                tc_mma(tmem + sb * kTile, ma + 2 * y, mb + 2 * y, mma_shape(128, 128, false, false), s > 0 || y > 0);
            }
          }
          tc_commit(smem_addr(&sh.q_free[sb]));
          tc_commit(smem_addr(&sh.s_full[sb]));
          if (t + 1 == x.tiles) tc_commit(smem_addr(&sh.a_free));
        }
        __syncwarp();
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == C::kWarps - 1 && !idle) {
    // every product is done before its memory is given back
    if (elect_one()) tc_commit(smem_addr(&sh.idle));
    __syncwarp();
    const bool done = warp_wait_for<false>(smem_addr(&sh.idle), 0, kWaitLimitNs);
    if (!done) w.live = false;
    tmem_free(tmem, C::kCols);
  }
  if (!w.live && lane == 0) status_or(a.r.d_status, CKV_STATUS_TIMEOUT);
  fill_behind<kTile>(a, sh.first_q, sh.req);
}

template <int kD>
int launch(const ScoreArgs& a, cudaStream_t s) {
  using C = StCfg<kD>;
  static_assert(C::kSmem + sizeof(StShared) <= 227 * 1024, "");
  const bool brief = a.wait_ns < kShortWaitNs;
  auto* kernel = brief ? q8_score_tc_kernel<kD, true> : q8_score_tc_kernel<kD, false>;
  static std::atomic<uint64_t> done[2];
  const int rc = allow_smem(reinterpret_cast<const void*>(kernel), C::kSmem, done[brief ? 1 : 0]);
  if (rc) return rc;
  uint32_t shift = 0;
  while ((1u << shift) < a.group) ++shift;
  return launch_pdl(kernel, dim3(static_cast<uint32_t>(sm_count())), dim3(C::kThreads), C::kSmem, s, a, shift);
}

}  // namespace

int launch_q8_score_tc(const ScoreArgs& a, cudaStream_t s) { return a.c.head_dim == 64 ? launch<64>(a, s) : launch<128>(a, s); }

}  // namespace ckv

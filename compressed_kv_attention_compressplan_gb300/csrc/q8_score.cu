// q8_score.cu -- what each block of the 8-bit paged cache can hold for a query:
// the blocks' bounds, and the scores that follow from them.
//
// Mathematics.  With hi_c and lo_c the largest and smallest code of channel c in a
// block, <q, k> of any of its entries is at most ks * sum_c max(q_c hi_c, q_c lo_c).
// As hi >= lo, the larger product is q_c hi_c for q_c > 0 and q_c lo_c otherwise, so the sum is
//     <max(q, 0), hi> + <min(q, 0), lo>,
// a matrix product of twice the depth: nothing is compared per channel.  The bounds are e4m3 codes of
// the block's own scale, hence exact, and exact again in fp16.  A query row is scaled by a
// power of two that puts its largest value in [2^14, 2^15) and rounded to fp16: exact for bf16 down to
// 2^-28 of it.  Products are exact, sums fp32.
#include <algorithm>

#include "async_copy.cuh"
#include "q8_score.cuh"

namespace ckv {
namespace {

// ------------------------------------------------------------------- bounds
constexpr int kBoundThreads = 256;

struct BoundArgs {
  Q8Cache c;
  uint8_t* bounds;
  const int64_t* rid;
  const int64_t* kv_lens;
  const int64_t* new_lens;
  uint32_t batch;
  const int32_t* table;
  uint32_t stride;
  uint32_t num_reqs;
  uint32_t* d_status;
};

// The bounds are looked for in the codes themselves.  An e4m3 code as the upper byte of a bf16 orders as the e4m3 value does, whatever
// the lower byte holds (it only decides between equal codes), and is finite but for NaN codes: so two channels are compared
// at once where they lie, and the two between them after one shift, without a conversion.  A NaN code is larger than every other of its
// sign, or a bf16 NaN that both operations hand on: it is in hi or in lo, and is copied to the other at the end.
__device__ __forceinline__ void widen(uint32_t w, uint32_t* hi, uint32_t* lo) {
  auto bf = [](uint32_t x) { return *reinterpret_cast<const __nv_bfloat162*>(&x); };
  auto word = [](__nv_bfloat162 x) { return *reinterpret_cast<const uint32_t*>(&x); };
  hi[0] = word(__hmax2_nan(bf(hi[0]), bf(w << 8)));
  lo[0] = word(__hmin2_nan(bf(lo[0]), bf(w << 8)));
  hi[1] = word(__hmax2_nan(bf(hi[1]), bf(w)));
  lo[1] = word(__hmin2_nan(bf(lo[1]), bf(w)));
}
__device__ __forceinline__ void codes_of(const uint32_t* hi, const uint32_t* lo, uint32_t* h, uint32_t* l) {
  *h = __byte_perm(hi[0], hi[1], 0x7351);  // the upper bytes: channels 0, 2 of the first word, 1, 3 of the second
  *l = __byte_perm(lo[0], lo[1], 0x7351);
  const uint32_t nan = q8_nan_bytes(*h) | q8_nan_bytes(*l);
  *h |= nan & 0x7F7F7F7Fu;
  *l |= nan & 0x7F7F7F7Fu;
}

// A warp takes an equal run of (block, head) pairs, one after the other: lane l holds 16 channels, chunk l % (kD / 16), of every (512 / kD)th
// entry.  The reads bound it: 237 MB (32 requests of up to 16384 new entries, eight kv heads of 128 channels, blocks of 64) in 47 us,
// 5.0 TB/s or 75 % of the copy rate.  One new entry for each of 64 requests takes 6.9, a
// launch and four dependent reads.  Pairs dealt out one by one to six CTAs an SM took 43 and 9.9 us; the codes as fp16, 47 and 7.6.
template <int kD>
__global__ __launch_bounds__(kBoundThreads, 4) void q8_bounds_kernel(const BoundArgs a) {
  constexpr uint32_t kChunks = kD / 16, kRows = 32 / kChunks;  // chunks of an entry, entries that a warp reads at once
  __shared__ unsigned long long s_unit[CKV_MAX_BATCH];
  __shared__ uint32_t s_first[CKV_MAX_BATCH], s_len[CKV_MAX_BATCH], s_rid[CKV_MAX_BATCH];
  __shared__ unsigned long long s_scan[kBoundThreads / 32 + 1];
  pdl_wait();
  pdl_release();
  const uint32_t T = a.c.block_tokens, H = a.c.heads;
  unsigned long long units = 0;
  for (uint32_t b0 = 0; b0 < a.batch; b0 += kBoundThreads) {
    const uint32_t b = b0 + threadIdx.x;
    unsigned long long n = 0;
    if (b < a.batch) {
      const int64_t r = a.rid[b], kl = a.kv_lens[b], nl = a.new_lens[b];
      const bool ok = r >= 0 && r < a.num_reqs && nl >= 0 && kl >= nl && kl <= 0x7FFFFFF0 && kl <= static_cast<int64_t>(a.stride) * T;
      if (!ok && blockIdx.x == 0) status_or(a.d_status, CKV_STATUS_BAD_LENGTH);
      if (ok && nl > 0) {
        const uint32_t first = static_cast<uint32_t>(kl - nl) / T;
        s_first[b] = first;
        s_len[b] = static_cast<uint32_t>(kl);
        s_rid[b] = static_cast<uint32_t>(r);
        n = (static_cast<uint32_t>(kl) + T - 1) / T - first;
      }
    }
    unsigned long long sum;
    const unsigned long long u0 = units + block_exclusive<kBoundThreads>(n, &sum, s_scan);
    if (b < a.batch) s_unit[b] = u0;
    units += sum;
  }
  __syncthreads();
  // An equal share of (block, head) pairs to a warp, the heads of a block one after the other.
  const int lane = threadIdx.x & 31;
  const uint32_t chunk = lane % kChunks, row = lane / kChunks;
  const unsigned long long pairs = units * H, warps = static_cast<unsigned long long>(gridDim.x) * (kBoundThreads / 32);
  const unsigned long long share = (pairs + warps - 1) / warps;
  const unsigned long long first = (static_cast<unsigned long long>(blockIdx.x) * (kBoundThreads / 32) + (threadIdx.x >> 5)) * share;
  if (first >= pairs) return;
  const unsigned long long u = first / H;
  uint32_t h = static_cast<uint32_t>(first - u * H), b = last_not_above(s_unit, a.batch, u);
  uint32_t j = s_first[b] + static_cast<uint32_t>(u - s_unit[b]);
  auto number = [&]() { return __ldg(a.table + static_cast<size_t>(s_rid[b]) * a.stride + j); };
  int32_t block = number();
  for (uint32_t left = static_cast<uint32_t>(min(share, pairs - first)); left > 0; --left) {
    const bool ok = static_cast<uint32_t>(block) < a.c.num_blocks;
    if (!ok && lane == 0) status_or(a.d_status, CKV_STATUS_BAD_INDEX);
    const uint32_t n = ok ? min(T, s_len[b] - j * T) : 0;
    const uint8_t* k = a.c.k + (static_cast<size_t>(ok ? block : 0) * H + h) * T * kD + chunk * 16;
    uint8_t* to = a.bounds + (static_cast<size_t>(ok ? block : 0) * H + h) * 2 * kD + chunk * 16;
    // the next pair's place; a block's number is asked for before this pair's work
    if (++h == H) {
      h = 0;
      if (left > 1) {
        if (++j >= (s_len[b] + T - 1) / T) {
          do ++b;
          while (b + 1 < a.batch && s_unit[b + 1] == s_unit[b]);
          j = s_first[b];
        }
        block = number();
      }
    }
    if (!ok) continue;
    uint32_t hi[8], lo[8];
#pragma unroll
    for (int z = 0; z < 8; ++z) {
      hi[z] = 0xFF80FF80u;  // -infinity
      lo[z] = 0x7F807F80u;
    }
#pragma unroll 8
    for (uint32_t r = row; r < n; r += kRows) {
      const uint4 v = ld_stream16(k + r * kD);
      widen(v.x, hi, lo);
      widen(v.y, hi + 2, lo + 2);
      widen(v.z, hi + 4, lo + 4);
      widen(v.w, hi + 6, lo + 6);
    }
    auto bf = [](uint32_t x) { return *reinterpret_cast<const __nv_bfloat162*>(&x); };
    auto word = [](__nv_bfloat162 x) { return *reinterpret_cast<const uint32_t*>(&x); };
#pragma unroll
    for (uint32_t s = kChunks; s < 32; s <<= 1) {
#pragma unroll
      for (int z = 0; z < 8; ++z) {
        hi[z] = word(__hmax2_nan(bf(hi[z]), bf(__shfl_xor_sync(0xFFFFFFFFu, hi[z], s))));
        lo[z] = word(__hmin2_nan(bf(lo[z]), bf(__shfl_xor_sync(0xFFFFFFFFu, lo[z], s))));
      }
    }
    if (row == 0) {
      uint32_t h4[4], l4[4];
#pragma unroll
      for (int z = 0; z < 4; ++z) codes_of(hi + 2 * z, lo + 2 * z, h4 + z, l4 + z);
      st16(to, make_uint4(h4[0], h4[1], h4[2], h4[3]));
      st16(to + kD, make_uint4(l4[0], l4[1], l4[2], l4[3]));
    }
  }
}

// ------------------------------------------------------------------- scores
// The product's rows are 16 blocks, a tile, and its columns eight query rows (query, head).  The tiles of every (request, kv
// head, queries that fit shared memory) are laid end to end and cut into one share a CTA; a CTA
// stages a segment's query rows once, and then its warps go over its tiles without waiting for one another, each with the
// next tile's bounds on their way into a ring of its own.  Lane (g, p) = (lane / 4, lane % 4) takes as the k of its fragments
// 16 consecutive channels, the 16 bytes of one copy, and copies what itself will read; the query rows in shared memory
// are read alike (sums over k may run in any order).  One query fragment serves both halves of the product: as max(q, 0)
// against hi and as min(q, 0) against lo.  From 256 channels on a block's channels are split over the warps of a set, which
// add their sums through shared memory.  Conversions and products bound it: a chunk of 128 channels takes 135 us where the 5th-generation
// tensor cores take 37.5 (see the launch).  What it is for: 64 requests of up to 16384 latent entries of 512 channels, one query of 64 heads each, 34 us
// (13 MB), of 128 heads 57; 2475 queries of 64 heads over such a cache 787 (50 GF), 1993 queries of 16 heads over four of 256 channels 95 (12 GF),
// of 128 heads over one of 128 channels 374 (47 GF).
constexpr int kScoreWarps = 8;
constexpr int kScoreThreads = 32 * kScoreWarps;
constexpr uint32_t kTileBlocks = 16;

// The requests, the tiles before each, and those of all.
__device__ __forceinline__ unsigned long long scan_tiles(const ScoreArgs& a, uint32_t* s_q, BlockReq* s_req, unsigned long long* s_tile,
                                                         unsigned long long* s_scan) {
  scan_queries<kScoreThreads>(a.r, s_q, s_req, s_scan);
  const uint32_t t_shift = __ffs(a.c.block_tokens) - 1;
  unsigned long long total = 0;
  for (uint32_t b0 = 0; b0 < a.r.batch; b0 += kScoreThreads) {
    const uint32_t b = b0 + threadIdx.x;
    unsigned long long n = 0;
    if (b < a.r.batch)
      n = static_cast<unsigned long long>((s_req[b].q_len + a.queries - 1) / a.queries) * a.c.heads * score_tiles<kTileBlocks>(s_req[b], a.r.ratio, t_shift);
    unsigned long long sum;
    const unsigned long long at = total + block_exclusive<kScoreThreads>(n, &sum, s_scan);
    if (b < a.r.batch) s_tile[b] = at;
    total += sum;
  }
  __syncthreads();
  return total;
}

// Few query rows (a decode step): a segment is a (request, kv head, eight query rows), and a share is a warp's, so that
// nothing waits for a CTA.  The query rows are fragments in registers; a warp's ring holds the bounds of three steps, a step
// being up to 128 channels of a tile.  The bounds' bytes and the way of one step bound it: 69 MB (64 requests of up to 65536 entries,
// eight kv heads of 128 channels) in 20.8 us, 3.3 TB/s; with a CTA's segments instead of a warp's 54 us.
template <int kD>
struct FewCfg {
  static constexpr int kDw = kD < 128 ? kD : 128;
  static constexpr int kParts = kD / kDw;
  static constexpr int kStages = 3;
  static constexpr uint32_t kCopies = kDw / 16;  // of 16 bytes, of a lane: kDw / 64 of two blocks and of two sides
  static constexpr uint32_t kStage = kCopies * 512 + 256;  // and two scales
  static constexpr uint32_t kRing = kScoreWarps * kStages * kStage;
  static uint32_t smem(uint32_t batch) { return kRing + batch * (8 + 16 + 4); }
};

// A place in the segments laid end to end.
struct ScorePlace {
  uint32_t b, h, i0, tile, tiles;  // request, kv head, its segment's first query, tile of a segment
};

template <int kD>
__global__ __launch_bounds__(kScoreThreads, 2) void q8_score_few_kernel(const ScoreArgs a) {
  using C = FewCfg<kD>;
  constexpr int kDw = C::kDw;
  extern __shared__ __align__(16) uint8_t smem[];
  BlockReq* s_req = reinterpret_cast<BlockReq*>(smem + C::kRing);
  unsigned long long* s_tile = reinterpret_cast<unsigned long long*>(s_req + a.r.batch);
  uint32_t* s_q = reinterpret_cast<uint32_t*>(s_tile + a.r.batch);
  __shared__ unsigned long long s_scan[kScoreThreads / 32 + 1];
  pdl_wait();
  pdl_release();
  const unsigned long long total = scan_tiles(a, s_q, s_req, s_tile, s_scan);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, p = lane & 3;
  const uint32_t H = a.c.heads, T = a.c.block_tokens, G = a.group, t_shift = __ffs(T) - 1, span_shift = __ffs(a.span) - 1;
  const unsigned long long warps = static_cast<unsigned long long>(gridDim.x) * kScoreWarps;
  const unsigned long long share = (total + warps - 1) / warps;
  const unsigned long long begin = (static_cast<unsigned long long>(blockIdx.x) * kScoreWarps + warp) * share;
  uint32_t left = begin < total ? static_cast<uint32_t>(min(share, total - begin)) : 0;  // tiles of this warp
  if (left > 0) {
    ScorePlace at;
    at.b = last_not_above(s_tile, a.r.batch, begin);
    {
      const BlockReq req = s_req[at.b];
      at.tiles = score_tiles<kTileBlocks>(req, a.r.ratio, t_shift);
      const unsigned long long rel = begin - s_tile[at.b], seg = rel / at.tiles;
      const uint32_t chunks = (req.q_len + a.queries - 1) / a.queries;
      at.tile = static_cast<uint32_t>(rel - seg * at.tiles);
      at.h = static_cast<uint32_t>(seg / chunks);
      at.i0 = static_cast<uint32_t>(seg % chunks) * a.queries;
    }
    auto next = [&](ScorePlace& x) {
      if (++x.tile < x.tiles) return;
      x.tile = 0;
      x.i0 += a.queries;
      if (x.i0 < s_req[x.b].q_len) return;
      x.i0 = 0;
      if (++x.h < H) return;
      x.h = 0;
      do ++x.b;
      while (x.b < a.r.batch && (x.tiles = score_tiles<kTileBlocks>(s_req[x.b], a.r.ratio, t_shift)) == 0);
    };
    // ---- copies, two steps ahead
    const uint32_t ring = smem_addr(smem) + warp * C::kStages * C::kStage;
    ScorePlace to = at;
    uint32_t to_left = left, to_part = 0, to_stage = 0;
    int32_t blk[2];
    bool here[2];
    auto look_up = [&]() {  // the block numbers of tile `to`
      const uint32_t b = to_left ? to.b : at.b;
      const BlockReq req = s_req[b];
      const uint32_t blocks = (seen_by(req, req.q_len - 1, a.r.ratio) + T - 1) >> t_shift;
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const uint32_t j = to.tile * kTileBlocks + g + 8 * r;
        here[r] = to_left && j < blocks;
        blk[r] = here[r] ? ld_ahead(a.table + static_cast<size_t>(req.rid) * a.stride + j) : -1;
      }
    };
    auto issue = [&]() {
      if (to_left) {
        const uint32_t dst = ring + to_stage * C::kStage;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const bool ok = static_cast<uint32_t>(blk[r]) < a.c.num_blocks;
          if (here[r] && !ok && p == 0 && to_part == 0) status_or(a.r.d_status, CKV_STATUS_BAD_INDEX);
          const size_t bh = static_cast<size_t>(ok ? blk[r] : 0) * H + to.h;
          const uint8_t* from = a.bounds + bh * 2 * kD + to_part * kDw + p * 16;
          const uint32_t n = ok ? 16u : 0u;
#pragma unroll
          for (int side = 0; side < 2; ++side) {
#pragma unroll
            for (int c = 0; c < kDw / 64; ++c)
              cp_async16(dst + ((side * 2 + r) * (kDw / 64) + c) * 512 + lane * 16, from + side * kD + c * 64, n);
          }
          const uint32_t ks = dst + C::kCopies * 512 + r * 128 + lane * 4;
          if (ok)
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(ks), "l"(a.c.k_scale + bh) : "memory");
          else
            asm volatile("st.shared.f32 [%0], %1;" ::"r"(ks), "f"(-1.0f) : "memory");
        }
        to_stage = to_stage + 1 == C::kStages ? 0 : to_stage + 1;
        if (++to_part == C::kParts) {
          to_part = 0;
          if (--to_left) next(to);
          look_up();
        }
      }
      cp_async_commit();
    };
    look_up();
    issue();
    issue();
    // ---- tiles
    uint32_t qf[kD / 16][2];  // this lane's row, as fp16
    float f[2];               // what undoes the scaling of rows 2p and 2p + 1; 0: no such row
    uint32_t lim[2] = {0, 0};    // blocks that the queries of those rows see
    float* out = nullptr;        // where the first one's scores go
    bool fresh = true;
    uint32_t stage = 0;
    for (; left > 0; --left) {
      if (fresh) {  // another segment's query rows
        const BlockReq req = s_req[at.b];
        const uint32_t i1 = min(req.q_len, at.i0 + a.queries);
        const uint32_t i = at.i0 + (g >> span_shift), head = g & (a.span - 1);
        const bool in = i < i1 && head < G;
        const __nv_bfloat16* src = a.q + (static_cast<size_t>(s_q[at.b] + (in ? i : at.i0)) * a.n_heads + at.h * G + (in ? head : 0)) * kD + p * 16;
        float m = 0.0f;
#pragma unroll 2
        for (int c = 0; c < kD / 64; ++c) {
          const uint4 x = ld_stream16_if(src + c * 64, in), y = ld_stream16_if(src + c * 64 + 8, in);
#pragma unroll
          for (int e = 0; e < 8; ++e) m = fmaxf(m, fmaxf(fabsf(unpack<__nv_bfloat16>(x, e)), fabsf(unpack<__nv_bfloat16>(y, e))));
        }
        m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
        m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
        const int ex = min(126, 14 - (static_cast<int>(__float_as_uint(m) >> 23) - 127));
        const float up = pow2f(ex), back = in ? row_factor(a, ex) : 0.0f;
#pragma unroll
        for (int c = 0; c < kD / 64; ++c) {  // loaded again: 128 registers would hold a row's 512 channels
          const uint4 x[2] = {ld_stream16_if(src + c * 64, in), ld_stream16_if(src + c * 64 + 8, in)};
#pragma unroll
          for (int z = 0; z < 4; ++z) {
#pragma unroll
            for (int y = 0; y < 2; ++y)
              qf[4 * c + z][y] = pack_f16x2(unpack<__nv_bfloat16>(x[z >> 1], (z & 1) * 4 + 2 * y) * up,
                                            unpack<__nv_bfloat16>(x[z >> 1], (z & 1) * 4 + 2 * y + 1) * up);
          }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          f[e] = __shfl_sync(0xFFFFFFFFu, back, (2 * p + e) * 4);
          const uint32_t n = at.i0 + ((2 * p + e) >> span_shift);
          lim[e] = ((2 * p + e) & (a.span - 1)) == 0 && n < i1 ? (seen_by(req, n, a.r.ratio) + T - 1) >> t_shift : 0xFFFFFFFFu;
        }
        out = a.scores + (static_cast<size_t>(s_q[at.b] + at.i0 + (2 * p >> span_shift)) * H + at.h) * a.width;
      }
      float s[2][4] = {};  // against hi and lo: blocks g (0, 1) and g + 8 (2, 3), rows 2p and 2p + 1
      float ks[2];
#pragma unroll
      for (int part = 0; part < C::kParts; ++part) {
        issue();
        cp_async_wait<2>();  // a lane reads what itself has copied: nothing else is waited for
        const uint32_t st = ring + stage * C::kStage + lane * 16;
        stage = stage + 1 == C::kStages ? 0 : stage + 1;
#pragma unroll
        for (int c = 0; c < kDw / 64; ++c) {
#pragma unroll
          for (int side = 0; side < 2; ++side) {
            const uint4 v = lds16(st + (side * 2 * (kDw / 64) + c) * 512), w = lds16(st + ((side * 2 + 1) * (kDw / 64) + c) * 512);
            const uint32_t x0[4] = {v.x, v.y, v.z, v.w}, x1[4] = {w.x, w.y, w.z, w.w};
            const __half2 zero = __float2half2_rn(0.0f);
#pragma unroll
            for (int z = 0; z < 4; ++z) {
              const uint32_t af[4] = {q8_lo_f16x2(x0[z]), q8_lo_f16x2(x1[z]), q8_hi_f16x2(x0[z]), q8_hi_f16x2(x1[z])};
              const __half2 q0 = as_half2(qf[part * (kDw / 16) + 4 * c + z][0]), q1 = as_half2(qf[part * (kDw / 16) + 4 * c + z][1]);
              if (side == 0)
                mma_f16(s[0], af, as_u32(__hmax2_nan(q0, zero)), as_u32(__hmax2_nan(q1, zero)));
              else
                mma_f16(s[1], af, as_u32(__hmin2_nan(q0, zero)), as_u32(__hmin2_nan(q1, zero)));
            }
          }
        }
        if (part == C::kParts - 1) {
#pragma unroll
          for (int r = 0; r < 2; ++r) asm volatile("ld.shared.f32 %0, [%1];" : "=f"(ks[r]) : "r"(st - lane * 12 + C::kCopies * 512 + r * 128) : "memory");
        }
      }
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float k = ks[r] * a.scale;
        float x0 = f[0] != 0.0f ? (s[0][2 * r] + s[1][2 * r]) * f[0] * k : -INFINITY;
        float x1 = f[1] != 0.0f ? (s[0][2 * r + 1] + s[1][2 * r + 1]) * f[1] * k : -INFINITY;
        const uint32_t j = at.tile * kTileBlocks + g + 8 * r;
        auto put = [&](float* to_row, uint32_t limit, float v) {
          if (limit != 0xFFFFFFFFu && j < a.width) to_row[j] = j < limit && ks[r] > 0.0f ? v : -INFINITY;
        };
        if (a.span > 1) {
          x0 = max_nan(x0, x1);
          if (a.span > 2) x0 = max_nan(x0, __shfl_xor_sync(0xFFFFFFFFu, x0, 1));
          if (a.span > 4) x0 = max_nan(x0, __shfl_xor_sync(0xFFFFFFFFu, x0, 2));
        } else {
          put(out + static_cast<size_t>(H) * a.width, lim[1], x1);
        }
        put(out, lim[0], x0);
      }
      const uint32_t b = at.b, h = at.h, i0 = at.i0;
      if (left > 1) next(at);
      fresh = at.b != b || at.h != h || at.i0 != i0;
    }
    cp_async_wait<0>();
  }
  fill_behind<kTileBlocks>(a, s_q, s_req);
}

template <int kD>
struct ScoreCfg {
  static constexpr int kNp = kD > 128 ? kD / 128 : 1;  // warps that share a block's channels
  static constexpr int kDw = kD / kNp;
  static constexpr int kSets = kScoreWarps / kNp;
  static constexpr int kCopies = kDw / 16;  // 16-byte copies of a lane: kDw / 64 of two blocks and of two sides
  static constexpr uint32_t kStage = kCopies * 512;
  static constexpr uint32_t kRing = kScoreWarps * 2 * kStage;
  static constexpr uint32_t kRowBytes = kD * 2 + 16;  // of a query row: rows of a fragment start 16 bytes apart modulo 128
  static constexpr uint32_t kMost = 218 * 1024;  // of 227 KB; sums of split channels take 8
  static uint32_t smem(uint32_t rows, uint32_t batch) { return kRing + rows * kRowBytes + rows * 8 + batch * (8 + 16 + 4); }
};

template <int kD>
__global__ __launch_bounds__(kScoreThreads, 2) void q8_score_kernel(const ScoreArgs a) {
  using C = ScoreCfg<kD>;
  constexpr int kNp = C::kNp, kDw = C::kDw;
  extern __shared__ __align__(16) uint8_t smem[];
  uint8_t* s_rows = smem + C::kRing;
  BlockReq* s_req = reinterpret_cast<BlockReq*>(s_rows + a.rows * C::kRowBytes);
  unsigned long long* s_tile = reinterpret_cast<unsigned long long*>(s_req + a.r.batch);  // tiles before each request
  uint32_t* s_q = reinterpret_cast<uint32_t*>(s_tile + a.r.batch);
  float* s_rf = reinterpret_cast<float*>(s_q + a.r.batch);      // of each row: what undoes its scaling, 0: no such row,
  uint32_t* s_lim = reinterpret_cast<uint32_t*>(s_rf + a.rows);  // and blocks that its query sees
  __shared__ unsigned long long s_scan[kScoreThreads / 32 + 1];
  __shared__ __align__(16) float s_part[kNp > 1 ? 2 : 1][kNp > 1 ? kScoreWarps : 1][kNp > 1 ? 128 : 1];
  pdl_wait();
  pdl_release();
  const unsigned long long total = scan_tiles(a, s_q, s_req, s_tile, s_scan);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, p = lane & 3, set = warp / kNp, part = warp % kNp;
  const uint32_t H = a.c.heads, T = a.c.block_tokens, G = a.group, t_shift = __ffs(T) - 1;
  const uint32_t span_shift = (a.span & (a.span - 1)) == 0 ? __ffs(a.span) - 1 : 32;  // 32: not a power of two
  // this CTA's share
  unsigned long long share = (total + gridDim.x - 1) / gridDim.x;
  share = (share + C::kSets - 1) / C::kSets * C::kSets;
  const unsigned long long end = min(total, (blockIdx.x + 1) * share);
  const uint32_t ring = smem_addr(smem) + warp * 2 * C::kStage + lane * 16;
  for (unsigned long long pos = blockIdx.x * share; pos < end;) {
    const uint32_t b = last_not_above(s_tile, a.r.batch, pos);
    const BlockReq req = s_req[b];
    const uint32_t q0 = s_q[b], tiles = score_tiles<kTileBlocks>(req, a.r.ratio, t_shift), chunks = (req.q_len + a.queries - 1) / a.queries;
    const unsigned long long rel = pos - s_tile[b], seg = rel / tiles;
    const uint32_t tile0 = static_cast<uint32_t>(rel - seg * tiles);
    const uint32_t tile1 = static_cast<uint32_t>(min(static_cast<unsigned long long>(tiles), tile0 + (end - pos)));
    const uint32_t h = static_cast<uint32_t>(seg / chunks), i0 = static_cast<uint32_t>(seg % chunks) * a.queries;
    const uint32_t i1 = min(req.q_len, i0 + a.queries);
    const int32_t* table = a.table + static_cast<size_t>(req.rid) * a.stride;
    pos += tile1 - tile0;
    auto blocks_of = [&](uint32_t i) { return (seen_by(req, i, a.r.ratio) + T - 1) >> t_shift; };
    const uint32_t most = blocks_of(i1 - 1);  // later queries see no less
    for (uint32_t piece = 0; piece < a.parts; ++piece) {
      const uint32_t r0 = piece * a.rows, rows = min(a.rows, (i1 - i0) * a.span - r0);
      // ---- the first tile's bounds are asked for; the block numbers a tile ahead of that
      auto block_at = [&](uint32_t tile, int r) -> int32_t {
        const uint32_t j = tile * kTileBlocks + g + 8 * r;
        return tile < tile1 && j < most ? ld_ahead(table + j) : -1;
      };
      int32_t blk[2], ahead[2];  // of the tile that is copied, and of the one behind it
      float ks_next[2], ks[2];
      bool ok_next[2], ok[2];
      auto issue = [&](uint32_t tile, uint32_t stage) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const uint32_t j = tile * kTileBlocks + g + 8 * r;
          ok_next[r] = static_cast<uint32_t>(blk[r]) < a.c.num_blocks;
          if (tile < tile1 && j < most && !ok_next[r] && part == 0 && p == 0) status_or(a.r.d_status, CKV_STATUS_BAD_INDEX);
          const size_t bh = static_cast<size_t>(ok_next[r] ? blk[r] : 0) * H + h;
          ks_next[r] = ld_ahead(a.c.k_scale + bh);
          const uint8_t* from = a.bounds + bh * 2 * kD + part * kDw + p * 16;
          const uint32_t to = ring + stage * C::kStage, n = ok_next[r] ? 16u : 0u;
#pragma unroll
          for (int side = 0; side < 2; ++side) {
#pragma unroll
            for (int c = 0; c < kDw / 64; ++c) cp_async16(to + ((side * 2 + r) * (kDw / 64) + c) * 512, from + side * kD + c * 64, n);
          }
        }
        cp_async_commit();
      };
      const uint32_t mine = tile0 + set;
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        blk[r] = block_at(mine, r);
        ahead[r] = block_at(mine + C::kSets, r);
      }
      issue(mine, 0);
      // ---- query rows as fp16
      __syncthreads();  // the rows before are read
      for (uint32_t r = warp; r < (rows + 7) / 8 * 8; r += kScoreWarps) {
        const uint32_t i = i0 + (r0 + r) / a.span, head = (r0 + r) % a.span;
        const bool in = r < rows && i < i1 && head < G;
        constexpr int kPer = kD / 32;  // consecutive channels of a lane
        const __nv_bfloat16* src = a.q + (static_cast<size_t>(q0 + i) * a.n_heads + h * G + head) * kD + lane * kPer;
        float v[kPer];
        if constexpr (kPer == 2) {
          const uint32_t w = in ? __ldg(reinterpret_cast<const uint32_t*>(src)) : 0;
          v[0] = bf16lo(w);
          v[1] = bf16hi(w);
        } else if constexpr (kPer == 4) {
          const uint2 w = in ? __ldg(reinterpret_cast<const uint2*>(src)) : make_uint2(0, 0);
          v[0] = bf16lo(w.x);
          v[1] = bf16hi(w.x);
          v[2] = bf16lo(w.y);
          v[3] = bf16hi(w.y);
        } else {
#pragma unroll
          for (int e = 0; e < kPer / 8; ++e) {
            const uint4 w = in ? ld_cached16(src + 8 * e) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int z = 0; z < 8; ++z) v[8 * e + z] = unpack<__nv_bfloat16>(w, z);
          }
        }
        float m = 0.0f;
#pragma unroll
        for (int z = 0; z < kPer; ++z) m = fmaxf(m, fabsf(v[z]));
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, s));
        const int ex = min(126, 14 - (static_cast<int>(__float_as_uint(m) >> 23) - 127));
        const float up = pow2f(ex);
#pragma unroll
        for (int z = 0; z < kPer; z += 2)
          *reinterpret_cast<uint32_t*>(s_rows + r * C::kRowBytes + (lane * kPer + z) * 2) = pack_f16x2(v[z] * up, v[z + 1] * up);
        if (lane == 0) {
          s_rf[r] = in ? row_factor(a, ex) : 0.0f;
          s_lim[r] = i < i1 ? blocks_of(i) : 0xFFFFFFFFu;
        }
      }
      __syncthreads();
      // ---- tiles
      uint32_t stage = 0;
      for (uint32_t tile = mine; tile < tile1; tile += C::kSets, stage ^= 1) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          ks[r] = ks_next[r];
          ok[r] = ok_next[r];
          blk[r] = ahead[r];
          ahead[r] = block_at(tile + 2 * C::kSets, r);
        }
        issue(tile + C::kSets, stage ^ 1);
        cp_async_wait<1>();  // a lane reads what itself has copied: nothing else is waited for
        uint32_t af[2][kDw / 16][4];  // hi and lo
#pragma unroll
        for (int side = 0; side < 2; ++side) {
#pragma unroll
          for (int c = 0; c < kDw / 64; ++c) {
            const uint4 v = lds16(ring + stage * C::kStage + (side * 2 * (kDw / 64) + c) * 512);
            const uint4 w = lds16(ring + stage * C::kStage + ((side * 2 + 1) * (kDw / 64) + c) * 512);
            const uint32_t x0[4] = {v.x, v.y, v.z, v.w}, x1[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int z = 0; z < 4; ++z) {
              af[side][4 * c + z][0] = q8_lo_f16x2(x0[z]);
              af[side][4 * c + z][1] = q8_lo_f16x2(x1[z]);
              af[side][4 * c + z][2] = q8_hi_f16x2(x0[z]);
              af[side][4 * c + z][3] = q8_hi_f16x2(x1[z]);
            }
          }
        }
        float top[2] = {-INFINITY, -INFINITY};  // groups of more than eight heads: over the rows of a query so far
        for (uint32_t t = 0; t < rows; t += 8) {
          float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};  // blocks g (0, 1) and g + 8 (2, 3), rows 2p and 2p + 1
          const uint8_t* row = s_rows + (t + g) * C::kRowBytes + (part * kDw + p * 16) * 2;
#pragma unroll
          for (int c = 0; c < kDw / 64; ++c) {
            const uint4 v = *reinterpret_cast<const uint4*>(row + c * 128), w = *reinterpret_cast<const uint4*>(row + c * 128 + 16);
            const uint32_t q[8] = {v.x, v.y, v.z, v.w, w.x, w.y, w.z, w.w};
            const __half2 zero = __float2half2_rn(0.0f);
#pragma unroll
            for (int z = 0; z < 4; ++z) {
              mma_f16(s, af[0][4 * c + z], as_u32(__hmax2_nan(as_half2(q[2 * z]), zero)), as_u32(__hmax2_nan(as_half2(q[2 * z + 1]), zero)));
              mma_f16(s, af[1][4 * c + z], as_u32(__hmin2_nan(as_half2(q[2 * z]), zero)), as_u32(__hmin2_nan(as_half2(q[2 * z + 1]), zero)));
            }
          }
          // where channels are split, warp `part` of a set finishes blocks g + 8 part
          constexpr int kMine = kNp > 1 ? 1 : 2;
          if constexpr (kNp > 1) {
            const uint32_t flip = (t >> 3) & 1;
            *reinterpret_cast<float4*>(&s_part[flip][warp][lane * 4]) = make_float4(s[0], s[1], s[2], s[3]);
            asm volatile("bar.sync %0, %1;" ::"r"(1 + set), "n"(32 * kNp) : "memory");
            if (part >= 2) continue;
            float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int w = 0; w < kNp; ++w) {
              const float2 y = *reinterpret_cast<const float2*>(&s_part[flip][set * kNp + w][lane * 4 + 2 * part]);
              sum.x += y.x;
              sum.y += y.y;
            }
            s[0] = sum.x;
            s[1] = sum.y;
          }
          const float f0 = s_rf[t + 2 * p], f1 = s_rf[t + 2 * p + 1];
          const uint32_t span = min(a.span, 8u);
#pragma unroll
          for (int r = 0; r < kMine; ++r) {
            const int at = kNp > 1 ? part : r;  // of the lane's two blocks
            const float k = (at ? ks[1] : ks[0]) * a.scale;
            const bool held = at ? ok[1] : ok[0];
            float x0 = f0 != 0.0f && held ? s[2 * r] * f0 * k : -INFINITY;
            float x1 = f1 != 0.0f && held ? s[2 * r + 1] * f1 * k : -INFINITY;
            const uint32_t j = tile * kTileBlocks + g + 8 * at;
            auto put = [&](uint32_t row, float v) {  // of this piece
              const uint32_t limit = s_lim[row];
              if (limit == 0xFFFFFFFFu || j >= a.width) return;
              const uint32_t i = i0 + (span_shift < 32 ? (r0 + row) >> span_shift : (r0 + row) / a.span);
              float* to = a.scores + (static_cast<size_t>(q0 + i) * H + h) * a.width + j;
              if (j >= limit) v = -INFINITY;
              if (piece > 0) v = max_nan(v, *to);  // what this lane wrote for the query's other heads
              *to = v;
            };
            if (span == 1) {
              put(t + 2 * p, x0);
              put(t + 2 * p + 1, x1);
              continue;
            }
            x0 = max_nan(x0, x1);
            if (span > 2) x0 = max_nan(x0, __shfl_xor_sync(0xFFFFFFFFu, x0, 1));
            if (span > 4) x0 = max_nan(x0, __shfl_xor_sync(0xFFFFFFFFu, x0, 2));
            if (a.span > 8) {
              top[r] = max_nan(top[r], x0);
              if ((span_shift < 32 ? (r0 + t + 8) & (a.span - 1) : (r0 + t + 8) % a.span) != 0 && t + 8 < rows) continue;
              x0 = top[r];
              top[r] = -INFINITY;
            }
            if (((2 * p) & (span - 1)) == 0) put(t + 2 * p, x0);
          }
        }
        // the next tile's sums come after every warp of the set has read this one's
        if (kNp > 1) asm volatile("bar.sync %0, %1;" ::"r"(1 + set), "n"(32 * kNp) : "memory");
      }
      cp_async_wait<0>();
    }
  }
  fill_behind<kTileBlocks>(a, s_q, s_req);
}

template <int kD>
int launch_scores(ScoreArgs a, cudaStream_t s) {
  using C = ScoreCfg<kD>;
  // Up to eight heads to a kv head, so that a segment's rows are whole queries (a batch may have fewer queries than requests), and up to eight rows
  // a request on average.  us of this kernel / of the one that takes more rows, four heads to a kv head, contexts of up to 32768 entries: 128 channels, 64
  // requests 15 / 51 at 8 rows, 42 / 50 at 32, 58 / 50 at 48, one request 6.1 / 9.0 at 8 and 9.3 / 9.5 at 128; 256 channels at 8 rows, 64 requests 11.1 / 14.6, one
  // 6.5 / 5.7; 512 channels 19 / 27 and 9.9 / 5.4.  So equal requests cross at some 40 rows; but one kernel takes a whole batch, and this one reads a request's bounds again
  // for every eight of its rows: 255 single tokens of 1024 entries beside a chunk of 257 queries that see 65536, eight rows on average, take 68 / 90,
  // 64 of them beside 256 such queries, twenty on average, 66 / 37.  (Chunks no longer than the rest: 200 tokens beside 512 queries of 8192 entries 37 / 68.)
  if (a.span <= 8 && static_cast<uint64_t>(a.r.num_q) * a.span <= 8ull * a.r.batch) {
    static std::atomic<uint64_t> few_done;
    auto* few = q8_score_few_kernel<kD>;
    const int rc = allow_smem(reinterpret_cast<const void*>(few), FewCfg<kD>::smem(CKV_MAX_BATCH), few_done);
    if (rc) return rc;
    a.queries = 8 / a.span;
    return launch_pdl(few, dim3(2 * sm_count()), dim3(kScoreThreads), FewCfg<kD>::smem(a.r.batch), s, a);
  }
  static std::atomic<uint64_t> done;
  auto* kernel = q8_score_kernel<kD>;
  // The tensor-core kernel takes 128 query rows at nearly the cost of sixteen (32 requests of up to 512 blocks, 8 kv heads of 128
  // channels, us of q8_score_kernel / there: 31.5 / 27.6 at 12 rows a request, 47 / 27.7 at 32, 85 / 28.8 at 64; one request of 1024 blocks 7.9 / 8.8
  // at 16 and 14.7 / 9.0 at 64; 64 channels 26.8 / 22.2 at 16).
  if constexpr (kD <= 128) {
    if (a.group <= 64) return launch_q8_score_tc(a, s);
  }
  // 64 query rows let two CTAs share an SM; up to 128 where a query has more
  a.rows = a.span <= 64 ? 64 / a.span * a.span : std::min<uint32_t>(128, a.span);
  if (C::smem(a.rows, a.r.batch) > C::kMost) a.rows = 64;  // 512 channels, and a batch near the largest
  a.queries = std::max<uint32_t>(1, a.rows / a.span);
  a.parts = (a.span + a.rows - 1) / a.rows;
  const int rc = allow_smem(reinterpret_cast<const void*>(kernel), C::kMost, done);
  if (rc) return rc;
  return launch_pdl(kernel, dim3(2 * sm_count()), dim3(kScoreThreads), C::smem(a.rows, a.r.batch), s, a);
}

}  // namespace
}  // namespace ckv

using namespace ckv;

extern "C" {

int ckv_q8_bounds(const ckv_q8_cache_t* cache, void* bounds, const int64_t* rid, const int64_t* kv_lens,
                  const int64_t* new_lens, uint32_t batch, const int32_t* block_table, uint64_t table_stride,
                  uint32_t num_reqs, uint32_t* d_status, ckv_stream_t stream) {
  BoundArgs a{};
  int rc = q8_cache_of(cache, &a.c);
  if (rc) return rc;
  if (batch > CKV_MAX_BATCH) return CKV_ERR_SIZE;
  if (batch == 0) return CKV_OK;
  rc = check_table(block_table, table_stride, num_reqs);
  if (rc) return rc;
  if (!aligned16(bounds) || !aligned_to(rid, 8) || !aligned_to(kv_lens, 8) || !aligned_to(new_lens, 8)) return CKV_ERR_POINTER;
  a.bounds = static_cast<uint8_t*>(bounds);
  a.rid = rid;
  a.kv_lens = kv_lens;
  a.new_lens = new_lens;
  a.batch = batch;
  a.table = block_table;
  a.stride = static_cast<uint32_t>(table_stride);
  a.num_reqs = num_reqs;
  a.d_status = d_status;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  // at most what fits the card at once; no more warps than the table has blocks of the batch
  const uint64_t most = (static_cast<uint64_t>(batch) * table_stride * a.c.heads + kBoundThreads / 32 - 1) / (kBoundThreads / 32);
  const dim3 grid(static_cast<uint32_t>(std::min<uint64_t>(most, 4ull * sm_count())));
  switch (a.c.head_dim) {
    case 64: return launch_pdl(q8_bounds_kernel<64>, grid, dim3(kBoundThreads), 0, s, a);
    case 128: return launch_pdl(q8_bounds_kernel<128>, grid, dim3(kBoundThreads), 0, s, a);
    case 256: return launch_pdl(q8_bounds_kernel<256>, grid, dim3(kBoundThreads), 0, s, a);
    default: return launch_pdl(q8_bounds_kernel<512>, grid, dim3(kBoundThreads), 0, s, a);
  }
}

int ckv_q8_block_scores(const ckv_q8_cache_t* cache, const void* bounds, uint32_t n_heads, uint32_t ratio, float scale,
                        const void* q, uint32_t num_q, const int64_t* rid, const int64_t* seq_lens,
                        const int64_t* extend_lens, const int64_t* kv_lens, uint32_t batch, const int32_t* block_table,
                        uint64_t table_stride, uint32_t num_reqs, uint32_t width, float* scores, uint32_t* d_status,
                        ckv_stream_t stream) {
  ScoreArgs a{};
  int rc = q8_cache_of(cache, &a.c);
  if (rc) return rc;
  if (!(scale > 0.0f) || !(scale < 1e30f)) return CKV_ERR_SIZE;
  if (num_q > CKV_MAX_TOKENS || n_heads == 0 || n_heads % a.c.heads != 0 || n_heads / a.c.heads > CKV_Q8_MAX_GROUP) return CKV_ERR_SIZE;
  if (width == 0 || width > 0x7FFFFFFFu) return CKV_ERR_SIZE;
  rc = check_lens(batch, ratio, seq_lens, extend_lens, kv_lens);
  if (rc) return rc;
  if (num_q == 0 || batch == 0) return CKV_OK;
  rc = check_table(block_table, table_stride, num_reqs);
  if (rc) return rc;
  if (!aligned16(bounds) || !aligned16(q) || !aligned_to(rid, 8) || !aligned_to(scores, 4)) return CKV_ERR_POINTER;
  const int64_t most = static_cast<int64_t>(std::min<uint64_t>(width, table_stride)) * a.c.block_tokens;
  a.r = {rid, seq_lens, extend_lens, kv_lens, batch, num_q, ratio, num_reqs, most, d_status};
  a.bounds = static_cast<const uint8_t*>(bounds);
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.n_heads = n_heads;
  a.group = n_heads / a.c.heads;
  a.span = 1;
  while (a.span < a.group && a.span < 8) a.span *= 2;
  if (a.group > 8) a.span = (a.group + 7) / 8 * 8;
  split_scale(scale, &a);
  a.table = block_table;
  a.stride = static_cast<uint32_t>(table_stride);
  a.width = width;
  a.scores = scores;
  a.wait_ns = wait_limit_ns();
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  switch (a.c.head_dim) {
    case 64: return launch_scores<64>(a, s);
    case 128: return launch_scores<128>(a, s);
    case 256: return launch_scores<256>(a, s);
    default: return launch_scores<512>(a, s);
  }
}

}  // extern "C"

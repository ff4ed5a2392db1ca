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

#include "q8_blocks.cuh"

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

__device__ __forceinline__ __half2 as_half2(uint32_t x) { return *reinterpret_cast<const __half2*>(&x); }
__device__ __forceinline__ uint32_t as_u32(__half2 x) { return *reinterpret_cast<const uint32_t*>(&x); }

// The e4m3 pairs that two fp16 pairs are (exact, NaN stays NaN).
__device__ __forceinline__ uint32_t e4m3_of(uint32_t lo, uint32_t hi) {
  uint16_t a, b;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(a) : "r"(lo));
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(b) : "r"(hi));
  return a | (static_cast<uint32_t>(b) << 16);
}

// A warp takes a (block, head): lane l holds 16 channels, chunk l % (kD / 16), of every (512 / kD)th entry.
template <int kD>
__global__ __launch_bounds__(kBoundThreads) void q8_bounds_kernel(const BoundArgs a) {
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
  const int lane = threadIdx.x & 31;
  const unsigned long long warps = static_cast<unsigned long long>(gridDim.x) * (kBoundThreads / 32);
  for (unsigned long long w = static_cast<unsigned long long>(blockIdx.x) * (kBoundThreads / 32) + (threadIdx.x >> 5); w < units * H;
       w += warps) {
    const unsigned long long u = w / H;
    const uint32_t h = static_cast<uint32_t>(w % H);
    const uint32_t b = last_not_above(s_unit, a.batch, u);
    const uint32_t j = s_first[b] + static_cast<uint32_t>(u - s_unit[b]);
    const int32_t block = __ldg(a.table + static_cast<size_t>(s_rid[b]) * a.stride + j);
    if (static_cast<uint32_t>(block) >= a.c.num_blocks) {
      if (lane == 0) status_or(a.d_status, CKV_STATUS_BAD_INDEX);
      continue;
    }
    const uint32_t n = min(T, s_len[b] - j * T), chunk = lane % kChunks, row = lane / kChunks;
    const uint8_t* k = a.c.k + (static_cast<size_t>(block) * H + h) * T * kD + chunk * 16;
    uint32_t hi[8], lo[8];  // fp16 pairs
#pragma unroll
    for (int z = 0; z < 8; ++z) {
      hi[z] = 0xFC00FC00u;  // -infinity
      lo[z] = 0x7C007C00u;
    }
#pragma unroll 8
    for (uint32_t r = row; r < n; r += kRows) {
      const uint4 v = ld_stream16(k + r * kD);
      const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int z = 0; z < 4; ++z) {
        const __half2 p = as_half2(q8_lo_f16x2(x[z])), q = as_half2(q8_hi_f16x2(x[z]));
        hi[2 * z] = as_u32(__hmax2_nan(as_half2(hi[2 * z]), p));
        lo[2 * z] = as_u32(__hmin2_nan(as_half2(lo[2 * z]), p));
        hi[2 * z + 1] = as_u32(__hmax2_nan(as_half2(hi[2 * z + 1]), q));
        lo[2 * z + 1] = as_u32(__hmin2_nan(as_half2(lo[2 * z + 1]), q));
      }
    }
#pragma unroll
    for (uint32_t s = kChunks; s < 32; s <<= 1) {
#pragma unroll
      for (int z = 0; z < 8; ++z) {
        hi[z] = as_u32(__hmax2_nan(as_half2(hi[z]), as_half2(__shfl_xor_sync(0xFFFFFFFFu, hi[z], s))));
        lo[z] = as_u32(__hmin2_nan(as_half2(lo[z]), as_half2(__shfl_xor_sync(0xFFFFFFFFu, lo[z], s))));
      }
    }
    if (row == 0) {
      uint8_t* to = a.bounds + (static_cast<size_t>(block) * H + h) * 2 * kD + chunk * 16;
      st16(to, make_uint4(e4m3_of(hi[0], hi[1]), e4m3_of(hi[2], hi[3]), e4m3_of(hi[4], hi[5]), e4m3_of(hi[6], hi[7])));
      st16(to + kD, make_uint4(e4m3_of(lo[0], lo[1]), e4m3_of(lo[2], lo[3]), e4m3_of(lo[4], lo[5]), e4m3_of(lo[6], lo[7])));
    }
  }
}

// ------------------------------------------------------------------- scores
// A CTA takes a run of blocks of a (request, kv head), and queries of it.  The product's rows are 16 blocks, a warp's for
// the unit's length, with their bounds as fp16 fragments in registers; its columns are eight query rows.
// Lane (g, p) = (lane / 4, lane % 4) takes as the k of its fragments 16 consecutive
// channels, the 16 bytes of one load, and the query rows in shared memory are read alike (sums over k may run in any order).  The same
// query fragment serves both halves of the product: as max(q, 0) against hi and as min(q, 0) against lo.  From
// 256 channels on a block's channels are split over the warps of a set, which add their sums through shared memory.
constexpr int kScoreWarps = 8;
constexpr int kScoreThreads = 32 * kScoreWarps;
constexpr uint32_t kStageRows = 64;  // query rows in shared memory at a time
constexpr uint32_t kUnitRows = 256;  // and of a unit

struct ScoreArgs {
  Q8Cache c;
  BlockReqs r;
  const uint8_t* bounds;
  const __nv_bfloat16* q;
  uint32_t n_heads, group;
  uint32_t span;     // rows that a query takes: the group, up to a power of two or a multiple of eight
  uint32_t queries;  // of a unit
  float scale;
  const int32_t* table;
  uint32_t stride;
  uint32_t width;
  float* scores;
};

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

template <int kD>
struct ScoreCfg {
  static constexpr int kNp = kD > 128 ? kD / 128 : 1;  // warps that share a block's channels
  static constexpr int kDw = kD / kNp;
  static constexpr int kSets = kScoreWarps / kNp;
  static constexpr uint32_t kRun = 16 * kSets;  // blocks of a unit
  static constexpr uint32_t kRowBytes = kD * 2 + 16;  // of a query row in shared memory: rows of a fragment start 16 bytes apart modulo 128
  static constexpr uint32_t kSmem = kStageRows * kRowBytes;
};

template <int kD>
__global__ __launch_bounds__(kScoreThreads) void q8_score_kernel(const ScoreArgs a) {
  using C = ScoreCfg<kD>;
  constexpr int kNp = C::kNp, kDw = C::kDw;
  extern __shared__ __align__(16) uint8_t s_rows[];
  __shared__ uint32_t s_q[CKV_MAX_BATCH];
  __shared__ BlockReq s_req[CKV_MAX_BATCH];
  __shared__ unsigned long long s_unit[CKV_MAX_BATCH];
  __shared__ unsigned long long s_scan[kScoreThreads / 32 + 1];
  __shared__ float s_rf[kStageRows];
  __shared__ __align__(16) float s_part[kNp > 1 ? 2 : 1][kNp > 1 ? kScoreWarps : 1][kNp > 1 ? 128 : 1];
  pdl_wait();
  pdl_release();
  scan_queries<kScoreThreads>(a.r, s_q, s_req, s_scan);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, p = lane & 3, set = warp / kNp, part = warp % kNp;
  const uint32_t H = a.c.heads, T = a.c.block_tokens, G = a.group, t_shift = __ffs(T) - 1;
  const uint32_t runs = (a.width + C::kRun - 1) / C::kRun;
  // units: by request, then head, queries and run
  unsigned long long units = 0;
  for (uint32_t b0 = 0; b0 < a.r.batch; b0 += kScoreThreads) {
    const uint32_t b = b0 + tid;
    const unsigned long long n =
        b < a.r.batch ? static_cast<unsigned long long>((s_req[b].q_len + a.queries - 1) / a.queries) * H * runs : 0;
    unsigned long long sum;
    const unsigned long long u0 = units + block_exclusive<kScoreThreads>(n, &sum, s_scan);
    if (b < a.r.batch) s_unit[b] = u0;
    units += sum;
  }
  __syncthreads();

  for (unsigned long long u = blockIdx.x; u < units; u += gridDim.x) {
    const uint32_t b = last_not_above(s_unit, a.r.batch, u);
    const BlockReq req = s_req[b];
    unsigned long long x = u - s_unit[b];
    const uint32_t run0 = static_cast<uint32_t>(x % runs) * C::kRun;
    x /= runs;
    const uint32_t chunks = (req.q_len + a.queries - 1) / a.queries;
    const uint32_t i0 = static_cast<uint32_t>(x % chunks) * a.queries, i1 = min(req.q_len, i0 + a.queries);
    const uint32_t h = static_cast<uint32_t>(x / chunks);
    auto row_at = [&](uint32_t i) { return a.scores + (static_cast<size_t>(s_q[b] + i) * H + h) * a.width; };
    auto blocks_of = [&](uint32_t i) { return (seen_by(req, i, a.r.ratio) + T - 1) >> t_shift; };
    const uint32_t most = blocks_of(i1 - 1);  // later queries see no less
    if (run0 >= most) {
      const uint32_t n = min(C::kRun, a.width - run0);
      for (uint32_t y = tid; y < (i1 - i0) * n; y += kScoreThreads) row_at(i0 + y / n)[run0 + y % n] = -INFINITY;
      continue;
    }
    // ---- this warp's 16 blocks: lane (g, p) holds those of rows g and g + 8
    uint32_t af[2][kDw / 16][4];  // hi and lo
    float ks[2];
    bool ok[2];
    {
      const uint8_t* at[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const uint32_t j = run0 + set * 16 + g + 8 * r;
        const int32_t blk = j < most ? __ldg(a.table + static_cast<size_t>(req.rid) * a.stride + j) : -1;
        ok[r] = static_cast<uint32_t>(blk) < a.c.num_blocks;
        if (j < most && !ok[r] && part == 0 && p == 0) status_or(a.r.d_status, CKV_STATUS_BAD_INDEX);
        const size_t bh = static_cast<size_t>(ok[r] ? blk : 0) * H + h;
        ks[r] = ok[r] ? __ldg(a.c.k_scale + bh) * a.scale : 0.0f;
        at[r] = a.bounds + bh * 2 * kD + part * kDw + p * 16;
      }
#pragma unroll
      for (int side = 0; side < 2; ++side) {
#pragma unroll
        for (int c = 0; c < kDw / 64; ++c) {
          const uint4 v = ld_stream16_if(at[0] + side * kD + c * 64, ok[0]), w = ld_stream16_if(at[1] + side * kD + c * 64, ok[1]);
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
    }
    float top[2] = {-INFINITY, -INFINITY};  // groups of more than eight heads: over the tiles of a query so far
    const uint32_t rows = (i1 - i0) * a.span;
    for (uint32_t r0 = 0; r0 < rows; r0 += kStageRows) {
      // ---- query rows as fp16
      __syncthreads();  // the rows before are read
      for (uint32_t r = warp; r < kStageRows; r += kScoreWarps) {
        const uint32_t i = i0 + (r0 + r) / a.span, head = (r0 + r) % a.span;
        const bool in = i < i1 && head < G;
        constexpr int kPer = kD / 32;  // consecutive channels of a lane
        const __nv_bfloat16* src = a.q + (static_cast<size_t>(s_q[b] + i) * a.n_heads + h * G + head) * kD + lane * kPer;
        float v[kPer];
        if (kPer == 2) {
          const uint32_t w = in ? __ldg(reinterpret_cast<const uint32_t*>(src)) : 0;
          v[0] = bf16lo(w);
          v[1] = bf16hi(w);
        } else if (kPer == 4) {
          const uint2 w = in ? __ldg(reinterpret_cast<const uint2*>(src)) : make_uint2(0, 0);
          v[0] = bf16lo(w.x);
          v[1 % kPer] = bf16hi(w.x);
          v[2 % kPer] = bf16lo(w.y);
          v[3 % kPer] = bf16hi(w.y);
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
        if (lane == 0) s_rf[r] = in ? pow2f(-ex) : 0.0f;  // 0: no such row
      }
      __syncthreads();
      // ---- products, eight rows at a time
      const uint32_t here = min(kStageRows, rows - r0);
      for (uint32_t t = 0; t < here; t += 8) {
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
        if (kNp > 1) {
          const uint32_t flip = (t >> 3) & 1;
          *reinterpret_cast<float4*>(&s_part[flip][warp][lane * 4 % (kNp > 1 ? 128 : 1)]) = make_float4(s[0], s[1], s[2], s[3]);
          asm volatile("bar.sync %0, %1;" ::"r"(1 + set), "n"(32 * kNp) : "memory");
          if (part >= 2) continue;
          float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
          for (int w = 0; w < kNp; ++w) {
            const float2 y = *reinterpret_cast<const float2*>(&s_part[flip][set * kNp + w][(lane * 4 + 2 * part) % (kNp > 1 ? 128 : 1)]);
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
          const float k = at ? ks[1] : ks[0];
          const bool held = at ? ok[1] : ok[0];
          float x0 = f0 != 0.0f && held ? s[2 * r] * f0 * k : -INFINITY;
          float x1 = f1 != 0.0f && held ? s[2 * r + 1] * f1 * k : -INFINITY;
          const uint32_t j = run0 + set * 16 + g + 8 * at;
          auto put = [&](uint32_t i, float v) {
            if (i < i1 && j < a.width) row_at(i)[j] = j < blocks_of(i) ? v : -INFINITY;
          };
          const uint32_t row0 = r0 + t;
          if (span == 1) {
            put(i0 + row0 + 2 * p, x0);
            put(i0 + row0 + 2 * p + 1, x1);
            continue;
          }
          x0 = max_nan(x0, x1);
          if (span > 2) x0 = max_nan(x0, __shfl_xor_sync(0xFFFFFFFFu, x0, 1));
          if (span > 4) x0 = max_nan(x0, __shfl_xor_sync(0xFFFFFFFFu, x0, 2));
          if (a.span > 8) {
            top[r] = max_nan(top[r], x0);
            if ((row0 + 8) % a.span != 0) continue;
            x0 = top[r];
            top[r] = -INFINITY;
          }
          if ((2 * p) % span == 0) put(i0 + (row0 + 2 * p) / a.span, x0);
        }
      }
    }
  }
}

template <int kD>
int launch_scores(const ScoreArgs& a, cudaStream_t s) {
  using C = ScoreCfg<kD>;
  static std::atomic<uint64_t> done;
  auto* kernel = q8_score_kernel<kD>;
  const int rc = allow_smem(reinterpret_cast<const void*>(kernel), C::kSmem, done);
  if (rc) return rc;
  return launch_pdl(kernel, dim3(2 * sm_count()), dim3(kScoreThreads), C::kSmem, s, a);
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
  a.queries = std::max<uint32_t>(1, kUnitRows / a.span);
  a.scale = scale;
  a.table = block_table;
  a.stride = static_cast<uint32_t>(table_stride);
  a.width = width;
  a.scores = scores;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  switch (a.c.head_dim) {
    case 64: return launch_scores<64>(a, s);
    case 128: return launch_scores<128>(a, s);
    case 256: return launch_scores<256>(a, s);
    default: return launch_scores<512>(a, s);
  }
}

}  // extern "C"

// q8_weigh.cu -- how much attention each cached entry received: for every
// entry of the batch's requests,
//     weights[slot] = decay * weights[slot] + sum over queries and heads of p,
//     p = 2^(scale log2(e) k_scale <q, k8> - lse log2(e)),
// with lse the attention's log-sum-exp, so p is the softmax weight itself and
// one pass over the keys does: the values are not read and no maximum is kept.
//
// An entry belongs to one CTA, which walks all rows and heads in a fixed order: no
// atomics, and results that repeat bit for bit.  Two kernels:
//
// Few rows (a decode step): the keys' bytes bound it.  A warp keeps a head's query
// fragments and streams its tiles of 16 entries through a ring of its own, as the split
// attention does, but with the entries as the product's 16 rows and the queries as its
// columns, eight or sixteen: a batch of up to eight rows a head then costs half the products
// and exponentials, and an entry's sum crosses four lanes.  The CTAs share the batch's tiles out evenly, and a CTA's warps take
// one head each and are summed in head order once per run of 512 entries.
//
// 32 requests, 132 MB of keys: 29.9 us, 65 % of the measured copy rate (30.5 with a copy for each tile's scale; then five stages a warp instead of
// four 31.4, six, i.e. one CTA to an SM, 39), the kernel below 90.
//
// Many rows (a window of queries): the products and exponentials bound it.  Up to 128
// channels the tensor cores take it (q8_weigh_tc.cu); from 256 on a warp holds 16 entries
// of a head as bf16 fragments (exact, and queries are bf16 already) and streams the
// request's rows past them.
#include <algorithm>

#include "q8_weigh.cuh"

namespace ckv {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kTile = 16;

__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int kD>
__global__ __launch_bounds__(kThreads) void q8_weigh_rows_kernel(const WeighArgs a) {
  constexpr int kKj = kD / 64;
  __shared__ uint32_t s_unit[CKV_MAX_BATCH];
  __shared__ uint32_t s_q[CKV_MAX_BATCH];
  __shared__ uint32_t s_scan[kWarps + 1];
  __shared__ unsigned long long s_scan64[kWarps + 1];
  __shared__ float s_sum[kWarps][kTile];
  pdl_wait();
  pdl_release();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, q = lane & 3;
  const uint32_t T = a.c.block_tokens, H = a.c.heads, G = a.group;
  const uint32_t unit_entries = kWarps / a.head_warps * kTile;

  const uint32_t units = scan_requests<kThreads>(a, unit_entries, s_unit, s_q, s_scan, s_scan64);
  for (uint32_t u = blockIdx.x; u < units; u += gridDim.x) {
    const uint32_t b = last_not_above(s_unit, a.batch, u);
    const uint32_t kv_len = static_cast<uint32_t>(a.kv_lens[b]);
    const uint32_t q_len = static_cast<uint32_t>(a.extend_lens[b]);
    const uint32_t phase = a.ratio - 1 - static_cast<uint32_t>(a.seq_lens[b]) % a.ratio;
    const uint32_t rows = q_len * G;
    const uint32_t e0 = (u - s_unit[b]) * unit_entries + warp / a.head_warps * kTile;
    float sum[2][2] = {};  // entries 8 n + 2q + {0, 1}
    int32_t block = -1;
    if (e0 < kv_len) {
      block = __ldg(a.table + static_cast<size_t>(a.rid[b]) * a.stride + e0 / T);
      if (static_cast<uint32_t>(block) >= a.c.num_blocks) {
        if (lane == 0) status_or(a.d_status, CKV_STATUS_BAD_INDEX);
        block = -1;
      }
    }
    if (block >= 0) {
      for (uint32_t h = warp % a.head_warps; h < H; h += a.head_warps) {
        uint32_t kf[2][kKj * 4][2];
        const size_t bh = static_cast<size_t>(block) * H + h;
        const uint8_t* k = a.c.k + (bh * T + e0 % T) * kD;
        const float f = a.scale_log2 * __ldg(a.c.k_scale + bh);
#pragma unroll
        for (int n = 0; n < 2; ++n) {
#pragma unroll
          for (int j = 0; j < kKj; ++j) {
            const uint4 w = ld_stream16_if(k + static_cast<size_t>(n * 8 + g) * kD + (j * 4 + q) * 16, true);
            const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int s = 0; s < 4; ++s) {
              kf[n][j * 4 + s][0] = f16x2_to_bf16x2(q8_lo_f16x2(x[s]));
              kf[n][j * 4 + s][1] = f16x2_to_bf16x2(q8_hi_f16x2(x[s]));
            }
          }
        }
        for (uint32_t r0 = 0; r0 < rows; r0 += 16) {
          float s[2][4] = {};
          float off[2];
          int64_t vis[2];
          const __nv_bfloat16* p[2];
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const uint32_t rho = min(r0 + g + 8 * r, rows - 1);
            const uint32_t i = rho / G, hg = rho % G;
            const size_t row = static_cast<size_t>(s_q[b] + i) * a.n_heads + h * G + hg;
            vis[r] = r0 + g + 8 * r < rows ? q8_visible(kv_len, q_len - 1 - i, phase, a.ratio) : 0;
            const float lse = __ldg(a.lse + row);
            off[r] = lse == -INFINITY ? -INFINITY : lse * -kLog2e;  // a row that saw nothing weighs nothing
            p[r] = a.q + row * kD;
          }
#pragma unroll
          for (int j = 0; j < kKj; ++j) {
            uint4 v[2][2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              v[r][0] = ld_cached16(p[r] + (j * 4 + q) * 16);
              v[r][1] = ld_cached16(p[r] + (j * 4 + q) * 16 + 8);
            }
#pragma unroll
            for (int st = 0; st < 4; ++st) {
              const uint4 x0 = v[0][st >> 1], x1 = v[1][st >> 1];
              uint32_t af[4];
              af[0] = st & 1 ? x0.z : x0.x;
              af[1] = st & 1 ? x1.z : x1.x;
              af[2] = st & 1 ? x0.w : x0.y;
              af[3] = st & 1 ? x1.w : x1.y;
              mma_bf16(s[0], af, kf[0][j * 4 + st][0], kf[0][j * 4 + st][1]);
              mma_bf16(s[1], af, kf[1][j * 4 + st][0], kf[1][j * 4 + st][1]);
            }
          }
#pragma unroll
          for (int n = 0; n < 2; ++n) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int64_t at = e0 + n * 8 + 2 * q + (e & 1);
              const float w = ex2(fmaf(s[n][e], f, off[e >> 1]));
              sum[n][e & 1] += at < vis[e >> 1] ? w : 0.0f;
            }
          }
        }
      }
    }
    // rows of the fragment (the lanes of one column), then the heads' warps in order
#pragma unroll
    for (int n = 0; n < 2; ++n) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) sum[n][e] += __shfl_xor_sync(0xFFFFFFFFu, sum[n][e], x);
        if (g == 0) s_sum[warp][n * 8 + 2 * q + e] = sum[n][e];
      }
    }
    __syncthreads();
    if (warp % a.head_warps == 0 && lane < kTile && block >= 0 && e0 + lane < kv_len) {
      float w = 0.0f;
      for (uint32_t x = 0; x < a.head_warps; ++x) w += s_sum[warp + x][lane];
      put_weight(a, block, e0 % T + lane, w);
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------- few rows
template <int kD>
struct StreamCfg {
  static constexpr int kStages = kD == 64 ? 8 : kD == 128 ? 4 : kD == 256 ? 5 : 3;
  static constexpr int kPerSm = kD <= 128 ? 2 : 1;
  static constexpr int kStageBytes = kTile * kD;
  static constexpr int kSmem = kWarps * kStages * kStageBytes;
  static constexpr int kRun = 32;  // tiles that are summed over the heads at once: one to a lane
};

// kCols: query rows of a pass, 8 or 16.
template <int kD, int kCols>
__global__ __launch_bounds__(kThreads, StreamCfg<kD>::kPerSm) void q8_weigh_stream_kernel(const WeighArgs a) {
  using C = StreamCfg<kD>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint32_t s_tile[CKV_MAX_BATCH];
  __shared__ uint32_t s_q[CKV_MAX_BATCH];
  __shared__ uint32_t s_scan[kWarps + 1];
  __shared__ unsigned long long s_scan64[kWarps + 1];
  __shared__ float s_sum[kWarps][C::kRun * kTile];
  pdl_wait();
  pdl_release();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, q = lane & 3;
  const uint32_t T = a.c.block_tokens, t_shift = __ffs(T) - 1, H = a.c.heads, G = a.group;
  const uint32_t head0 = warp % a.head_warps, part = warp / a.head_warps, parts = kWarps / a.head_warps;
  const uint32_t ring = static_cast<uint32_t>(__cvta_generic_to_shared(smem)) + warp * C::kStages * C::kStageBytes;
  const uint32_t tiles = scan_requests<kThreads>(a, kTile, s_tile, s_q, s_scan, s_scan64);
  // this CTA's share of the batch's tiles, request after request, in runs of at most kRun
  const uint32_t from = static_cast<uint32_t>(static_cast<uint64_t>(tiles) * blockIdx.x / gridDim.x);
  const uint32_t to = static_cast<uint32_t>(static_cast<uint64_t>(tiles) * (blockIdx.x + 1) / gridDim.x);
  for (uint32_t t0 = from; t0 < to;) {
    const uint32_t b = last_not_above(s_tile, a.batch, t0);
    const uint32_t end = b + 1 < a.batch ? s_tile[b + 1] : tiles;
    const uint32_t run = min(min(end, to) - t0, static_cast<uint32_t>(C::kRun));
    const uint32_t first = (t0 - s_tile[b]) * kTile;
    const uint32_t kv_len = static_cast<uint32_t>(a.kv_lens[b]);
    const uint32_t q_len = static_cast<uint32_t>(a.extend_lens[b]);
    const uint32_t phase = a.ratio - 1 - static_cast<uint32_t>(a.seq_lens[b]) % a.ratio;
    const uint32_t rows = q_len * G;
    const int32_t* table = a.table + static_cast<size_t>(a.rid[b]) * a.stride;
    const uint32_t mine = run > part ? (run - part + parts - 1) / parts : 0;  // tiles part, part + parts, ...
    // lane t keeps tile t's block number
    const int32_t blk = __ldg(table + (min(first + lane * kTile, kv_len - 1) >> t_shift));
    const bool blk_ok = static_cast<uint32_t>(blk) < a.c.num_blocks;
    if (!blk_ok && static_cast<uint32_t>(lane) < run) status_or(a.d_status, CKV_STATUS_BAD_INDEX);
    for (uint32_t i = lane; i < C::kRun * kTile; i += 32) s_sum[warp][i] = 0.0f;
    __syncwarp();
    for (uint32_t h = head0; h < H; h += a.head_warps) {
      const float scale = ld_ahead(a.c.k_scale + static_cast<size_t>(blk_ok ? blk : 0) * H + h);  // lane t's tile's
      for (uint32_t r0 = 0; r0 < rows; r0 += kCols) {
        auto issue = [&](uint32_t i) {
          if (i < mine) {
            const uint32_t t = part + i * parts, e = first + t * kTile;
            const int32_t bk = __shfl_sync(0xFFFFFFFFu, blk, t);
            const bool ok = static_cast<uint32_t>(bk) < a.c.num_blocks;
            const size_t bh = static_cast<size_t>(ok ? bk : 0) * H + h;
            const uint8_t* k = a.c.k + ((bh << t_shift) + (e & (T - 1))) * kD;
            const uint32_t dst = ring + (i % C::kStages) * C::kStageBytes;
#pragma unroll
            for (int x = 0; x < kD / 32; ++x) {
              const uint32_t c = x * 32 + lane, tok = c / (kD / 16), cc = c % (kD / 16);
              cp_async16(dst + tile_off<kD>(tok, cc), k + tok * kD + cc * 16, ok ? 16u : 0u);
            }
          }
          cp_async_commit();
        };
#pragma unroll
        for (int s = 0; s < C::kStages - 1; ++s) issue(s);
        // column g of column tile c is row r0 + 8 c + g; a lane's results are columns 2q and 2q + 1
        uint32_t qf[kD / 16][4];  // [..][c] and [..][2 + c]: the two halves of a k step
        float f[kCols / 8][2], off[kCols / 8][2];
        int64_t vis[kCols / 8][2];
#pragma unroll
        for (int c = 0; c < kCols / 8; ++c) {
          const uint32_t row = r0 + 8 * c + g;
          const bool in = row < rows;
          const uint32_t rho = in ? row : 0, i = rho / G, hg = rho % G;
          const size_t at = static_cast<size_t>(s_q[b] + i) * a.n_heads + h * G + hg;
          const float lse = in ? __ldg(a.lse + at) : -INFINITY;
          const float fg = load_query<kD>(a.q + at * kD, in, q, c, qf) * a.scale_log2;
          const float og = lse == -INFINITY ? -INFINITY : lse * -kLog2e;  // a row that saw nothing weighs nothing
          const int vg = in ? static_cast<int>(q8_visible(kv_len, q_len - 1 - i, phase, a.ratio)) : 0;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            f[c][e] = __shfl_sync(0xFFFFFFFFu, fg, (2 * q + e) * 4);
            off[c][e] = __shfl_sync(0xFFFFFFFFu, og, (2 * q + e) * 4);
            vis[c][e] = __shfl_sync(0xFFFFFFFFu, vg, (2 * q + e) * 4);
          }
        }
        for (uint32_t i = 0; i < mine; ++i) {
          cp_async_wait<C::kStages - 2>();
          __syncwarp();  // every lane's copies of this tile are in; every lane has read the tile before it
          issue(i + C::kStages - 1);
          const uint32_t st = ring + (i % C::kStages) * C::kStageBytes, t = part + i * parts;
          const float ks = __shfl_sync(0xFFFFFFFFu, scale, t);
          float s[kCols / 8][4] = {};
#pragma unroll
          for (int j = 0; j < kD / 64; ++j) {
            const int cc = lane_chunk<kD>(j, q);
            const uint4 lo = lds16(st + tile_off<kD>(g, cc)), hi = lds16(st + tile_off<kD>(8 + g, cc));
            const uint32_t x[4] = {lo.x, lo.y, lo.z, lo.w}, y[4] = {hi.x, hi.y, hi.z, hi.w};
#pragma unroll
            for (int z = 0; z < 4; ++z) {
              const uint32_t kf[4] = {q8_lo_f16x2(x[z]), q8_lo_f16x2(y[z]), q8_hi_f16x2(x[z]), q8_hi_f16x2(y[z])};
#pragma unroll
              for (int c = 0; c < kCols / 8; ++c) mma_f16(s[c], kf, qf[j * 4 + z][c], qf[j * 4 + z][2 + c]);
            }
          }
          float sum[2] = {0.0f, 0.0f};  // entries g and 8 + g
#pragma unroll
          for (int c = 0; c < kCols / 8; ++c) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int64_t at = first + t * kTile + (e >> 1) * 8 + g;
              const float w = ex2(fmaf(s[c][e], f[c][e & 1] * ks, off[c][e & 1]));
              sum[e >> 1] += at < vis[c][e & 1] ? w : 0.0f;
            }
          }
#pragma unroll
          for (int x = 1; x < 4; x <<= 1) {
            sum[0] += __shfl_xor_sync(0xFFFFFFFFu, sum[0], x);
            sum[1] += __shfl_xor_sync(0xFFFFFFFFu, sum[1], x);
          }
          if (q == 0) {  // one lane to an entry, the same one every time
            s_sum[warp][t * kTile + g] += sum[0];
            s_sum[warp][t * kTile + 8 + g] += sum[1];
          }
        }
        cp_async_wait<0>();
        __syncwarp();
      }
    }
    __syncthreads();
    for (uint32_t i = tid; i < run * kTile; i += kThreads) {
      const uint32_t e = first + i;
      if (e < kv_len) {
        const int32_t block = __ldg(table + (e >> t_shift));
        if (static_cast<uint32_t>(block) < a.c.num_blocks) {
          const uint32_t w0 = (i / kTile) % parts * a.head_warps;
          float w = 0.0f;
          for (uint32_t x = 0; x < a.head_warps; ++x) w += s_sum[w0 + x][i];
          put_weight(a, block, e & (T - 1), w);
        }
      }
    }
    __syncthreads();
    t0 += run;
  }
}

template <int kD>
int launch_weigh(const WeighArgs& a, cudaStream_t s) {
  // Rows of a request and kv head: up to 64 on average the keys are streamed, once for every 8 or 16 of them.
  const uint64_t all = static_cast<uint64_t>(a.num_q) * a.group;
  // By rows of a request and kv head (us, streaming / the other kernel, 32 to 64 requests of 4096 entries): 64 channels 59 / 63 at 64 and
  // 84 / 64 at 96; 128 channels 98 / 100 and 142 / 100; 256 channels 68 / 73 and 96 / 96; 512 channels 148 / 144 and 209 / 190
  // (there the two cross a little under 64).  Eight
  // columns against sixteen for at most eight rows: 18.1 / 20.9, 31.5 / 32.3, 21.4 / 24.1, 42 / 48.
  if (all <= 64ull * a.batch) {
    using C = StreamCfg<kD>;
    const bool narrow = all <= 8ull * a.batch;
    auto* kernel = narrow ? q8_weigh_stream_kernel<kD, 8> : q8_weigh_stream_kernel<kD, 16>;
    static std::atomic<uint64_t> done[2];
    const int rc = allow_smem(reinterpret_cast<const void*>(kernel), C::kSmem, done[narrow]);
    if (rc) return rc;
    return launch_pdl(kernel, dim3(static_cast<uint32_t>(C::kPerSm * sm_count())), dim3(kThreads), C::kSmem, s, a);
  }
  if (kD <= 128) return launch_q8_weigh_tc(a, s);
  return launch_pdl(q8_weigh_rows_kernel<kD < 256 ? 256 : kD>, dim3(2u * static_cast<uint32_t>(sm_count())), dim3(kThreads), 0, s, a);
}

}  // namespace
}  // namespace ckv

using namespace ckv;

extern "C" int ckv_q8_weigh(const ckv_q8_cache_t* cache, uint32_t n_heads, uint32_t ratio, float scale, float decay,
                            const void* q, const float* lse, uint32_t num_q, const int64_t* rid,
                            const int64_t* seq_lens, const int64_t* extend_lens, const int64_t* kv_lens,
                            uint32_t batch, const int32_t* block_table, uint64_t table_stride, uint32_t num_reqs,
                            float* weights, uint32_t* d_status, ckv_stream_t stream) {
  WeighArgs a{};
  int rc = q8_cache_of(cache, &a.c);
  if (rc) return rc;
  if (ratio == 0 || ratio > 65536) return CKV_ERR_RATIO;
  if (!(scale > 0.0f) || !(scale < 1e30f) || !(decay >= 0.0f) || !(decay <= 1.0f)) return CKV_ERR_SIZE;
  if (batch > CKV_MAX_BATCH || num_q > CKV_MAX_TOKENS) return CKV_ERR_SIZE;
  if (n_heads == 0 || n_heads % a.c.heads != 0 || n_heads / a.c.heads > CKV_Q8_MAX_GROUP) return CKV_ERR_SIZE;
  a.group = n_heads / a.c.heads;
  if (static_cast<uint64_t>(num_q) * a.group > 0x7FFFFFFFull) return CKV_ERR_SIZE;  // row numbers are 32-bit
  if (batch == 0 || num_q == 0) return CKV_OK;
  rc = check_table(block_table, table_stride, num_reqs);
  if (rc) return rc;
  if (!aligned16(q) || !aligned_to(lse, 4) || !aligned_to(weights, 4) || !aligned_to(rid, 8) ||
      !aligned_to(seq_lens, 8) || !aligned_to(extend_lens, 8) || !aligned_to(kv_lens, 8))
    return CKV_ERR_POINTER;
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.lse = lse;
  a.num_q = num_q;
  a.n_heads = n_heads;
  a.ratio = ratio;
  a.scale_log2 = scale * kLog2e;
  a.decay = decay;
  a.weights = weights;
  a.rid = rid;
  a.seq_lens = seq_lens;
  a.extend_lens = extend_lens;
  a.kv_lens = kv_lens;
  a.batch = batch;
  a.table = block_table;
  a.stride = static_cast<uint32_t>(table_stride);
  a.num_reqs = num_reqs;
  a.head_warps = 1;
  while (a.head_warps * 2 <= std::min<uint32_t>(a.c.heads, kWarps)) a.head_warps *= 2;
  a.wait_ns = wait_limit_ns();
  a.d_status = d_status;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  switch (a.c.head_dim) {
    case 64: return launch_weigh<64>(a, s);
    case 128: return launch_weigh<128>(a, s);
    case 256: return launch_weigh<256>(a, s);
    default: return launch_weigh<512>(a, s);
  }
}

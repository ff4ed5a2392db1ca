// q8_weigh_tc.cu -- the cached entries' attention weights when a request brings many
// rows (a window of queries), on the 5th-generation tensor cores.
//
// A unit is 128 entries of a request with all its heads and rows:
//     S^T [128 entries x 128 rows] = K8 Q^T   per head and chunk of rows,
// so an entry is a lane of tensor memory, a thread owns it, and its weight
//     sum over rows of 2^(scale log2(e) k_scale S - lse log2(e))
// is one register: no lane or warp exchanges anything until the unit's four column
// groups are added at its end.  Keys become bf16 (exact) and queries are bf16 already.
//
// Roles.  Sixteen warps for the exponentials, four that convert keys, four that copy queries four chunks ahead (row by row:
// a chunk's rows lie in as many pieces as it has queries), one for the products.
//
// Bound.  128 channels: a chunk's products take 512 cycles, its exponentials 512.  Measured: 18 MB of keys and 8.9 GF
// in 28 us, some 10 k cycles for a unit of four chunks: copying a chunk's queries takes 2 k.  Keys and queries by the same eight
// warps took 31.6 us; the next unit's weights and scales asked for only at its start, 29.0.
#include <algorithm>

#include "q8_tc.cuh"
#include "q8_weigh.cuh"

namespace ckv {
namespace {

constexpr int kChunk = 128;  // rows

template <int kD>
struct WtCfg {
  static constexpr int kSlices = kD / 64;
  static constexpr int kExpWarps = 16;  // four groups of four; a group takes 32 rows of a chunk
  static constexpr int kKeyWarps = 4, kQueryWarps = 4;
  static constexpr int kWarps = kExpWarps + kKeyWarps + kQueryWarps + 1;
  static constexpr int kLoads = kEntries / (8 * kKeyWarps);  // entries of a key thread
  static_assert(kChunk == 32 * kQueryWarps, "a row to a lane");
  static constexpr int kThreads = 32 * kWarps;
  static constexpr uint32_t kTileBytes = kSlices * kSlice;  // 128 rows of kD bf16 values
  static constexpr int kQStages = 4;
  static constexpr uint32_t kBytes = (2 + kQStages) * kTileBytes + 1024;  // two stages of keys, the queries', the alignment
  static constexpr uint32_t kSmem = kBytes < 120 * 1024 ? 120 * 1024 : kBytes;  // one CTA to an SM: see the attention
  static constexpr uint32_t kCols = 256;
};

template <int kD>
struct alignas(16) WtShared {
  static constexpr int kQ = WtCfg<kD>::kQStages;
  uint64_t k_full[2], k_free[2], q_full[kQ], q_free[kQ], s_full[2], s_free[2], idle;
  alignas(16) float off[kQ][kChunk];
  int vis[kQ][kChunk];
  float part[2][3][128];
  uint32_t unit[CKV_MAX_BATCH];
  uint32_t first_q[CKV_MAX_BATCH];
  uint4 meta[CKV_MAX_BATCH];
  unsigned long long scan64[WtCfg<kD>::kWarps + 1];
  uint32_t scan[WtCfg<kD>::kWarps + 1];
  uint32_t tmem;
};

// bf16 operands
constexpr uint32_t kBf16 = (1u << 7) | (1u << 10);

template <int kD, bool kShort>
__global__ __launch_bounds__(WtCfg<kD>::kThreads, 1) void q8_weigh_tc_kernel(const WeighArgs a) {
  using C = WtCfg<kD>;
  extern __shared__ uint8_t raw[];
  __shared__ WtShared<kD> sh;
  pdl_wait();
  pdl_release();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t T = a.c.block_tokens, t_shift = __ffs(T) - 1, H = a.c.heads, G = a.group;
  const uint32_t units = scan_requests<C::kThreads>(a, kEntries, sh.unit, sh.first_q, sh.scan, sh.scan64, sh.meta);
  if (blockIdx.x >= units) return;
  const uint32_t base = (smem_addr(raw) + 1023) & ~1023u;
  const uint32_t k_at = base, q_at = base + 2 * C::kTileBytes;
  if (warp == C::kWarps - 1) tmem_alloc(smem_addr(&sh.tmem), C::kCols);
  if (tid == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(smem_addr(&sh.k_full[s]), C::kKeyWarps);
      mbar_init(smem_addr(&sh.k_free[s]), 1);
      mbar_init(smem_addr(&sh.s_full[s]), 1);
      mbar_init(smem_addr(&sh.s_free[s]), C::kExpWarps);
    }
    for (int s = 0; s < C::kQStages; ++s) {
      mbar_init(smem_addr(&sh.q_full[s]), 33 * C::kQueryWarps);  // every thread's copies, and a warp's lse and counts
      mbar_init(smem_addr(&sh.q_free[s]), C::kExpWarps);
    }
    mbar_init(smem_addr(&sh.idle), 1);
    fence_mbar_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  Waiter w{static_cast<long long>(a.wait_ns) * 2, true};

  // every role walks the same (unit, head, chunk) sequence; kc and qc count keys' tiles and chunks
  uint32_t kc = 0, qc = 0;
  if (warp >= C::kExpWarps && warp < C::kExpWarps + C::kKeyWarps) {
    // ---- keys into bf16, a head ahead of the products; the next unit's block numbers are asked for a unit ahead
    const int lw = warp - C::kExpWarps, q = lane & 3;
    constexpr int kStep = 8 * C::kKeyWarps;
    const uint32_t tok = lw * 8 + (lane >> 2), sw = tok & 7;  // entries tok, tok + kStep, ...
    int32_t blk[C::kLoads];
    uint32_t kv_len = 0, e0 = 0;
    auto ask = [&](uint32_t u) {
      kv_len = 0;
      if (u >= units) return;
      const uint32_t b = last_not_above(sh.unit, a.batch, u);
      const uint4 meta = sh.meta[b];
      kv_len = meta.x;
      e0 = (u - sh.unit[b]) * kEntries;
      const int32_t* table = a.table + static_cast<size_t>(meta.w) * a.stride;
#pragma unroll
      for (int i = 0; i < C::kLoads; ++i) blk[i] = ld_ahead(table + (min(e0 + tok + kStep * i, kv_len - 1) >> t_shift));
    };
    const uint8_t* src[C::kLoads];
    uint32_t ok = 0;
    auto open = [&]() {
      ok = 0;
#pragma unroll
      for (int i = 0; i < C::kLoads; ++i) {
        const uint32_t e = e0 + tok + kStep * i;
        const bool in = e < kv_len && static_cast<uint32_t>(blk[i]) < a.c.num_blocks;
        src[i] = a.c.k + ((static_cast<size_t>(in ? blk[i] : 0) * H << t_shift) + (e & (T - 1))) * kD + q * 16;
        ok |= (in ? 1u : 0u) << i;
      }
    };
    uint4 buf[C::kSlices][C::kLoads];
    auto load = [&](uint32_t h) {
#pragma unroll
      for (int s = 0; s < C::kSlices; ++s) {
#pragma unroll
        for (int i = 0; i < C::kLoads; ++i)
          buf[s][i] = ld_stream16_if(src[i] + (static_cast<size_t>(h) << t_shift) * kD + s * 64, ok >> i & 1);
      }
    };
    ask(blockIdx.x);
    open();
    load(0);
    for (uint32_t u = blockIdx.x; u < units; u += gridDim.x) {
      for (uint32_t h = 0; h < H; ++h, ++kc) {
        const uint32_t ks = kc & 1;
        w.wait<kShort>(&sh.k_free[ks], ((kc >> 1) & 1) ^ 1);
#pragma unroll
        for (int s = 0; s < C::kSlices; ++s) {
#pragma unroll
          for (int i = 0; i < C::kLoads; ++i) {
            const uint32_t at = k_at + ks * C::kTileBytes + s * kSlice + (tok + kStep * i) * 128;
            const uint32_t x[4] = {buf[s][i].x, buf[s][i].y, buf[s][i].z, buf[s][i].w};
#pragma unroll
            for (int y = 0; y < 2; ++y)
              asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at + (((2 * q + y) ^ sw) << 4)),
                           "r"(f16x2_to_bf16x2(q8_lo_f16x2(x[2 * y]))), "r"(f16x2_to_bf16x2(q8_hi_f16x2(x[2 * y]))),
                           "r"(f16x2_to_bf16x2(q8_lo_f16x2(x[2 * y + 1]))), "r"(f16x2_to_bf16x2(q8_hi_f16x2(x[2 * y + 1])))
                           : "memory");
          }
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&sh.k_full[ks]));
        if (h == 0) ask(u + gridDim.x);
        if (h + 1 < H) {
          load(h + 1);
        } else {
          open();
          load(0);  // the next unit's
        }
      }
    }
  } else if (warp >= C::kExpWarps && warp < C::kWarps - 1) {
    // ---- queries as they are, four chunks ahead.  Lane l keeps row l of this warp's 32 of a chunk: its place (a division, so
    // once a chunk), its query and its lse, which is asked for a chunk ahead.
    const int lw = warp - C::kExpWarps - C::kKeyWarps;
    uint32_t query_next = 0;
    unsigned long long row_next = 0;
    auto place = [&](uint32_t b, uint32_t h, uint32_t c) {
      const uint32_t rho = min(c * kChunk + lw * 32 + lane, sh.meta[b].y * G - 1);
      query_next = rho / G;
      row_next = static_cast<unsigned long long>(sh.first_q[b] + query_next) * a.n_heads + h * G + (rho - query_next * G);
    };
    uint32_t b = last_not_above(sh.unit, a.batch, blockIdx.x);
    place(b, 0, 0);
    float lse_next = ld_ahead(a.lse + row_next);
    for (uint32_t u = blockIdx.x; u < units; u += gridDim.x) {
      const uint4 meta = sh.meta[b];
      const uint32_t rows = meta.y * G, chunks = (rows + kChunk - 1) / kChunk;
      const uint32_t b_next = u + gridDim.x < units ? last_not_above(sh.unit, a.batch, u + gridDim.x) : b;
      for (uint32_t h = 0; h < H; ++h) {
        for (uint32_t c = 0; c < chunks; ++c, ++qc) {
          const uint32_t qs = qc % C::kQStages, query = query_next;
          const unsigned long long row = row_next;
          const float lse = lse_next;
          if (c + 1 < chunks)
            place(b, h, c + 1);
          else if (h + 1 < H)
            place(b, h + 1, 0);
          else
            place(b_next, 0, 0);
          lse_next = ld_ahead(a.lse + row_next);
          w.wait<kShort>(&sh.q_free[qs], ((qc / C::kQStages) & 1) ^ 1);
          // this warp's 32 rows, 16 bytes a lane at a time; they arrive at the barrier when they have landed
          constexpr int kRowChunks = kD / 8;  // 16-byte chunks of a row
#pragma unroll
          for (int x = 0; x < kRowChunks; ++x) {
            const uint32_t i = x * 32 + lane, r = i / kRowChunks, n = lw * 32 + r, cc = i % kRowChunks;
            const unsigned long long from = __shfl_sync(0xFFFFFFFFu, row, r);
            cp_async16(q_at + qs * C::kTileBytes + (cc >> 3) * kSlice + n * 128 + (((cc & 7) ^ (n & 7)) << 4),
                       a.q + from * kD + cc * 8, 16u);
          }
          cp_async_arrive(smem_addr(&sh.q_full[qs]));
          const uint32_t n = lw * 32 + lane, at = c * kChunk + n;
          const int64_t see = at < rows ? q8_visible(meta.x, meta.y - 1 - query, meta.z, a.ratio) : 0;
          sh.vis[qs][n] = static_cast<int>(see);
          // a row that saw nothing weighs nothing, nor does one past the last
          sh.off[qs][n] = at >= rows || lse == -INFINITY ? -INFINITY : lse * -kLog2e;
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_addr(&sh.q_full[qs]));
        }
      }
      b = b_next;
    }
    // none of these copies may land after the CTA is gone
    cp_async_commit();
    cp_async_wait<0>();
  } else if (warp < C::kExpWarps) {
    const int group = warp >> 2, quarter = warp & 3, entry = quarter * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    // A unit's blocks are asked for a unit ahead, and its first scale and its weights so far before the last head of the unit before.
    auto block_of = [&](uint32_t u) -> int32_t {
      if (u >= units) return -1;
      const uint32_t b = last_not_above(sh.unit, a.batch, u);
      const uint4 meta = sh.meta[b];
      return ld_ahead(a.table + static_cast<size_t>(meta.w) * a.stride +
                      (min((u - sh.unit[b]) * kEntries + entry, meta.x - 1) >> t_shift));
    };
    auto exists = [&](int32_t blk) { return static_cast<uint32_t>(blk) < a.c.num_blocks; };
    auto scales_of = [&](int32_t blk) { return a.c.k_scale + static_cast<size_t>(exists(blk) ? blk : 0) * H; };
    // a unit starts where a block does, so an entry's slot follows from its place in the unit
    auto weight_of = [&](int32_t blk) {
      float* at = a.weights + (static_cast<size_t>(exists(blk) ? blk : 0) << t_shift) + (entry & (T - 1));
      return group == 0 && a.decay != 0.0f ? *static_cast<volatile float*>(at) : 0.0f;
    };
    int32_t blk_next = block_of(blockIdx.x);
    float scale_next = ld_ahead(scales_of(blk_next)), weight_next = weight_of(blk_next);
    uint32_t turn = 0;
    for (uint32_t u = blockIdx.x; u < units; u += gridDim.x, turn ^= 1) {
      const uint32_t b = last_not_above(sh.unit, a.batch, u);
      const uint4 meta = sh.meta[b];
      const uint32_t chunks = (meta.y * G + kChunk - 1) / kChunk;
      const uint32_t kv_len = meta.x, e0 = (u - sh.unit[b]) * kEntries, e = e0 + entry;
      const int32_t blk = blk_next;
      float next = scale_next;
      const float before = weight_next;
      blk_next = block_of(u + gridDim.x);
      const bool valid = exists(blk);
      if (!valid && e < kv_len && group == 0) status_or(a.d_status, CKV_STATUS_BAD_INDEX);
      const float* scales = scales_of(blk);
      F2 sum = f2_pack(0.0f, 0.0f);
      // the request's first row sees least: where it sees the whole tile, all do
      const bool edge = static_cast<int64_t>(e0) + kEntries > q8_visible(kv_len, meta.y - 1, meta.z, a.ratio);
      for (uint32_t h = 0; h < H; ++h) {
        const float f = next * a.scale_log2;
        next = ld_ahead(scales + min(h + 1, H - 1));
        if (h + 1 == H) {
          scale_next = ld_ahead(scales_of(blk_next));
          weight_next = weight_of(blk_next);
        }
        const F2 f2 = f2_pack(f, f);
        for (uint32_t c = 0; c < chunks; ++c, ++qc) {
          const uint32_t sb = qc & 1, qs = qc % C::kQStages;
          w.wait<kShort>(&sh.s_full[sb], (qc >> 1) & 1);
          w.wait<kShort>(&sh.q_full[qs], (qc / C::kQStages) & 1);  // long since; for the sight of off and vis
          tc_fence_after();
          float s[32];
          tmem_load32(tmem + lanes + sb * kChunk + group * 32, s);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_addr(&sh.s_free[sb]));
          const float* off = sh.off[qs] + group * 32;
          const int* vis = sh.vis[qs] + group * 32;
#pragma unroll
          for (int x = 0; x < 32; x += 4) {
            const float4 o = *reinterpret_cast<const float4*>(off + x);
            float t0, t1, t2, t3;
            f2_unpack(f2_fma(f2_pack(s[x], s[x + 1]), f2, f2_pack(o.x, o.y)), t0, t1);
            f2_unpack(f2_fma(f2_pack(s[x + 2], s[x + 3]), f2, f2_pack(o.z, o.w)), t2, t3);
            float w0 = ex2(t0), w1 = ex2(t1), w2 = ex2(t2), w3 = ex2(t3);
            if (edge) {
              w0 = static_cast<int>(e) < vis[x] ? w0 : 0.0f;
              w1 = static_cast<int>(e) < vis[x + 1] ? w1 : 0.0f;
              w2 = static_cast<int>(e) < vis[x + 2] ? w2 : 0.0f;
              w3 = static_cast<int>(e) < vis[x + 3] ? w3 : 0.0f;
            }
            sum = f2_add(sum, f2_add(f2_pack(w0, w1), f2_pack(w2, w3)));
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_addr(&sh.q_free[qs]));
        }
      }
      float s0, s1;
      f2_unpack(sum, s0, s1);
      float(*part)[128] = sh.part[turn];  // two turns: no group is a whole unit ahead of another
      if (group > 0) part[group - 1][entry] = s0 + s1;
      asm volatile("bar.sync 1, 512;" ::: "memory");
      if (group == 0 && e < kv_len && valid) {
        const float w = ((s0 + s1) + part[0][entry]) + (part[1][entry] + part[2][entry]);
        a.weights[(static_cast<size_t>(blk) << t_shift) + (e & (T - 1))] = a.decay == 0.0f ? w : fmaf(a.decay, before, w);
      }
    }
  } else {
    for (uint32_t u = blockIdx.x; u < units; u += gridDim.x) {
      const uint32_t b = last_not_above(sh.unit, a.batch, u);
      const uint4 meta = sh.meta[b];
      const uint32_t chunks = (meta.y * G + kChunk - 1) / kChunk;
      for (uint32_t h = 0; h < H; ++h, ++kc) {
        const uint32_t ks = kc & 1;
        w.wait<kShort>(&sh.k_full[ks], (kc >> 1) & 1);
        for (uint32_t c = 0; c < chunks; ++c, ++qc) {
          const uint32_t sb = qc & 1, qs = qc % C::kQStages;
          w.wait<kShort>(&sh.q_full[qs], (qc / C::kQStages) & 1);
          w.wait<kShort>(&sh.s_free[sb], ((qc >> 1) & 1) ^ 1);
          fence_async_smem();  // other threads' copies come without a fence of theirs
          tc_fence_after();
          if (elect_one()) {
            if (w.live) {
#pragma unroll
              for (int s = 0; s < C::kSlices; ++s) {
                const uint64_t ka = smem_operand(k_at + ks * C::kTileBytes + s * kSlice, 0);
                const uint64_t qb = smem_operand(q_at + qs * C::kTileBytes + s * kSlice, 0);
#pragma unroll
                for (int x = 0; x < 4; ++x)
                  tc_mma(tmem + sb * kChunk, ka + 2 * x, qb + 2 * x, mma_shape(128, kChunk, false, false) | kBf16,
                         s > 0 || x > 0);
              }
            }
            tc_commit(smem_addr(&sh.s_full[sb]));
            if (c + 1 == chunks) tc_commit(smem_addr(&sh.k_free[ks]));
          }
          __syncwarp();
        }
      }
    }
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
  if (!w.live && lane == 0) status_or(a.d_status, CKV_STATUS_TIMEOUT);
}

template <int kD>
int launch(const WeighArgs& a, cudaStream_t s) {
  using C = WtCfg<kD>;
  const bool brief = a.wait_ns < kShortWaitNs;
  auto* kernel = brief ? q8_weigh_tc_kernel<kD, true> : q8_weigh_tc_kernel<kD, false>;
  static std::atomic<uint64_t> done[2];
  const int rc = allow_smem(reinterpret_cast<const void*>(kernel), C::kSmem, done[brief ? 1 : 0]);
  if (rc) return rc;
  return launch_pdl(kernel, dim3(static_cast<uint32_t>(sm_count())), dim3(C::kThreads), C::kSmem, s, a);
}

}  // namespace

int launch_q8_weigh_tc(const WeighArgs& a, cudaStream_t s) {
  return a.c.head_dim == 64 ? launch<64>(a, s) : launch<128>(a, s);
}

}  // namespace ckv

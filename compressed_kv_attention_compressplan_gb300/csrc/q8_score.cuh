// q8_score.cuh -- what the kernels for the blocks' scores share.
#pragma once

#include <algorithm>
#include <cmath>

#include "q8_blocks.cuh"

namespace ckv {

__device__ __forceinline__ __half2 as_half2(uint32_t x) { return *reinterpret_cast<const __half2*>(&x); }
__device__ __forceinline__ uint32_t as_u32(__half2 x) { return *reinterpret_cast<const uint32_t*>(&x); }

struct ScoreArgs {
  Q8Cache c;
  BlockReqs r;
  const uint8_t* bounds;
  const __nv_bfloat16* q;
  uint32_t n_heads, group;
  uint32_t span;     // rows that a query takes: the group, up to a power of two or a multiple of eight
  uint32_t rows;     // query rows in shared memory: whole queries, or a part of one
  uint32_t queries;  // of a segment
  uint32_t parts;    // of a query that has more rows
  float scale, row_scale;  // the score's scale, as the blocks' and the rows' factors of it
  const int32_t* table;
  uint32_t stride;
  uint32_t width;
  float* scores;
  uint64_t wait_ns;
};

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// A score is s 2^-ex k_scale scale, s being the sum over a query row that was scaled by 2^ex.  These factors pass fp32's range where a
// score need not: 2^-ex s is up to 2^18 times the row's largest value (448 by 512 channels), and k_scale may bring it back; and scale alone may take the others'
// product out.  So a row's factor leaves 2^18 out, the block's makes up for it, and of a scale that would not let every
// k_scale times it be a normal number the rest goes to the rows: it is above one only where every block's factor is, and under one only where
// none is.  One product for a row and one for a block are then in range as long as the score is; a row of values under 2^-102 pays for the
// 2^18 with a subnormal product's steps, 2^-30 of its largest value and more.
constexpr int kHeadroom = 18;
inline void split_scale(float scale, ScoreArgs* a) {
  int e;
  const float m = std::frexp(scale, &e);
  const int kept = std::min(std::max(e, -126 - kHeadroom - kQ8ExpMin + 1), 126 - kHeadroom - kQ8ExpMax);
  a->scale = std::ldexp(m, kept + kHeadroom);
  a->row_scale = std::ldexp(1.0f, e - kept - kHeadroom);
}
__device__ __forceinline__ float row_factor(const ScoreArgs& a, int ex) {  // never 0, nor infinite
  return fminf(fmaxf(pow2f(-ex) * a.row_scale, 0x1p-149f), 0x1p127f);
}

// Tiles of the blocks that a request's queries see.
template <uint32_t kTile>
__device__ __forceinline__ uint32_t score_tiles(const BlockReq& r, uint32_t ratio, uint32_t t_shift) {
  if (r.q_len == 0) return 0;
  const uint32_t blocks = (seen_by(r, r.q_len - 1, ratio) + (1u << t_shift) - 1) >> t_shift;  // later queries see no less
  return (blocks + kTile - 1) / kTile;
}

// -infinity for the blocks behind a request's last tile.
template <uint32_t kTile>
__device__ __forceinline__ void fill_behind(const ScoreArgs& a, const uint32_t* s_q, const BlockReq* s_req) {
  const uint32_t H = a.c.heads, lane = threadIdx.x & 31, t_shift = __ffs(a.c.block_tokens) - 1, warps = blockDim.x / 32;
  const uint64_t rows = static_cast<uint64_t>(a.r.num_q) * H, step = gridDim.x * static_cast<uint64_t>(warps);
  for (uint64_t row = blockIdx.x * static_cast<uint64_t>(warps) + (threadIdx.x >> 5); row < rows; row += step) {
    BlockReq req;
    uint32_t i;
    if (!request_of(static_cast<uint32_t>(row / H), s_q, s_req, a.r.batch, &req, &i)) continue;
    for (uint32_t j = score_tiles<kTile>(req, a.r.ratio, t_shift) * kTile + lane; j < a.width; j += 32) a.scores[row * a.width + j] = -INFINITY;
  }
}

// The tensor-core kernel, for many query rows of up to 128 channels, at most 64 heads to a kv head.
int launch_q8_score_tc(const ScoreArgs& a, cudaStream_t s);

}  // namespace ckv

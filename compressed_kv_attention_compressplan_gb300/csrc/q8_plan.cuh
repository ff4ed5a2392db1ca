// q8_plan.cuh -- the attention plan over the 8-bit paged cache: how a step's
// (request, row tile) work is cut into equal shares, and where it lies.
//
// Work.  The rows of a request for one kv head are its q_len * group (query,
// head) pairs; a tile is `rows` consecutive ones, and its cost is the entries
// its last row sees, in units of entries, plus a fixed start-up.
// The tiles' costs are laid end to end and cut at multiples of one quota, so
// every CTA of a kv head gets the same number of entries whatever the lengths
// are (one wave, no tail); a tile that a cut crosses leaves partial results,
// which the combine kernel joins.  One plan serves every layer of a step.
//
// Buffer: header | first item of each CTA | first item of each split tile | items.
#pragma once

#include "q8.cuh"

namespace ckv {

struct Q8Item {  // 48 bytes
  uint32_t rid;
  uint32_t q_start;   // ragged query of the request's first row
  uint32_t q_len;
  uint32_t row0;      // the tile's first row
  uint32_t kv_begin;  // entries of this item
  uint32_t kv_end;
  uint32_t kv_len;    // of the request
  uint32_t phase;     // see q8_visible
  int32_t part;       // first partial slot of the tile; -1: this item is the whole tile
  uint32_t chunk;     // this item's number among the tile's
  uint32_t chunks;
  uint32_t reserved;
};
static_assert(sizeof(Q8Item) == 48, "");

struct Q8Header {  // 64 bytes
  uint32_t items;
  uint32_t ctas;
  uint32_t parts;
  uint32_t splits;
  uint32_t rows;  // the geometry the plan was made for; the attention checks it
  uint32_t group;
  uint32_t num_q;
  uint32_t ratio;
  uint32_t cap_ctas;
  uint32_t batch;
  uint32_t most;  // parts of the tile that has most
  uint32_t reserved[5];
};
static_assert(sizeof(Q8Header) == 64, "");

struct Q8Geom {
  bool tc;             // the tensor-core kernel takes it, not the split kernel
  uint32_t start_cost; // entries that starting a tile costs; a multiple of 16
  uint32_t rows;       // rows of a tile
  uint32_t group;      // query heads of a kv head
  uint32_t ctas;       // CTAs of a kv head
  uint32_t min_quota;  // entries
  uint32_t grain;      // entries are counted in these, and the quota is a multiple: 16, or the tensor-core kernels' tile
  uint32_t cap_items;
  uint32_t cap_parts;
  uint64_t off_first, off_split, off_items, bytes;
  uint64_t workspace;
};

// From sizes alone (and the device's SM count), the same for the plan and the
// attention call.  CKV_OK or CKV_ERR_SIZE.
int q8_attn_geom(const Q8Cache& c, uint32_t batch, uint32_t num_q, uint32_t n_heads, Q8Geom* g);

// Arguments of the attention kernels.
struct AttnArgs {
  Q8Cache c;
  Q8Geom g;
  const __nv_bfloat16* q;
  uint32_t batch;
  uint32_t num_q;
  uint32_t n_heads;
  uint32_t ratio;
  float scale_log2;
  const int32_t* table;
  uint32_t stride;
  uint32_t num_reqs;
  const uint8_t* plan;
  int out_f32;
  void* out;
  float* lse;
  float* part_o;    // [part][kv head][row][head_dim]
  float2* part_ml;  // [part][kv head][row]
  uint64_t wait_ns;
  uint32_t* d_status;
};

__device__ __forceinline__ bool item_fits(const Q8Item& item, const AttnArgs& a) {
  return item.rid < a.num_reqs && static_cast<uint64_t>(item.q_start) + item.q_len <= a.num_q &&
         item.row0 < static_cast<uint64_t>(item.q_len) * a.g.group &&
         item.kv_len <= static_cast<uint64_t>(a.stride) * a.c.block_tokens && item.kv_end <= item.kv_len &&
         (item.part < 0 || (static_cast<uint64_t>(item.part) + item.chunks <= a.g.cap_parts && item.chunk < item.chunks));
}

__device__ __forceinline__ bool plan_fits(const Q8Header* h, const AttnArgs& a) {
  return h->rows == a.g.rows && h->group == a.g.group && h->num_q == a.num_q && h->ratio == a.ratio &&
         h->cap_ctas == a.g.ctas && h->batch == a.batch;
}

// Takes the NaNs out of a word of four channels of entry e, noting the first entry with one for each channel.
__device__ __forceinline__ uint32_t without_nan(uint32_t w, int e, int* s_nan, int* s_any_nan) {
  const uint32_t bad = q8_nan_bytes(w);
  if (bad) {
    for (int z = 0; z < 4; ++z)
      if (bad >> (8 * z) & 1) atomicMin(s_nan + z, e);
    *s_any_nan = 1;
  }
  return w & ~bad;
}

// The tensor-core kernels, for tiles of many rows (g.tc); the parts that they leave are joined by the caller.
int launch_q8_attn_tc(const AttnArgs& a, cudaStream_t s);    // 256 channels and more
int launch_q8_attn_rows(const AttnArgs& a, cudaStream_t s);  // up to 128 channels

}  // namespace ckv

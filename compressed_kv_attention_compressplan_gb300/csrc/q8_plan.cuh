// q8_plan.cuh -- the attention plan over the 8-bit paged cache: how a step's
// (request, row tile) work is cut into equal shares, and where it lies.
//
// Work.  The rows of a request for one kv head are its q_len * group (query,
// head) pairs; a tile is `rows` consecutive ones, and its cost is the entries
// its last row sees, in units of entries, plus a fixed start-up of kQ8StartCost.
// The tiles' costs are laid end to end and cut at multiples of one quota, so
// every CTA of a kv head gets the same number of entries whatever the lengths
// are (one wave, no tail); a tile that a cut crosses leaves partial results,
// which the combine kernel joins.  One plan serves every layer of a step.
//
// Buffer: header | first item of each CTA | first item of each split tile | items.
#pragma once

#include "q8.cuh"

namespace ckv {

constexpr uint32_t kQ8StartCost = 32;  // entries; a multiple of 16

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
  uint32_t reserved[7];
};
static_assert(sizeof(Q8Header) == 64, "");

struct Q8Geom {
  uint32_t rows;       // rows of a tile
  uint32_t group;      // query heads of a kv head
  uint32_t ctas;       // CTAs of a kv head
  uint32_t min_quota;  // entries
  uint32_t round;      // the quota is a multiple of this
  uint32_t cap_items;
  uint32_t cap_parts;
  uint64_t off_first, off_split, off_items, bytes;
  uint64_t workspace;
};

// From sizes alone (and the device's SM count), the same for the plan and the
// attention call.  CKV_OK or CKV_ERR_SIZE.
int q8_attn_geom(const Q8Cache& c, uint32_t batch, uint32_t num_q, uint32_t n_heads, Q8Geom* g);

}  // namespace ckv

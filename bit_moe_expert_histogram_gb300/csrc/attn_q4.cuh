// What the kernels of a cache in 4 bits share: the rows' layout and the write
// and read kernels' arguments.
#pragma once
#include "attn_batch.cuh"

namespace moe {

// 16-bit units of a row of D elements (codes, four scales, four biases), 0
// for a D that has no layout
__host__ __device__ constexpr int q4_units(int D) { return D == 64 || D == 128 ? D / 4 + 8 : 0; }

struct CacheQ4Args {
  const int32_t* table;  // [n_slots][max_blocks]
  const int32_t* lens;   // [n_slots]
  const int32_t* n;      // [n_slots] or null: T
  void* k;               // [n_phys][n_kv][64][units]
  void* v;
  int n_slots, T, max_blocks, n_phys, n_kv;
  Ctrl* ctrl;
};

struct AttnQ4Args {
  const uint16_t* q;  // token (s, t) starts at q_stride * (s * T + t)
  int64_t q_stride;
  const char* k;      // [n_phys][n_kv][64][q4_units(D) * 2 bytes]
  const char* v;
  const int32_t* table;  // [n_slots][max_blocks]
  const int32_t* lens;
  const int32_t* n_new;  // [n_slots] or null: T
  int n_slots, T, n_q, n_kv, max_blocks, n_phys;
  int group;          // n_q / n_kv
  int row_shift;      // rows of a tile: 8 or 16
  int tiles;          // that a slot's and head's rows make
  int pairs;          // slots, heads and tiles
  int pair_cost;      // units of the line that a pair counts beside its own
  uint16_t* o;        // [n_slots][T][n_q][D]
  float* part;        // [CTA][2]: what the CTA's ends cut
  float* pieces;      // [CTA][warp]: what a warp's start cuts, where shared memory has no room
  unsigned* count;    // [CTA][16]: arrivals at 32 items of the pair that the CTA's end cuts
  Ctrl* ctrl;
};

}  // namespace moe

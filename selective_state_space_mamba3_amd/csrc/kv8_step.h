// What the decode step over an 8-bit cache hands to its kernels; each element type's are compiled apart.
#pragma once

#include "kv8.h"

namespace m3 {

struct Kv8StepArgs {
  HeadView q, k, v;  // k, v: p NULL where the cache holds the new tokens already
  Kv8Cache kc, vc;
  const int32_t *lengths, *table;
  HeadOut out;
  float* ws;  // as JoinArgs
  uint32_t B, T, H, G, D, capacity, window, sinks, log_block, num_pages, page_size, max_pages, scale_blocks;
  uint32_t splits, col_blocks;
  uint32_t step_pages, step_rows;  // from one tile to the next, in whole pages and rows
  float scale_log2;
};

// `waves` to a workgroup (4 or 8), `tiles` of 16 columns to a workgroup (1 or 2).
template <class T>
hipError_t launch_kv8_step(const Kv8StepArgs& a, uint32_t waves, uint32_t tiles, hipStream_t stream);

}  // namespace m3

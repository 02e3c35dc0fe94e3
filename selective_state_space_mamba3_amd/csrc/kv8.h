// Internal launch interface of the 8-bit key / value cache: tokens quantised
// into it, read back, and attended to by the decode step.  Geometry, pointers
// and strides arriving here were validated by abi.cpp.
#pragma once

#include "attn.h"

namespace m3 {

struct Kv8Geom {
  uint32_t B, T, capacity, H, G, D, block, window, sinks, dtype;  // T: tokens of a row, the longest with offsets
  uint32_t num_pages, page_size, max_pages, total;
  float scale;
};
// Codes [page, row, head, d] and the exponent bytes of their blocks [page, head, block], contiguous.
// `vec`: every 8 codes from a multiple of 8 stand in one aligned 8-byte word.
struct Kv8Cache {
  uint8_t *codes, *scales;
  int64_t page, row, head;
  uint32_t vec;
};
struct Kv8Operands {
  HeadView q, k, v;  // k, v: the new tokens, p NULL where the step finds them in the cache
  Kv8Cache kc, vc;
  const int32_t *lengths, *offsets, *table;  // lengths: first positions
  HeadOut out, out_v;                        // the read's keys and values, or the step's result
  float* ws;
};

inline uint32_t log_block(const Kv8Geom& g) { return g.block == 16 ? 4 : g.block == 32 ? 5 : g.block == 64 ? 6 : 7; }
inline uint32_t scale_blocks(const Kv8Geom& g) { return (g.page_size + g.block - 1) / g.block; }  // of a page's head

uint64_t kv8_write_workgroups(const Kv8Geom& g);
uint64_t kv8_read_workgroups(const Kv8Geom& g);
uint64_t attn_step_kv8_workgroups(const Kv8Geom& g);
size_t attn_step_kv8_workspace_floats(const Kv8Geom& g);

hipError_t launch_kv8_write(const Kv8Geom& g, const Kv8Operands& o, hipStream_t stream);
hipError_t launch_kv8_read(const Kv8Geom& g, const Kv8Operands& o, hipStream_t stream);
hipError_t launch_attn_step_kv8(const Kv8Geom& g, const Kv8Operands& o, hipStream_t stream);

}  // namespace m3

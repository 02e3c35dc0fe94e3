// The decode step over an 8-bit key / value cache: how its rows are dealt over workgroups.
#include "attn_join.h"
#include "kv8_step.h"

#include <algorithm>

namespace m3 {

namespace {

// 32 columns to a workgroup where there are more than 16; float32's pieces of them leave room for 16 from 65 on.
uint32_t column_tiles(const Kv8Geom& g) { return g.H / g.G * g.T > 16 && !(g.dtype == kF32 && g.D > 64) ? 2 : 1; }
uint32_t column_blocks(const Kv8Geom& g) {
  const uint32_t n = 16 * column_tiles(g);
  return (g.H / g.G * g.T + n - 1) / n;
}
struct Plan {
  uint32_t waves, splits;
};
// A workgroup to a row, of four waves where there are many rows, else of eight.  Where that leaves half of the
// places on the chip empty, rows are cut into stretches, none shorter than two chunks for each wave at the longest row.
// (Up to 64 columns registers leave room for two workgroups of eight waves on a compute unit, 117 to 119 of them for
// 16-bit types, 109 for float32 up to 32 columns; between 33 and 64 float32 takes 133, and one of its workgroups runs
// at a time, though as many stretches are cut.)
// (Even shares of all rows' tiles, for rows of different lengths, were no better where rows are few, and worse than
// whole rows where they are many: 64 rows of 1024 to 4096 positions, four float16 tokens of 32 heads of 128 over 4:
// 54 us whole, 72 and a join in even shares.  211 rows of up to 20 positions, 8 heads of 128 over 4: 18 us with four
// waves, 30 with eight.)
Plan plan(const Kv8Geom& g) {
  const uint64_t rows = (uint64_t)g.B * g.G * column_blocks(g);
  const uint64_t seen = g.window ? std::min((uint64_t)g.capacity, (uint64_t)g.window + g.T + g.sinks) : g.capacity;
  const uint64_t slots = g.D <= 64 && column_tiles(g) == 1 ? 512 : 256, tile = 256;
  if (2 * rows > slots || seen <= tile) return {rows < 1024 && seen > tile ? 8u : 4u, 1};
  const uint64_t want = slots / rows, most = (seen + 2 * tile - 1) / (2 * tile);
  return {8, (uint32_t)std::min({want, most, (uint64_t)kMaxSplits})};
}

}  // namespace

uint64_t attn_step_kv8_workgroups(const Kv8Geom& g) {
  const uint64_t splits = plan(g).splits, rows = (uint64_t)g.B * g.T;
  // (counted as if of 256 threads)
  return std::max({2 * ((g.B * splits + 7) / 8 * 8 * g.G * column_blocks(g)),
                   splits > 1 ? join_workgroups(rows, g.H, g.D) : 0, kv8_write_workgroups(g)});
}

size_t attn_step_kv8_workspace_floats(const Kv8Geom& g) {
  const uint32_t splits = plan(g).splits;
  return splits == 1 ? 0 : join_floats((uint64_t)g.B * g.T, g.H, g.D, splits);
}

hipError_t launch_attn_step_kv8(const Kv8Geom& g, const Kv8Operands& o, hipStream_t stream) {
  // Several workgroups read a row's heads where it has more columns than one takes: then the tokens are written
  // before any of them begins.
  const bool apart = column_blocks(g) > 1 && o.k.p != nullptr;
  if (apart) {
    const hipError_t e = launch_kv8_write(g, o, stream);
    if (e != hipSuccess) return e;
  }
  const Plan p = plan(g);
  const uint32_t tile = 32 * p.waves;
  const Kv8StepArgs a{o.q, apart ? HeadView{} : o.k, apart ? HeadView{} : o.v, o.kc, o.vc, o.lengths, o.table, o.out,
                      o.ws, g.B, g.T, g.H, g.G, g.D, g.capacity, g.window, g.sinks, log_block(g), g.num_pages,
                      g.page_size, g.max_pages, scale_blocks(g), p.splits, column_blocks(g), tile / g.page_size,
                      tile % g.page_size, g.scale * kLog2e};
  const uint32_t columns = column_tiles(g);
  if (g.dtype == kF32) return launch_kv8_step<float>(a, p.waves, columns, stream);
  if (g.dtype == kF16) return launch_kv8_step<_Float16>(a, p.waves, columns, stream);
  return launch_kv8_step<__bf16>(a, p.waves, columns, stream);
}

}  // namespace m3

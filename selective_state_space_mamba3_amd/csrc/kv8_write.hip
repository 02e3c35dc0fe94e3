// Keys and values quantised as they are written into an 8-bit cache.
//
// Each block of `block` positions of a head has one scale 2^e, the least that
// holds the largest magnitude of what is written to it; a block that already
// holds older tokens keeps its scale unless that grows, and then its codes
// are rounded to the new one.  Powers of two: the products are exact, so that
// a code depends on nothing but the token and e, growing scales cost only what
// leaves the subnormals, and e4m3's own exponent makes a finer scale worth nothing
// but the last of 18 binary places.
//
// One group of threads takes a block of one head, of the keys or of the
// values: its new tokens are read once and stay in registers while their
// largest magnitude is found.  Bound by memory: 65536 tokens of 4 heads of 128,
// float16: 43 us (4.7 TB/s); 256 rows of one token, 8 heads of 64: 5 us, all of it latency.
#include "kv8_common.h"

#include <algorithm>

namespace m3 {

namespace {

struct WriteArgs {
  HeadView x[2];
  Kv8Cache c[2];
  const int32_t *lengths, *offsets, *table;
  uint32_t B, T, G, D, capacity, log_block, num_pages, page_size, max_pages, total;
  uint32_t blocks, scale_blocks;  // blocks of a row that a call can touch; scales of a page's head
  uint32_t items;
};

constexpr int kThreads = 256;

// GROUP threads to a block of a head (one wave or the workgroup), PIECES
// pieces of 8 elements to a thread.
template <class T, int GROUP, int PIECES, bool VEC>
__global__ __launch_bounds__(kThreads) void kv8_write_kernel(const WriteArgs a) {
  __shared__ float red[kThreads / 64];
  const uint32_t tid = threadIdx.x % GROUP;
  uint32_t at = blockIdx.x * (kThreads / GROUP) + threadIdx.x / GROUP;
  if constexpr (GROUP == 64) at = __builtin_amdgcn_readfirstlane(at);
  if (at >= a.items) return;
  const uint32_t g = at % a.G;
  at /= a.G;
  const uint32_t kv = at % 2;
  at /= 2;
  const uint32_t b = at / a.blocks, nth = at % a.blocks;

  int64_t x0;
  int n;
  seq_range(a.offsets, b, a.T, a.total, &x0, &n);
  n = min(n, (int)a.T);
  const int len = a.lengths[b];
  if (len < 0 || (int64_t)len + n > (int64_t)a.capacity) return;
  const int first = (int)(((uint32_t)len >> a.log_block) + nth) << a.log_block;  // the block's first position
  const int begin = max(first, len), end = min(first + (1 << a.log_block), len + n);
  if (begin >= end) return;
  const Kv8Cache& c = a.c[kv];
  const HeadView& x = a.x[kv];
  const T* rows = static_cast<const T*>(x.p) + (x0 + (begin - len)) * x.row + (int64_t)g * x.head;

  // piece i of the new tokens: token i / per_row, columns 8 (i % per_row) ...
  const uint32_t per_row = (a.D + 7) / 8, pieces = (uint32_t)(end - begin) * per_row;
  const uint32_t inverse = (65535 + per_row) / per_row;  // i / per_row = i * inverse >> 16 for i < 2^12
  Raw8<T> raw[PIECES];
#pragma unroll
  for (int p = 0; p < PIECES; ++p) {
    const uint32_t i = tid + p * GROUP, token = i * inverse >> 16;
    raw[p] = Raw8<T>{};
    if (i < pieces) raw[p] = read_elements<T, VEC>(rows + (int64_t)token * x.row, 8 * (i - token * per_row), a.D);
  }
  // (the block's place is found while they are on their way)
  const Slot slot = find_slot(a.table, b, (uint32_t)first, a.page_size, a.max_pages, a.num_pages);
  if (slot.page < 0) return;
  uint8_t* codes = c.codes + slot.page * c.page + (int64_t)slot.row * c.row + (int64_t)g * c.head;
  uint8_t* scale = c.scales + ((size_t)slot.page * a.G + g) * a.scale_blocks + (slot.row >> a.log_block);
  const int had = begin > first ? held_exponent(*scale) : kLeastExp;
  float amax = 0.f;
#pragma unroll
  for (int p = 0; p < PIECES; ++p) amax = max_finite8<T>(raw[p], amax);
  amax = wave_max_nn(amax);
  if constexpr (GROUP > 64) {
    if (tid % 64 == 0) red[tid / 64] = amax;
    __syncthreads();
    amax = __builtin_fmaxf(max3(red[0], red[1], red[2]), red[3]);
  }
  const int e = max(least_exponent(amax), had);
  if (tid == 0) *scale = (uint8_t)(e + kExpBias);

  // codes of older tokens, where the scale grew (below 2^-126 nothing is left of any of them)
  if (begin > first && e > had) {
    const float down = power_of_two(max(had - e, -126));
    for (uint32_t i = tid; i < (uint32_t)(begin - first) * per_row; i += GROUP) {
      const uint32_t token = i * inverse >> 16, col = 8 * (i - token * per_row);
      uint8_t* p = codes + (int64_t)token * c.row;
      write_codes<VEC>(p, col, a.D, rescale8(read_codes<VEC>(p, col, a.D), down));
    }
  }
  const float inv = power_of_two(-e);
#pragma unroll
  for (int p = 0; p < PIECES; ++p) {
    const uint32_t i = tid + p * GROUP, token = i * inverse >> 16;
    if (i >= pieces) break;
    write_codes<VEC>(codes + (int64_t)(begin - first + (int)token) * c.row, 8 * (i - token * per_row), a.D,
                     quantise8<T>(raw[p], inv));
  }
}

// The blocks of a row that its tokens can touch, and the pieces of one block.
uint32_t touched_blocks(const Kv8Geom& g) { return (g.T - 1 + g.block - 1) / g.block + 1; }
uint32_t block_pieces(const Kv8Geom& g) { return std::min(g.T, g.block) * ((g.D + 7) / 8); }
uint64_t write_items(const Kv8Geom& g) { return (uint64_t)g.B * touched_blocks(g) * 2 * g.G; }
// A wave to a block where its tokens fit eight pieces of 8 to a lane, else the workgroup.  (4 x 2048 tokens of 8 heads
// of 64, blocks of 64: 8.8 us by waves, 10.3 by workgroups.)
bool by_wave(const Kv8Geom& g) { return block_pieces(g) <= 8 * 64; }

template <class T, int GROUP, int PIECES>
hipError_t launch_pieces(const Kv8Geom& g, const WriteArgs& a, hipStream_t stream) {
  const dim3 grid((uint32_t)kv8_write_workgroups(g));
  if (a.x[0].vec && a.x[1].vec && a.c[0].vec && a.c[1].vec)
    kv8_write_kernel<T, GROUP, PIECES, true><<<grid, kThreads, 0, stream>>>(a);
  else
    kv8_write_kernel<T, GROUP, PIECES, false><<<grid, kThreads, 0, stream>>>(a);
  return hipGetLastError();
}
// As many pieces to a lane as a full block needs: loads that are left out cost as much as others (105 rows of up to 220
// tokens, 8 heads of 80, blocks of 16: 13.8 us with four, 15.2 with eight).
template <class T>
hipError_t launch(const Kv8Geom& g, const WriteArgs& a, hipStream_t stream) {
  const uint32_t pieces = block_pieces(g);
  if (!by_wave(g)) return launch_pieces<T, 256, 8>(g, a, stream);
  if (pieces > 4 * 64) return launch_pieces<T, 64, 8>(g, a, stream);
  return pieces > 64 ? launch_pieces<T, 64, 4>(g, a, stream) : launch_pieces<T, 64, 1>(g, a, stream);
}

}  // namespace

uint64_t kv8_write_workgroups(const Kv8Geom& g) { return by_wave(g) ? (write_items(g) + 3) / 4 : write_items(g); }

hipError_t launch_kv8_write(const Kv8Geom& g, const Kv8Operands& o, hipStream_t stream) {
  const WriteArgs a{{o.k, o.v}, {o.kc, o.vc}, o.lengths, o.offsets, o.table, g.B, g.T, g.G, g.D, g.capacity,
                    log_block(g), g.num_pages, g.page_size, g.max_pages, g.total, touched_blocks(g),
                    scale_blocks(g), (uint32_t)write_items(g)};
  if (g.dtype == kF32) return launch<float>(g, a, stream);
  if (g.dtype == kF16) return launch<_Float16>(g, a, stream);
  return launch<__bf16>(g, a, stream);
}

}  // namespace m3

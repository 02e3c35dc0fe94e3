// Positions of an 8-bit cache read back as rows of keys and values, for the
// attention over whole sequences of a prompt that goes on.
//
// A wave takes 16 positions of a row, all heads of them (or some, where that
// makes too few waves): they lie in one page and in one block, so that its
// address is found once.  Neighbouring lanes hold a row's pieces of eight, and
// four rows of a lane are on their way at a time.  Bound by memory: each code is
// read once, each element written once (65536 positions of 4 heads of 128 to
// bfloat16: 43 us, 4.7 TB/s).
#include "kv8_common.h"

namespace m3 {

namespace {

struct ReadArgs {
  Kv8Cache c[2];
  const int32_t *starts, *offsets, *table;
  HeadOut y[2];
  uint32_t B, T, G, D, capacity, log_block, num_pages, page_size, max_pages, total, scale_blocks;
  uint32_t groups, heads;  // workgroups to a row, and heads to a wave
};

constexpr int kThreads = 256, kRun = 16, kAhead = 4;

template <class T, bool VEC>
__global__ __launch_bounds__(kThreads) void kv8_read_kernel(const ReadArgs a) {
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x % 64;
  const uint32_t b = blockIdx.x / a.groups, nth = blockIdx.x % a.groups * (kThreads / 64) + wave, kv = blockIdx.y % 2;
  const uint32_t head0 = blockIdx.y / 2 * a.heads, heads = min(a.heads, a.G - head0);
  int64_t y0;
  int n;
  seq_range(a.offsets, b, a.T, a.total, &y0, &n);
  n = min(n, (int)a.T);
  const int64_t start = a.starts == nullptr ? 0 : a.starts[b];
  // runs of 16 from a multiple of 16 (rounded down, below zero as well)
  const int64_t first = (start & ~(int64_t)(kRun - 1)) + (int64_t)nth * kRun;
  const int64_t begin = max(first, start), end = min(first + kRun, start + n);
  if (begin >= end) return;
  Slot slot{-1, 0};
  if (first >= 0 && first < (int64_t)a.capacity)
    slot = find_slot(a.table, b, (uint32_t)first, a.page_size, a.max_pages, a.num_pages);
  const int page = max(__builtin_amdgcn_readfirstlane(slot.page), 0);
  const uint32_t row = __builtin_amdgcn_readfirstlane(slot.row);
  const Kv8Cache& c = a.c[kv];
  const HeadOut& y = a.y[kv];
  const uint8_t* codes = c.codes + page * c.page + (int64_t)row * c.row;
  const uint8_t* scales = c.scales + (size_t)page * a.G * a.scale_blocks + (row >> a.log_block);
  T* out = static_cast<T*>(y.p) + (y0 + (first - start)) * y.row;
  // positions of the run that are asked for, and those of them that there are
  const int lo = (int)(begin - first), hi = (int)(end - first),
            there = slot.page < 0 ? 0 : (int)min((int64_t)hi, (int64_t)a.capacity - first);

  const uint32_t per_row = (a.D + 7) / 8, at_once = 64 / per_row, mine = lane / per_row, col = lane % per_row * 8;
  if (mine >= at_once) return;
  const uint32_t rows = kRun * heads;  // row i: head i / 16 of them, position i % 16
  for (uint32_t i0 = mine; i0 < rows; i0 += kAhead * at_once) {
    uintx2 w[kAhead];
    uint32_t byte[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const uint32_t i = i0 + k * at_once, g = head0 + i / kRun;
      const int r = (int)(i % kRun);
      w[k] = uintx2{};
      byte[k] = 1;
      if (i < rows && r >= lo && r < there) {
        w[k] = read_codes<VEC>(codes + (int64_t)r * c.row + (int64_t)g * c.head, col, a.D);
        byte[k] = scales[(size_t)g * a.scale_blocks];
      }
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const uint32_t i = i0 + k * at_once, g = head0 + i / kRun;
      const int r = (int)(i % kRun);
      if (i >= rows || r < lo || r >= hi) continue;
      const float s = scale_value(byte[k]);
      floatx4 f[2] = {values4(w[k][0]) * s, values4(w[k][1]) * s};
      if constexpr (__is_same(T, _Float16)) {
        // a code may stand for more than float16 holds (65504 itself rounds to 65536): its largest value then
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float v = f[e / 4][e % 4];
          f[e / 4][e % 4] = __builtin_fabsf(v) > 65504.f ? __builtin_copysignf(65504.f, v) : v;
        }
      }
      write_elements<T, VEC>(out + (int64_t)r * y.row + (int64_t)g * y.head, col, a.D, f);
    }
  }
}

uint32_t read_groups(const Kv8Geom& g) {
  const uint32_t runs = (g.T + 2 * kRun - 2) / kRun, waves = kThreads / 64;
  return (runs + waves - 1) / waves;
}
// Heads to a wave: all of them where there are waves for the whole chip (9 rows of up to 2047 positions, 8 heads of
// 64: 13.4 us with all).
uint32_t read_heads(const Kv8Geom& g) {
  const uint64_t waves = 2ull * g.B * read_groups(g) * (kThreads / 64), parts = (8192 + waves - 1) / waves;
  return parts >= g.G ? 1 : (uint32_t)((g.G + parts - 1) / parts);
}

template <class T>
hipError_t launch(const ReadArgs& a, hipStream_t stream) {
  const dim3 grid(a.B * a.groups, 2 * ((a.G + a.heads - 1) / a.heads));
  if (a.c[0].vec && a.c[1].vec && a.y[0].vec && a.y[1].vec)
    kv8_read_kernel<T, true><<<grid, kThreads, 0, stream>>>(a);
  else
    kv8_read_kernel<T, false><<<grid, kThreads, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace

uint64_t kv8_read_workgroups(const Kv8Geom& g) {
  const uint32_t heads = read_heads(g);
  return 2ull * g.B * read_groups(g) * ((g.G + heads - 1) / heads);
}

hipError_t launch_kv8_read(const Kv8Geom& g, const Kv8Operands& o, hipStream_t stream) {
  const ReadArgs a{{o.kc, o.vc}, o.lengths, o.offsets, o.table, {o.out, o.out_v}, g.B, g.T, g.G, g.D, g.capacity,
                   log_block(g), g.num_pages, g.page_size, g.max_pages, g.total, scale_blocks(g), read_groups(g),
                   read_heads(g)};
  if (g.dtype == kF32) return launch<float>(a, stream);
  if (g.dtype == kF16) return launch<_Float16>(a, stream);
  return launch<__bf16>(a, stream);
}

}  // namespace m3

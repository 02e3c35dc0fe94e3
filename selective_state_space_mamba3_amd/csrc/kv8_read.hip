// Positions of an 8-bit cache read back as rows of keys and values, for the
// attention over whole sequences of a prompt that goes on.
//
// A workgroup takes 16 positions of a row, all heads of them, keys and values:
// they lie in one page and in one block, so that its address and scales are
// found once.  Bound by memory: each code is read once, each element written once.
#include "kv8_common.h"

namespace m3 {

namespace {

struct ReadArgs {
  Kv8Cache c[2];
  const int32_t *starts, *offsets, *table;
  HeadOut y[2];
  uint32_t B, T, G, D, capacity, block, num_pages, page_size, max_pages, total, runs, scale_blocks;
};

constexpr int kThreads = 256, kRun = 16;

template <class T, bool VEC>
__global__ __launch_bounds__(kThreads) void kv8_read_kernel(const ReadArgs a) {
  const uint32_t b = blockIdx.x / a.runs, nth = blockIdx.x % a.runs, kv = blockIdx.y;
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
  const Kv8Cache& c = a.c[kv];
  const HeadOut& y = a.y[kv];
  const uint8_t* codes = c.codes + max(slot.page, 0) * c.page + (int64_t)slot.row * c.row;
  const uint8_t* scales = c.scales + (size_t)max(slot.page, 0) * a.G * a.scale_blocks + slot.row / a.block;
  const uint32_t per_row = (a.D + 7) / 8, rows = (uint32_t)(end - begin), pieces = rows * a.G * per_row;
  for (uint32_t i = threadIdx.x; i < pieces; i += kThreads) {
    const uint32_t col = i % per_row * 8, rg = i / per_row, g = rg % a.G, r = rg / a.G;
    const int64_t j = begin + r;
    T* out = static_cast<T*>(y.p) + (y0 + (j - start)) * y.row + (int64_t)g * y.head;
    float f[8] = {};
    if (slot.page >= 0 && j < (int64_t)a.capacity) {
      const uint8_t* p = codes + (j - first) * c.row + (int64_t)g * c.head + col;
      uintx2 w = {};
      if constexpr (VEC) {
        w = *reinterpret_cast<const uintx2*>(p);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (col + e < a.D) w[e / 4] |= (uint32_t)p[e] << 8 * (e % 4);
      }
      const float s = scale_value(scales[(size_t)g * a.scale_blocks]);
      const floatx4 lo = values4(w[0]) * s, hi = values4(w[1]) * s;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        f[e] = lo[e];
        f[4 + e] = hi[e];
      }
      if constexpr (__is_same(T, _Float16)) {
        // a code may stand for more than float16 holds (65504 itself rounds to 65536): its largest value then
#pragma unroll
        for (int e = 0; e < 8; ++e)
          f[e] = __builtin_fabsf(f[e]) > 65504.f ? __builtin_copysignf(65504.f, f[e]) : f[e];
      }
    }
    store4<T, VEC>(out, col, a.D, f[0], f[1], f[2], f[3]);
    store4<T, VEC>(out, col + 4, a.D, f[4], f[5], f[6], f[7]);
  }
}

uint32_t read_runs(const Kv8Geom& g) { return (g.T + 2 * kRun - 2) / kRun; }

template <class T>
hipError_t launch(const ReadArgs& a, hipStream_t stream) {
  const dim3 grid(a.B * a.runs, 2);
  if (a.c[0].vec && a.c[1].vec && a.y[0].vec && a.y[1].vec)
    kv8_read_kernel<T, true><<<grid, kThreads, 0, stream>>>(a);
  else
    kv8_read_kernel<T, false><<<grid, kThreads, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace

uint64_t kv8_read_workgroups(const Kv8Geom& g) { return 2ull * g.B * read_runs(g); }

hipError_t launch_kv8_read(const Kv8Geom& g, const Kv8Operands& o, hipStream_t stream) {
  const ReadArgs a{{o.kc, o.vc}, o.lengths, o.offsets, o.table, {o.out, o.out_v}, g.B, g.T, g.G, g.D, g.capacity,
                   g.block, g.num_pages, g.page_size, g.max_pages, g.total, read_runs(g),
                   (g.page_size + g.block - 1) / g.block};
  if (g.dtype == kF32) return launch<float>(a, stream);
  if (g.dtype == kF16) return launch<_Float16>(a, stream);
  return launch<__bf16>(a, stream);
}

}  // namespace m3

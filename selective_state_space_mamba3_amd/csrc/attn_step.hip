// Single-token attention over a key / value cache, dense or in pages.  The
// token's key and value go into the cache at position lengths[b], and its query
// attends to the lengths[b] + 1 (or the last `window`) positions.
//
// Bound by reading the cache once.  A workgroup takes the heads of one group
// (16 at a time: the columns of a 16x16x32 product) over one stretch of one
// sequence; its four waves walk that stretch in chunks of 32 positions, each on
// its own.  Keys go from memory straight into the operand registers of
// S^T = K Q^T; values pass through the wave's own piece of LDS, which turns
// them round for O^T += V^T P^T.  A long sequence is split over many
// workgroups, whose (maximum, sum, O) a second kernel joins.
//
// 256 rows of up to 2048 positions, 8 groups of 64, bf16: 152 us, 4.5 TB/s of cache rows, where
// a large copy reaches 4.9.  One row of 65536 positions, 4 groups of 128, pages of 64: 34 us
// (5.3 TB/s in the 25 us of the first kernel, 4 us for the join).
#include "attn_common.h"

#include <algorithm>

namespace m3 {

namespace {

struct StepArgs {
  HeadView q, k, v;
  StepCache kc, vc;
  const int32_t *lengths, *table;
  HeadOut out;
  float* ws;  // (maximum, sum) [B, H, splits, 2], then O [B, H, splits, D]
  uint32_t B, H, G, D, capacity, window, num_pages, page_size, max_pages, splits, head_blocks;
  float scale_log2;
};

constexpr int kThreads = 256, kWaves = 4, kChunk = 32;

// [lo, hi) of the positions that row b attends to; none if the row is inactive
// (a length below zero or one that leaves no room for the token).
__device__ __forceinline__ void row_range(const StepArgs& a, int len, int* lo, int* hi) {
  const bool active = len >= 0 && len < (int)a.capacity;
  *hi = active ? len + 1 : 0;
  *lo = active && a.window && len + 1 > (int)a.window ? len + 1 - (int)a.window : 0;
}

template <class T, bool VEC>
__device__ __forceinline__ Raw8<T> read8(const T* p, uint32_t col, uint32_t D) {
  Raw8<T> out;
  if constexpr (VEC) {
    out = *reinterpret_cast<const Raw8<T>*>(p + (col < D ? col : 0));
  } else {
    T e[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = col + i < D ? p[col + i] : (T)0.f;
    __builtin_memcpy(&out, e, sizeof out);
  }
  return out;
}

template <class T, int DP, bool VEC>
__global__ __launch_bounds__(kThreads, sizeof(T) == 4 ? 1 : 2) void attn_step_kernel(const StepArgs a) {
  constexpr int DS = DP / 32, DB = DP / 16, VN = kChunk * DP / 8 / 64;
  using L = Tile<T, DP, kChunk>;
  // values of each wave's chunk, then the waves' sums
  constexpr int kTileBytes = kWaves * L::words * 2, kJoinBytes = kWaves * 16 * (DP + 2) * 4;
  __shared__ __align__(16) unsigned char raw[kTileBytes > kJoinBytes ? kTileBytes : kJoinBytes];

  uint32_t at = blockIdx.x;
  const uint32_t split = at % a.splits;
  at /= a.splits;
  const uint32_t hb = at % a.head_blocks;
  at /= a.head_blocks;
  const uint32_t g = at % a.G, b = at / a.G;
  const uint32_t share = a.H / a.G, heads = min(16u, share - 16 * hb), h0 = g * share + 16 * hb;
  const int tid = threadIdx.x, lane = tid % 64, wave = __builtin_amdgcn_readfirstlane(tid / 64), quad = lane / 16, col = lane % 16;
  uint16_t* vl = reinterpret_cast<uint16_t*>(raw) + wave * L::words;

  const int len = a.lengths[b];
  int lo, hi;
  row_range(a, len, &lo, &hi);
  // the split's stretch, whole chunks for each wave
  const int each = ((hi - lo + (int)a.splits - 1) / (int)a.splits + kChunk * kWaves - 1) / (kChunk * kWaves) *
                   (kChunk * kWaves);
  const int begin = min(hi, lo + (int)split * each), end = min(hi, begin + each);

  const T* kb = static_cast<const T*>(a.kc.p) + (int64_t)g * a.kc.head;
  const T* vb = static_cast<const T*>(a.vc.p) + (int64_t)g * a.vc.head;
  const T* knew = static_cast<const T*>(a.k.p) + (int64_t)b * a.k.row + (int64_t)g * a.k.head;
  const T* vnew = static_cast<const T*>(a.v.p) + (int64_t)b * a.v.row + (int64_t)g * a.v.head;

  // page and row of a position, page -1 where the table names no page
  auto find = [&](int j, int64_t* page, int* row) {
    const uint32_t p = (uint32_t)j / a.page_size;
    *row = (int)((uint32_t)j - p * a.page_size);
    const int id = a.table == nullptr ? (int)b : a.table[(size_t)b * a.max_pages + p];
    *page = id >= 0 && id < (int)a.num_pages ? id : -1;
  };

  // the token's own key and value: written by the workgroup whose stretch holds
  // the position; readers take them from the arguments, never from the cache
  if (hb == 0 && end > begin && end == hi && hi == len + 1) {
    int64_t page;
    int row;
    find(len, &page, &row);
    if (page >= 0)
      for (uint32_t d = tid; d < a.D; d += kThreads) {
        static_cast<T*>(a.kc.p)[page * a.kc.page + row * a.kc.row + (int64_t)g * a.kc.head + d] = knew[d];
        static_cast<T*>(a.vc.p)[page * a.vc.page + row * a.vc.row + (int64_t)g * a.vc.head + d] = vnew[d];
      }
  }

  Frag<T> qf[DS];
#pragma unroll
  for (int s = 0; s < DS; ++s) {
    const uint32_t c = 32 * s + 8 * quad;
    Raw8<T> r = {};
    if (col < (int)heads && c < a.D)
      r = read8<T, VEC>(static_cast<const T*>(a.q.p) + (int64_t)b * a.q.row + (int64_t)(h0 + col) * a.q.head, c, a.D);
    qf[s] = raw_frag<T>(r);
  }

  // A chunk of positions on its way from memory: the table entry is read one
  // chunk before the rows it names, and the rows one chunk before their use.
  auto entry = [&](int j0) {
    const int j = j0 + lane % 32;
    return a.table != nullptr && j < end ? a.table[(size_t)b * a.max_pages + (uint32_t)j / a.page_size] : (int)b;
  };
  struct Chunk {
    Raw8<T> k[2][DS], v[VN];
    uint32_t there;  // which positions there are
  };
  auto read = [&](Chunk& c, int j0, int id) {
    // lane l finds position j0 + l % 32 for all
    const int j = j0 + lane % 32, row = (int)((uint32_t)j % a.page_size);
    const bool mine = j == len && j < end, page = j < end && id >= 0 && id < (int)a.num_pages;
    c.there = (uint32_t)__ballot(mine || page);
    // a position that is not there is read from the token's own row, and dropped below
    const T* kp = mine || !page ? knew : kb + id * a.kc.page + row * a.kc.row;
    const T* vp = mine || !page ? vnew : vb + id * a.vc.page + row * a.vc.row;
    auto from = [&](const T* p, int at) {
      const uint64_t u = (uint64_t)p;
      return (const T*)((uint64_t)(uint32_t)__shfl((int)u, at) | (uint64_t)(uint32_t)__shfl((int)(u >> 32), at) << 32);
    };
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const T* p = from(kp, 16 * u + col);
#pragma unroll
      for (int s = 0; s < DS; ++s) c.k[u][s] = read8<T, VEC>(p, 32 * s + 8 * quad, a.D);
    }
#pragma unroll
    for (int i = 0; i < VN; ++i) {
      const int e = lane + 64 * i;
      c.v[i] = read8<T, VEC>(from(vp, e / (DP / 8)), e % (DP / 8) * 8, a.D);
    }
  };

  floatx4 acc[DB] = {};
  float m = -kInf, sum = 0.f;
  constexpr int kStep = kChunk * kWaves;
  Chunk now, next;
  int j0 = begin + wave * kChunk, id = 0;
  if (j0 < end) {
    read(now, j0, entry(j0));
    id = entry(j0 + kStep);
  }
  for (; j0 < end; j0 += kStep, now = next) {
    if (j0 + kStep < end) {
      read(next, j0 + kStep, id);
      id = entry(j0 + 2 * kStep);
    }
    Raw8<T>(&kr)[2][DS] = now.k;
    Raw8<T>(&vr)[VN] = now.v;
    const uint32_t there = now.there;
    if (there != 0xffffffffu) {
#pragma unroll
      for (int i = 0; i < VN; ++i)
        if (!(there >> (lane + 64 * i) / (DP / 8) & 1)) vr[i] = Raw8<T>{};
    }

    floatx4 s2[2] = {};
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int s = 0; s < DS; ++s) {
        if (32 * s + 8 * quad >= (int)a.D) kr[u][s] = Raw8<T>{};
        s2[u] = mma16<T>(raw_frag<T>(kr[u][s]), qf[s], s2[u]);
      }
    float top = -kInf;
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        s2[u][r] = there >> (16 * u + 4 * quad + r) & 1 ? s2[u][r] * a.scale_log2 : -kInf;
        top = __builtin_fmaxf(top, s2[u][r]);
      }
    top = max_xor32(max_xor16(top));
    if (__any(top > m)) {
      const float to = __builtin_fmaxf(m, top), f = to == -kInf ? 1.f : __builtin_amdgcn_exp2f(m - to);
      sum *= f;
#pragma unroll
      for (int db = 0; db < DB; ++db) acc[db] *= f;
      m = to;
    }
    const float base = m == -kInf ? 0.f : m;
    float p8[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      p8[e] = __builtin_amdgcn_exp2f(s2[e / 4][e % 4] - base);
      sum += p8[e];
    }
    const Frag<T> pf = make_frag<T>(p8);

    // the wave's own LDS: in order within the wave, no barrier
#pragma unroll
    for (int i = 0; i < VN; ++i) {
      const int c = lane + 64 * i;
      const Frag<T> f = raw_frag<T>(vr[i]);
#pragma unroll
      for (int p = 0; p < Pieces<T>::n; ++p)
        *reinterpret_cast<uintx4*>(vl + p * L::plane + L::at(c / (DP / 8), c % (DP / 8) * 8)) = f.p[p];
    }
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int db = 0; db < DB; ++db) {
      const uint16_t *p = vl + L::at(4 * quad + col / 4, 16 * db + 4 * (col % 4)),
                     *p16 = vl + 16 * L::ld + L::at(4 * quad + col / 4, 16 * db + 4 * (col % 4));
      Frag<T> vf;
#pragma unroll
      for (int i = 0; i < Pieces<T>::n; ++i) {
        const uintx2 x = lds_tr4(p + i * L::plane), y = lds_tr4(p16 + i * L::plane);
        vf.p[i] = uintx4{x[0], x[1], y[0], y[1]};
      }
      acc[db] = mma16<T>(vf, pf, acc[db]);
    }
    __builtin_amdgcn_wave_barrier();
  }

  // join the four waves
  sum = sum_xor32(sum_xor16(sum));
  __syncthreads();
  float* join = reinterpret_cast<float*>(raw);  // [wave][head][DP + 2]
  {
    float* mine = join + (wave * 16 + col) * (DP + 2);
    if (quad == 0) {
      mine[0] = m;
      mine[1] = sum;
    }
#pragma unroll
    for (int db = 0; db < DB; ++db)
#pragma unroll
      for (int r = 0; r < 4; ++r) mine[2 + 16 * db + 4 * quad + r] = acc[db][r];
  }
  __syncthreads();
  for (uint32_t e = tid; e < heads * a.D; e += kThreads) {
    const uint32_t hh = e / a.D, d = e % a.D;
    float top = -kInf;
    for (int w = 0; w < kWaves; ++w) top = __builtin_fmaxf(top, join[(w * 16 + hh) * (DP + 2)]);
    float s = 0.f, o = 0.f;
    for (int w = 0; w < kWaves; ++w) {
      const float* p = join + (w * 16 + hh) * (DP + 2);
      const float f = top == -kInf ? 1.f : __builtin_amdgcn_exp2f(p[0] - top);
      s = fmaf(p[1], f, s);
      o = fmaf(p[2 + d], f, o);
    }
    if (a.splits == 1) {
      static_cast<T*>(a.out.p)[(int64_t)b * a.out.row + (int64_t)(h0 + hh) * a.out.head + d] = (T)(s == 0.f ? 0.f : o / s);
    } else {
      const size_t at = ((size_t)b * a.H + h0 + hh) * a.splits + split;
      if (d == 0) *reinterpret_cast<floatx2*>(a.ws + 2 * at) = floatx2{top, s};
      a.ws[2 * (size_t)a.B * a.H * a.splits + at * a.D + d] = o;
    }
  }
}

// Joins the splits of one row and head, 32 columns to a workgroup: eight lanes
// of four columns, and the splits dealt over 32 groups of them.  All of it is
// latency, so the first sums are on their way before the maxima are known, and the
// columns are spread over workgroups (128 splits of 32 heads of 128:
// 18 us with a workgroup to a head).
constexpr int kMaxSplits = 512, kJoinCols = 32;
template <class T, bool VEC>
__global__ __launch_bounds__(kThreads) void attn_step_join(const StepArgs a) {
  constexpr int kGroups = kThreads / 8, kAhead = 4;
  __shared__ float factor[kMaxSplits], red[2][kWaves];
  __shared__ __align__(16) float cols[kGroups][kJoinCols + 4];
  const int tid = threadIdx.x, lane = tid % 64, wave = tid / 64, grp = tid / 8;
  const uint32_t slices = (a.D + kJoinCols - 1) / kJoinCols, bh = blockIdx.x / slices;
  const uint32_t b = bh / a.H, h = bh % a.H, n = a.splits, col = blockIdx.x % slices * kJoinCols + tid % 8 * 4;
  const size_t at = (size_t)bh * n;
  const floatx2* ms = reinterpret_cast<const floatx2*>(a.ws) + at;
  const float* o = a.ws + 2 * (size_t)a.B * a.H * n + at * a.D;
  const auto part = [&](uint32_t i) {
    floatx4 v = {};
    if (i >= n) return v;
    const float* p = o + (size_t)i * a.D;
    if constexpr (VEC) {
      if (col < a.D) v = *reinterpret_cast<const floatx4*>(p + col);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (col + e < a.D) v[e] = p[col + e];
    }
    return v;
  };
  floatx2 mine[kMaxSplits / kThreads];
#pragma unroll
  for (int i = 0; i < kMaxSplits / kThreads; ++i)
    mine[i] = tid + i * kThreads < (int)n ? ms[tid + i * kThreads] : floatx2{-kInf, 0.f};
  floatx4 ahead[kAhead];
#pragma unroll
  for (int i = 0; i < kAhead; ++i) ahead[i] = part(grp + i * kGroups);

  float top = mine[0][0];
#pragma unroll
  for (int i = 1; i < kMaxSplits / kThreads; ++i) top = __builtin_fmaxf(top, mine[i][0]);
  for (int x = 1; x < 64; x *= 2) top = __builtin_fmaxf(top, __shfl_xor(top, x));
  if (lane == 0) red[0][wave] = top;
  __syncthreads();
  top = __builtin_fmaxf(max3(red[0][0], red[0][1], red[0][2]), red[0][3]);
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < kMaxSplits / kThreads; ++i) {
    const float f = top == -kInf ? 1.f : __builtin_amdgcn_exp2f(mine[i][0] - top);
    factor[tid + i * kThreads] = f;
    s = fmaf(mine[i][1], f, s);
  }
  for (int x = 1; x < 64; x *= 2) s += __shfl_xor(s, x);
  if (lane == 0) red[1][wave] = s;
  __syncthreads();
  s = (red[1][0] + red[1][1]) + (red[1][2] + red[1][3]);
  floatx4 sum = {};
#pragma unroll
  for (int i = 0; i < kAhead; ++i) sum += ahead[i] * factor[grp + i * kGroups];
  for (uint32_t i = grp + kAhead * kGroups; i < n; i += kGroups) sum += part(i) * factor[i];
  *reinterpret_cast<floatx4*>(&cols[grp][tid % 8 * 4]) = sum;
  __syncthreads();
  const uint32_t d = blockIdx.x % slices * kJoinCols + tid;
  if (tid < kJoinCols && d < a.D) {
    float v = 0.f;
#pragma unroll
    for (int k = 0; k < kGroups; ++k) v += cols[k][tid];
    static_cast<T*>(a.out.p)[(int64_t)b * a.out.row + (int64_t)h * a.out.head + d] = (T)(s == 0.f ? 0.f : v / s);
  }
}

// Stretches of a sequence: enough workgroups for two on each compute unit,
// none shorter than two chunks for each wave at the cache's full length.
uint32_t plan_splits(const AttnGeom& g) {
  const uint32_t head_blocks = (g.H / g.G + 15) / 16;
  const uint64_t rows = (uint64_t)g.B * g.G * head_blocks;
  const uint32_t seen = g.window && g.window < g.Lk ? g.window : g.Lk;
  const uint64_t want = (512 + rows - 1) / rows, most = (seen + 2 * kChunk * kWaves - 1) / (2 * kChunk * kWaves);
  return (uint32_t)(want < most ? want : most);
}

template <class T>
hipError_t launch(const AttnGeom& g, const StepArgs& a, hipStream_t stream) {
  const dim3 grid(a.splits * a.head_blocks * g.G * g.B);
  const bool vec = a.q.vec && a.k.vec && a.v.vec && a.kc.vec && a.vc.vec;
#define M3_CALL(DP)                                                           \
  (vec ? attn_step_kernel<T, DP, true><<<grid, kThreads, 0, stream>>>(a)      \
       : attn_step_kernel<T, DP, false><<<grid, kThreads, 0, stream>>>(a),    \
   hipGetLastError())
  const hipError_t e = M3_HEAD_DIM_SWITCH(g.D, M3_CALL);
#undef M3_CALL
  if (e != hipSuccess || a.splits == 1) return e;
  const dim3 join(g.B * g.H * ((g.D + kJoinCols - 1) / kJoinCols));
  // (the sums stand behind 2 B H splits floats and are D apart)
  if (g.D % 4 == 0 && g.B * g.H * a.splits % 2 == 0)
    attn_step_join<T, true><<<join, kThreads, 0, stream>>>(a);
  else
    attn_step_join<T, false><<<join, kThreads, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace

uint64_t attn_step_workgroups(const AttnGeom& g) {
  const uint64_t splits = plan_splits(g), heads = (uint64_t)g.B * g.H;
  return std::max((uint64_t)g.B * g.G * ((g.H / g.G + 15) / 16) * splits,
                  splits > 1 ? heads * ((g.D + kJoinCols - 1) / kJoinCols) : 0);
}

size_t attn_step_workspace_floats(const AttnGeom& g) {
  const uint32_t splits = plan_splits(g);
  return splits == 1 ? 0 : (size_t)g.B * g.H * splits * (g.D + 2);
}

hipError_t launch_attn_step(const AttnGeom& g, const AttnStepOperands& o, hipStream_t stream) {
  StepArgs a{o.q, o.k, o.v, o.kc, o.vc, o.lengths, o.table, o.out, o.ws, g.B, g.H, g.G, g.D, g.Lk, g.window,
             o.num_pages, o.page_size, o.max_pages, plan_splits(g), (g.H / g.G + 15) / 16, g.scale * kLog2e};
  if (g.dtype == kF32) return launch<float>(g, a, stream);
  if (g.dtype == kF16) return launch<_Float16>(g, a, stream);
  return launch<__bf16>(g, a, stream);
}

}  // namespace m3

// The decode step over an 8-bit key / value cache: one or a few new tokens of
// each row, their queries against the positions that they see.
//
// Bound by reading the cache once.  A workgroup takes the heads of one group
// and all new tokens of a row (16 NT columns of a 16x16x32 product) over one
// stretch of the row's positions; its four waves walk that stretch in tiles of 128,
// 32 positions each, on their own.  Codes go from memory straight into
// registers and become the operands of S^T = K Q^T and O^T += V^T P^T there:
// e4m3 times a power of two is exact in bfloat16, so both take bfloat16
// products whatever the queries' type, which are split in two pieces (float16) or
// three (float32), as are their probabilities.  A value's fragment wants
// eight positions of one column: a lane reads the same few columns of each of its
// eight rows, and byte permutes turn them round; no LDS is needed.
#include "attn_join.h"
#include "kv8_common.h"

#include <algorithm>

namespace m3 {

namespace {

struct StepArgs {
  HeadView q;
  Kv8Cache kc, vc;
  const int32_t *lengths, *table;
  HeadOut out;
  float* ws;  // as JoinArgs
  uint32_t B, T, H, G, D, capacity, window, sinks, block, num_pages, page_size, max_pages, scale_blocks;
  uint32_t splits, col_blocks;
  float scale_log2;
};

constexpr int kThreads = 256, kWaves = 4, kChunk = 32, kTile = kChunk * kWaves;

// Queries and probabilities as bfloat16 pieces: float16 fits two exactly, float32 three.
template <class T>
struct QPieces {
  static constexpr int n = sizeof(T) == 4 ? 3 : __is_same(T, _Float16) ? 2 : 1;
};
template <int N>
struct Bf16Pieces {
  uintx4 p[N];
};
template <int N>
__device__ __forceinline__ Bf16Pieces<N> pieces_of(const float* v) {
  Bf16Pieces<N> f;
  if constexpr (N == 3) {
    split8_bf16x3(v, f.p[0], f.p[1], f.p[2]);
  } else {
    float rest[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const unsigned h = pack2<__bf16>(v[2 * i], v[2 * i + 1]);
      f.p[0][i] = h;
      rest[2 * i] = v[2 * i] - __uint_as_float(h << 16);
      rest[2 * i + 1] = v[2 * i + 1] - __uint_as_float(h & 0xffff0000u);
    }
    if constexpr (N == 2) {
#pragma unroll
      for (int i = 0; i < 4; ++i) f.p[1][i] = pack2<__bf16>(rest[2 * i], rest[2 * i + 1]);
    }
  }
  return f;
}
// Smallest pieces first.
template <int N>
__device__ __forceinline__ floatx4 mma_exact(uintx4 a, const Bf16Pieces<N>& b, floatx4 c) {
#pragma unroll
  for (int i = N - 1; i >= 0; --i) c = mfma_bf16(a, b.p[i], c);
  return c;
}

// Eight codes of one row as a fragment.
__device__ __forceinline__ uintx4 widen8(uintx2 w, float scale) {
  uintx4 f;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    f[2 * i] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[i], scale, false));
    f[2 * i + 1] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[i], scale, true));
  }
  return f;
}

// The columns of a value row that lane i of 16 reads, and the bytes of them in each of its words: DP / 16
// neighbours, which for 96 are four of the first 64 and two of the last 32.
template <int DP>
__device__ __forceinline__ int value_column(int i, int db) {
  if constexpr (DP == 96) return db < 4 ? 4 * i + db : 64 + 2 * i + db - 4;
  return i * (DP / 16) + db;
}

// One chunk of 32 positions in registers: two halves of 16, each in one page and one block.
template <int DP>
struct Chunk {
  static constexpr int DS = DP / 32, VW = (DP + 63) / 64;  // value words of a row and lane
  uintx2 k[2][DS];
  uint32_t v[2][4][VW];
  uint32_t ks[2], vs[2];  // scale bytes
  int there[2];           // how many of a half's positions there are
};

// Whether any byte is one of e4m3's two NaN codes.
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) { return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; }

template <class T, int DP, int NT, bool VEC>
__global__ __launch_bounds__(kThreads, 2) void attn_step_kv8_kernel(const StepArgs a) {
  constexpr int DS = DP / 32, DB = DP / 16, VW = Chunk<DP>::VW, QN = QPieces<T>::n;
  __shared__ __align__(16) float join[kWaves * 16 * (DP + 2)];

  // All groups of a row's stretch go to one XCD: their rows share cache lines.
  const uint32_t inner = a.G * a.col_blocks, turn = blockIdx.x / 8;
  const uint32_t unit = turn / inner * 8 + blockIdx.x % 8;
  if (unit >= a.B * a.splits) return;
  const uint32_t g = turn % inner / a.col_blocks, cb = turn % inner % a.col_blocks;
  const uint32_t b = unit / a.splits, split = unit % a.splits;
  const uint32_t share = a.H / a.G, columns = share * a.T, c0 = cb * 16 * NT;
  const int tid = threadIdx.x, lane = tid % 64, wave = __builtin_amdgcn_readfirstlane(tid / 64), quad = lane / 16,
            col = lane % 16;

  // Positions that the row's queries see: [0, sinks) and [lo, hi), in tiles.
  const int len = __builtin_amdgcn_readfirstlane(a.lengths[b]);
  const bool active = len >= 0 && (int64_t)len + a.T <= (int64_t)a.capacity;
  const int hi = active ? len + (int)a.T : 0;
  const int lo = active && a.window && len + 1 > (int)a.window ? len + 1 - (int)a.window : 0;
  const int sinks = min((int)a.sinks, lo);
  const int sink_tiles = (sinks + kTile - 1) / kTile, window_tile = max(lo / kTile, sink_tiles);
  const int tiles = sink_tiles + (hi + kTile - 1) / kTile - window_tile;
  const int each = (tiles + (int)a.splits - 1) / (int)a.splits;
  const int t0 = min(tiles, (int)split * each), t1 = min(tiles, t0 + each);

  // This lane's columns: token and head.
  int token[NT], head[NT];
  Bf16Pieces<QN> qf[NT][DS];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const uint32_t c = c0 + 16 * n + col;
    token[n] = (int)(c / share);
    head[n] = (int)(g * share + c % share);
#pragma unroll
    for (int s = 0; s < DS; ++s) {
      float f[8] = {};
      const uint32_t d = 32 * s + 8 * quad;
      if (c < columns && d < a.D) {
        const T* p = static_cast<const T*>(a.q.p) + ((int64_t)b * a.T + token[n]) * a.q.row + (int64_t)head[n] * a.q.head;
        if (a.q.vec) {
          raw_floats<T>(*reinterpret_cast<const Raw8<T>*>(p + d), f);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) f[e] = d + e < a.D ? to_float(p[d + e]) : 0.f;
        }
      }
      qf[n][s] = pieces_of<QN>(f);
    }
  }

  // Byte offsets of this lane's codes in a half of 16 rows.
  uint32_t ko[DS], vo[4][VW];
#pragma unroll
  for (int s = 0; s < DS; ++s) {
    const uint32_t d = 32 * s + 8 * quad;
    ko[s] = d < a.D ? (uint32_t)col * (uint32_t)a.kc.row + d : kOutside;
  }
#pragma unroll
  for (int r = 0; r < 4; ++r)
#pragma unroll
    for (int w = 0; w < VW; ++w) {
      const uint32_t d = value_column<DP>(col, 4 * w);
      vo[r][w] = d < a.D ? (uint32_t)(4 * quad + r) * (uint32_t)a.vc.row + d : kOutside;
    }

  auto read = [&](Chunk<DP>& c, int j0) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int j = j0 + 16 * u;
      const bool seen = j < hi && (j + 15 >= lo || j < sinks);
      Slot slot{-1, 0};
      if (seen) slot = find_slot(a.table, b, (uint32_t)j, a.page_size, a.max_pages, a.num_pages);
      const int page = __builtin_amdgcn_readfirstlane(slot.page);
      const uint32_t row = __builtin_amdgcn_readfirstlane(slot.row);
      const int rows = page >= 0 ? min(16, hi - j) : 0, at = max(page, 0);
      c.there[u] = rows;
      const rsrc_t kr = make_rsrc(a.kc.codes + at * a.kc.page + (int64_t)row * a.kc.row + (int64_t)g * a.kc.head,
                                  rows ? (uint32_t)(rows - 1) * (uint32_t)a.kc.row + a.D : 0);
      const rsrc_t vr = make_rsrc(a.vc.codes + at * a.vc.page + (int64_t)row * a.vc.row + (int64_t)g * a.vc.head,
                                  rows ? (uint32_t)(rows - 1) * (uint32_t)a.vc.row + a.D : 0);
      const size_t block = ((size_t)at * a.G + g) * a.scale_blocks + row / a.block;
      c.ks[u] = rows ? a.kc.scales[block] : kExpBias;
      c.vs[u] = rows ? a.vc.scales[block] : kExpBias;
#pragma unroll
      for (int s = 0; s < DS; ++s) {
        if constexpr (VEC) {
          c.k[u][s] = __builtin_bit_cast(uintx2, __builtin_amdgcn_raw_buffer_load_b64(kr, ko[s], 0, 0));
        } else {
          c.k[u][s] = uintx2{};
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const uint32_t o = 32 * s + 8 * quad + e < a.D ? ko[s] + e : kOutside;
            c.k[u][s][e / 4] |= (uint32_t)(uint8_t)__builtin_amdgcn_raw_buffer_load_b8(kr, o, 0, 0) << 8 * (e % 4);
          }
        }
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        if constexpr (!VEC) {
#pragma unroll
          for (int w = 0; w < VW; ++w) {
            c.v[u][r][w] = 0;
#pragma unroll
            for (int e = 0; e < 4 && 4 * w + e < DB; ++e) {
              const uint32_t d = value_column<DP>(col, 4 * w + e), o = d < a.D ? vo[r][w] + e : kOutside;
              c.v[u][r][w] |= (uint32_t)(uint8_t)__builtin_amdgcn_raw_buffer_load_b8(vr, o, 0, 0) << 8 * e;
            }
          }
        } else if constexpr (DP == 128) {
          const uintx2 x = __builtin_bit_cast(uintx2, __builtin_amdgcn_raw_buffer_load_b64(vr, vo[r][0], 0, 0));
          c.v[u][r][0] = x[0];
          c.v[u][r][1] = x[1];
        } else if constexpr (DP == 32) {
          c.v[u][r][0] = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(vr, vo[r][0], 0, 0);
        } else {
          c.v[u][r][0] = (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(vr, vo[r][0], 0, 0);
          if constexpr (DP == 96) c.v[u][r][1] = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(vr, vo[r][1], 0, 0);
        }
      }
    }
  };

  floatx4 acc[NT][DB] = {};
  float m[NT], sum[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    m[n] = -kInf;
    sum[n] = 0.f;
  }
  auto start = [&](int t) { return (t < sink_tiles ? t : t - sink_tiles + window_tile) * kTile + wave * kChunk; };
  Chunk<DP> now, next;
  if (t0 < t1) read(now, start(t0));
  for (int t = t0; t < t1; ++t, now = next) {
    const int j0 = start(t);
    if (t + 1 < t1) read(next, start(t + 1));
    if (now.there[0] + now.there[1] == 0) continue;
    // whether every query sees all of the chunk
    const bool whole = now.there[0] == 16 && now.there[1] == 16 && j0 + kChunk - 1 <= len &&
                       (!a.window || j0 > hi - 1 - (int)a.window || j0 + kChunk <= (int)a.sinks);

    uintx4 kf[2][DS];
    const float ks[2] = {scale_value(now.ks[0]), scale_value(now.ks[1])},
                vs[2] = {scale_value(now.vs[0]), scale_value(now.vs[1])};
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int s = 0; s < DS; ++s) kf[u][s] = widen8(now.k[u][s], ks[u]);

    Bf16Pieces<QN> pf[NT];
    bool hidden[NT][8];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      floatx4 s2[2] = {};
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int s = 0; s < DS; ++s) s2[u] = mma_exact<QN>(kf[u][s], qf[n][s], s2[u]);
      float z[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) z[e] = s2[e / 4][e % 4] * a.scale_log2;
      if (!whole) {
        const int last = len + token[n];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int r = 4 * quad + e % 4, j = j0 + 16 * (e / 4) + r;
          hidden[n][e] = r >= now.there[e / 4] || j > last ||
                         (a.window && j <= last - (int)a.window && j >= (int)a.sinks);
          z[e] = hidden[n][e] ? -kInf : z[e];
        }
      }
      float top = z[0];
#pragma unroll
      for (int e = 1; e < 8; ++e) top = __builtin_fmaxf(top, z[e]);
      top = max_xor32(max_xor16(top));
      if (__any(top > m[n])) {
        const float to = __builtin_fmaxf(m[n], top), f = to == -kInf ? 1.f : __builtin_amdgcn_exp2f(m[n] - to);
        sum[n] *= f;
#pragma unroll
        for (int db = 0; db < DB; ++db) acc[n][db] *= f;
        m[n] = to;
      }
      const float base = m[n] == -kInf ? 0.f : m[n];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        z[e] = __builtin_amdgcn_exp2f(z[e] - base);
        sum[n] += z[e];
      }
      pf[n] = pieces_of<QN>(z);
    }

    // A NaN among values that some of the queries do not see must not reach those: it is taken out of the product
    // and given to the queries that see it.
    bool odd = false;
    if (!whole) {
      uint32_t bad = 0;
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
          for (int w = 0; w < VW; ++w) bad |= nan_bytes(now.v[u][r][w]);
      odd = __any(bad != 0);
    }

#pragma unroll
    for (int w = 0; w < VW; ++w) {
      // columns 4 w .. 4 w + 3 of the lane's: two of them in each permuted word, for two rows
      uint32_t x[2][2][2];  // [half][rows 0 1 or 2 3][columns 0 1 or 2 3]
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const uint32_t p = now.v[u][2 * r][w], q = now.v[u][2 * r + 1][w];
          x[u][r][0] = __builtin_amdgcn_perm(q, p, 0x05010400u);
          x[u][r][1] = __builtin_amdgcn_perm(q, p, 0x07030602u);
        }
#pragma unroll
      for (int d = 0; d < 4 && 4 * w + d < DB; ++d) {
        const int db = 4 * w + d;
        uintx4 vf, mark = {};
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            uint32_t codes = x[u][r][d / 2];
            if (odd) {
              const uint32_t bad = nan_bytes(codes) >> 7;  // 1 in each NaN's byte
              codes &= ~(bad * 0xffu);
              const uint32_t two = d % 2 ? bad >> 16 : bad;
              mark[2 * u + r] = (two & 1u ? 0x3f80u : 0u) | (two & 0x100u ? 0x3f800000u : 0u);
            }
            vf[2 * u + r] = __builtin_bit_cast(
                unsigned, d % 2 ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes, vs[u], true)
                                : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes, vs[u], false));
          }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          acc[n][db] = mma_exact<QN>(vf, pf[n], acc[n][db]);
          if (odd) {
            uintx4 sees;
#pragma unroll
            for (int i = 0; i < 4; ++i)
              sees[i] = (hidden[n][2 * i] ? 0u : 0x3f80u) | (hidden[n][2 * i + 1] ? 0u : 0x3f800000u);
            const floatx4 count = mfma_bf16(mark, sees, floatx4{});
#pragma unroll
            for (int r = 0; r < 4; ++r) acc[n][db][r] = count[r] > 0.f ? __builtin_nanf("") : acc[n][db][r];
          }
        }
      }
    }
  }

  // join the four waves, 16 columns at a time
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    if (c0 + 16 * n >= columns) break;
    if (n) __syncthreads();
    const float s = sum_xor32(sum_xor16(sum[n]));
    float* mine = join + (wave * 16 + col) * (DP + 2);
    if (quad == 0) {
      mine[0] = m[n];
      mine[1] = s;
    }
#pragma unroll
    for (int db = 0; db < DB; ++db)
#pragma unroll
      for (int r = 0; r < 4; ++r) mine[2 + value_column<DP>(4 * quad + r, db)] = acc[n][db][r];
    __syncthreads();
    const uint32_t many = min(16u, columns - (c0 + 16 * n));
    for (uint32_t e = tid; e < many * a.D; e += kThreads) {
      const uint32_t c = e / a.D, d = e % a.D, at = c0 + 16 * n + c;
      float top = -kInf;
      for (int w = 0; w < kWaves; ++w) top = __builtin_fmaxf(top, join[(w * 16 + c) * (DP + 2)]);
      float l = 0.f, o = 0.f;
      for (int w = 0; w < kWaves; ++w) {
        const float* p = join + (w * 16 + c) * (DP + 2);
        const float f = top == -kInf ? 1.f : __builtin_amdgcn_exp2f(p[0] - top);
        l = fmaf(p[1], f, l);
        o = fmaf(p[2 + d], f, o);
      }
      const size_t row = (size_t)b * a.T + at / share, h = g * share + at % share;
      if (a.splits == 1) {
        static_cast<T*>(a.out.p)[(int64_t)row * a.out.row + (int64_t)h * a.out.head + d] = (T)(l == 0.f ? 0.f : o / l);
      } else {
        const size_t part = (row * a.H + h) * a.splits + split;
        if (d == 0) *reinterpret_cast<floatx2*>(a.ws + 2 * part) = floatx2{top, l};
        a.ws[2 * (size_t)a.B * a.T * a.H * a.splits + part * a.D + d] = o;
      }
    }
  }
}

uint32_t column_tiles(const Kv8Geom& g) { return g.H / g.G * g.T > 16 ? 2 : 1; }
uint32_t column_blocks(const Kv8Geom& g) {
  const uint32_t n = 16 * column_tiles(g);
  return (g.H / g.G * g.T + n - 1) / n;
}
// Stretches of a row: enough workgroups for two on each compute unit, none
// shorter than two chunks for each wave at the longest row.
uint32_t plan_splits(const Kv8Geom& g) {
  const uint64_t rows = (uint64_t)g.B * g.G * column_blocks(g);
  const uint64_t seen = g.window ? std::min((uint64_t)g.capacity, (uint64_t)g.window + g.T + g.sinks) : g.capacity;
  const uint64_t want = (512 + rows - 1) / rows, most = (seen + 2 * kTile - 1) / (2 * kTile);
  return (uint32_t)std::min({want, most, (uint64_t)kMaxSplits});
}

template <class T, int NT>
hipError_t launch_tiles(const Kv8Geom& g, const StepArgs& a, hipStream_t stream) {
  const dim3 grid((uint32_t)((g.B * a.splits + 7) / 8 * 8 * g.G * a.col_blocks));
  const bool vec = a.kc.vec && a.vc.vec;
#define M3_CALL(DP)                                                                \
  (vec ? attn_step_kv8_kernel<T, DP, NT, true><<<grid, kThreads, 0, stream>>>(a)   \
       : attn_step_kv8_kernel<T, DP, NT, false><<<grid, kThreads, 0, stream>>>(a), \
   hipGetLastError())
  return M3_HEAD_DIM_SWITCH(g.D, M3_CALL);
#undef M3_CALL
}
template <class T>
hipError_t launch(const Kv8Geom& g, const StepArgs& a, hipStream_t stream) {
  const hipError_t e = column_tiles(g) == 1 ? launch_tiles<T, 1>(g, a, stream) : launch_tiles<T, 2>(g, a, stream);
  if (e != hipSuccess || a.splits == 1) return e;
  return launch_join<T>(JoinArgs{a.ws, a.out, g.B * g.T, g.H, g.D, a.splits}, stream);
}

}  // namespace

uint64_t attn_step_kv8_workgroups(const Kv8Geom& g) {
  const uint64_t splits = plan_splits(g), rows = (uint64_t)g.B * g.T;
  return std::max({(g.B * splits + 7) / 8 * 8 * g.G * column_blocks(g), splits > 1 ? join_workgroups(rows, g.H, g.D) : 0,
                   kv8_write_workgroups(g)});
}

size_t attn_step_kv8_workspace_floats(const Kv8Geom& g) {
  const uint32_t splits = plan_splits(g);
  return splits == 1 ? 0 : join_floats((uint64_t)g.B * g.T, g.H, g.D, splits);
}

hipError_t launch_attn_step_kv8(const Kv8Geom& g, const Kv8Operands& o, hipStream_t stream) {
  if (o.k.p != nullptr) {
    const hipError_t e = launch_kv8_write(g, o, stream);
    if (e != hipSuccess) return e;
  }
  const StepArgs a{o.q, o.kc, o.vc, o.lengths, o.table, o.out, o.ws, g.B, g.T, g.H, g.G, g.D, g.capacity, g.window,
                   g.sinks, g.block, g.num_pages, g.page_size, g.max_pages, (g.page_size + g.block - 1) / g.block,
                   plan_splits(g), column_blocks(g), g.scale * kLog2e};
  if (g.dtype == kF32) return launch<float>(g, a, stream);
  if (g.dtype == kF16) return launch<_Float16>(g, a, stream);
  return launch<__bf16>(g, a, stream);
}

}  // namespace m3

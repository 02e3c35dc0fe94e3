// The decode step over an 8-bit key / value cache: one or a few new tokens of
// each row, their queries against the positions that they see.
//
// Bound by reading the cache once.  A workgroup takes the heads of one group
// and all new tokens of a row (16 NT columns of a 16x16x32 product) over one
// stretch of the row's positions; its waves walk that stretch in chunks of 32
// positions, each on its own.  Codes go from memory straight into
// registers and become the operands of S^T = K Q^T and O^T += V^T P^T there:
// a code is exact in bfloat16 and float16, and a value, code times a power of
// two, in bfloat16.  A value's fragment wants eight positions of one column: a
// lane reads the same few columns of each of its eight rows, and byte permutes
// turn them round; no LDS is needed.  Each half of a chunk lies in one page and
// one block, so that addresses and scales are the wave's, and a buffer
// resource that ends with the row's last position leaves out what is not there.
//
// 256 rows of up to 2048 positions, 24 heads of 64 over 8, bf16: 73.7 us (4.7 TB/s; a large copy reaches 5.0),
// 67 if the cache holds the tokens already.  One row of 65536, 32 heads of 128 over 4, pages of 64: 18.0 us,
// then 3.9 for the join.  64 rows of up to 4096, four float16 tokens, 32 heads of 128 over 4: 54 us (bfloat16 55),
// which are the longest row's, a compute unit to each of its groups: 12.7 for the first 256 positions, then 2.3 for
// each 256, though no other row had any (two waves to a SIMD; it is not memory that holds them).  A third chunk on
// its way did not pay: at 64 columns a wave to a SIMD is lost (73 -> 79 us), at 128 the row of 65536 took 22.5
// for 20.
#pragma once

#include "attn_join.h"
#include "kv8_common.h"
#include "kv8_step.h"

namespace m3 {

namespace {

constexpr int kChunk = 32;

// Queries and probabilities, as operands: bfloat16 queries are their own operand, and so are float16 ones (codes
// are exact in float16 too); float32 fits three bfloat16 pieces, in queries and probabilities.  For 16-bit results
// probabilities are two bfloat16 pieces, 16 bits at any size: one would cost bfloat16 results as much again as their
// own rounding, for some 1 % of the time.
template <class T>
struct Operands {
  static constexpr bool half = __is_same(T, _Float16);
  static constexpr int q = sizeof(T) == 4 ? 3 : 1, p = sizeof(T) == 4 ? 3 : 2;
};
template <int N>
struct Pieced {
  uintx4 p[N];
};
template <int N>
__device__ __forceinline__ Pieced<N> bf16_pieces(const float* v) {
  Pieced<N> f;
  if constexpr (N == 3) {
    split8_bf16x3(v, f.p[0], f.p[1], f.p[2]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const unsigned h = pack2<__bf16>(v[2 * i], v[2 * i + 1]);
      f.p[0][i] = h;
      if constexpr (N == 2)
        f.p[1][i] = pack2<__bf16>(v[2 * i] - __uint_as_float(h << 16), v[2 * i + 1] - __uint_as_float(h & 0xffff0000u));
    }
  }
  return f;
}
// Products of bfloat16 pieces, smallest first.
template <int N>
__device__ __forceinline__ floatx4 mma_pieces(uintx4 a, const Pieced<N>& b, floatx4 c) {
#pragma unroll
  for (int i = N - 1; i >= 0; --i) c = mfma_bf16(a, b.p[i], c);
  return c;
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

// Where a wave reads: position, and the page and row of the two halves of its chunk.
struct Place {
  int t, j;            // tile and first position
  uint32_t page, row;  // of the first half, as entry of the table and row of the page
};

// Bit 7 of the bytes that are no finite number: the NaN codes, and at a scale byte b from 247 on codes from 8 (262 - b)
// on, which stand for 2^128 and more (m3_kv8_write leaves none, but memory that it never wrote may hold them).
__device__ __forceinline__ uint32_t past_finite(uint32_t b) {
  return 0x01010101u * (uint32_t)max(1, 8 * (int)min(b, 254u) - 1968);
}
__device__ __forceinline__ uint32_t not_finite(uint32_t w, uint32_t past) {
  return ((w & 0x7f7f7f7fu) + past) & 0x80808080u;
}

// A word that this kernel does not write, through the scalar cache.  (The kernel's stores keep the compiler from it,
// and a vector load is waited for behind all rows that were asked for before.)
__device__ __forceinline__ int scalar_load(const int32_t* p) {
  return *(const __attribute__((address_space(4))) int32_t*)(uintptr_t)p;
}

// a / b for numbers below 2^24, which takes a few instructions.  (Nothing that a launch can hold is larger.)
__device__ __forceinline__ uint32_t divide(uint32_t a, uint32_t b) { return (a & 0xffffffu) / (b & 0xffffffu); }

// A value that all lanes share, in a scalar register.  (Divisions run on the vector unit, and the compiler would leave
// there what follows from them.)
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return (uint32_t)__builtin_amdgcn_readfirstlane((int)v); }

// One wave writes a row's new tokens [begin, end) into their block of one head, as kv8_write_kernel does.
template <class T, bool VEC>
__device__ __forceinline__ void write_block(const HeadView& x, const Kv8Cache& c, const Kv8StepArgs& a, uint32_t b,
                                            uint32_t g, int len, int first, int lane) {
  const int block = 1 << a.log_block, begin = max(first, len), end = min(first + block, len + (int)a.T);
  const T* rows = static_cast<const T*>(x.p) + ((int64_t)b * a.T + (begin - len)) * x.row + (int64_t)g * x.head;
  const uint32_t per_row = (a.D + 7) / 8, pieces = (uint32_t)(end - begin) * per_row;
  auto piece = [&](uint32_t i) {
    const uint32_t token = divide(i, per_row);
    return read_elements<T, VEC>(rows + (int64_t)token * x.row, 8 * (i - token * per_row), a.D);
  };
  // a lane's first piece stays in registers: most often there are no others
  Raw8<T> mine = {};
  if (lane < (int)pieces) mine = piece(lane);
  const uint32_t entry = uniform((uint32_t)first / a.page_size), row = (uint32_t)first - entry * a.page_size;
  const int page = a.table == nullptr ? (int)b : scalar_load(a.table + (size_t)b * a.max_pages + entry);
  if (page < 0 || page >= (int)a.num_pages) return;
  uint8_t* codes = c.codes + page * c.page + (int64_t)row * c.row + (int64_t)g * c.head;
  uint8_t* scale = c.scales + ((size_t)page * a.G + g) * a.scale_blocks + (row >> a.log_block);
  const int had = begin > first ? held_exponent(*scale) : kLeastExp;
  float amax = max_finite8<T>(mine, 0.f);
  for (uint32_t i = lane + 64; i < pieces; i += 64) amax = max_finite8<T>(piece(i), amax);
  const int e = max(least_exponent(wave_max_nn(amax)), had);
  if (lane == 0) *scale = (uint8_t)(e + kExpBias);
  if (begin > first && e > had) {
    const float down = power_of_two(max(had - e, -126));
    for (uint32_t i = lane; i < (uint32_t)(begin - first) * per_row; i += 64) {
      const uint32_t token = divide(i, per_row), col = 8 * (i - token * per_row);
      uint8_t* p = codes + (int64_t)token * c.row;
      write_codes<VEC>(p, col, a.D, rescale8(read_codes<VEC>(p, col, a.D), down));
    }
  }
  const float inv = power_of_two(-e);
  for (uint32_t i = lane; i < pieces; i += 64) {
    if (i >= 64) mine = piece(i);
    const uint32_t token = divide(i, per_row), col = 8 * (i - token * per_row);
    write_codes<VEC>(codes + (int64_t)(begin - first + (int)token) * c.row, col, a.D, quantise8<T>(mine, inv));
  }
}

template <class T, int DP, int NT, int NW, bool VEC>
__global__ __launch_bounds__(64 * NW, NW == 4 ? 2 : 1) void attn_step_kv8_kernel(const Kv8StepArgs a) {
  constexpr int DS = DP / 32, DB = DP / 16, VW = Chunk<DP>::VW, QN = Operands<T>::q, PN = Operands<T>::p;
  constexpr int kTile = kChunk * NW, kThreads = 64 * NW, kWaves = NW;
  constexpr int kJoinRow = DP + 4;
  __shared__ __align__(16) float join[kWaves * 16 * kJoinRow];
  __shared__ floatx2 join_ms[kWaves][16];

  // All groups of a row's stretch go to one XCD: their rows share cache lines.
  const uint32_t inner = a.G * a.col_blocks, turn = blockIdx.x / 8;
  const uint32_t eight = uniform(divide(turn, inner)), unit = eight * 8 + blockIdx.x % 8;
  if (unit >= a.B * a.splits) return;
  const uint32_t g = uniform(divide(turn - eight * inner, a.col_blocks)), cb = turn - eight * inner - g * a.col_blocks;
  const uint32_t b = uniform(divide(unit, a.splits)), split = unit - b * a.splits;
  const uint32_t share = uniform(divide(a.H, a.G)), columns = share * a.T, c0 = cb * 16 * NT;
  const int tid = threadIdx.x, lane = tid % 64, wave = __builtin_amdgcn_readfirstlane(tid / 64), quad = lane / 16,
            col = lane % 16;

  const int len = scalar_load(a.lengths + b);
  // Positions that the row's queries see: [0, sinks) and [lo, hi), in tiles.
  const bool active = len >= 0 && (int64_t)len + a.T <= (int64_t)a.capacity;
  const int hi = active ? len + (int)a.T : 0;
  const int lo = active && a.window && len + 1 > (int)a.window ? len + 1 - (int)a.window : 0;
  const int sinks = min((int)a.sinks, lo);
  const int sink_tiles = (sinks + kTile - 1) / kTile, window_tile = max(lo / kTile, sink_tiles);
  const int tiles = sink_tiles + (hi + kTile - 1) / kTile - window_tile;
  const int each = (int)uniform(divide((uint32_t)(tiles + (int)a.splits - 1), a.splits));
  const int t0 = min(tiles, (int)split * each), t1 = min(tiles, t0 + each);

  // The row's new tokens go into the cache first: the workgroup whose stretch holds a block writes it, two waves to a
  // block.  (A block lies in one tile, and nobody else reads that tile of this head.)  The first of those tiles is
  // read behind a barrier that the writers meet when their stores are done, which is enough: writer and readers share
  // a compute unit and its first-level cache.  (A fence over the device writes the second-level cache back: 71 us
  // became 584; a barrier that waits for every wave's loads empties them before the last tile: 79.)
  const int block = 1 << a.log_block, first_new = len / block * block;
  auto turn_of = [&](int j) {
    const int tile = j / kTile;
    return tile < sink_tiles ? tile : tile - window_tile + sink_tiles;
  };
  int gate = -1;
  if (a.k.p != nullptr && hi > 0) {
    gate = max(t0, turn_of(first_new));
    if (gate >= t1 || turn_of(hi - 1) < t0) gate = -1;
  }
  auto write_tokens = [&] {
    int item = 0;
    for (int first = first_new; first < hi; first += block) {
      const int t = turn_of(first);
      if (t < t0 || t >= t1) continue;
#pragma unroll
      for (int kv = 0; kv < 2; ++kv, ++item) {
        if (kWaves - 1 - item % kWaves != wave) continue;  // the last waves have least to read in the last tile
        const bool words = (kv ? a.v.vec : a.k.vec) && (kv ? a.vc.vec : a.kc.vec);
        if (words)
          write_block<T, true>(kv ? a.v : a.k, kv ? a.vc : a.kc, a, b, g, len, first, lane);
        else
          write_block<T, false>(kv ? a.v : a.k, kv ? a.vc : a.kc, a, b, g, len, first, lane);
      }
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  };
  if (gate >= 0) write_tokens();

  auto place_of = [&](int t) {
    const int j = (t < sink_tiles ? t : t - sink_tiles + window_tile) * kTile + wave * kChunk;
    const uint32_t p = uniform((uint32_t)j / a.page_size);
    return Place{t, j, p, (uint32_t)j - p * a.page_size};
  };
  const Place jump = place_of(max(t0, sink_tiles));  // where the window begins
  auto after = [&](const Place& p) {
    if (p.t + 1 == sink_tiles) return jump;
    Place n{p.t + 1, p.j + kTile, p.page + a.step_pages, p.row + a.step_rows};
    if (n.row >= a.page_size) {
      n.row -= a.page_size;
      ++n.page;
    }
    return n;
  };
  // pages of a chunk's halves; entries behind the row's last position are read as its last one and dropped later
  struct Pages {
    int id[2];
  };
  const int32_t* table = a.table == nullptr ? nullptr : a.table + (size_t)b * a.max_pages;
  auto pages_at = [&](const Place& p) {
    Pages out{{(int)b, (int)b}};
    if (table != nullptr) {
      const uint32_t most = a.max_pages - 1;
      out.id[0] = scalar_load(table + min(p.page, most));
      out.id[1] = scalar_load(table + min(p.row + 16 >= a.page_size ? p.page + 1 : p.page, most));
    }
    return out;
  };

  Place at = place_of(t0);
  Pages pages = pages_at(at);

  // This lane's columns: token and head.
  int token[NT];
  Pieced<QN> qf[NT][DS];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const uint32_t c = c0 + 16 * n + col, t = divide(c, share), head = g * share + c - t * share;
    token[n] = (int)t;
#pragma unroll
    for (int s = 0; s < DS; ++s) {
      const uint32_t d = 32 * s + 8 * quad;
      Raw8<T> raw = {};
      if (c < columns && d < a.D) {
        const T* p = static_cast<const T*>(a.q.p) + ((int64_t)b * a.T + token[n]) * a.q.row + (int64_t)head * a.q.head;
        if (a.q.vec) {
          raw = *reinterpret_cast<const Raw8<T>*>(p + d);
        } else {
          T e8[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) e8[e] = d + e < a.D ? p[d + e] : (T)0.f;
          __builtin_memcpy(&raw, e8, sizeof raw);
        }
      }
      if constexpr (QN == 1) {
        qf[n][s].p[0] = raw.v[0];
      } else {
        float f[8];
        raw_floats<T>(raw, f);
        qf[n][s] = bf16_pieces<QN>(f);
      }
    }
  }

  // Infinities among a query's elements become NaN.  And queries times codes, which are up to 2^9 and 2^119 times what a key is, have to stay in float32 where the scores do: a
  // query with an element from 2^65 on is multiplied as 2^-16 of itself (what that takes from elements below 2^-110 is
  // nothing beside it), and 2^128 2^-16 448 of 128 columns is below 2^128.  No float16 comes near.
  float scale_log2[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) scale_log2[n] = a.scale_log2;
  auto limit_queries = [&] {
    constexpr bool half = Operands<T>::half;
    // nothing of elements below 2^65
    const auto limited = [](uint32_t w) { return half ? nonfinite_pair<T>(w) : w & w << 1 & 0x40004000u; };
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      uint32_t top = 0;
#pragma unroll
      for (int s = 0; s < DS; ++s)
#pragma unroll
        for (int i = 0; i < 4; ++i) top |= limited(qf[n][s].p[0][i]);
      const uint64_t lanes = __ballot(top != 0);
      if (lanes == 0 || (lanes >> col & 0x0001000100010001u) == 0) continue;
#pragma unroll
      for (int s = 0; s < DS; ++s) nan_for_infinities<T>(qf[n][s]);
      if constexpr (half) continue;
      scale_log2[n] = a.scale_log2 * 0x1p16f;
#pragma unroll
      for (int s = 0; s < DS; ++s)
#pragma unroll
        for (int p = 0; p < QN; ++p)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t w = qf[n][s].p[p][i];
            qf[n][s].p[p][i] = pack2<__bf16>(__uint_as_float(w << 16) * 0x1p-16f, __uint_as_float(w & 0xffff0000u) * 0x1p-16f);
          }
    }
  };

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

  uint32_t nothing = 0;
  asm("" : "+v"(nothing));
  auto read = [&](Chunk<DP>& c, const Place& p, const Pages& pages) {
    const uint32_t turned = p.row + 16 >= a.page_size ? p.row + 16 - a.page_size : p.row + 16;
    int page[2];
    uint32_t row[2];
    // Scales first: the compiler waits for them at the end of the loop, and what was asked for later stays on its way.
    // (Their address is the lanes' own to it: one in scalar registers would be waited for at once.)
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int j = p.j + 16 * u, id = pages.id[u];
      const bool seen = p.t < t1 && j < hi && (j + 15 >= lo || j < sinks) && id >= 0 && id < (int)a.num_pages;
      c.there[u] = seen ? min(16, hi - j) : 0;
      page[u] = seen ? id : 0;
      row[u] = seen ? (u ? turned : p.row) : 0;
      const size_t block = ((size_t)page[u] * a.G + g) * a.scale_blocks + (row[u] >> a.log_block);
      c.ks[u] = (a.kc.scales + block)[nothing];
      c.vs[u] = (a.vc.scales + block)[nothing];
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int rows = c.there[u];
      auto half_of = [&](const Kv8Cache& cache) {
        return make_rsrc(cache.codes + page[u] * cache.page + (int64_t)row[u] * cache.row + (int64_t)g * cache.head,
                         rows ? (uint32_t)(rows - 1) * (uint32_t)cache.row + a.D : 0);
      };
      const rsrc_t kr = half_of(a.kc), vr = half_of(a.vc);
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

  // Values' fragment db: eight positions of one of the lane's columns, from words of neighbouring rows whose
  // bytes x = (column 0 of rows r and r + 1, column 1 of them).
  struct Turned {
    uint32_t x[2][2][2];  // [half][rows 0 1 or 2 3][columns 0 1 or 2 3]
  };
  auto turn_word = [&](const Chunk<DP>& c, int w) {
    Turned y;
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const uint32_t p = c.v[u][2 * r][w], q = c.v[u][2 * r + 1][w];
        y.x[u][r][0] = __builtin_amdgcn_perm(q, p, 0x05010400u);
        y.x[u][r][1] = __builtin_amdgcn_perm(q, p, 0x07030602u);
      }
    return y;
  };
  auto widen = [&](uint32_t codes, int half, float scale) {
    return __builtin_bit_cast(unsigned, half ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes, scale, true)
                                             : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes, scale, false));
  };

  bool far = false;  // whether any column's maximum is as large
  const auto far_off = [](float m) { return __builtin_fabsf(m) >= 0x1p24f && __builtin_fabsf(m) < kInf; };
  auto use = [&](Chunk<DP>& c, int j0) {
    if (c.there[0] + c.there[1] == 0) return;
    floatx4 s2[NT][2] = {};
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int s = 0; s < DS; ++s) {
        uintx4 kf;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if constexpr (Operands<T>::half) {
            const uint32_t w = c.k[u][s][i];
            kf[2 * i] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.f, false));
            kf[2 * i + 1] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.f, true));
          } else {
            kf[2 * i] = widen(c.k[u][s][i], 0, 1.f);
            kf[2 * i + 1] = widen(c.k[u][s][i], 1, 1.f);
          }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          if constexpr (Operands<T>::half)
            s2[n][u] = mma16<_Float16>(Frag<_Float16>{kf}, Frag<_Float16>{qf[n][s].p[0]}, s2[n][u]);
          else
            s2[n][u] = mma_pieces<QN>(kf, qf[n][s], s2[n][u]);
        }
      }

    // Where not every query sees all of the chunk:
    if (!(c.there[0] == 16 && c.there[1] == 16 && j0 + kChunk - 1 <= len &&
          (!a.window || j0 > hi - 1 - (int)a.window || j0 + kChunk <= (int)a.sinks))) {
      const uint32_t past[2] = {past_finite(uniform(c.vs[0])), past_finite(uniform(c.vs[1]))};
      uint32_t bad = 0;
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
          for (int w = 0; w < VW; ++w) bad |= not_finite(c.v[u][r][w], past[u]);
      const bool any = __any(bad != 0);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int last = len + token[n];
        uintx4 sees;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int r = 4 * quad + e % 4, j = j0 + 16 * (e / 4) + r;
          const bool hidden = r >= c.there[e / 4] || j > last ||
                              (a.window && j <= last - (int)a.window && j >= (int)a.sinks);
          s2[n][e / 4][e % 4] = hidden ? -kInf : s2[n][e / 4][e % 4];
          const uint32_t one = hidden ? 0u : e % 2 ? 0x3f800000u : 0x3f80u;
          sees[e / 2] = e % 2 ? sees[e / 2] | one : one;
        }
        // What is no finite number among the values must not reach the queries that do not see it (nothing times it is
        // NaN): those that do get a NaN from a product of marks, and it is taken out of the words.
        if (any) {
#pragma unroll
          for (int w = 0; w < VW; ++w) {
            const Turned y = turn_word(c, w);
#pragma unroll
            for (int d = 0; d < 4 && 4 * w + d < DB; ++d) {
              uintx4 mark;
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const uint32_t at = not_finite(y.x[i / 2][i % 2][d / 2], past[i / 2]) >> (d % 2 ? 16 : 0);
                mark[i] = (at & 0x80u ? 0x3f80u : 0u) | (at & 0x8000u ? 0x3f800000u : 0u);
              }
              const floatx4 count = mfma_bf16(mark, sees, floatx4{});
#pragma unroll
              for (int r = 0; r < 4; ++r)
                acc[n][4 * w + d][r] = count[r] > 0.f ? __builtin_nanf("") : acc[n][4 * w + d][r];
            }
          }
        }
      }
      if (any) {
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int w = 0; w < VW; ++w) c.v[u][r][w] &= ~((not_finite(c.v[u][r][w], past[u]) >> 7) * 0xffu);
      }
    }

    const float vs[2] = {scale_value(c.vs[0]), scale_value(c.vs[1])};
    Pieced<PN> pf[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      // (never zero, which would make a NaN of a hidden score's infinity, nor infinite, which would of a score of zero)
      auto scale_of = [&](uint32_t byte) {
        return __builtin_amdgcn_fmed3f(scale_value(byte) * scale_log2[n], 0x1p-149f, 0x1.fffffep127f);
      };
      const float scale[2] = {scale_of(c.ks[0]), scale_of(c.ks[1])};
      float z[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) z[e] = s2[n][e / 4][e % 4];
      // The running maximum follows a query's scores only when one passes it by 2^8: what is summed stays far from
      // the limits of float32, and the sums are rarely multiplied.
      const float top = __builtin_fmaxf(scale[0] * __builtin_fmaxf(max3(z[0], z[1], z[2]), z[3]),
                                        scale[1] * __builtin_fmaxf(max3(z[4], z[5], z[6]), z[7]));
      if (__any(top > m[n] + 8.f)) {
        const float all = max_xor32(max_xor16(top)), to = all > m[n] + 8.f ? all : m[n];
        const float f = to == -kInf ? 1.f : __builtin_amdgcn_exp2f(m[n] - to);
        sum[n] *= f;
#pragma unroll
        for (int db = 0; db < DB; ++db) acc[n][db] *= f;
        m[n] = to;
        far = far || __any(far_off(to));
      }
      const float base = m[n] == -kInf ? 0.f : m[n];
      float arg[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) arg[e] = __builtin_fmaf(z[e], scale[e / 4], -base);
      // Of a maximum that large the rounding is no small number, and the scores have to be rounded as it was.
      if (far) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float score = z[e] * scale[e / 4];
          asm("" : "+v"(score));  // (kept out of a fused multiply-and-add)
          arg[e] = far_off(m[n]) ? score - base : arg[e];
        }
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        z[e] = __builtin_amdgcn_exp2f(arg[e]);
        sum[n] += z[e];
      }
      pf[n] = bf16_pieces<PN>(z);
    }

#pragma unroll
    for (int w = 0; w < VW; ++w) {
      const Turned y = turn_word(c, w);
#pragma unroll
      for (int d = 0; d < 4 && 4 * w + d < DB; ++d) {
        uintx4 vf;
#pragma unroll
        for (int i = 0; i < 4; ++i) vf[i] = widen(y.x[i / 2][i % 2][d / 2], d % 2, vs[i / 2]);
#pragma unroll
        for (int n = 0; n < NT; ++n) acc[n][4 * w + d] = mma_pieces<PN>(vf, pf[n], acc[n][4 * w + d]);
      }
    }
  };

  // Rows are read one chunk before their use, and the table entries of their pages one chunk before that.
  Chunk<DP> even, odd;
  int j_even, j_odd;
  auto read_next = [&](Chunk<DP>& c, int& j) {
    if (at.t == gate) asm volatile("s_barrier" ::: "memory");
    j = at.j;
    read(c, at, pages);
    at = after(at);
    pages = pages_at(at);
  };
  read_next(even, j_even);
  limit_queries();
  for (int t = t0; t < t1; t += 2) {
    read_next(odd, j_odd);
    use(even, j_even);
    read_next(even, j_even);
    use(odd, j_odd);
  }

  // join the waves, 16 columns at a time
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    if (c0 + 16 * n >= columns) break;
    if (n) __syncthreads();
    const float s = sum_xor32(sum_xor16(sum[n]));
    if (quad == 0) join_ms[wave][col] = floatx2{m[n], s};
    float* mine = join + (wave * 16 + col) * kJoinRow;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      if constexpr (DB % 4 == 0) {
#pragma unroll
        for (int db = 0; db < DB; db += 4)
          *reinterpret_cast<floatx4*>(mine + value_column<DP>(4 * quad + r, db)) =
              floatx4{acc[n][db][r], acc[n][db + 1][r], acc[n][db + 2][r], acc[n][db + 3][r]};
      } else {
#pragma unroll
        for (int db = 0; db < DB; ++db) mine[value_column<DP>(4 * quad + r, db)] = acc[n][db][r];
      }
    }
    __syncthreads();
    const uint32_t many = min(16u, columns - (c0 + 16 * n)), quads = (a.D + 3) / 4;
    for (uint32_t e = tid; e < many * quads; e += kThreads) {
      const uint32_t c = divide(e, quads), d = (e - c * quads) * 4, at = c0 + 16 * n + c;
      float top = -kInf, l = 0.f, f[kWaves];
      floatx4 o = {};
#pragma unroll
      for (int w = 0; w < kWaves; ++w) top = __builtin_fmaxf(top, join_ms[w][c][0]);
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        const floatx2 ms = join_ms[w][c];
        f[w] = top == -kInf ? 1.f : __builtin_amdgcn_exp2f(ms[0] - top);
        l = fmaf(ms[1], f[w], l);
      }
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        const floatx4 p = *reinterpret_cast<const floatx4*>(join + (w * 16 + c) * kJoinRow + d);
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = fmaf(p[i], f[w], o[i]);
      }
      const uint32_t t = divide(at, share), head = g * share + at - t * share;
      if (a.splits == 1) {
        T* out = static_cast<T*>(a.out.p) + ((int64_t)b * a.T + t) * a.out.row + (int64_t)head * a.out.head;
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = l == 0.f ? 0.f : o[i] / l;
        if (a.out.vec)
          store4<T, true>(out, d, a.D, o[0], o[1], o[2], o[3]);
        else
          store4<T, false>(out, d, a.D, o[0], o[1], o[2], o[3]);
      } else {
        const size_t part = (((size_t)b * a.T + t) * a.H + head) * a.splits + split;
        if (d == 0) *reinterpret_cast<floatx2*>(a.ws + 2 * part) = floatx2{top, l};
        float* sums = a.ws + 2 * (size_t)a.B * a.T * a.H * a.splits + part * a.D;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (d + i < a.D) sums[d + i] = o[i];
      }
    }
  }
}

template <class T, int NT, int NW>
hipError_t launch_tiles(const Kv8StepArgs& a, hipStream_t stream) {
  const dim3 grid((a.B * a.splits + 7) / 8 * 8 * a.G * a.col_blocks);
  const bool vec = a.kc.vec && a.vc.vec;
#define M3_CALL(DP)                                                                   \
  (vec ? attn_step_kv8_kernel<T, DP, NT, NW, true><<<grid, 64 * NW, 0, stream>>>(a)   \
       : attn_step_kv8_kernel<T, DP, NT, NW, false><<<grid, 64 * NW, 0, stream>>>(a), \
   hipGetLastError())
  if constexpr (sizeof(T) == 4 && NT == 2)  // (the plan takes one tile of float32 columns from 65 on)
    return a.D <= 32 ? M3_CALL(32) : M3_CALL(64);
  else
    return M3_HEAD_DIM_SWITCH(a.D, M3_CALL);
#undef M3_CALL
}

}  // namespace

template <class T>
hipError_t launch_kv8_step(const Kv8StepArgs& a, uint32_t waves, uint32_t tiles, hipStream_t stream) {
  const hipError_t e = waves == 4 ? (tiles == 1 ? launch_tiles<T, 1, 4>(a, stream) : launch_tiles<T, 2, 4>(a, stream))
                                  : (tiles == 1 ? launch_tiles<T, 1, 8>(a, stream) : launch_tiles<T, 2, 8>(a, stream));
  if (e != hipSuccess || a.splits == 1) return e;
  const JoinArgs join{a.ws, a.out, a.B * a.T, a.H, a.D, a.splits};
  return a.splits <= 8 ? launch_join_few<T>(join, stream) : launch_join<T>(join, stream);
}

}  // namespace m3

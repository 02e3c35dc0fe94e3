// Device helpers of the attention kernels: matrix fragments of the three
// element types, tiles in LDS, and loads that zero what lies outside a sequence.
#pragma once

#include "attn.h"
#include "common.h"

namespace m3 {

typedef float floatx16 __attribute__((ext_vector_type(16)));
typedef short shortx4 __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.44269504088896341f;
constexpr float kLn2 = 0.693147180559945309f;
constexpr float kInf = __builtin_inff();
// A byte offset past every buffer resource made here (their sizes stay below 2^31).
constexpr uint32_t kOutside = 0x80000000u;

// A matrix operand of 8 contraction slots per lane.  16-bit types are one
// piece; float32 is three bf16 pieces (split8_bf16x3), which mma multiplies in
// six products at float32 precision: 2.7 times the rate of the float32 matrix
// instruction, and the same kernels serve all three types.
template <class T>
struct Pieces {
  static constexpr int n = sizeof(T) == 4 ? 3 : 1;
};
template <class T>
struct Frag {
  uintx4 p[Pieces<T>::n];
};

// v_mfma_f32_32x32x16: lane l supplies row (column) l % 32 of A (B) and eight
// contraction slots; register r of the result in lane l is
// D[8 (r / 4) + 4 (l / 32) + r % 4][l % 32].
__device__ __forceinline__ floatx16 mma32_bf16(uintx4 a, uintx4 b, floatx16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0,
                                                 0);
}
template <class T>
__device__ __forceinline__ floatx16 mma32(const Frag<T>& a, const Frag<T>& b, floatx16 c) {
  if constexpr (sizeof(T) == 4) {
    c = mma32_bf16(a.p[1], b.p[1], c);
    c = mma32_bf16(a.p[0], b.p[2], c);
    c = mma32_bf16(a.p[2], b.p[0], c);
    c = mma32_bf16(a.p[0], b.p[1], c);
    c = mma32_bf16(a.p[1], b.p[0], c);
    return mma32_bf16(a.p[0], b.p[0], c);
  } else if constexpr (__is_same(T, _Float16)) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(halfx8, a.p[0]),
                                                  __builtin_bit_cast(halfx8, b.p[0]), c, 0, 0, 0);
  } else {
    return mma32_bf16(a.p[0], b.p[0], c);
  }
}
// v_mfma_f32_16x16x32: as mfma_bf16 of common.h.
template <class T>
__device__ __forceinline__ floatx4 mma16(const Frag<T>& a, const Frag<T>& b, floatx4 c) {
  if constexpr (sizeof(T) == 4) {
    return mfma_bf16x6(a.p[0], a.p[1], a.p[2], b.p[0], b.p[1], b.p[2], c);
  } else if constexpr (__is_same(T, _Float16)) {
    return mfma_f16(a.p[0], b.p[0], c);
  } else {
    return mfma_bf16(a.p[0], b.p[0], c);
  }
}

__device__ __forceinline__ float to_float(__bf16 v) { return (float)v; }
__device__ __forceinline__ float to_float(_Float16 v) { return (float)v; }
__device__ __forceinline__ float to_float(float v) { return v; }

// Round two floats to nearest in one 16-bit pair.
template <class T>
__device__ __forceinline__ unsigned pack2(float a, float b) {
  typedef T pair __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(unsigned, __builtin_convertvector((floatx2){a, b}, pair));
}
// Eight float32 values as an operand: one rounding to a 16-bit type, or the split.
template <class T>
__device__ __forceinline__ Frag<T> make_frag(const float* v) {
  Frag<T> f;
  if constexpr (sizeof(T) == 4)
    split8_bf16x3(v, f.p[0], f.p[1], f.p[2]);
  else
    f.p[0] = uintx4{pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]), pack2<T>(v[4], v[5]), pack2<T>(v[6], v[7])};
  return f;
}
// Bit 15 of those of two 16-bit elements (bfloat16 pieces of float32) that are no finite number.
template <class T>
__device__ __forceinline__ uint32_t nonfinite_pair(uint32_t w) {
  constexpr bool half = __is_same(T, _Float16);
  return ((w & (half ? 0x7c007c00u : 0x7f807f80u)) + (half ? 0x04000400u : 0x00800080u)) & 0x80008000u;
}
// A query's operand with NaN in the place of infinities: the scores of such a query are infinite or NaN, and minus
// infinity is what hidden keys have.
template <class T, class Operand>
__device__ __forceinline__ void nan_for_infinities(Operand& f) {
#pragma unroll
  for (int i = 0; i < 4; ++i) f.p[0][i] |= nonfinite_pair<T>(f.p[0][i]) >> (__is_same(T, _Float16) ? 6 : 9);
}
// Registers 8 t .. 8 t + 7 of a 32x32 result as the operand of contraction
// step t over its rows: lane half h holds rows 16 t + 8 (i / 4) + 4 h + i % 4 in
// slot i, the rows that frag_cols reads for the same step, so the result of one
// product feeds the next without leaving its lanes.
template <class T>
__device__ __forceinline__ Frag<T> acc_frag(const floatx16& s, int t) {
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = s[8 * t + i];
  return make_frag<T>(v);
}

// Eight neighbouring elements of one row as they stand in memory.
template <class T>
struct Raw8 {
  uintx4 v[sizeof(T) / 2];
};
// Elements col .. col + 7 of a row that starts `off` bytes into the resource;
// rows past the resource and columns past D read as zero.
template <class T, bool VEC>
__device__ __forceinline__ Raw8<T> load8(rsrc_t r, uint32_t off, uint32_t col, uint32_t D) {
  Raw8<T> out;
  if constexpr (VEC) {
    const uint32_t at = col < D ? off + col * (uint32_t)sizeof(T) : kOutside;
#pragma unroll
    for (int i = 0; i < (int)(sizeof(T) / 2); ++i)
      out.v[i] = __builtin_bit_cast(uintx4, __builtin_amdgcn_raw_buffer_load_b128(r, at + 16 * i, 0, 0));
  } else {
    unsigned w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t at = col + e < D ? off + (col + e) * (uint32_t)sizeof(T) : kOutside;
      if constexpr (sizeof(T) == 4)
        w[e] = (unsigned)__builtin_amdgcn_raw_buffer_load_b32(r, at, 0, 0);
      else
        w[e] = (unsigned short)__builtin_amdgcn_raw_buffer_load_b16(r, at, 0, 0);
    }
    if constexpr (sizeof(T) == 4) {
      out.v[0] = uintx4{w[0], w[1], w[2], w[3]};
      out.v[1] = uintx4{w[4], w[5], w[6], w[7]};
    } else {
      out.v[0] = uintx4{w[0] | w[1] << 16, w[2] | w[3] << 16, w[4] | w[5] << 16, w[6] | w[7] << 16};
    }
  }
  return out;
}
template <class T>
__device__ __forceinline__ void raw_floats(const Raw8<T>& r, float* f) {
  typedef T vec8 __attribute__((ext_vector_type(8)));
  const vec8 v = __builtin_bit_cast(vec8, r);
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = to_float(v[i]);
}
template <class T>
__device__ __forceinline__ Frag<T> raw_frag(const Raw8<T>& r) {
  Frag<T> f;
  if constexpr (sizeof(T) == 4) {
    float v[8];
    raw_floats<T>(r, v);
    return make_frag<T>(v);
  } else {
    f.p[0] = r.v[0];
  }
  return f;
}

// Resource over `rows` rows of a view from row r0 of head h: every row past
// the last reads as zero (the row stride is at least D).
template <class T, class View>
__device__ __forceinline__ rsrc_t rows_rsrc(const View& w, int64_t r0, uint32_t h, int rows, uint32_t D) {
  const T* base = static_cast<const T*>(w.p) + r0 * w.row + (int64_t)h * w.head;
  const uint32_t bytes = rows > 0 ? (uint32_t)((rows - 1) * w.row + D) * (uint32_t)sizeof(T) : 0u;
  return make_rsrc(base, bytes);
}

// The tile of a matrix in LDS: ROWS rows of DP 16-bit columns for each piece, as
// 16-byte words.  Word c of row r stands at place c ^ turn(r) of its row, so that
// both ways of reading meet each of the 64 banks once: the 16 lanes of a row
// read (one word of 16 rows) and the 32 lanes of a transposed read (four words
// of four rows).  With padded rows one of the two ran into conflicts (half of
// the LDS cycles at DP = 128).
template <class T, int DP, int ROWS>
struct Tile {
  static constexpr int ld = DP == 96 ? 128 : DP;
  static constexpr int plane = ROWS * ld;
  static constexpr int words = Pieces<T>::n * plane;  // 16-bit words
  static __device__ __forceinline__ int turn(int r) {
    if constexpr (ld == 32) return (r >> 2) & 3;                           // four rows pass the banks once
    if constexpr (ld == 64) return ((r >> 1) & 1) << 2 | ((r >> 2) & 3);   // two rows
    return (r & 3) << 2 | ((r >> 2) & 3);                                  // one row
  }
  // Place of column `col` (its word's first, or within the word) of row r.
  static __device__ __forceinline__ int at(int r, int col) { return r * ld + (((col >> 3) ^ turn(r)) << 3) + (col & 7); }
};

// ds_read_b64_tr_b16: sixteen lanes read a block of 4 rows of 16 columns, 8
// bytes each, and lane t receives column t of the four rows.
__device__ __forceinline__ uintx2 lds_tr4(const uint16_t* p) {
  return __builtin_bit_cast(
      uintx2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) shortx4*)(p)));
}

// Where a lane reads a tile (LDS bytes).  The turn is an exclusive or on a
// row's words, so another column of the same rows is one more exclusive or, and
// another row, piece or tile of the same shape (`tile` 16-bit words further on) an offset in the
// instruction: at most one vector instruction to a read, none where the
// columns' addresses stay in registers.  (Tiles start at multiples of 256
// bytes, row0 is a multiple of 16.)
struct TileAt {
  uint32_t rows, cols;
};
constexpr int kTileAlign = 256;
template <class T, int DP, int ROWS>
__device__ __forceinline__ TileAt tile_at(const uint16_t* tile, int lane) {
  using L = Tile<T, DP, ROWS>;
  const uint32_t base = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const uint16_t*)tile;
  const int t = lane % 16;
  return {base + 2 * (uint32_t)L::at(lane % 32, 8 * (lane / 32)),
          base + 2 * (uint32_t)L::at(4 * (lane / 32) + t / 4, (lane & 16) + 4 * (t % 4))};
}
// Row operand: lane l takes row row0 + l % 32, columns col0 + 8 (l / 32) .. + 7.
template <class T, int DP, int ROWS>
__device__ __forceinline__ Frag<T> frag_rows(TileAt at, int row0, int col0, int tile = 0) {
  using L = Tile<T, DP, ROWS>;
  Frag<T> f;
#pragma unroll
  for (int i = 0; i < Pieces<T>::n; ++i)
    f.p[i] = *(__attribute__((address_space(3))) const uintx4*)(uintptr_t)((at.rows ^ 2 * (uint32_t)col0) +
                                                                           2 * (tile + row0 * L::ld + i * L::plane));
  return f;
}
// Column operand: lane l takes column col0 + l % 32, in slot i row
// row0 + 8 (i / 4) + 4 (l / 32) + i % 4 (the slots of acc_frag); eight rows on
// the turn differs by its second bit.
template <class T, int DP, int ROWS>
__device__ __forceinline__ Frag<T> frag_cols(TileAt at, int row0, int col0, int tile = 0) {
  using L = Tile<T, DP, ROWS>;
  typedef __attribute__((address_space(3))) shortx4* Lds4;
  const uint32_t p = at.cols ^ 2 * (uint32_t)col0, q = p ^ 32;
  Frag<T> f;
#pragma unroll
  for (int i = 0; i < Pieces<T>::n; ++i) {
    const uintx2 lo = __builtin_bit_cast(uintx2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                                     (Lds4)(uintptr_t)(p + 2 * (tile + row0 * L::ld + i * L::plane))));
    const uintx2 hi = __builtin_bit_cast(uintx2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                                     (Lds4)(uintptr_t)(q + 2 * (tile + (row0 + 8) * L::ld + i * L::plane))));
    f.p[i] = uintx4{lo[0], lo[1], hi[0], hi[1]};
  }
  return f;
}

// A workgroup's copy of ROWS rows on its way from memory to LDS, in registers.
template <class T, int DP, int ROWS, int THREADS, bool VEC>
struct Stage {
  static constexpr int per_row = DP / 8;
  static constexpr int n = (ROWS * per_row + THREADS - 1) / THREADS;
  Raw8<T> r[n];

  __device__ __forceinline__ void load(rsrc_t rs, uint32_t stride_bytes, uint32_t D, int tid) {
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const int c = tid + i * THREADS;
      r[i] = load8<T, VEC>(rs, c < ROWS * per_row ? (c / per_row) * stride_bytes : kOutside, (c % per_row) * 8, D);
    }
  }
  __device__ __forceinline__ void store(uint16_t* tile, int tid) const {
    using L = Tile<T, DP, ROWS>;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const int c = tid + i * THREADS;
      if (ROWS * per_row % THREADS != 0 && c >= ROWS * per_row) break;
      const Frag<T> f = raw_frag<T>(r[i]);
#pragma unroll
      for (int p = 0; p < Pieces<T>::n; ++p)
        *reinterpret_cast<uintx4*>(tile + p * L::plane + L::at(c / per_row, (c % per_row) * 8)) = f.p[p];
    }
  }
  // Whether any piece of any element is an infinity or NaN (a float32 value from here on rounds to bf16's infinity).
  static constexpr float kLargest = sizeof(T) == 4 ? 0x1.ffp127f : kInf;
  __device__ __forceinline__ bool nonfinite() const {
    bool bad = false;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      float f[8];
      raw_floats<T>(r[i], f);
#pragma unroll
      for (int e = 0; e < 8; ++e) bad |= !(__builtin_fabsf(f[e]) < kLargest);
    }
    return bad;
  }
};

// Maximum of three (v_max3_f32; a NaN operand is passed over).
__device__ __forceinline__ float max3(float a, float b, float c) {
  return __builtin_fmaxf(__builtin_fmaxf(a, b), c);
}
// Maximum and sum over lanes l and l ^ 32.
__device__ __forceinline__ float max_xor32(float v) {
  auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __builtin_fmaxf(__uint_as_float(s[0]), __uint_as_float(s[1]));
}
__device__ __forceinline__ float sum_xor32(float v) {
  auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(s[0]) + __uint_as_float(s[1]);
}
__device__ __forceinline__ float max_xor16(float v) {
  auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __builtin_fmaxf(__uint_as_float(s[0]), __uint_as_float(s[1]));
}
__device__ __forceinline__ float sum_xor16(float v) {
  auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(s[0]) + __uint_as_float(s[1]);
}

// Four neighbouring results of one row, columns col .. col + 3 (a multiple of
// four), rounded once to the element type.
template <class T, bool VEC>
__device__ __forceinline__ void store4(T* row, uint32_t col, uint32_t D, float a, float b, float c, float d) {
  // keeps the last product out of a fused multiply-and-round, so that every
  // variant of a kernel rounds alike
  asm("" : "+v"(a), "+v"(b), "+v"(c), "+v"(d));
  if constexpr (VEC) {
    if (col >= D) return;
    if constexpr (sizeof(T) == 4)
      *reinterpret_cast<floatx4*>(row + col) = floatx4{a, b, c, d};
    else
      *reinterpret_cast<uintx2*>(row + col) = uintx2{pack2<T>(a, b), pack2<T>(c, d)};
  } else {
    if (col < D) row[col] = (T)a;
    if (col + 1 < D) row[col + 1] = (T)b;
    if (col + 2 < D) row[col + 2] = (T)c;
    if (col + 3 < D) row[col + 3] = (T)d;
  }
}

// One sequence's rows: where its queries and keys start, how many there are,
// and how far the causal diagonal is moved (the last query stands on the last key).
struct Seq {
  int64_t q0, k0;
  int lq, lk, shift;
};
// Offsets come from device memory, which the host cannot check: they are
// clamped to the rows that exist, so a wrong one cannot read or write outside.
__device__ __forceinline__ void seq_range(const int32_t* offsets, uint32_t b, uint32_t len, uint32_t total, int64_t* at,
                                          int* n) {
  if (offsets == nullptr) {
    *at = (int64_t)b * len;
    *n = (int)len;
    return;
  }
  const int s = min(max(offsets[b], 0), (int)total), e = min(max(offsets[b + 1], s), (int)total);
  *at = s;
  *n = e - s;
}

// The sequence that holds a row; false for a row of none, or one past the
// longest length that the launch covers.
__device__ __forceinline__ bool find_seq(const int32_t* offsets, uint32_t B, uint32_t len, uint32_t total, int64_t row,
                                         uint32_t* b) {
  if (offsets == nullptr) {
    *b = (uint32_t)(row / len);
    return *b < B;
  }
  // the last whose start is not behind the row
  uint32_t lo = 0, hi = B;
  while (hi - lo > 1) {
    const uint32_t mid = (lo + hi) / 2;
    (offsets[mid] <= row ? lo : hi) = mid;
  }
  *b = lo;
  int64_t at;
  int n;
  seq_range(offsets, lo, len, total, &at, &n);
  return row >= at && row < at + n && row < at + (int64_t)len;
}

// Keys of one of `splits` workgroups that share [lo, hi), whole tiles of BN.
__device__ __forceinline__ void split_keys(int splits, int split, int BN, int* lo, int* hi) {
  if (splits == 1 || *lo >= *hi) return;
  const int per = ((*hi - *lo + BN - 1) / BN + splits - 1) / splits * BN;
  const int begin = min((int64_t)*hi, (int64_t)*lo + (int64_t)split * per);
  *hi = min((int64_t)*hi, (int64_t)begin + per);
  *lo = begin;
}

// Workgroups that share the keys of one block of queries, where the blocks
// alone leave compute units without work: enough for two to each of the 256 units,
// `least` keys each.  Their partial results cost a pass of their own (4 us).  (bf16, forward:
// one head, 2874 queries over 2883 keys: 20 us, 78 us unsplit.  1024 queries over 4096 keys without a mask,
// 23 heads of 64, 184 blocks in two halves: 56 us; 24 heads, 192 blocks unsplit: 75 us, and no more up to 256
// blocks, so that from 192 on some work of the last units is still left undone; heads of 128: 85 and 110 us.)
inline uint32_t key_splits(uint64_t blocks, uint64_t seen, uint64_t least) {
  if (blocks >= 192) return 1;
  const uint64_t want = 512 / blocks, most = seen / least, n = want < most ? want : most;
  return n < 1 ? 1 : n > 16 ? 16 : (uint32_t)n;
}

// The run of keys that query i of a sequence sees: `first` and how many, so that
// a key is seen where (unsigned)(key - first) < n (one subtraction, one comparison, no branch).
struct Seen {
  int first;
  uint32_t n;
};
__device__ __forceinline__ Seen seen_keys(int i, int shift, int lk, bool causal, int window) {
  const int end = causal ? min(lk, i + shift + 1) : lk, first = window ? max(0, i + shift - window + 1) : 0;
  return {first, (uint32_t)max(0, end - first)};
}
// The run of queries that see key j.
__device__ __forceinline__ Seen seen_by(int j, int shift, int lq, bool causal, int window) {
  const int first = causal ? max(0, j - shift) : 0;
  const int end = window ? (int)min((int64_t)lq, (int64_t)j - shift + window) : lq;
  return {first, (uint32_t)max(0, end - first)};
}

// Asks the scheduler for N groups of one matrix instruction, V vector and X
// transcendental instructions: the vector work that does not depend on the
// products runs in their shadow (32 cycles each).
template <int N, int V, int X>
__device__ __forceinline__ void interleave() {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    __builtin_amdgcn_sched_group_barrier(0x002, V, 0);
    __builtin_amdgcn_sched_group_barrier(0x400, X, 0);
  }
}

// Head size as the kernels are compiled for it, the next of 32, 64, 96, 128.
#define M3_HEAD_DIM_SWITCH(D, call) \
  ((D) <= 32 ? call(32) : (D) <= 64 ? call(64) : (D) <= 96 ? call(96) : call(128))

}  // namespace m3

// Softmax attention, forward: o_i = sum_j p_ij v_j with p = softmax over the
// allowed keys of scale q_i . k_j, and lse_i = log sum_j exp(scale q_i . k_j).
//
// One workgroup of four waves takes 128 or 256 queries of one head; each wave
// owns 32 or 64 of them and walks the keys in tiles that the workgroup stages in LDS.  A wave
// computes S^T = K Q^T, so that a lane holds the scores of one query: the
// running maximum and sum need one exchange between the two lane halves, and
// the rounded probabilities are, in the registers they stand in, the operand of
// O^T += V^T P^T (V read from LDS transposed).
//
// Bound by the matrix and vector units together: a 32 x 32 block of scores takes
// 256 (D = 64) or 512 (D = 128) cycles of matrix instructions and about 350 of vector ones (a
// multiply-add, an exponential, a sum, half a maximum and half a rounding for each score), and
// the two waves of a SIMD hide only part of the one behind the other.  One prompt of 16384
// queries, 16 heads of 128 over 2: 1.19 ms, 923 TFLOP/s, where a large library product of bf16
// reaches 1249; 4 x 2048 tokens, 24 heads of 64 over 8: 87 us, 591 TFLOP/s.
#include "attn_common.h"

#include <algorithm>
#include <type_traits>

namespace m3 {

namespace {

struct FwdArgs {
  HeadView q, k, v;
  HeadOut out;
  float* lse;
  const int32_t *q_offsets, *kv_offsets;
  uint32_t B, Lq, Lk, H, G, D, total_q, total_k, causal, window;
  uint32_t tiles;     // query tiles of the longest sequence
  uint32_t splits;    // workgroups that share a tile's keys
  float* partial;     // of several: O [splits, B, Lq, H, D], then (maximum, sum) [splits, B, Lq, H]
  float scale_log2;   // scale log2(e): the softmax runs on exp2
};

// The running maximum is only moved when a score passes it by more than this
// (in powers of two): until then the sums hold factors of at most 2^8, exact
// in float32 and within float16's range for the rounded probabilities, and the
// accumulators need no rescaling.
constexpr float kSlack = 8.f;

constexpr int kThreads = 256;

template <class T, int DP>
constexpr int key_tile() {
  return sizeof(T) == 4 ? 32 : 64;  // float32 tiles hold three pieces of each element
}

// Waves of a SIMD that have to fit: two where the registers allow it (256 each,
// none of them accumulator registers, which cost a move on each use).
template <class T, int DP, int QB>
constexpr int min_waves() {
  return sizeof(T) == 4 ? (DP <= 96 ? 2 : 1) : DP * QB <= 128 ? 2 : 1;
}

// QB blocks of 32 queries to a wave.  Two share each key and value operand read
// from LDS, whose bandwidth the kernel otherwise runs into; one is for float32
// (registers) and for sequences too short to fill the larger tile.
template <class T, int DP, int QB, bool VEC>
__global__ __launch_bounds__(kThreads, (min_waves<T, DP, QB>())) void attn_fwd_kernel(const FwdArgs a) {
  constexpr int BN = key_tile<T, DP>(), kQueries = 4 * 32 * QB;
  constexpr int KB = BN / 32, DS = DP / 16, DB = DP / 32;
  using L = Tile<T, DP, BN>;
  // Float32 heads above 64 take 96 KB for two buffers, one workgroup to a compute unit.
  // Up to 96 columns a single buffer and 256 registers let two in (8 x 1000 tokens, 8 heads of
  // 80, no mask: 153 us, 193 us); at 128 the registers spill (4 x 1400 tokens, 8 heads over 2: 234 us, 144 us).
  constexpr int kBufs = sizeof(T) == 4 && DP == 96 ? 1 : 2;
  __shared__ __align__(kTileAlign) uint16_t lds[kBufs][2][L::words];  // [buffer][K, V]

  const uint32_t pairs = a.H * a.B;
  // Late query tiles see the most keys, so they go first.  Head and sequence
  // pairs are dealt to the XCDs in runs, so that the heads of a group share
  // their keys in one L2 (where a tile has one workgroup; several splits of a tile
  // stand next to one another instead, on as many XCDs).
  const uint32_t split = blockIdx.x % a.splits;
  uint32_t i = blockIdx.x / a.splits, pair;
  if (pairs % 8 == 0) {
    const uint32_t per = pairs / 8;
    pair = (i % 8) * per + (i / 8) % per;
    i = i / 8 / per;
  } else {
    pair = i % pairs;
    i = i / pairs;
  }
  const uint32_t h = pair / a.B, b = pair % a.B, g = h / (a.H / a.G);
  const int tile_q = (int)(a.tiles - 1 - i) * kQueries;
  int64_t q0, k0;
  int lq, lk;
  seq_range(a.q_offsets, b, a.Lq, a.total_q, &q0, &lq);
  seq_range(a.kv_offsets, b, a.Lk, a.total_k, &k0, &lk);
  if (tile_q >= lq) return;
  const int shift = lk - lq;

  const int tid = threadIdx.x, lane = tid % 64, wave = __builtin_amdgcn_readfirstlane(tid / 64), half = lane / 32;
  const int wq = tile_q + wave * 32 * QB;  // the wave's first query
  const int last = min(tile_q + kQueries, lq) - 1;
  Seen seen[QB];  // of query wq + 32 qb + lane % 32
#pragma unroll
  for (int qb = 0; qb < QB; ++qb)
    seen[qb] = seen_keys(wq + 32 * qb + lane % 32, shift, lk, a.causal, (int)a.window);
  int lo = 0, hi = lk;
  if (a.causal) {
    hi = min(lk, last + shift + 1);
    if (a.window) lo = max(0, tile_q + shift - (int)a.window + 1) / BN * BN;
  }
  split_keys((int)a.splits, (int)split, BN, &lo, &hi);

  Frag<T> qf[QB][DS];
#pragma unroll
  for (int qb = 0; qb < QB; ++qb) {
    const rsrc_t r = rows_rsrc<T>(a.q, q0 + wq + 32 * qb, h, min(32, lq - wq - 32 * qb), a.D);
#pragma unroll
    for (int s = 0; s < DS; ++s)
      qf[qb][s] =
          raw_frag<T>(load8<T, VEC>(r, (lane % 32) * (uint32_t)(a.q.row * sizeof(T)), 16 * s + 8 * half, a.D));
  }

  floatx16 acc[QB][DB] = {};
  float m[QB], sum[QB];  // the lane's running maximum (powers of two) and its half of the sum
#pragma unroll
  for (int qb = 0; qb < QB; ++qb) {
    m[qb] = -kInf;
    sum[qb] = 0.f;
  }

  Stage<T, DP, BN, kThreads, VEC> sk, sv;
  auto fetch = [&](int kt) {
    const int rows = min(BN, lk - kt);
    sk.load(rows_rsrc<T>(a.k, k0 + kt, g, rows, a.D), (uint32_t)(a.k.row * sizeof(T)), a.D, tid);
    sv.load(rows_rsrc<T>(a.v, k0 + kt, g, rows, a.D), (uint32_t)(a.v.row * sizeof(T)), a.D, tid);
  };
  if (lo < hi) fetch(lo);
  const TileAt at = tile_at<T, DP, BN>(lds[0][0], lane);
  // One tile of keys, in buffer `buf`: a constant, so that the reads of both
  // buffers share their address registers.
  const auto walk = [&](int kt, auto buffer) __attribute__((always_inline)) {
    constexpr int buf = kBufs == 1 ? 0 : decltype(buffer)::value;
    if (kBufs == 1) __syncthreads();  // the last tile has been read
    uint16_t *kl = lds[buf][0], *vl = lds[buf][1];
    sk.store(kl, tid);
    sv.store(vl, tid);
    // tiles that the diagonal or the window's edge crosses hide some of their keys from some queries
    if (a.causal && (kt + BN - 1 > tile_q + shift || (a.window && kt <= last + shift - (int)a.window))) {
      // A hidden value must not reach the output as 0 x NaN: where such a
      // tile of V holds an infinity or NaN, the queries that see it take it
      // directly, and the products get a zero in its place.
      if (__syncthreads_or(sv.nonfinite())) {
        for (int j = 0; j < BN; ++j)
#pragma unroll
          for (int qb = 0; qb < QB; ++qb)
#pragma unroll
            for (int db = 0; db < DB; ++db)
#pragma unroll
              for (int r = 0; r < 16; ++r) {
                const uint16_t u = vl[L::at(j, 32 * db + 8 * (r / 4) + 4 * half + r % 4)];
                float x;
                if constexpr (__is_same(T, _Float16))
                  x = (float)__builtin_bit_cast(_Float16, u);
                else
                  x = __uint_as_float((uint32_t)u << 16);
                const bool take = !(__builtin_fabsf(x) < kInf) & ((uint32_t)(kt + j - seen[qb].first) < seen[qb].n);
                acc[qb][db][r] += take ? x : 0.f;
              }
        __syncthreads();
        for (int e = tid; e < L::plane; e += kThreads) {
          const uint16_t top = __is_same(T, _Float16) ? 0x7c00 : 0x7f80;
          if ((vl[e] & top) == top)
            for (int p = 0; p < Pieces<T>::n; ++p) vl[e + p * L::plane] = 0;
        }
        __syncthreads();
      }
    } else {
      __syncthreads();
    }
    if (kt + BN < hi) fetch(kt + BN);
    const int wlast = wq + 32 * QB - 1;
    if (a.causal && (kt > wlast + shift || (a.window && kt + BN <= wq + shift - (int)a.window + 1)))
      return;  // nothing in it for this wave
    const bool edge = kt + BN > lk || (a.causal && (kt + BN - 1 > wq + shift ||
                                                    (a.window && kt <= wlast + shift - (int)a.window)));

    floatx16 s[KB][QB];
    const auto scores = [&](int kb) {
#pragma unroll
      for (int qb = 0; qb < QB; ++qb) s[kb][qb] = floatx16{};
#pragma unroll
      for (int d = 0; d < DS; ++d) {
        const Frag<T> kf = frag_rows<T, DP, BN>(at, 32 * kb, 16 * d, 2 * buf * L::words);
#pragma unroll
        for (int qb = 0; qb < QB; ++qb) s[kb][qb] = mma32<T>(kf, qf[qb][d], s[kb][qb]);
      }
    };
    // hides what the mask hides and moves the running maximum where the scores have left it behind
    const auto level = [&](int kb) {
      if (edge) {
#pragma unroll
        for (int qb = 0; qb < QB; ++qb)
#pragma unroll
          for (int r = 0; r < 16; ++r) {
            const int key = kt + 32 * kb + 8 * (r / 4) + 4 * half + r % 4;
            s[kb][qb][r] = (uint32_t)(key - seen[qb].first) < seen[qb].n ? s[kb][qb][r] : -kInf;
          }
      }
      float top[QB];
      bool move = false;
#pragma unroll
      for (int qb = 0; qb < QB; ++qb) {
        top[qb] = s[kb][qb][0];
#pragma unroll
        for (int r = 1; r < 15; r += 2) top[qb] = max3(top[qb], s[kb][qb][r], s[kb][qb][r + 1]);
        top[qb] = max_xor32(__builtin_fmaxf(top[qb], s[kb][qb][15])) * a.scale_log2;
        move |= top[qb] > m[qb] + kSlack;
      }
      if (__any(move)) {
#pragma unroll
        for (int qb = 0; qb < QB; ++qb) {
          // (a query's own scores alone decide, so that its bits do not depend on its neighbours)
          const float to = top[qb] > m[qb] + kSlack ? top[qb] : m[qb];
          // no key yet: the sums are zero, or an infinity that a hidden tile's edge has put there already
          const float f = m[qb] == -kInf ? 1.f : __builtin_amdgcn_exp2f(m[qb] - to);
          sum[qb] *= f;
#pragma unroll
          for (int db = 0; db < DB; ++db) acc[qb][db] *= f;
          m[qb] = to;
        }
      }
    };
    scores(0);
    level(0);
    // The next block's scores are multiplied while this block's probabilities
    // are made: matrix and vector instructions alternate in one wave.
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
      if (kb + 1 < KB) scores(kb + 1);
      Frag<T> pf[2][QB];
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int qb = 0; qb < QB; ++qb) {
          const float base = m[qb] == -kInf ? 0.f : m[qb];  // no key seen yet: every score is -inf
#pragma unroll
          for (int r = 8 * t; r < 8 * t + 8; ++r) {
            s[kb][qb][r] = __builtin_amdgcn_exp2f(fmaf(s[kb][qb][r], a.scale_log2, -base));
            sum[qb] += s[kb][qb][r];
          }
          pf[t][qb] = acc_frag<T>(s[kb][qb], t);
        }
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int db = 0; db < DB; ++db) {
          const Frag<T> vf = frag_cols<T, DP, BN>(at, 32 * kb + 16 * t, 32 * db, (2 * buf + 1) * L::words);
#pragma unroll
          for (int qb = 0; qb < QB; ++qb) acc[qb][db] = mma32<T>(vf, pf[t][qb], acc[qb][db]);
        }
      if constexpr (sizeof(T) == 2) {
        if (kb + 1 < KB) interleave<DS * QB, 40 / DS, 16 / DS>();
        interleave<DB * QB, 40 / DB, 16 / DB>();
      }
      if (kb + 1 < KB) level(kb + 1);
    }
  };
  for (int kt = lo; kt < hi; kt += 2 * BN) {
    walk(kt, std::integral_constant<int, 0>());
    if (kt + BN < hi) walk(kt + BN, std::integral_constant<int, 1>());
  }

#pragma unroll
  for (int qb = 0; qb < QB; ++qb) {
    const int qi = wq + 32 * qb + lane % 32;
    const float total = sum_xor32(sum[qb]);
    if (qi >= lq) continue;
    if (a.splits > 1) {
      if (qi >= (int)a.Lq) continue;  // a sequence longer than it may be
      const size_t at = (((size_t)split * a.B + b) * a.Lq + qi) * a.H + h;
#pragma unroll
      for (int db = 0; db < DB; ++db)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          store4<float, VEC>(a.partial + at * a.D, 32 * db + 8 * j + 4 * half, a.D, acc[qb][db][4 * j],
                             acc[qb][db][4 * j + 1], acc[qb][db][4 * j + 2], acc[qb][db][4 * j + 3]);
      if (half == 0) {
        float* ms = a.partial + (size_t)a.splits * a.B * a.Lq * a.H * a.D + 2 * at;
        ms[0] = m[qb];
        ms[1] = total;
      }
      continue;
    }
    const float inv = total == 0.f ? 0.f : 1.f / total;  // a query that sees no key: zero, lse = -inf
    T* row = static_cast<T*>(a.out.p) + (q0 + qi) * a.out.row + (int64_t)h * a.out.head;
#pragma unroll
    for (int db = 0; db < DB; ++db)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        store4<T, VEC>(row, 32 * db + 8 * j + 4 * half, a.D, acc[qb][db][4 * j] * inv,
                  acc[qb][db][4 * j + 1] * inv, acc[qb][db][4 * j + 2] * inv, acc[qb][db][4 * j + 3] * inv);
    if (half == 0)
      a.lse[(q0 + qi) * a.H + h] = total == 0.f ? -kInf : (m[qb] + __builtin_amdgcn_logf(total)) * kLn2;
  }
}

// Joins the splits: a thread takes four columns of one query and head.
template <class T, bool VEC>
__global__ __launch_bounds__(kThreads) void attn_fwd_join(const FwdArgs a) {
  const uint32_t pieces = (a.D + 3) / 4;
  const size_t e = (size_t)blockIdx.x * kThreads + threadIdx.x, n = (size_t)a.B * a.Lq * a.H, at = e / pieces;
  if (at >= n) return;
  const uint32_t col = e % pieces * 4, h = at % a.H, qi = at / a.H % a.Lq, b = (uint32_t)(at / a.H / a.Lq);
  int64_t q0;
  int lq;
  seq_range(a.q_offsets, b, a.Lq, a.total_q, &q0, &lq);
  if ((int)qi >= lq) return;
  const float* ms = a.partial + (size_t)a.splits * n * a.D;
  float top = -kInf;
  for (uint32_t s = 0; s < a.splits; ++s) top = __builtin_fmaxf(top, ms[2 * (s * n + at)]);
  float sum = 0.f, o[4] = {};
#pragma unroll 4
  for (uint32_t s = 0; s < a.splits; ++s) {
    const float* p = a.partial + (s * n + at) * a.D + col;
    const float f = top == -kInf ? 1.f : __builtin_amdgcn_exp2f(ms[2 * (s * n + at)] - top);
    sum = fmaf(ms[2 * (s * n + at) + 1], f, sum);
    floatx4 x = {};
    if constexpr (VEC) {
      x = *reinterpret_cast<const floatx4*>(p);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (col + i < a.D) x[i] = p[i];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = fmaf(x[i], f, o[i]);
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  store4<T, VEC>(static_cast<T*>(a.out.p) + (q0 + qi) * a.out.row + (int64_t)h * a.out.head, col, a.D, o[0] * inv, o[1] * inv,
                 o[2] * inv, o[3] * inv);
  if (col == 0) a.lse[(q0 + qi) * a.H + h] = sum == 0.f ? -kInf : (top + __builtin_amdgcn_logf(sum)) * kLn2;
}

// Two blocks of queries to a wave where they alone fill the compute units (and
// the registers hold them), and the workgroups that share a tile's keys.
struct Plan {
  uint32_t qb, tiles, splits;
};
Plan plan(const AttnGeom& g) {
  const uint64_t pairs = (uint64_t)g.H * g.B;
  const auto tiles = [&](uint64_t qb) { return (g.Lq + 128 * qb - 1) / (128 * qb); };
  const uint32_t qb = g.dtype != kF32 && g.D <= 64 && tiles(2) * pairs >= 256 ? 2 : 1;
  const uint32_t seen = g.window && g.window < g.Lk ? g.window : g.Lk;
  return {qb, (uint32_t)tiles(qb), key_splits(tiles(qb) * pairs, seen, g.dtype == kF32 ? 128 : 256)};
}

template <class T, int DP, int QB>
hipError_t launch_q(const AttnGeom& g, const FwdArgs& a, hipStream_t stream) {
  const dim3 grid(a.tiles * g.H * g.B * a.splits);
  const bool vec = a.q.vec && a.k.vec && a.v.vec && a.out.vec;
  if (vec)
    attn_fwd_kernel<T, DP, QB, true><<<grid, kThreads, 0, stream>>>(a);
  else
    attn_fwd_kernel<T, DP, QB, false><<<grid, kThreads, 0, stream>>>(a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.splits == 1) return e;
  const size_t n = (size_t)g.Lq * g.B * g.H * ((g.D + 3) / 4);
  const dim3 join((uint32_t)((n + kThreads - 1) / kThreads));
  if (vec)
    attn_fwd_join<T, true><<<join, kThreads, 0, stream>>>(a);
  else
    attn_fwd_join<T, false><<<join, kThreads, 0, stream>>>(a);
  return hipGetLastError();
}

template <class T, int DP>
hipError_t launch_d(const AttnGeom& g, const FwdArgs& a, hipStream_t stream) {
  if constexpr (sizeof(T) == 2 && DP <= 64)
    if (plan(g).qb == 2) return launch_q<T, DP, 2>(g, a, stream);
  return launch_q<T, DP, 1>(g, a, stream);
}

template <class T>
hipError_t launch(const AttnGeom& g, const FwdArgs& a, hipStream_t stream) {
#define M3_CALL(DP) launch_d<T, DP>(g, a, stream)
  return M3_HEAD_DIM_SWITCH(g.D, M3_CALL);
#undef M3_CALL
}

}  // namespace

size_t attn_fwd_workspace_floats(const AttnGeom& g) {
  const Plan p = plan(g);
  return p.splits == 1 ? 0 : (size_t)p.splits * g.Lq * g.B * g.H * (g.D + 2);
}

uint64_t attn_fwd_workgroups(const AttnGeom& g) {
  const Plan p = plan(g);
  const uint64_t pairs = (uint64_t)g.H * g.B, join = (pairs * g.Lq * ((g.D + 3) / 4) + kThreads - 1) / kThreads;
  return std::max<uint64_t>(pairs * p.tiles * p.splits, p.splits > 1 ? join : 0);
}

hipError_t launch_attn_fwd(const AttnGeom& g, const AttnOperands& o, hipStream_t stream) {
  const Plan p = plan(g);
  FwdArgs a{o.q,       o.k,      o.v,      o.out,   o.lse,   o.q_offsets, o.kv_offsets, g.B, g.Lq, g.Lk, g.H, g.G, g.D,
            g.total_q, g.total_k, g.causal, g.window, p.tiles, p.splits, o.ws, g.scale * kLog2e};
  if (g.dtype == kF32) return launch<float>(g, a, stream);
  if (g.dtype == kF16) return launch<_Float16>(g, a, stream);
  return launch<__bf16>(g, a, stream);
}

}  // namespace m3

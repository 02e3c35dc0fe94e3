// Softmax attention, forward: o_i = sum_j p_ij v_j with p = softmax over the
// allowed keys of scale q_i . k_j, and lse_i = log sum_j exp(scale q_i . k_j).
//
// One workgroup of four waves takes 128 queries of one head; each wave owns 32
// of them and walks the keys in tiles that the workgroup stages in LDS.  A wave
// computes S^T = K Q^T, so that a lane holds the scores of one query: the
// running maximum and sum need one exchange between the two lane halves, and
// the rounded probabilities are, in the registers they stand in, the operand of
// O^T += V^T P^T (V read from LDS transposed).
#include "attn_common.h"

namespace m3 {

namespace {

struct FwdArgs {
  HeadView q, k, v;
  HeadOut out;
  float* lse;
  const int32_t *q_offsets, *kv_offsets;
  uint32_t B, Lq, Lk, H, G, D, total_q, total_k, causal, window;
  uint32_t tiles;     // query tiles of the longest sequence
  float scale_log2;   // scale log2(e): the softmax runs on exp2
};

constexpr int kThreads = 256;
constexpr int kQueries = 128;  // of a workgroup

// The running maximum is only moved when a score passes it by more than this
// (in powers of two): until then the sums hold factors of at most 2^8, exact
// in float32 and within float16's range for the rounded probabilities, and the
// accumulators need no rescaling.
constexpr float kSlack = 8.f;

template <class T, int DP>
constexpr int key_tile() {
  return sizeof(T) == 4 ? 32 : 64;  // float32 tiles hold three pieces of each element
}

template <class T, int DP>
__global__ __launch_bounds__(kThreads) void attn_fwd_kernel(const FwdArgs a) {
  constexpr int BN = key_tile<T, DP>();
  constexpr int KB = BN / 32, DS = DP / 16, DB = DP / 32;
  using L = Tile<T, DP, BN>;
  __shared__ uint16_t lds[2][2][L::words];  // [buffer][K, V]

  const uint32_t pairs = a.H * a.B;
  // Late query tiles see the most keys, so they go first.  Head and sequence
  // pairs are dealt to the XCDs in runs, so that the heads of a group share
  // their keys in one L2.
  uint32_t i = blockIdx.x, pair;
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
  const int wq = tile_q + wave * 32;  // the wave's first query
  const int qi = wq + lane % 32;      // the lane's query
  const int last = min(tile_q + kQueries, lq) - 1;
  const Seen seen = seen_keys(qi, shift, lk, a.causal, (int)a.window);
  const auto hidden = [seen](int key) { return (uint32_t)(key - seen.first) >= seen.n; };
  int lo = 0, hi = lk;
  if (a.causal) {
    hi = min(lk, last + shift + 1);
    if (a.window) lo = max(0, tile_q + shift - (int)a.window + 1) / BN * BN;
  }

  Frag<T> qf[DS];
  {
    const rsrc_t r = rows_rsrc<T>(a.q, q0 + wq, h, min(32, lq - wq), a.D);
#pragma unroll
    for (int s = 0; s < DS; ++s)
      qf[s] = raw_frag<T>(load8<T>(r, (lane % 32) * (uint32_t)(a.q.row * sizeof(T)), 16 * s + 8 * half, a.D, a.q.vec));
  }

  floatx16 acc[DB] = {};
  float m = -kInf, sum = 0.f;  // the lane's running maximum (powers of two) and its half of the sum

  Stage<T, DP, BN, kThreads> sk, sv;
  auto fetch = [&](int kt) {
    const int rows = min(BN, lk - kt);
    sk.load(rows_rsrc<T>(a.k, k0 + kt, g, rows, a.D), (uint32_t)(a.k.row * sizeof(T)), a.D, a.k.vec, tid);
    sv.load(rows_rsrc<T>(a.v, k0 + kt, g, rows, a.D), (uint32_t)(a.v.row * sizeof(T)), a.D, a.v.vec, tid);
  };
  if (lo < hi) fetch(lo);
  int buf = 0;
  for (int kt = lo; kt < hi; kt += BN, buf ^= 1) {
    uint16_t *kl = lds[buf][0], *vl = lds[buf][1];
    sk.store(kl, tid);
    sv.store(vl, tid);
    // tiles that the diagonal or the window's edge crosses hide some of their keys from some queries
    const bool edge = a.causal && (kt + BN - 1 > tile_q + shift || (a.window && kt <= last + shift - (int)a.window));
    if (edge) {
      // A hidden value must not reach the output as 0 x NaN: where such a
      // tile of V holds an infinity or NaN, the queries that see it take it
      // directly, and the products get a zero in its place.
      if (__syncthreads_or(sv.nonfinite())) {
        for (int j = 0; j < BN; ++j)
#pragma unroll
          for (int db = 0; db < DB; ++db)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
              const uint16_t u = vl[j * L::ld + 32 * db + 8 * (r / 4) + 4 * half + r % 4];
              float x;
              if constexpr (__is_same(T, _Float16))
                x = (float)__builtin_bit_cast(_Float16, u);
              else
                x = __uint_as_float((uint32_t)u << 16);
              if (!(__builtin_fabsf(x) < kInf) && !hidden(kt + j)) acc[db][r] += x;
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
    if (a.causal && (kt > wq + 31 + shift || (a.window && kt + BN <= wq + shift - (int)a.window + 1)))
      continue;  // nothing in it for this wave

    floatx16 s[KB] = {};
#pragma unroll
    for (int d = 0; d < DS; ++d)
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) s[kb] = mma32<T>(frag_rows<T, DP, BN>(kl, 32 * kb, 16 * d, lane), qf[d], s[kb]);

    float top = -kInf;
    if (edge || kt + BN > lk) {
#pragma unroll
      for (int kb = 0; kb < KB; ++kb)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          s[kb][r] = hidden(kt + 32 * kb + 8 * (r / 4) + 4 * half + r % 4) ? -kInf : s[kb][r] * a.scale_log2;
          top = __builtin_fmaxf(top, s[kb][r]);
        }
    } else {
#pragma unroll
      for (int kb = 0; kb < KB; ++kb)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          s[kb][r] *= a.scale_log2;
          top = __builtin_fmaxf(top, s[kb][r]);
        }
    }
    top = max_xor32(top);
    if (__any(top > m + kSlack || (m == -kInf && top > -kInf))) {
      const float to = __builtin_fmaxf(m, top);
      const float f = to == -kInf ? 1.f : __builtin_amdgcn_exp2f(m - to);
      sum *= f;
#pragma unroll
      for (int db = 0; db < DB; ++db) acc[db] *= f;
      m = to;
    }
    const float base = m == -kInf ? 0.f : m;  // no key allowed yet: every score is -inf
#pragma unroll
    for (int kb = 0; kb < KB; ++kb)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        s[kb][r] = __builtin_amdgcn_exp2f(s[kb][r] - base);
        sum += s[kb][r];
      }
#pragma unroll
    for (int kb = 0; kb < KB; ++kb)
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const Frag<T> pf = acc_frag<T>(s[kb], t);
#pragma unroll
        for (int db = 0; db < DB; ++db)
          acc[db] = mma32<T>(frag_cols<T, DP, BN>(vl, 32 * kb + 16 * t, 32 * db, lane), pf, acc[db]);
      }
  }

  if (qi >= lq) return;
  sum = sum_xor32(sum);
  const float inv = sum == 0.f ? 0.f : 1.f / sum;  // a query that sees no key: zero, lse = -inf
  T* row = static_cast<T*>(a.out.p) + (q0 + qi) * a.out.row + (int64_t)h * a.out.head;
#pragma unroll
  for (int db = 0; db < DB; ++db)
#pragma unroll
    for (int j = 0; j < 4; ++j)
      store4<T>(row, 32 * db + 8 * j + 4 * half, a.D, a.out.vec, acc[db][4 * j] * inv, acc[db][4 * j + 1] * inv,
                acc[db][4 * j + 2] * inv, acc[db][4 * j + 3] * inv);
  if (half == 0) a.lse[(q0 + qi) * a.H + h] = sum == 0.f ? -kInf : (m + __builtin_amdgcn_logf(sum)) * kLn2;
}

template <class T>
hipError_t launch(const AttnGeom& g, const FwdArgs& a, hipStream_t stream) {
  const dim3 grid(a.tiles * g.H * g.B);
#define M3_CALL(DP) (attn_fwd_kernel<T, DP><<<grid, kThreads, 0, stream>>>(a), hipGetLastError())
  return M3_HEAD_DIM_SWITCH(g.D, M3_CALL);
#undef M3_CALL
}

}  // namespace

size_t attn_fwd_workspace_floats(const AttnGeom&) { return 0; }

hipError_t launch_attn_fwd(const AttnGeom& g, const AttnOperands& o, hipStream_t stream) {
  FwdArgs a{o.q,  o.k,  o.v, o.out, o.lse, o.q_offsets, o.kv_offsets, g.B, g.Lq, g.Lk, g.H, g.G, g.D, g.total_q,
            g.total_k, g.causal, g.window, (g.Lq + kQueries - 1) / kQueries, g.scale * kLog2e};
  if (g.dtype == kF32) return launch<float>(g, a, stream);
  if (g.dtype == kF16) return launch<_Float16>(g, a, stream);
  return launch<__bf16>(g, a, stream);
}

}  // namespace m3

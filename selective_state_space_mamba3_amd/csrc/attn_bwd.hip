// Softmax attention, backward.  With p_ij = exp(scale q_i . k_j - lse_i) made
// again from the scores and the forward pass's lse,
//   delta_i = do_i . o_i,   ds_ij = p_ij (do_i . v_j - delta_i),
//   dq_i = scale sum_j ds_ij k_j,   dk_j = scale sum_i ds_ij q_i,   dv_j = sum_i p_ij do_i,
// the last two summed over the heads that share the key head as well.
//
// Two kernels, each owning its outputs: attn_bwd_dq walks the keys for a block
// of queries (and leaves delta and the base-2 lse behind), attn_bwd_dkv walks the
// queries of every sharing head for a block of keys.  The scores and dO V^T are
// computed in both, seven matrix products where five would do; in exchange no
// sum goes through atomics, so the results do not depend on the order of the
// workgroups.  P and dS are rounded once to the operands' type for the products
// they enter (float32: split, no rounding to speak of) and summed in float32.
//
// Bound by the matrix units' share of two waves to a SIMD: the products that are
// run keep them busy for 49 % (dq, D = 64) and less of the time; neither reading operands
// ahead, nor fewer vector instructions, nor more waves moved the time of dq any further.
// 4 x 2048 tokens, 24 heads of 64 over 8, bf16: 249 us, 518 TFLOP/s of the five products (under the
// profiler, at lower clocks, dq 102, dkv 158, the join of its parts 14).  Six packed sequences up to 1999, 16
// heads of 128 over 2, float16: 436 us (161, 316, 25).  8 x 512 tokens, 24 heads of 64 over 8, bf16:
// 74 us (25, 37, 14).
#include "attn_common.h"

#include <algorithm>

namespace m3 {

namespace {

struct BwdArgs {
  HeadView q, k, v, o, dout;
  HeadOut dq, dk, dv;
  const float* lse;
  float* lse2;   // [H, total_q] lse log2(e), +inf where a query saw no key
  float* delta;  // [H, total_q]
  const int32_t *q_offsets, *kv_offsets;
  uint32_t B, Lq, Lk, H, G, D, total_q, total_k, causal, window;
  uint32_t tiles;  // of the longest sequence
  uint32_t parts;  // dkv: workgroups that may share the queries of one block of keys
  int steps;       // dkv: query tiles of one workgroup
  float* partial;  // [2 (dk, dv), parts, total_k, G, D] where there are several
  uint32_t splits;     // dq: workgroups that share the keys of one block of queries
  float* partial_q;    // [splits, total_q, H, D] where there are several
  float scale, scale_log2;
};

constexpr int kThreads = 256;
constexpr int kRows = 128;  // queries (dq) or keys (dkv) of a workgroup

template <class T, int DP>
constexpr int inner_tile() {
  return sizeof(T) == 4 || DP > 64 ? 32 : 64;
}

// Waves of a SIMD that have to fit: two where 256 registers hold the operands and sums.
template <class T, int DP>
constexpr int dq_waves() {
  return sizeof(T) == 4 && DP > 64 ? 1 : 2;
}
template <class T, int DP>
constexpr bool values_in_lds() {
  return sizeof(T) == 2 ? DP > 64 : DP == 64;
}
template <class T, int DP>
constexpr int dkv_waves() {
  return sizeof(T) == 4 && DP > 64 ? 1 : 2;
}

// float16 has five bits of exponent: P is about one over the number of keys and dS = P (dP - delta) smaller
// yet, so both would fall below its normal range (2^-14), or to zero, long before the gradients do (dq over 2048
// keys from a dout of 1e-3: off by 2.8e-3, of which 5e-4 is the rounding of the result).  So they are
// rounded as multiples: P times 2^14 (P is at most one), dS times a power of two of each query (dq) or key
// (dkv) that starts high and comes down, with the sum that it belongs to, where a block passes 2^15: to where
// its largest value stands at 2^10, which leaves room for later ones.  Every value down to 2^-24 of the largest
// then keeps its eleven bits.  The powers are undone in float32 at the end.  (4 x 2048 tokens, 24 heads of 64
// over 8: 279 us, 261 unscaled; 16 heads of 128 over 2: 405 us, 397.)
template <class T>
constexpr bool scaled() {
  return __is_same(T, _Float16);
}
constexpr int kUpP = 14, kUpStart = 40;
// The power of two that brings a lane's block (and that of lane ^ 32) down, one where it fits.
__device__ __forceinline__ float down(const floatx16& s) {
  float top = 0.f;
#pragma unroll
  for (int r = 0; r < 16; r += 2) top = max3_abs(s[r], s[r + 1], top);
  top = max_xor32(top);
  return top > 0x1p15f ? __builtin_amdgcn_ldexpf(1.f, 11 - __builtin_amdgcn_frexp_expf(top)) : 1.f;
}

// delta = sum_j p_ij dp_ij is taken from the forward pass's out, which is rounded to the operands' type.
// Beside dS's own rounding that error falls with the root of the number of keys that a query sees: dq (bf16,
// heads of 64) is off by 3.6e-3 instead of 2.3e-3 over two keys, 2.8e-3 over four, 2.5e-3 over sixteen, 2.43e-3
// instead of 2.35e-3 over 32.  So queries that see at most this many keys get theirs from the float32
// probabilities, in a short walk over those keys; which queries those are depends on nothing but their own
// sequence's mask.  Causal sequences pay for it in their first tile (no difference measured); a window of 32 over
// 4 x 2048 tokens, 24 heads of 64 over 8, takes 107 us instead of 96.
constexpr uint32_t kFewKeys = 32;

template <class T, int DP, bool VEC>
__global__ __launch_bounds__(kThreads, (dq_waves<T, DP>())) void attn_bwd_dq(const BwdArgs a) {
  constexpr int BN = inner_tile<T, DP>();
  constexpr int KB = BN / 32, DS = DP / 16, DB = DP / 32;
  using L = Tile<T, DP, BN>;
  __shared__ __align__(kTileAlign) uint16_t lds[sizeof(T) == 4 ? 1 : 2][2][L::words];

  const uint32_t pairs = a.H * a.B;
  const uint32_t split = blockIdx.x % a.splits;
  uint32_t i = blockIdx.x / a.splits, pair;
  if (pairs % 8 == 0) {  // as in the forward pass: late tiles first, without splits a group's heads on one XCD
    const uint32_t per = pairs / 8;
    pair = (i % 8) * per + (i / 8) % per;
    i = i / 8 / per;
  } else {
    pair = i % pairs;
    i = i / pairs;
  }
  const uint32_t h = pair / a.B, b = pair % a.B, g = h / (a.H / a.G);
  const int tile_q = (int)(a.tiles - 1 - i) * kRows;
  int64_t q0, k0;
  int lq, lk;
  seq_range(a.q_offsets, b, a.Lq, a.total_q, &q0, &lq);
  seq_range(a.kv_offsets, b, a.Lk, a.total_k, &k0, &lk);
  if (tile_q >= lq) return;
  const int shift = lk - lq;

  const int tid = threadIdx.x, lane = tid % 64, wave = __builtin_amdgcn_readfirstlane(tid / 64), half = lane / 32;
  const int wq = tile_q + wave * 32, qi = wq + lane % 32;
  const int last = min(tile_q + kRows, lq) - 1;
  const Seen seen = seen_keys(qi, shift, lk, a.causal, (int)a.window);
  int lo = 0, hi = lk;
  if (a.causal) {
    hi = min(lk, last + shift + 1);
    if (a.window) lo = max(0, tile_q + shift - (int)a.window + 1) / BN * BN;
  }
  // the keys of the block's queries that see few: all where every query sees few, or the first ones
  const bool all_few = lk <= (int)kFewKeys || (a.window && a.window <= kFewKeys);
  const int few_lo = lo;
  const int few_hi = sizeof(T) == 4 ? lo
                     : all_few      ? hi
                     : a.causal && tile_q + shift < (int)kFewKeys ? min(hi, (int)kFewKeys) : lo;
  split_keys((int)a.splits, (int)split, BN, &lo, &hi);

  Frag<T> qf[DS], df[DS];
  float delta = 0.f;
  {
    const int rows = min(32, lq - wq);
    const rsrc_t rq = rows_rsrc<T>(a.q, q0 + wq, h, rows, a.D);
    const rsrc_t rd = rows_rsrc<T>(a.dout, q0 + wq, h, rows, a.D);
    const rsrc_t ro = rows_rsrc<T>(a.o, q0 + wq, h, rows, a.D);
#pragma unroll
    for (int s = 0; s < DS; ++s) {
      const uint32_t row = lane % 32, col = 16 * s + 8 * half;
      qf[s] = raw_frag<T>(load8<T, VEC>(rq, row * (uint32_t)(a.q.row * sizeof(T)), col, a.D));
      const Raw8<T> d = load8<T, VEC>(rd, row * (uint32_t)(a.dout.row * sizeof(T)), col, a.D);
      const Raw8<T> o = load8<T, VEC>(ro, row * (uint32_t)(a.o.row * sizeof(T)), col, a.D);
      float x[8], y[8];
      raw_floats<T>(d, x);
      raw_floats<T>(o, y);
#pragma unroll
      for (int e = 0; e < 8; ++e) delta = fmaf(x[e], y[e], delta);
      df[s] = raw_frag<T>(d);
    }
  }
  delta = sum_xor32(delta);
  float lse2 = kInf;
  if (qi < lq) {
    const float l = a.lse[(q0 + qi) * a.H + h];
    lse2 = l == -kInf ? kInf : l * kLog2e;  // exp2(s - inf) = 0 on a row without keys
  }

  floatx16 acc[DB] = {};
  Stage<T, DP, BN, kThreads, VEC> sk, sv;
  auto fetch = [&](int kt) {
    const int rows = min(BN, lk - kt);
    sk.load(rows_rsrc<T>(a.k, k0 + kt, g, rows, a.D), (uint32_t)(a.k.row * sizeof(T)), a.D, tid);
    sv.load(rows_rsrc<T>(a.v, k0 + kt, g, rows, a.D), (uint32_t)(a.v.row * sizeof(T)), a.D, tid);
  };
  if constexpr (sizeof(T) == 2) {
    if (few_lo < few_hi) {
      float exact = 0.f;
      for (int kt = few_lo; kt < few_hi; kt += BN) {
        fetch(kt);
        __syncthreads();  // the last tile has been read
        sk.store(lds[0][0], tid);
        sv.store(lds[0][1], tid);
        __syncthreads();
        const TileAt kl_at = tile_at<T, DP, BN>(lds[0][0], lane), vl_at = tile_at<T, DP, BN>(lds[0][1], lane);
#pragma unroll 1
        for (int kb = 0; kb < KB; ++kb) {
          floatx16 s = {}, dp = {};
#pragma unroll
          for (int d = 0; d < DS; ++d) {
            s = mma32<T>(frag_rows<T, DP, BN>(kl_at, 0, 16 * d, 32 * kb * L::ld), qf[d], s);
            dp = mma32<T>(frag_rows<T, DP, BN>(vl_at, 0, 16 * d, 32 * kb * L::ld), df[d], dp);
          }
#pragma unroll
          for (int r = 0; r < 16; ++r) {
            const int key = kt + 32 * kb + 8 * (r / 4) + 4 * half + r % 4;
            const float x = __builtin_amdgcn_exp2f(fmaf(s[r], a.scale_log2, -lse2)) * dp[r];
            exact += (uint32_t)(key - seen.first) < seen.n ? x : 0.f;
          }
        }
      }
      __syncthreads();
      exact = sum_xor32(exact);
      if (seen.n <= kFewKeys) delta = exact;
    }
  }
  if (qi < lq && half == 0 && split == 0) {
    a.lse2[(int64_t)h * a.total_q + q0 + qi] = lse2;
    a.delta[(int64_t)h * a.total_q + q0 + qi] = delta;
  }

  float up = 1.f;  // what dS stands multiplied by
  float base = -lse2;
  if constexpr (scaled<T>()) {
    up = __builtin_amdgcn_ldexpf(1.f, kUpStart);
    base += (float)kUpStart;  // (rounds p by 2^-19 of itself at most, where its operand has 2^-11)
  }
  if (lo < hi) fetch(lo);
  int buf = 0;
  for (int kt = lo; kt < hi; kt += BN, buf ^= sizeof(T) == 4 ? 0 : 1) {
    if (sizeof(T) == 4) __syncthreads();  // one buffer: the last tile has been read
    uint16_t *kl = lds[buf][0], *vl = lds[buf][1];
    sk.store(kl, tid);
    sv.store(vl, tid);
    __syncthreads();
    if (kt + BN < hi) fetch(kt + BN);
    if (a.causal && (kt > wq + 31 + shift || (a.window && kt + BN <= wq + shift - (int)a.window + 1)))
      continue;  // nothing in it for this wave
    const bool edge = kt + BN > lk || (a.causal && (kt + BN - 1 > wq + shift ||
                                                    (a.window && kt <= wq + 31 + shift - (int)a.window)));
    const TileAt kl_at = tile_at<T, DP, BN>(kl, lane), vl_at = tile_at<T, DP, BN>(vl, lane);
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
      floatx16 s = {}, dp = {};
#pragma unroll
      for (int d = 0; d < DS; ++d) {
        s = mma32<T>(frag_rows<T, DP, BN>(kl_at, 32 * kb, 16 * d), qf[d], s);
        dp = mma32<T>(frag_rows<T, DP, BN>(vl_at, 32 * kb, 16 * d), df[d], dp);
      }
#pragma unroll
      for (int r = 0; r < 16; ++r)
        s[r] = __builtin_amdgcn_exp2f(fmaf(s[r], a.scale_log2, base)) * (dp[r] - delta);
      if (edge) {
        int first = seen.first;  // opaque, for a branch: most tiles have no edge, and selects would cost each of them
        asm volatile("" : "+v"(first));
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const int key = kt + 32 * kb + 8 * (r / 4) + 4 * half + r % 4;
          s[r] = (uint32_t)(key - first) < seen.n ? s[r] : 0.f;
        }
      }
      if constexpr (scaled<T>()) {
        const float f = down(s);
        if (__any(f != 1.f)) {
          s *= f;
#pragma unroll
          for (int db = 0; db < DB; ++db) acc[db] *= f;
          up *= f;
          base += (float)(__builtin_amdgcn_frexp_expf(f) - 1);
        }
      }
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const Frag<T> f = acc_frag<T>(s, t);
#pragma unroll
        for (int db = 0; db < DB; ++db) acc[db] = mma32<T>(frag_cols<T, DP, BN>(kl_at, 32 * kb + 16 * t, 32 * db), f, acc[db]);
      }
    }
  }

  if constexpr (scaled<T>()) {
#pragma unroll
    for (int db = 0; db < DB; ++db) acc[db] *= 1.f / up;
  }
  if (qi >= lq) return;
  if (a.splits > 1) {
    float* row = a.partial_q + (((size_t)split * a.total_q + q0 + qi) * a.H + h) * a.D;
#pragma unroll
    for (int db = 0; db < DB; ++db)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        store4<float, VEC>(row, 32 * db + 8 * j + 4 * half, a.D, acc[db][4 * j], acc[db][4 * j + 1], acc[db][4 * j + 2],
                           acc[db][4 * j + 3]);
    return;
  }
  T* row = static_cast<T*>(a.dq.p) + (q0 + qi) * a.dq.row + (int64_t)h * a.dq.head;
#pragma unroll
  for (int db = 0; db < DB; ++db)
#pragma unroll
    for (int j = 0; j < 4; ++j)
      store4<T, VEC>(row, 32 * db + 8 * j + 4 * half, a.D, acc[db][4 * j] * a.scale, acc[db][4 * j + 1] * a.scale,
                acc[db][4 * j + 2] * a.scale, acc[db][4 * j + 3] * a.scale);
}

// The queries that see any key of the block at tile_k, as tiles of BN for every
// sharing head: per_head tiles of a head from query lo, `all` together.
struct Run {
  int lo, per_head, all;
};
__device__ __forceinline__ Run query_run(const BwdArgs& a, int tile_k, int lq, int lk, int BN) {
  const int shift = lk - lq, last = min(tile_k + kRows, lk) - 1;
  int lo = 0, hi = lq;
  if (a.causal) {
    lo = max(0, tile_k - shift) / BN * BN;
    if (a.window) hi = min((int64_t)lq, (int64_t)last - shift + a.window);
  }
  const int per_head = lo < hi ? (hi - lo + BN - 1) / BN : 0;
  return {lo, per_head, per_head * (int)(a.H / a.G)};
}
// Workgroups that work on the block: one at least, which writes zeros where no
// query sees it; the last of them takes what is left.
__device__ __forceinline__ uint32_t parts_of(const BwdArgs& a, int all) {
  return min(a.parts, (uint32_t)max(1, (all + a.steps - 1) / a.steps));
}

// Each wave owns 32 keys.  S = Q K^T puts one key in each lane, its queries in the
// registers: P and dS are then the operands of dV^T += dO^T P and dK^T += Q^T dS.
template <class T, int DP, bool VEC>
__global__ __launch_bounds__(kThreads, (dkv_waves<T, DP>())) void attn_bwd_dkv(const BwdArgs a) {
  constexpr int BN = inner_tile<T, DP>();
  constexpr int QB = BN / 32, DS = DP / 16, DB = DP / 32;
  using L = Tile<T, DP, BN>;
  constexpr int kBufs = sizeof(T) == 4 ? 1 : 2;
  __shared__ __align__(kTileAlign) uint16_t lds[kBufs][2][L::words];  // Q, dO
  __shared__ __align__(16) float stats[kBufs][2][BN];         // lse2, -delta
  // The sums of 32 keys take 128 registers at DP = 128, their keys 32: with the
  // values beside them there would be one wave to a SIMD and moves between the register files
  // on each use, so the values stay in LDS (4 x 2048 queries, 16 heads of 128 over 2, without a
  // mask: 332 us with this and cheaper addresses, 539 us before).  float32 at DP = 64 is the
  // same case (4 x 1200 tokens, 24 heads of 64 over 8, the whole call: 432 us, 482 us with
  // the values in registers); wider float32 heads do not fit two waves either way.
  constexpr bool kValuesInLds = values_in_lds<T, DP>();
  __shared__ __align__(kTileAlign) uint16_t values[kValuesInLds ? Tile<T, DP, kRows>::words : 8];

  const uint32_t pairs = a.G * a.B;
  uint32_t i = blockIdx.x, pair;
  if (pairs % 8 == 0) {
    const uint32_t per = pairs / 8;
    pair = (i % 8) * per + (i / 8) % per;
    i = i / 8 / per;
  } else {
    pair = i % pairs;
    i = i / pairs;
  }
  const uint32_t g = pair / a.B, b = pair % a.B, share = a.H / a.G, part = i % a.parts;
  const int tile_k = (int)(i / a.parts) * kRows;  // early keys are seen by the most queries: they go first
  int64_t q0, k0;
  int lq, lk;
  seq_range(a.q_offsets, b, a.Lq, a.total_q, &q0, &lq);
  seq_range(a.kv_offsets, b, a.Lk, a.total_k, &k0, &lk);
  if (tile_k >= lk) return;
  const int shift = lk - lq;

  const int tid = threadIdx.x, lane = tid % 64, wave = __builtin_amdgcn_readfirstlane(tid / 64), half = lane / 32;
  const int wk = tile_k + wave * 32, ki = wk + lane % 32;
  const Seen seen = seen_by(ki, shift, lq, a.causal, (int)a.window);
  const Run run = query_run(a, tile_k, lq, lk, BN);
  const uint32_t parts = parts_of(a, run.all);
  if (part >= parts) return;
  const int lo = run.lo, per_head = run.per_head;
  const int begin = (int)part * a.steps, steps = part + 1 == parts ? run.all : begin + a.steps;

  Frag<T> kf[DS], vf[kValuesInLds ? 1 : DS];
  {
    const int rows = min(32, lk - wk);
    const rsrc_t rk = rows_rsrc<T>(a.k, k0 + wk, g, rows, a.D);
    const rsrc_t rv = rows_rsrc<T>(a.v, k0 + wk, g, rows, a.D);
#pragma unroll
    for (int s = 0; s < DS; ++s) {
      const uint32_t row = lane % 32, col = 16 * s + 8 * half;
      kf[s] = raw_frag<T>(load8<T, VEC>(rk, row * (uint32_t)(a.k.row * sizeof(T)), col, a.D));
      if constexpr (!kValuesInLds) vf[s] = raw_frag<T>(load8<T, VEC>(rv, row * (uint32_t)(a.v.row * sizeof(T)), col, a.D));
    }
  }

  if constexpr (kValuesInLds) {  // read after the first tile's barrier
    Stage<T, DP, kRows, kThreads, VEC> sv;
    sv.load(rows_rsrc<T>(a.v, k0 + tile_k, g, min(kRows, lk - tile_k), a.D), (uint32_t)(a.v.row * sizeof(T)), a.D, tid);
    sv.store(values, tid);
  }
  const TileAt values_at = tile_at<T, DP, kRows>(values + (kValuesInLds ? 32 * wave * L::ld : 0), lane);

  floatx16 dk[DB] = {}, dv[DB] = {};
  float up = __builtin_amdgcn_ldexpf(1.f, kUpStart - kUpP);  // (float16) what dS stands multiplied by, beside P's factor
  Stage<T, DP, BN, kThreads, VEC> sq, sd;
  float stat = 0.f;
  // Places that follow from the thread are made again on each step where they
  // would not stay in registers: a spilled one costs more than its reload, whose
  // wait covers the rows on their way as well.
  const auto again = [](int v) {
    if constexpr (kValuesInLds) asm volatile("" : "+v"(v));
    return v;
  };
  // Q's rows set out after the scores where the registers are short until then.
  constexpr bool kLateQ = kValuesInLds;
  auto fetch_q = [&](int step) {
    const int tid = again(threadIdx.x);
    const uint32_t h = g * share + (uint32_t)(step / per_head);
    const int qt = lo + step % per_head * BN;
    sq.load(rows_rsrc<T>(a.q, q0 + qt, h, min(BN, lq - qt), a.D), (uint32_t)(a.q.row * sizeof(T)), a.D, tid);
  };
  auto fetch = [&](int step) {
    const int tid = again(threadIdx.x);
    const uint32_t h = g * share + (uint32_t)(step / per_head);
    const int qt = lo + step % per_head * BN, rows = min(BN, lq - qt);
    sd.load(rows_rsrc<T>(a.dout, q0 + qt, h, rows, a.D), (uint32_t)(a.dout.row * sizeof(T)), a.D, tid);
    if (tid < 2 * BN) {
      const int r = tid % BN;
      const float* from = tid < BN ? a.lse2 : a.delta;
      // a query past the end has p = exp2(s - inf) = 0
      stat = r < rows ? from[(int64_t)h * a.total_q + q0 + qt + r] : tid < BN ? kInf : 0.f;
      if (tid >= BN)
        stat = -stat;
      else if constexpr (scaled<T>())
        stat -= (float)kUpP;  // P as a multiple of 2^14
    }
  };
  if (begin < steps) {
    fetch(begin);
    fetch_q(begin);
  }
  for (int step = begin; step < steps; ++step) {
    const int buf = kBufs == 1 ? 0 : step & 1;
    if (kBufs == 1) __syncthreads();
    const int tid = again(threadIdx.x), lane = tid % 64, half = lane / 32;
    uint16_t *ql = lds[buf][0], *dl = lds[buf][1];
    sq.store(ql, tid);
    sd.store(dl, tid);
    if (tid < 2 * BN) stats[buf][tid / BN][tid % BN] = stat;
    __syncthreads();
    if (step + 1 < steps) {
      fetch(step + 1);
      if (!kLateQ) fetch_q(step + 1);
    }
    const int qt = lo + step % per_head * BN;
    const TileAt ql_at = tile_at<T, DP, BN>(ql, lane), dl_at = tile_at<T, DP, BN>(dl, lane);
    const bool edge = a.causal && (qt + shift < wk + 31 || (a.window && qt + BN - 1 + shift - (int)a.window >= wk));
#pragma unroll
    for (int qb = 0; qb < QB; ++qb) {
      floatx16 s = {}, dp;
#pragma unroll
      for (int j = 0; j < 4; ++j) {  // dP - delta as a sum that starts at -delta
        const floatx4 d4 = lds_read4(&stats[buf][1][32 * qb + 8 * j + 4 * half]);
#pragma unroll
        for (int e = 0; e < 4; ++e) dp[4 * j + e] = d4[e];
      }
#pragma unroll
      for (int d = 0; d < DS; ++d) s = mma32<T>(frag_rows<T, DP, BN>(ql_at, 32 * qb, 16 * d), kf[d], s);
#pragma unroll
      for (int d = 0; d < DS; ++d) {
        const Frag<T> row = frag_rows<T, DP, BN>(dl_at, 32 * qb, 16 * d);
        if constexpr (kValuesInLds)
          dp = mma32<T>(row, frag_rows<T, DP, kRows>(values_at, 0, 16 * d), dp);
        else
          dp = mma32<T>(row, vf[d], dp);
      }
      if (kLateQ && qb == QB - 1 && step + 1 < steps) fetch_q(step + 1);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const floatx4 l4 = lds_read4(&stats[buf][0][32 * qb + 8 * j + 4 * half]);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          s[4 * j + e] = __builtin_amdgcn_exp2f(fmaf(s[4 * j + e], a.scale_log2, -l4[e]));
      }
      if (edge) {
        int first = seen.first;  // a branch, as above
        asm volatile("" : "+v"(first));
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const int row = qt + 32 * qb + 8 * (r / 4) + 4 * half + r % 4;
          const bool there = (uint32_t)(row - first) < seen.n;
          s[r] = there ? s[r] : 0.f;
          dp[r] = there ? dp[r] : 0.f;  // (a hidden one may have overflowed)
        }
      }
      if constexpr (scaled<T>()) {
#pragma unroll
        for (int r = 0; r < 16; ++r) dp[r] = dp[r] * up * s[r];
        const float f = down(dp);
        if (__any(f != 1.f)) {
          dp *= f;
#pragma unroll
          for (int db = 0; db < DB; ++db) dk[db] *= f;
          up *= f;
        }
      } else {
#pragma unroll
        for (int r = 0; r < 16; ++r) dp[r] *= s[r];
      }
      Frag<T> pf[2], df[2];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        pf[t] = acc_frag<T>(s, t);
        df[t] = acc_frag<T>(dp, t);
      }
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int db = 0; db < DB; ++db)
          dv[db] = mma32<T>(frag_cols<T, DP, BN>(dl_at, 32 * qb + 16 * t, 32 * db), pf[t], dv[db]);
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int db = 0; db < DB; ++db)
          dk[db] = mma32<T>(frag_cols<T, DP, BN>(ql_at, 32 * qb + 16 * t, 32 * db), df[t], dk[db]);
    }
  }

  if constexpr (scaled<T>()) {
    const float rest = 1.f / up;
#pragma unroll
    for (int db = 0; db < DB; ++db) {
      dv[db] *= __builtin_amdgcn_ldexpf(1.f, -kUpP);
      dk[db] *= __builtin_amdgcn_ldexpf(1.f, -kUpP) * rest;
    }
  }
  if (ki >= lk) return;
  if (parts > 1) {
    const size_t size = (size_t)a.total_k * a.G * a.D;
    float* rk = a.partial + part * size + ((size_t)(k0 + ki) * a.G + g) * a.D;
    float* rv = rk + a.parts * size;
#pragma unroll
    for (int db = 0; db < DB; ++db)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t col = 32 * db + 8 * j + 4 * half;
        store4<float, VEC>(rk, col, a.D, dk[db][4 * j], dk[db][4 * j + 1], dk[db][4 * j + 2], dk[db][4 * j + 3]);
        store4<float, VEC>(rv, col, a.D, dv[db][4 * j], dv[db][4 * j + 1], dv[db][4 * j + 2], dv[db][4 * j + 3]);
      }
    return;
  }
  T* rk = static_cast<T*>(a.dk.p) + (k0 + ki) * a.dk.row + (int64_t)g * a.dk.head;
  T* rv = static_cast<T*>(a.dv.p) + (k0 + ki) * a.dv.row + (int64_t)g * a.dv.head;
#pragma unroll
  for (int db = 0; db < DB; ++db)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t col = 32 * db + 8 * j + 4 * half;
      store4<T, VEC>(rk, col, a.D, dk[db][4 * j] * a.scale, dk[db][4 * j + 1] * a.scale, dk[db][4 * j + 2] * a.scale,
                     dk[db][4 * j + 3] * a.scale);
      store4<T, VEC>(rv, col, a.D, dv[db][4 * j], dv[db][4 * j + 1], dv[db][4 * j + 2], dv[db][4 * j + 3]);
    }
}

// Adds the parts of each block of keys that has several, in order, and rounds
// once: a thread takes four columns of one row and head.
template <class T, int DP, bool VEC>
__global__ __launch_bounds__(kThreads) void attn_bwd_join(const BwdArgs a) {
  const uint32_t pieces = (a.D + 3) / 4;
  const size_t e = (size_t)blockIdx.x * kThreads + threadIdx.x;
  const uint32_t col = e % pieces * 4, g = e / pieces % a.G;
  const int64_t row = (int64_t)(e / pieces / a.G);
  if (row >= a.total_k) return;
  uint32_t b;
  if (!find_seq(a.kv_offsets, a.B, a.Lk, a.total_k, row, &b)) return;
  int64_t q0, k0;
  int lq, lk;
  seq_range(a.q_offsets, b, a.Lq, a.total_q, &q0, &lq);
  seq_range(a.kv_offsets, b, a.Lk, a.total_k, &k0, &lk);
  const uint32_t parts = parts_of(a, query_run(a, (int)(row - k0) / kRows * kRows, lq, lk, inner_tile<T, DP>()).all);
  if (parts == 1) return;
  const size_t size = (size_t)a.total_k * a.G * a.D;
  const float* from = a.partial + ((size_t)row * a.G + g) * a.D + col;
  float dk[4] = {}, dv[4] = {};
  for (uint32_t p = 0; p < parts; ++p) {
    if constexpr (VEC) {
      const floatx4 x = *reinterpret_cast<const floatx4*>(from + p * size),
                    y = *reinterpret_cast<const floatx4*>(from + (a.parts + p) * size);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        dk[i] += x[i];
        dv[i] += y[i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (col + i < a.D) {
          dk[i] += from[p * size + i];
          dv[i] += from[(a.parts + p) * size + i];
        }
    }
  }
  store4<T, VEC>(static_cast<T*>(a.dk.p) + row * a.dk.row + (int64_t)g * a.dk.head, col, a.D, dk[0] * a.scale,
                 dk[1] * a.scale, dk[2] * a.scale, dk[3] * a.scale);
  store4<T, VEC>(static_cast<T*>(a.dv.p) + row * a.dv.row + (int64_t)g * a.dv.head, col, a.D, dv[0], dv[1], dv[2],
                 dv[3]);
}

// Adds the splits of dq in order and rounds once.
template <class T, bool VEC>
__global__ __launch_bounds__(kThreads) void attn_bwd_join_dq(const BwdArgs a) {
  const uint32_t pieces = (a.D + 3) / 4;
  const size_t e = (size_t)blockIdx.x * kThreads + threadIdx.x;
  const uint32_t col = e % pieces * 4, h = e / pieces % a.H;
  const int64_t row = (int64_t)(e / pieces / a.H);
  uint32_t b;
  if (row >= a.total_q || !find_seq(a.q_offsets, a.B, a.Lq, a.total_q, row, &b)) return;
  const size_t size = (size_t)a.total_q * a.H * a.D;
  const float* from = a.partial_q + ((size_t)row * a.H + h) * a.D + col;
  float dq[4] = {};
#pragma unroll 4
  for (uint32_t p = 0; p < a.splits; ++p) {
    if constexpr (VEC) {
      const floatx4 x = *reinterpret_cast<const floatx4*>(from + p * size);
#pragma unroll
      for (int i = 0; i < 4; ++i) dq[i] += x[i];
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (col + i < a.D) dq[i] += from[p * size + i];
    }
  }
  store4<T, VEC>(static_cast<T*>(a.dq.p) + row * a.dq.row + (int64_t)h * a.dq.head, col, a.D, dq[0] * a.scale,
                 dq[1] * a.scale, dq[2] * a.scale, dq[3] * a.scale);
}

uint32_t dq_splits(const AttnGeom& g) {
  const uint32_t seen = g.window && g.window < g.Lk ? g.window : g.Lk;
  return key_splits((uint64_t)((g.Lq + kRows - 1) / kRows) * g.H * g.B, seen, g.dtype == kF32 ? 64 : 256);
}

// The query tiles of one workgroup of dkv and how many share the longest block
// of keys.  Causal and ragged sequences give some blocks many times the queries
// of others, and a launch lasts as long as its longest workgroup; so each takes
// `steps` tiles, about half of what an even deal would give each of the 512
// workgroups that run at once, with the sums of a block's workgroups in the
// workspace and one more pass that adds them.  (4 x 2048 tokens, 24 heads of 64 over 8: 195 us
// and 14 for the join where one workgroup to a block took 224, both before the loop's
// later changes; a third or a quarter of the even deal costs more in the join than it
// saves.)  At most sixteen parts: their sums
// are written and read once each.
struct Plan {
  uint32_t parts;
  int steps;
};
Plan plan(const AttnGeom& g) {
  const uint64_t bn = g.dtype == kF32 || g.D > 64 ? 32 : 64;  // inner_tile
  const auto tiles = [](uint64_t n, uint64_t of) { return (n + of - 1) / of; };
  const uint64_t mq = tiles(g.total_q, g.B), mk = tiles(g.total_k, g.B);  // a mean sequence
  uint64_t seen = tiles(mq, bn);
  if (g.window && g.window < mk)
    seen = std::min(seen, tiles(g.window + kRows, bn));
  else if (g.causal)
    seen = (seen + 1) / 2;
  const uint64_t share = g.H / g.G, work = tiles(mk, kRows) * seen * share * g.G * g.B;
  const uint64_t longest = share * tiles(g.Lq, bn);
  uint64_t steps = std::max(tiles(work, 2 * 512), g.dtype == kF32 ? 2 : 256 / bn);
  steps = std::max(steps, tiles(longest, 16));
  steps = std::min(std::max<uint64_t>(steps, 1), (uint64_t)1 << 30);
  const uint64_t parts = std::max<uint64_t>(1, tiles(longest, steps));
  if (parts * tiles(g.Lk, kRows) * g.G * g.B > 1u << 24) return {1, 1 << 30};  // the launch is full without them
  return {(uint32_t)parts, (int)steps};
}

template <class T, int DP, bool VEC>
hipError_t launch_d(const AttnGeom& g, BwdArgs a, hipStream_t stream) {
  if (g.total_q > 0) {
    a.tiles = (g.Lq + kRows - 1) / kRows;
    attn_bwd_dq<T, DP, VEC><<<dim3(a.tiles * g.H * g.B * a.splits), kThreads, 0, stream>>>(a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (a.splits > 1) {
      const size_t n = (size_t)g.total_q * g.H * ((g.D + 3) / 4);
      attn_bwd_join_dq<T, VEC><<<dim3((uint32_t)((n + kThreads - 1) / kThreads)), kThreads, 0, stream>>>(a);
      e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
  }
  if (g.total_k > 0) {
    a.tiles = (g.Lk + kRows - 1) / kRows;
    attn_bwd_dkv<T, DP, VEC><<<dim3(a.tiles * a.parts * g.G * g.B), kThreads, 0, stream>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.parts == 1) return e;
    const size_t n = (size_t)g.total_k * g.G * ((g.D + 3) / 4);
    attn_bwd_join<T, DP, VEC><<<dim3((uint32_t)((n + kThreads - 1) / kThreads)), kThreads, 0, stream>>>(a);
  }
  return hipGetLastError();
}

template <class T>
hipError_t launch(const AttnGeom& g, const BwdArgs& a, hipStream_t stream) {
  const bool vec = a.q.vec && a.k.vec && a.v.vec && a.o.vec && a.dout.vec && a.dq.vec && a.dk.vec && a.dv.vec;
#define M3_CALL(DP) (vec ? launch_d<T, DP, true>(g, a, stream) : launch_d<T, DP, false>(g, a, stream))
  return M3_HEAD_DIM_SWITCH(g.D, M3_CALL);
#undef M3_CALL
}

// The workspace: lse2 and delta, the parts of dk and dv, then the splits of dq,
// each from a 16-byte boundary.
struct Workspace {
  size_t parts, splits, end;
};
Workspace layout(const AttnGeom& g) {
  const auto up = [](size_t n) { return (n + 3) / 4 * 4; };
  const uint32_t parts = plan(g).parts, splits = dq_splits(g);
  Workspace w;
  w.parts = up(2 * (size_t)g.total_q * g.H);
  w.splits = w.parts + (parts > 1 ? up(2 * parts * (size_t)g.total_k * g.G * g.D) : 0);
  w.end = w.splits + (splits > 1 ? splits * (size_t)g.total_q * g.H * g.D : 0);
  return w;
}

}  // namespace

size_t attn_bwd_workspace_floats(const AttnGeom& g) { return layout(g).end; }

uint64_t attn_bwd_workgroups(const AttnGeom& g) {
  const uint64_t parts = plan(g).parts, splits = dq_splits(g), pieces = (g.D + 3) / 4;
  const auto tiles = [](uint64_t n, uint64_t of) { return (n + of - 1) / of; };
  return std::max({tiles(g.Lq, kRows) * g.H * g.B * splits, tiles(g.Lk, kRows) * g.G * g.B * parts,
                   splits > 1 ? tiles((uint64_t)g.total_q * g.H * pieces, kThreads) : 0,
                   parts > 1 ? tiles((uint64_t)g.total_k * g.G * pieces, kThreads) : 0});
}

hipError_t launch_attn_bwd(const AttnGeom& g, const AttnOperands& o, hipStream_t stream) {
  const Workspace w = layout(g);
  const Plan p = plan(g);
  BwdArgs a{o.q, o.k, o.v, o.o, o.dout, o.dq, o.dk, o.dv, o.lse, o.ws, o.ws + (size_t)g.total_q * g.H, o.q_offsets,
            o.kv_offsets, g.B, g.Lq, g.Lk, g.H, g.G, g.D, g.total_q, g.total_k, g.causal, g.window, 0, p.parts, p.steps,
            o.ws + w.parts, dq_splits(g), o.ws + w.splits, g.scale, g.scale * kLog2e};
  if (g.dtype == kF32) return launch<float>(g, a, stream);
  if (g.dtype == kF16) return launch<_Float16>(g, a, stream);
  return launch<__bf16>(g, a, stream);
}

}  // namespace m3

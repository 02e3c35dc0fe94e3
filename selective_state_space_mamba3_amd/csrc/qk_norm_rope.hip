// Per-head RMS norm and position rotation of queries and keys in one pass:
//   n = w x / sqrt(mean(x^2) + eps);  for a < A, theta = position inv_freq[a],
//   (y_a, y_{a+A}) = R(theta) (n_a, n_{a+A});  y_d = n_d for d >= 2A.
// Backward, with u = R(theta)^T g on the pairs, r = 1 / sqrt(mean(x^2) + eps):
//   dx = r (u w - x r^2 mean(u w x)),   dw = sum over rows and heads of u x r.
//
// Bound by memory: each element is read once and written once.  A head is
// spread over a few lanes, each holding V columns below A and their partners
// V columns above (or two pieces of the columns that are not rotated), so the
// rotation needs no exchange and the mean a short one.  A workgroup first makes the
// sines of its rows (angles in float64: a far position times a frequency has
// no float32 digits to spare), which all the heads of a row share.
//
// 8192 rows of 24 + 8 heads of 64, bf16: 14.7 us forward (4.6 TB/s), 30.8 us backward (3.3 TB/s with
// the pass that adds the weights' gradient), where a large copy reaches 4.9 TB/s.
#include "attn_common.h"

#include <algorithm>

namespace m3 {

namespace {

struct RopeArgs {
  HeadView q, k, gq, gk;
  HeadOut oq, ok;
  const int32_t* positions;
  const float *inv_freq, *qw, *kw;
  float* partial;
  uint32_t rows, H, G, D, A;
  uint32_t lanes;     // of a head, a power of two
  uint32_t rows_per;  // rows of one workgroup and round
  float eps;
};

constexpr int kThreads = 256;
constexpr int kMaxRows = 16;  // of one round
constexpr uint32_t kMaxBlocks = 1024;  // of the backward pass
constexpr uint32_t kSpread = 512;      // workgroups that a launch should have before one takes more rows

// The two pieces of V columns that lane `c` of a head holds, -1 for none.
// Rotated columns come in pairs; the others follow, two pieces at a time.
template <int V>
__device__ __forceinline__ void pieces(uint32_t c, uint32_t A, uint32_t D, int* p0, int* p1, bool* turned) {
  const uint32_t pairs = A / V, rest = (D - 2 * A) / V;
  if (c < pairs) {
    *p0 = c * V;
    *p1 = A + c * V;
    *turned = true;
    return;
  }
  const uint32_t e = 2 * (c - pairs);
  *p0 = e < rest ? (int)(2 * A + e * V) : -1;
  *p1 = e + 1 < rest ? (int)(2 * A + (e + 1) * V) : -1;
  *turned = false;
}

// V neighbouring elements as they stand in memory: whole words of 16 (8) bytes.
template <class T, int V>
struct alignas(V * sizeof(T) > 16 ? 16 : V * sizeof(T)) Piece {
  T e[V];
};
template <class T, int V>
__device__ __forceinline__ Piece<T, V> load_piece(const T* row, int at) {
  Piece<T, V> p = {};
  if (at >= 0) p = *reinterpret_cast<const Piece<T, V>*>(row + at);
  return p;
}
template <class T, int V>
__device__ __forceinline__ void floats(const Piece<T, V>& p, float* f) {
#pragma unroll
  for (int i = 0; i < V; ++i) f[i] = to_float(p.e[i]);
}
// Weights of V columns; a vector of them has any alignment.
template <int V>
__device__ __forceinline__ void load_weights(const float* w, int at, float* f) {
#pragma unroll
  for (int i = 0; i < V; ++i) f[i] = 0.f;
  if (at >= 0) __builtin_memcpy(f, w + at, V * sizeof(float));
}
template <class T, int V>
__device__ __forceinline__ void store_piece(T* row, int at, const float* f) {
  if (at < 0) return;
  if constexpr (sizeof(T) == 2 && V > 1) {
    unsigned w[V / 2];
#pragma unroll
    for (int i = 0; i < V / 2; ++i) w[i] = pack2<T>(f[2 * i], f[2 * i + 1]);
    *reinterpret_cast<Piece<T, V>*>(row + at) = __builtin_bit_cast(Piece<T, V>, w);
  } else {
    Piece<T, V> p;
#pragma unroll
    for (int i = 0; i < V; ++i) p.e[i] = (T)f[i];
    *reinterpret_cast<Piece<T, V>*>(row + at) = p;
  }
}

__device__ __forceinline__ float group_sum(float v, uint32_t lanes) {
  for (uint32_t m = 1; m < lanes; m *= 2) v += __shfl_xor(v, m);
  return v;
}

// LDS: (cos, sin) of each row of the round and angle.
__device__ __forceinline__ void make_turns(const RopeArgs& a, uint32_t r0, uint32_t n, floatx2* turn, int tid) {
  for (uint32_t e = tid; e < n * a.A; e += kThreads) {
    float s, c;
    sincos_acc_d((double)a.positions[r0 + e / a.A] * (double)a.inv_freq[e % a.A], &s, &c);
    turn[e] = floatx2{c, s};
  }
}

// A lane's heads are read kBatch at a time, the first of them before the sines
// are made, so that the reads' latency and the sines' pass together.
constexpr int kBatch = 4;
template <class T, int V>
__global__ __launch_bounds__(kThreads) void qk_norm_rope_kernel(const RopeArgs a) {
  __shared__ floatx2 turn[kMaxRows * 64];
  const int tid = threadIdx.x;
  const uint32_t c = tid % a.lanes, slot = tid / a.lanes, slots = kThreads / a.lanes;
  const uint32_t heads = a.H + a.G;
  int p0, p1;
  bool turned;
  pieces<V>(c, a.A, a.D, &p0, &p1, &turned);
  const uint32_t r0 = blockIdx.x * a.rows_per, n = min(a.rows_per, a.rows - r0);
  Piece<T, V> lo[kBatch], hi[kBatch];
  const auto read = [&](uint32_t e0) {
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const uint32_t e = e0 + j * slots;
      if (e >= n * heads) break;
      const uint32_t row = e / heads, hh = e % heads;
      const HeadView& in = hh < a.H ? a.q : a.k;
      const T* x = static_cast<const T*>(in.p) + (int64_t)(r0 + row) * in.row +
                   (int64_t)(hh < a.H ? hh : hh - a.H) * in.head;
      lo[j] = load_piece<T, V>(x, p0);
      hi[j] = load_piece<T, V>(x, p1);
    }
  };
  read(slot);
  make_turns(a, r0, n, turn, tid);
  __syncthreads();
  for (uint32_t e0 = slot; e0 < n * heads; e0 += kBatch * slots) {
    if (e0 != slot) read(e0);
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const uint32_t e = e0 + j * slots;
      if (e >= n * heads) break;
      const uint32_t row = e / heads, hh = e % heads;
      const bool is_q = hh < a.H;
      const HeadOut& out = is_q ? a.oq : a.ok;
      T* y = static_cast<T*>(out.p) + (int64_t)(r0 + row) * out.row + (int64_t)(is_q ? hh : hh - a.H) * out.head;
      float l[V], h[V], wl[V], wh[V], sq = 0.f;
      floats<T, V>(lo[j], l);
      floats<T, V>(hi[j], h);
      load_weights<V>(is_q ? a.qw : a.kw, p0, wl);
      load_weights<V>(is_q ? a.qw : a.kw, p1, wh);
#pragma unroll
      for (int i = 0; i < V; ++i) sq = fmaf(l[i], l[i], fmaf(h[i], h[i], sq));
      const float r = 1.f / sqrtf(group_sum(sq, a.lanes) / (float)a.D + a.eps);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        l[i] *= r * wl[i];
        h[i] *= r * wh[i];
        if (turned) {
          const floatx2 t = turn[row * a.A + p0 + i];
          const float u = l[i] * t[0] - h[i] * t[1];
          h[i] = l[i] * t[1] + h[i] * t[0];
          l[i] = u;
        }
      }
      store_piece<T, V>(y, p0, l);
      store_piece<T, V>(y, p1, h);
    }
  }
}

// Columns of a lane's piece in the backward pass: with eight, the inputs, their
// successors and the weight sums take 160 registers and three workgroups of a compute
// unit's four (28 us at 8192 rows of 32 heads of 64, 25 us with four).
constexpr int kBwdCols = 4;
// Backward.  Each workgroup strides over the rows; a lane keeps the weight
// gradient of its columns in float32 over the few heads it meets, and the
// sums over lanes, then over workgroups, run in a fixed order (the last in float64).
template <class T, int V>
__global__ __launch_bounds__(kThreads) void qk_norm_rope_bwd_kernel(const RopeArgs a) {
  __shared__ floatx2 turn[kMaxRows * 64];
  __shared__ float sums[kThreads * 2 * V];
  const int tid = threadIdx.x;
  const uint32_t c = tid % a.lanes, slot = tid / a.lanes, slots = kThreads / a.lanes;
  int p0, p1;
  bool turned;
  pieces<V>(c, a.A, a.D, &p0, &p1, &turned);
  float dw[2][2 * V] = {};  // of the query and the key weight
  struct Item {
    Piece<T, V> x0, x1, g0, g1;
  };
  for (uint32_t r0 = blockIdx.x * a.rows_per; r0 < a.rows; r0 += gridDim.x * a.rows_per) {
    const uint32_t n = min(a.rows_per, a.rows - r0);
    const auto read = [&](int which, uint32_t e) {
      const HeadView &in = which ? a.k : a.q, &gr = which ? a.gk : a.gq;
      const uint32_t heads = which ? a.G : a.H;
      Item it = {};
      if (e < n * heads) {
        const uint32_t row = e / heads, h = e % heads;
        const T* x = static_cast<const T*>(in.p) + (int64_t)(r0 + row) * in.row + (int64_t)h * in.head;
        const T* gp = static_cast<const T*>(gr.p) + (int64_t)(r0 + row) * gr.row + (int64_t)h * gr.head;
        it = {load_piece<T, V>(x, p0), load_piece<T, V>(x, p1), load_piece<T, V>(gp, p0), load_piece<T, V>(gp, p1)};
      }
      return it;
    };
    // a lane's next head is on its way while it works on one, the first while the sines are made
    Item next = read(0, slot);
    __syncthreads();
    make_turns(a, r0, n, turn, tid);
    __syncthreads();
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      const HeadOut& out = which ? a.ok : a.oq;
      const uint32_t heads = which ? a.G : a.H;
      float w0[V], w1[V];
      load_weights<V>(which ? a.kw : a.qw, p0, w0);
      load_weights<V>(which ? a.kw : a.qw, p1, w1);
      for (uint32_t e = slot; e < n * heads; e += slots) {
        const Item it = next;
        if (which == 0 && e + slots >= n * heads)
          next = read(1, slot);
        else
          next = read(which, e + slots);
        const uint32_t row = e / heads, h = e % heads;
        T* y = static_cast<T*>(out.p) + (int64_t)(r0 + row) * out.row + (int64_t)h * out.head;
        float x0[V], x1[V], u0[V], u1[V], sq = 0.f, dot = 0.f;
        floats<T, V>(it.x0, x0);
        floats<T, V>(it.x1, x1);
        floats<T, V>(it.g0, u0);
        floats<T, V>(it.g1, u1);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          if (turned) {
            const floatx2 t = turn[row * a.A + p0 + i];
            const float l = u0[i] * t[0] + u1[i] * t[1];
            u1[i] = u1[i] * t[0] - u0[i] * t[1];
            u0[i] = l;
          }
          sq = fmaf(x0[i], x0[i], fmaf(x1[i], x1[i], sq));
          dot = fmaf(u0[i] * w0[i], x0[i], fmaf(u1[i] * w1[i], x1[i], dot));
        }
        const float r = 1.f / sqrtf(group_sum(sq, a.lanes) / (float)a.D + a.eps);
        const float f = group_sum(dot, a.lanes) / (float)a.D * r * r;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          dw[which][i] = fmaf(u0[i], x0[i] * r, dw[which][i]);
          dw[which][V + i] = fmaf(u1[i], x1[i] * r, dw[which][V + i]);
          u0[i] = r * (u0[i] * w0[i] - x0[i] * f);
          u1[i] = r * (u1[i] * w1[i] - x1[i] * f);
        }
        store_piece<T, V>(y, p0, u0);
        store_piece<T, V>(y, p1, u1);
      }
      // a lane without a query head read its key head here
      if (which == 0 && slot >= n * heads) next = read(1, slot);
    }
  }
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2 * V; ++i) sums[i * kThreads + tid] = dw[which][i];
    __syncthreads();
    // column (lane c, piece value i) summed over the slots
    for (uint32_t e = tid; e < a.lanes * 2 * V; e += kThreads) {
      const uint32_t cc = e % a.lanes, i = e / a.lanes;
      int q0, q1;
      bool t;
      pieces<V>(cc, a.A, a.D, &q0, &q1, &t);
      const int at = i < V ? q0 : q1;
      float s = 0.f;
      for (uint32_t k = 0; k < slots; ++k) s += sums[i * kThreads + k * a.lanes + cc];
      if (at >= 0) a.partial[((size_t)blockIdx.x * 2 + which) * a.D + at + i % V] = s;
    }
  }
}

// Adds the workgroups' sums in float64, in a fixed order: 16 columns by 64 runs of workgroups.
constexpr int kSumThreads = 1024;
__global__ __launch_bounds__(kSumThreads) void sum_partials_kernel(const float* partial, uint32_t blocks, uint32_t D,
                                                                   float* dqw, float* dkw) {
  __shared__ double sums[kSumThreads];
  const uint32_t c = threadIdx.x % 16, run = threadIdx.x / 16, col = blockIdx.x * 16 + c;  // of 2 D
  double s = 0.;
  if (col < 2 * D)
#pragma unroll 8
    for (uint32_t b = run; b < blocks; b += 64) s += (double)partial[(size_t)b * 2 * D + col];
  sums[threadIdx.x] = s;
  for (int half = 32; half; half /= 2) {
    __syncthreads();
    if (run < (uint32_t)half) sums[threadIdx.x] += sums[threadIdx.x + 16 * half];
  }
  if (run == 0 && col < 2 * D) (col < D ? dqw[col] : dkw[col - D]) = (float)sums[c];
}

uint32_t pow2_at_least(uint32_t n) {
  uint32_t p = 1;
  while (p < n) p *= 2;
  return p;
}

RopeArgs make_args(const RopeGeom& g, const RopeOperands& o, uint32_t V) {
  RopeArgs a{o.q, o.k, o.gq, o.gk, o.oq, o.ok, o.positions, o.inv_freq, o.qw, o.kw, o.partial, g.rows, g.H, g.G, g.D,
             g.A, 0, 0, g.eps};
  a.lanes = pow2_at_least(g.A / V + ((g.D - 2 * g.A) / V + 1) / 2);
  return a;
}

// Eight columns at a time where every piece is whole and aligned, one otherwise.
bool wide_ok(const RopeGeom& g, const RopeOperands& o, bool bwd) {
  return g.D % 8 == 0 && g.A % 8 == 0 && o.q.vec && o.k.vec && o.oq.vec && o.ok.vec &&
         (!bwd || (o.gq.vec && o.gk.vec));
}

uint32_t ceil_div(uint32_t n, uint32_t of) { return n / of + (n % of != 0); }

// Rows of a forward workgroup: as many as its lanes take in one batch (their
// angles then keep every lane at work too), fewer where that would leave compute
// units without a workgroup.
uint32_t fwd_rows(uint32_t rows, uint32_t lanes, uint32_t heads) {
  const uint32_t most = std::min<uint32_t>(kBatch * (kThreads / lanes) / heads, kMaxRows);
  return std::max(1u, std::min(most, ceil_div(rows, kSpread)));
}
// Backward: a round for each of at most four workgroups to a compute unit, and
// more rounds past 16 rows.  (8192 rows of 32 heads of 64: 1024 workgroups of 8 rows 25 us,
// 512 of 16 rows 33 us, 2048 of 4 rows 27 us.)
uint32_t bwd_rows(uint32_t rows) {
  return std::max(1u, std::min<uint32_t>(kMaxRows, ceil_div(rows, kMaxBlocks)));
}
uint32_t bwd_blocks(uint32_t rows) { return std::min(ceil_div(rows, bwd_rows(rows)), kMaxBlocks); }

template <class T>
hipError_t launch(const RopeGeom& g, const RopeOperands& o, bool bwd, hipStream_t stream) {
  const bool wide = wide_ok(g, o, bwd);
  RopeArgs a = make_args(g, o, !wide ? 1 : bwd ? kBwdCols : 8);
  if (!bwd) {
    a.rows_per = fwd_rows(g.rows, a.lanes, g.H + g.G);
    const dim3 grid(ceil_div(g.rows, a.rows_per));
    if (wide)
      qk_norm_rope_kernel<T, 8><<<grid, kThreads, 0, stream>>>(a);
    else
      qk_norm_rope_kernel<T, 1><<<grid, kThreads, 0, stream>>>(a);
    return hipGetLastError();
  }
  a.rows_per = bwd_rows(g.rows);
  const uint32_t blocks = bwd_blocks(g.rows);
  if (wide)
    qk_norm_rope_bwd_kernel<T, kBwdCols><<<dim3(blocks), kThreads, 0, stream>>>(a);
  else
    qk_norm_rope_bwd_kernel<T, 1><<<dim3(blocks), kThreads, 0, stream>>>(a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  sum_partials_kernel<<<dim3((2 * g.D + 15) / 16), kSumThreads, 0, stream>>>(o.partial, blocks, g.D, o.dqw, o.dkw);
  return hipGetLastError();
}

hipError_t dispatch(const RopeGeom& g, const RopeOperands& o, bool bwd, hipStream_t stream) {
  if (g.dtype == kF32) return launch<float>(g, o, bwd, stream);
  if (g.dtype == kF16) return launch<_Float16>(g, o, bwd, stream);
  return launch<__bf16>(g, o, bwd, stream);
}

}  // namespace

uint64_t qk_norm_rope_workgroups(const RopeGeom& g, const RopeOperands& o) {
  const RopeArgs a = make_args(g, o, wide_ok(g, o, false) ? 8 : 1);
  return ceil_div(g.rows, fwd_rows(g.rows, a.lanes, g.H + g.G));
}

hipError_t launch_qk_norm_rope(const RopeGeom& g, const RopeOperands& o, hipStream_t stream) {
  return dispatch(g, o, false, stream);
}
size_t qk_norm_rope_bwd_workspace_floats(const RopeGeom& g) { return (size_t)bwd_blocks(g.rows) * 2 * g.D; }
hipError_t launch_qk_norm_rope_bwd(const RopeGeom& g, const RopeOperands& o, hipStream_t stream) {
  return dispatch(g, o, true, stream);
}

}  // namespace m3

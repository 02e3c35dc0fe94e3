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
#include "attn_common.h"

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

template <class T, int V>
__device__ __forceinline__ void load_piece(const T* row, int at, float* f) {
  if (at < 0) {
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = 0.f;
    return;
  }
  if constexpr (V == 8) {
    raw_floats<T>(*reinterpret_cast<const Raw8<T>*>(row + at), f);
  } else {
    f[0] = to_float(row[at]);
  }
}
template <class T, int V>
__device__ __forceinline__ void store_piece(T* row, int at, const float* f) {
  if (at < 0) return;
  if constexpr (V == 8) {
    Raw8<T> r;
    if constexpr (sizeof(T) == 4) {
      r.v[0] = uintx4{__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3])};
      r.v[1] = uintx4{__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]), __float_as_uint(f[7])};
    } else {
      r.v[0] = uintx4{pack2<T>(f[0], f[1]), pack2<T>(f[2], f[3]), pack2<T>(f[4], f[5]), pack2<T>(f[6], f[7])};
    }
    *reinterpret_cast<Raw8<T>*>(row + at) = r;
  } else {
    row[at] = (T)f[0];
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
  make_turns(a, r0, n, turn, tid);
  __syncthreads();
  for (uint32_t e = slot; e < n * heads; e += slots) {
    const uint32_t row = e / heads, hh = e % heads;
    const bool is_q = hh < a.H;
    const HeadView& in = is_q ? a.q : a.k;
    const HeadOut& out = is_q ? a.oq : a.ok;
    const uint32_t h = is_q ? hh : hh - a.H;
    const T* x = static_cast<const T*>(in.p) + (int64_t)(r0 + row) * in.row + (int64_t)h * in.head;
    T* y = static_cast<T*>(out.p) + (int64_t)(r0 + row) * out.row + (int64_t)h * out.head;
    const float* w = is_q ? a.qw : a.kw;
    float lo[V], hi[V], sq = 0.f;
    load_piece<T, V>(x, p0, lo);
    load_piece<T, V>(x, p1, hi);
#pragma unroll
    for (int i = 0; i < V; ++i) sq = fmaf(lo[i], lo[i], fmaf(hi[i], hi[i], sq));
    const float r = 1.f / sqrtf(group_sum(sq, a.lanes) / (float)a.D + a.eps);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (p0 >= 0) lo[i] *= r * w[p0 + i];
      if (p1 >= 0) hi[i] *= r * w[p1 + i];
      if (turned) {
        const floatx2 t = turn[row * a.A + p0 + i];
        const float l = lo[i] * t[0] - hi[i] * t[1];
        hi[i] = lo[i] * t[1] + hi[i] * t[0];
        lo[i] = l;
      }
    }
    store_piece<T, V>(y, p0, lo);
    store_piece<T, V>(y, p1, hi);
  }
}

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
  for (uint32_t r0 = blockIdx.x * a.rows_per; r0 < a.rows; r0 += gridDim.x * a.rows_per) {
    const uint32_t n = min(a.rows_per, a.rows - r0);
    __syncthreads();
    make_turns(a, r0, n, turn, tid);
    __syncthreads();
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      const HeadView &in = which ? a.k : a.q, &gr = which ? a.gk : a.gq;
      const HeadOut& out = which ? a.ok : a.oq;
      const float* w = which ? a.kw : a.qw;
      const uint32_t heads = which ? a.G : a.H;
      for (uint32_t e = slot; e < n * heads; e += slots) {
        const uint32_t row = e / heads, h = e % heads;
        const T* x = static_cast<const T*>(in.p) + (int64_t)(r0 + row) * in.row + (int64_t)h * in.head;
        const T* gp = static_cast<const T*>(gr.p) + (int64_t)(r0 + row) * gr.row + (int64_t)h * gr.head;
        T* y = static_cast<T*>(out.p) + (int64_t)(r0 + row) * out.row + (int64_t)h * out.head;
        float x0[V], x1[V], u0[V], u1[V], sq = 0.f, dot = 0.f;
        load_piece<T, V>(x, p0, x0);
        load_piece<T, V>(x, p1, x1);
        load_piece<T, V>(gp, p0, u0);
        load_piece<T, V>(gp, p1, u1);
        float w0[V], w1[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
          w0[i] = p0 >= 0 ? w[p0 + i] : 0.f;
          w1[i] = p1 >= 0 ? w[p1 + i] : 0.f;
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

RopeArgs make_args(const RopeGeom& g, const RopeOperands& o, bool wide) {
  const uint32_t V = wide ? 8 : 1;
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

// Rows of one round: enough that the key heads alone give each lane group one.
uint32_t round_rows(uint32_t lanes, uint32_t heads) {
  const uint32_t slots = kThreads / lanes, n = (slots + heads - 1) / heads;
  return n < kMaxRows ? n : kMaxRows;
}

// Workgroups of the backward pass: a round each, at most four for each compute unit.
uint32_t bwd_blocks(uint32_t rows, uint32_t rows_per) {
  const uint32_t n = (rows + rows_per - 1) / rows_per;
  return n < kMaxBlocks ? n : kMaxBlocks;
}

template <class T>
hipError_t launch(const RopeGeom& g, const RopeOperands& o, bool bwd, hipStream_t stream) {
  const bool wide = wide_ok(g, o, bwd);
  RopeArgs a = make_args(g, o, wide);
  if (!bwd) {
    a.rows_per = round_rows(a.lanes, g.H + g.G);
    const dim3 grid((g.rows + a.rows_per - 1) / a.rows_per);
    if (wide)
      qk_norm_rope_kernel<T, 8><<<grid, kThreads, 0, stream>>>(a);
    else
      qk_norm_rope_kernel<T, 1><<<grid, kThreads, 0, stream>>>(a);
    return hipGetLastError();
  }
  a.rows_per = round_rows(a.lanes, g.G);
  const uint32_t blocks = bwd_blocks(g.rows, a.rows_per);
  if (wide)
    qk_norm_rope_bwd_kernel<T, 8><<<dim3(blocks), kThreads, 0, stream>>>(a);
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

hipError_t launch_qk_norm_rope(const RopeGeom& g, const RopeOperands& o, hipStream_t stream) {
  return dispatch(g, o, false, stream);
}
size_t qk_norm_rope_bwd_workspace_floats(const RopeGeom& g) { return (size_t)bwd_blocks(g.rows, 1) * 2 * g.D; }
hipError_t launch_qk_norm_rope_bwd(const RopeGeom& g, const RopeOperands& o, hipStream_t stream) {
  return dispatch(g, o, true, stream);
}

}  // namespace m3

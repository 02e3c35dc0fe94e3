// The second kernel of a decode step whose rows are split over workgroups.
#pragma once

#include "attn_common.h"

namespace m3 {

namespace {

// Partial results: (maximum, sum) [rows, H, splits, 2], then O [rows, H, splits, D].
struct JoinArgs {
  const float* ws;
  HeadOut out;
  uint32_t rows, H, D, splits;
};

// Joins the splits of one row and head, 32 columns to a workgroup: eight lanes
// of four columns, and the splits dealt over 32 groups of them.  All of it is
// latency, so the first sums are on their way before the maxima are known, and the
// columns are spread over workgroups (128 splits of 32 heads of 128:
// 18 us with a workgroup to a head).
constexpr int kMaxSplits = 512, kJoinCols = 32, kJoinThreads = 256, kJoinWaves = 4;
template <class T, bool VEC>
__global__ __launch_bounds__(kJoinThreads) void attn_step_join(const JoinArgs a) {
  constexpr int kGroups = kJoinThreads / 8, kAhead = 4;
  __shared__ float factor[kMaxSplits], red[2][kJoinWaves];
  __shared__ __align__(16) float cols[kGroups][kJoinCols + 4];
  const int tid = threadIdx.x, lane = tid % 64, wave = tid / 64, grp = tid / 8;
  const uint32_t slices = (a.D + kJoinCols - 1) / kJoinCols, bh = blockIdx.x / slices;
  const uint32_t row = bh / a.H, h = bh % a.H, n = a.splits, col = blockIdx.x % slices * kJoinCols + tid % 8 * 4;
  const size_t at = (size_t)bh * n;
  const floatx2* ms = reinterpret_cast<const floatx2*>(a.ws) + at;
  const float* o = a.ws + 2 * (size_t)a.rows * a.H * n + at * a.D;
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
  floatx2 mine[kMaxSplits / kJoinThreads];
#pragma unroll
  for (int i = 0; i < kMaxSplits / kJoinThreads; ++i)
    mine[i] = tid + i * kJoinThreads < (int)n ? ms[tid + i * kJoinThreads] : floatx2{-kInf, 0.f};
  floatx4 ahead[kAhead];
#pragma unroll
  for (int i = 0; i < kAhead; ++i) ahead[i] = part(grp + i * kGroups);

  float top = mine[0][0];
#pragma unroll
  for (int i = 1; i < kMaxSplits / kJoinThreads; ++i) top = __builtin_fmaxf(top, mine[i][0]);
  for (int x = 1; x < 64; x *= 2) top = __builtin_fmaxf(top, __shfl_xor(top, x));
  if (lane == 0) red[0][wave] = top;
  __syncthreads();
  top = __builtin_fmaxf(max3(red[0][0], red[0][1], red[0][2]), red[0][3]);
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < kMaxSplits / kJoinThreads; ++i) {
    const float f = top == -kInf ? 1.f : __builtin_amdgcn_exp2f(mine[i][0] - top);
    factor[tid + i * kJoinThreads] = f;
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
    static_cast<T*>(a.out.p)[(int64_t)row * a.out.row + (int64_t)h * a.out.head + d] = (T)(s == 0.f ? 0.f : v / s);
  }
}

// The same for few splits of many rows: a wave to a row and head, its halves taking turns at the splits.  (Two splits
// of 256 rows of 32 heads of 128: 37 us by the kernel above.)
template <class T>
__global__ __launch_bounds__(kJoinThreads) void attn_step_join_few(const JoinArgs a) {
  const int lane = threadIdx.x % 64, half = lane / 32;
  const uint32_t bh = blockIdx.x * kJoinWaves + __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  if (bh >= a.rows * a.H) return;
  const uint32_t row = bh / a.H, h = bh % a.H, n = a.splits, col = lane % 32 * 4;
  const size_t at = (size_t)bh * n;
  const floatx2* ms = reinterpret_cast<const floatx2*>(a.ws) + at;
  const float* o = a.ws + 2 * (size_t)a.rows * a.H * n + at * a.D;
  float top = -kInf, s = 0.f;
  for (uint32_t i = 0; i < n; ++i) top = __builtin_fmaxf(top, ms[i][0]);
  floatx4 sum = {};
  for (uint32_t i = half; i < n; i += 2) {
    const floatx2 part = ms[i];
    const float f = top == -kInf ? 1.f : __builtin_amdgcn_exp2f(part[0] - top);
    s = fmaf(part[1], f, s);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (col + e < a.D) sum[e] = fmaf(o[(size_t)i * a.D + col + e], f, sum[e]);
  }
  s = sum_xor32(s);
#pragma unroll
  for (int e = 0; e < 4; ++e) sum[e] = s == 0.f ? 0.f : sum_xor32(sum[e]) / s;
  if (half == 0)
    store4<T, false>(static_cast<T*>(a.out.p) + (int64_t)row * a.out.row + (int64_t)h * a.out.head, col, a.D, sum[0],
                     sum[1], sum[2], sum[3]);
}

inline uint64_t join_workgroups(uint64_t rows, uint32_t H, uint32_t D) {
  return rows * H * ((D + kJoinCols - 1) / kJoinCols);
}
template <class T>
hipError_t launch_join_few(const JoinArgs& a, hipStream_t stream) {
  attn_step_join_few<T><<<dim3((a.rows * a.H + kJoinWaves - 1) / kJoinWaves), kJoinThreads, 0, stream>>>(a);
  return hipGetLastError();
}
inline size_t join_floats(uint64_t rows, uint32_t H, uint32_t D, uint32_t splits) {
  return (size_t)rows * H * splits * (D + 2);
}

template <class T>
hipError_t launch_join(const JoinArgs& a, hipStream_t stream) {
  const dim3 grid((uint32_t)join_workgroups(a.rows, a.H, a.D));
  // (the sums stand behind 2 rows H splits floats and are D apart)
  if (a.D % 4 == 0 && (uint64_t)a.rows * a.H * a.splits % 2 == 0)
    attn_step_join<T, true><<<grid, kJoinThreads, 0, stream>>>(a);
  else
    attn_step_join<T, false><<<grid, kJoinThreads, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace

}  // namespace m3

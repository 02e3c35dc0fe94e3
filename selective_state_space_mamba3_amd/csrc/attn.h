// Internal launch interface of the attention layer's operators: per-head norm
// with rotation, attention forward and backward, the single-token step.
// Geometry, pointers and strides arriving here were validated by abi.cpp.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace m3 {

enum : uint32_t { kF32 = 0, kBF16 = 1, kF16 = 2 };

// Rows of heads: element (r, h, d) stands at p[r row + h head + d].  `vec`
// says that every 8-element piece (8 columns from a multiple of 8) can be read or
// written as aligned 16-byte words.
struct HeadView {
  const void* p;
  int64_t row, head;
  uint32_t vec;
};
struct HeadOut {
  void* p;
  int64_t row, head;
  uint32_t vec;
};

struct RopeGeom {
  uint32_t rows, H, G, D, A, dtype;
  float eps;
};
struct RopeOperands {
  HeadView q, k, gq, gk;  // gq, gk: backward only
  const int32_t* positions;
  const float *inv_freq, *qw, *kw;
  HeadOut oq, ok;  // y forward, dx backward
  float *dqw, *dkw;
  float* partial;  // backward: weight-gradient sums of each workgroup
};

struct AttnGeom {
  uint32_t B, Lq, Lk, H, G, D, causal, window, dtype;
  uint32_t total_q, total_k;
  float scale;
};
struct AttnOperands {
  HeadView q, k, v, o, dout;
  const int32_t *q_offsets, *kv_offsets;
  HeadOut out, dq, dk, dv;
  float* lse;
  float* ws;
};

struct StepCache {
  void* p;
  int64_t page, row, head;
  uint32_t vec;
};
struct AttnStepOperands {
  HeadView q, k, v;
  StepCache kc, vc;
  const int32_t *lengths, *table;
  uint32_t num_pages, page_size, max_pages;
  HeadOut out;
  float* ws;
};

// The largest launch of a call, in workgroups of 256 threads; a launch holds fewer than 2^32 threads.
constexpr uint64_t kMaxWorkgroups = 0xffffffffull / 256;
uint64_t qk_norm_rope_workgroups(const RopeGeom& g, const RopeOperands& o);
uint64_t attn_fwd_workgroups(const AttnGeom& g);
uint64_t attn_bwd_workgroups(const AttnGeom& g);
uint64_t attn_step_workgroups(const AttnGeom& g);

hipError_t launch_qk_norm_rope(const RopeGeom& g, const RopeOperands& o, hipStream_t stream);
size_t qk_norm_rope_bwd_workspace_floats(const RopeGeom& g);
hipError_t launch_qk_norm_rope_bwd(const RopeGeom& g, const RopeOperands& o, hipStream_t stream);

size_t attn_fwd_workspace_floats(const AttnGeom& g);
hipError_t launch_attn_fwd(const AttnGeom& g, const AttnOperands& o, hipStream_t stream);
size_t attn_bwd_workspace_floats(const AttnGeom& g);
hipError_t launch_attn_bwd(const AttnGeom& g, const AttnOperands& o, hipStream_t stream);
size_t attn_step_workspace_floats(const AttnGeom& g);
hipError_t launch_attn_step(const AttnGeom& g, const AttnStepOperands& o, hipStream_t stream);

}  // namespace m3

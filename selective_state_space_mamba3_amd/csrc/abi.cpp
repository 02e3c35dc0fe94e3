// C ABI of the Mamba-3 forward path: validation and dispatch.
//
// Validation mirrors the rules of the oarust 0.8.6 page
// src/rs/ml/matrix/mamba3.rs: Geometry::resolve (SISO), MimoGeometry::resolve
// (MIMO, without its P*N <= 4096 capacity cap), PreprocessGeometry::resolve
// and the sequence_length == 1 rule of dispatch_mamba3_siso_step, plus the
// u32 element-count limits those functions apply.  Every rule is checked on
// the host before any HIP call, so a rejected call touches no device memory
// and does not initialise the HIP runtime.
#include "../../include/m3.h"
#include "attn.h"
#include "kv8.h"
#include "launch.h"

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <initializer_list>
#include <mutex>
#include <utility>

namespace {

thread_local char g_err[512] = "";

int fail(int code, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_err, sizeof g_err, fmt, ap);
  va_end(ap);
  return code;
}

void clear_error() { g_err[0] = '\0'; }

constexpr uint64_t kU32 = 0xffffffffull;

// Product of extents, false on overflow of uint32 (the stable shader ABI width).
bool count_u32(std::initializer_list<uint64_t> ext) {
  uint64_t c = 1;
  for (uint64_t e : ext) {
    if (e != 0 && c > kU32 / e) return false;
    c *= e;
  }
  return c <= kU32;
}

struct Resolved {
  m3::ScanGeom g;
};

// Shared rule set of the scan geometry, one rule at a time, so that the
// message names the rule that failed.  `mimo` selects the multi-input rules
// (rank 1..8 and an optional output norm) instead of the single-input ones
// (rank exactly 1, no output norm).
int resolve_scan(const char* op, const m3_ssm_config& cfg, bool mimo, m3::ScanGeom* out) {
  const uint32_t G = cfg.num_groups == 0 ? cfg.num_heads : cfg.num_groups;
  const struct {
    const char* name;
    uint32_t v;
  } flags[] = {{"has_z", cfg.has_z}, {"has_d", cfg.has_d}, {"has_output_norm", cfg.has_output_norm}};
  for (const auto& f : flags)
    if (f.v > 1) return fail(M3_ERR_INVALID_ARGUMENT, "%s: flag %s is %u; a flag is 0 or 1", op, f.name, f.v);
  const struct {
    const char* name;
    uint32_t v;
  } extents[] = {{"batch_size", cfg.batch_size}, {"sequence_length", cfg.sequence_length},
                 {"num_heads", cfg.num_heads}, {"head_dim", cfg.head_dim}, {"state_size", cfg.state_size}};
  for (const auto& e : extents)
    if (e.v == 0) return fail(M3_ERR_INVALID_ARGUMENT, "%s: %s is 0; every extent must be at least 1", op, e.name);
  if (cfg.num_heads % G != 0)
    return fail(M3_ERR_INVALID_ARGUMENT, "%s: num_groups %u does not divide num_heads %u", op, G, cfg.num_heads);
  if (cfg.head_dim > 128)
    return fail(M3_ERR_INVALID_ARGUMENT, "%s: head_dim %u is above the limit of 128", op, cfg.head_dim);
  if (cfg.state_size > 128)
    return fail(M3_ERR_INVALID_ARGUMENT, "%s: state_size %u is above the limit of 128", op, cfg.state_size);
  if (cfg.num_rope_angles > 64)
    return fail(M3_ERR_INVALID_ARGUMENT, "%s: num_rope_angles %u is above the limit of 64", op,
                cfg.num_rope_angles);
  if (2ull * cfg.num_rope_angles > cfg.state_size)
    return fail(M3_ERR_INVALID_ARGUMENT,
                "%s: the %u rotary pairs need 2 * num_rope_angles = %u state coordinates, but state_size is %u",
                op, cfg.num_rope_angles, 2 * cfg.num_rope_angles, cfg.state_size);
  if (mimo) {
    if (cfg.mimo_rank < 1 || cfg.mimo_rank > 8)
      return fail(M3_ERR_INVALID_ARGUMENT, "%s: mimo_rank %u is outside 1..8", op, cfg.mimo_rank);
  } else {
    if (cfg.mimo_rank != 1)
      return fail(M3_ERR_INVALID_ARGUMENT, "%s: mimo_rank is %u; the single-input scan takes rank 1 only", op,
                  cfg.mimo_rank);
    if (cfg.has_output_norm != 0)
      return fail(M3_ERR_INVALID_ARGUMENT,
                  "%s: has_output_norm is set; the output norm belongs to the multi-input scan only", op);
  }
  const uint64_t B = cfg.batch_size, L = cfg.sequence_length, H = cfg.num_heads, P = cfg.head_dim,
                 N = cfg.state_size, A = cfg.num_rope_angles, R = mimo ? cfg.mimo_rank : 1;
  const struct {
    const char* name;
    bool ok;
  } counts[] = {{"c / b", count_u32({B, L, R * G, N})}, {"x / z / out", count_u32({B, L, H, P})},
                {"adt / dt / trap", count_u32({B, L, H})}, {"angle", count_u32({B, L, A})},
                {"c_bias / b_bias", count_u32({H, R, N})}, {"mimo weight", count_u32({H, R, P})},
                {"batch * heads", count_u32({B, H})}};
  for (const auto& c : counts)
    if (!c.ok)
      return fail(M3_ERR_INVALID_ARGUMENT, "%s: the %s element count does not fit in u32", op, c.name);
  out->B = cfg.batch_size;
  out->L = cfg.sequence_length;
  out->H = cfg.num_heads;
  out->G = G;
  out->P = cfg.head_dim;
  out->N = cfg.state_size;
  out->A = cfg.num_rope_angles;
  out->R = (uint32_t)R;
  out->has_z = cfg.has_z;
  out->has_d = cfg.has_d;
  out->has_norm = mimo ? cfg.has_output_norm : 0;
  return M3_OK;
}

int check_ptrs(const char* op, std::initializer_list<std::pair<const char*, const void*>> ptrs) {
  for (const auto& pr : ptrs)
    if (pr.second == nullptr) return fail(M3_ERR_INVALID_ARGUMENT, "%s: operand %s is NULL", op, pr.first);
  return M3_OK;
}

int hip_status(const char* op, hipError_t e) {
  if (e == hipSuccess) return M3_OK;
  return fail(M3_ERR_HIP, "%s: HIP error %d (%s)", op, (int)e, hipGetErrorString(e));
}

}  // namespace

extern "C" {

const char* m3_last_error(void) { return g_err; }

void m3_set_profile_events(void* start_event, void* stop_event) {
  m3::ProfileEvents& pe = m3::profile_events();
  const bool on = start_event != nullptr && stop_event != nullptr;
  pe.start = on ? static_cast<hipEvent_t>(start_event) : nullptr;
  pe.stop = on ? static_cast<hipEvent_t>(stop_event) : nullptr;
}

const char* m3_version(void) { return "m3 0.2.0 gfx950"; }

void m3_set_scan_segments(uint32_t segments) { m3::set_forced_segments(segments); }

}  // extern "C"

namespace {

// Preprocess geometry rules shared by the forward and the backward, checked
// one at a time so that the message names the rule that failed.
int resolve_pre(const char* op, uint32_t rows, const m3_preprocess_config& cfg, m3::PreGeom* out) {
  const struct {
    const char* name;
    uint32_t v;
  } extents[] = {{"rows", rows}, {"inner_size", cfg.inner_size}, {"state_size", cfg.state_size},
                 {"num_heads", cfg.num_heads}, {"num_groups", cfg.num_groups}, {"mimo_rank", cfg.mimo_rank}};
  for (const auto& e : extents)
    if (e.v == 0) return fail(M3_ERR_INVALID_ARGUMENT, "%s: %s is 0; every extent must be at least 1", op, e.name);
  if (2ull * cfg.num_rope_angles > cfg.state_size)
    return fail(M3_ERR_INVALID_ARGUMENT,
                "%s: the %u rotary pairs need 2 * num_rope_angles = %u state coordinates, but state_size is %u",
                op, cfg.num_rope_angles, 2 * cfg.num_rope_angles, cfg.state_size);
  const struct {
    const char* name;
    float v;
  } bounds[] = {{"epsilon", cfg.epsilon}, {"dt_min", cfg.dt_min}, {"dt_max", cfg.dt_max}, {"a_floor", cfg.a_floor}};
  for (const auto& b : bounds)
    if (!std::isfinite(b.v)) return fail(M3_ERR_INVALID_ARGUMENT, "%s: %s is not a finite number", op, b.name);
  // dt_max needs no sign rule of its own: it is at least dt_min
  for (const auto& b : {bounds[0], bounds[1], bounds[3]})
    if (b.v <= 0.f)
      return fail(M3_ERR_INVALID_ARGUMENT, "%s: %s is %g; it must be above zero", op, b.name, (double)b.v);
  if (cfg.dt_min > cfg.dt_max)
    return fail(M3_ERR_INVALID_ARGUMENT, "%s: dt_min %g is above dt_max %g", op, (double)cfg.dt_min,
                (double)cfg.dt_max);
  const uint64_t I = cfg.inner_size, N = cfg.state_size, H = cfg.num_heads,
                 A = cfg.num_rope_angles, GR = (uint64_t)cfg.num_groups * cfg.mimo_rank;
  const uint64_t M = GR * N;
  const uint64_t W = 2 * I + 2 * M + 3 * H + A;
  if (GR > kU32 || M > kU32 || W > kU32 || !count_u32({rows, W}) || !count_u32({rows, I}) ||
      !count_u32({rows, M}) || !count_u32({rows, H}) || !count_u32({rows, A}))
    return fail(M3_ERR_INVALID_ARGUMENT, "%s: projected width or an element count exceeds u32", op);
  *out = m3::PreGeom{rows, cfg.inner_size, cfg.state_size, cfg.num_heads, cfg.num_rope_angles,
                     cfg.num_groups, cfg.mimo_rank, cfg.epsilon, cfg.dt_min, cfg.dt_max, cfg.a_floor};
  return M3_OK;
}

}  // namespace

extern "C" {

int m3_preprocess(const float* projected, const float* dt_bias, uint32_t rows,
                  m3_preprocess_config cfg, float* x, float* z, float* bh, float* ch, float* dt,
                  float* adt, float* trap, float* angle, void* stream) {
  const char* op = "m3_preprocess";
  clear_error();
  m3::PreGeom g{};
  int st = resolve_pre(op, rows, cfg, &g);
  if (st) return st;
  st = check_ptrs(op, {{"projected", projected}, {"dt_bias", dt_bias}, {"x", x}, {"z", z},
                       {"bh", bh}, {"ch", ch}, {"dt", dt}, {"adt", adt}, {"trap", trap}});
  if (st) return st;
  if (g.A > 0 && angle == nullptr) return fail(M3_ERR_INVALID_ARGUMENT, "%s: operand angle is NULL", op);
  m3::PreOperands o{projected, dt_bias, x, z, bh, ch, dt, adt, trap, angle};
  return hip_status(op, m3::launch_preprocess(g, o, static_cast<hipStream_t>(stream)));
}

int m3_preprocess_bwd(const float* projected, const float* dt_bias, uint32_t rows,
                      m3_preprocess_config cfg, const float* g_x, const float* g_z, const float* g_bh,
                      const float* g_ch, const float* g_dt, const float* g_adt, const float* g_trap,
                      const float* g_angle, float* d_projected, float* d_dt_bias, void* stream) {
  const char* op = "m3_preprocess_bwd";
  clear_error();
  m3::PreGeom g{};
  int st = resolve_pre(op, rows, cfg, &g);
  if (st) return st;
  st = check_ptrs(op, {{"projected", projected}, {"dt_bias", dt_bias}, {"d_projected", d_projected},
                       {"d_dt_bias", d_dt_bias}});
  if (st) return st;
  m3::PreBwdOperands o{projected, dt_bias, g_x, g_z, g_bh, g_ch, g_dt, g_adt, g_trap,
                       g.A > 0 ? g_angle : nullptr, d_projected, d_dt_bias};
  return hip_status(op, m3::launch_preprocess_bwd(g, o, static_cast<hipStream_t>(stream)));
}

size_t m3_siso_bwd_workspace_bytes(m3_ssm_config cfg) {
  m3::ScanGeom g{};
  if (resolve_scan("m3_siso_bwd_workspace_bytes", cfg, false, &g) != M3_OK) return 0;
  return m3::siso_bwd_workspace_floats(g) * sizeof(float);
}

int m3_siso_bwd(const float* dout, const float* c, const float* b, const float* x, const float* z,
                const float* adt, const float* dt, const float* trap, const float* angle,
                const float* c_bias, const float* b_bias, const float* d, m3_ssm_config cfg,
                float* d_c, float* d_b, float* d_x, float* d_z, float* d_adt, float* d_dt,
                float* d_trap, float* d_angle, float* d_c_bias, float* d_b_bias, float* d_d,
                void* workspace, size_t workspace_bytes, void* stream) {
  const char* op = "m3_siso_bwd";
  clear_error();
  m3::ScanGeom g{};
  int st = resolve_scan(op, cfg, false, &g);
  if (st) return st;
  st = check_ptrs(op, {{"dout", dout}, {"c", c}, {"b", b}, {"x", x}, {"z", z}, {"adt", adt},
                       {"dt", dt}, {"trap", trap}, {"c_bias", c_bias}, {"b_bias", b_bias}, {"d", d},
                       {"d_c", d_c}, {"d_b", d_b}, {"d_x", d_x}, {"d_z", d_z}, {"d_adt", d_adt},
                       {"d_dt", d_dt}, {"d_trap", d_trap}, {"d_c_bias", d_c_bias},
                       {"d_b_bias", d_b_bias}, {"d_d", d_d}});
  if (st) return st;
  if (g.A > 0 && (angle == nullptr || d_angle == nullptr))
    return fail(M3_ERR_INVALID_ARGUMENT, "%s: operand angle or d_angle is NULL", op);
  if (!m3::siso_bwd_fits(g))
    return fail(M3_ERR_UNSUPPORTED, "%s: %u heads per group with state_size %u exceed the LDS of the "
                "backward group reduction", op, g.H / g.G, g.N);
  const size_t need = m3::siso_bwd_workspace_floats(g) * sizeof(float);
  if (workspace == nullptr || workspace_bytes < need)
    return fail(M3_ERR_INVALID_ARGUMENT, "%s: workspace of %zu bytes required, %zu given", op, need,
                workspace == nullptr ? (size_t)0 : workspace_bytes);
  m3::ScanOperands o{c, b, x, z, adt, dt, trap, angle, c_bias, b_bias, d,
                     nullptr, nullptr, nullptr, nullptr, nullptr};
  m3::BwdOperands go{dout, d_c, d_b, d_x, d_z, d_adt, d_dt, d_trap, d_angle, d_c_bias, d_b_bias, d_d};
  return hip_status(op, m3::launch_siso_bwd(g, o, go, workspace, static_cast<hipStream_t>(stream)));
}

}  // extern "C"

namespace {

// Fused preprocess -> scan: the two configs must describe one geometry.
struct PackedPlan {
  m3::ScanGeom g;
  m3::PreGeom pg;
  m3::ScanPlan plan;
  size_t o_bh, o_ch, o_dt, o_adt, o_scan, total_bytes;
  uint32_t W, I, M;
};

int resolve_packed(const char* op, const m3_preprocess_config& pcfg, const m3_ssm_config& cfg, PackedPlan* pp) {
  int st = resolve_scan(op, cfg, false, &pp->g);
  if (st) return st;
  const m3::ScanGeom& g = pp->g;
  if (!count_u32({g.B, g.L})) return fail(M3_ERR_INVALID_ARGUMENT, "%s: batch_size * sequence_length exceeds u32", op);
  st = resolve_pre(op, g.B * g.L, pcfg, &pp->pg);
  if (st) return st;
  if ((uint64_t)pcfg.inner_size != (uint64_t)g.H * g.P)
    return fail(M3_ERR_INVALID_ARGUMENT, "%s: inner_size %u differs from num_heads * head_dim = %u", op,
                pcfg.inner_size, g.H * g.P);
  const struct {
    const char* name;
    uint32_t pre, scan;
  } same[] = {{"state_size", pcfg.state_size, g.N}, {"num_heads", pcfg.num_heads, g.H},
              {"num_rope_angles", pcfg.num_rope_angles, g.A}, {"num_groups", pcfg.num_groups, g.G}};
  for (const auto& m : same)
    if (m.pre != m.scan)
      return fail(M3_ERR_INVALID_ARGUMENT, "%s: %s is %u in the preprocess config but %u in the scan config", op,
                  m.name, m.pre, m.scan);
  if (pcfg.mimo_rank != 1)
    return fail(M3_ERR_INVALID_ARGUMENT, "%s: the preprocess config has mimo_rank %u; the fused call is rank 1",
                op, pcfg.mimo_rank);
  pp->I = pcfg.inner_size;
  pp->M = g.G * g.N;
  pp->W = 2 * pp->I + 2 * pp->M + 3 * g.H + g.A;
  pp->plan = m3::plan_siso(g);
  const size_t rows = (size_t)g.B * g.L;
  size_t off = 0;
  auto take = [&](size_t floats) {
    const size_t o = off;
    off += (floats + 63) / 64 * 64;  // 256-byte aligned pieces
    return o;
  };
  pp->o_bh = take(rows * pp->M);
  pp->o_ch = take(rows * pp->M);
  pp->o_dt = take(rows * g.H);
  pp->o_adt = take(rows * g.H);
  pp->o_scan = off;
  pp->total_bytes = off * sizeof(float) + m3::plan_workspace_bytes(pp->plan);
  return M3_OK;
}

}  // namespace

extern "C" {

size_t m3_siso_fwd_packed_workspace_bytes(m3_preprocess_config pcfg, m3_ssm_config cfg) {
  PackedPlan pp{};
  if (resolve_packed("m3_siso_fwd_packed_workspace_bytes", pcfg, cfg, &pp) != M3_OK) return 0;
  return pp.total_bytes;
}

int m3_siso_fwd_packed(const float* projected, const float* dt_bias, const float* c_bias,
                       const float* b_bias, const float* d, m3_preprocess_config pcfg,
                       m3_ssm_config cfg, float* out, void* workspace, size_t workspace_bytes,
                       void* stream) {
  const char* op = "m3_siso_fwd_packed";
  clear_error();
  PackedPlan pp{};
  int st = resolve_packed(op, pcfg, cfg, &pp);
  if (st) return st;
  st = check_ptrs(op, {{"projected", projected}, {"dt_bias", dt_bias}, {"c_bias", c_bias},
                       {"b_bias", b_bias}, {"d", d}, {"out", out}, {"workspace", workspace}});
  if (st) return st;
  if (workspace_bytes < pp.total_bytes)
    return fail(M3_ERR_INVALID_ARGUMENT, "%s: workspace of %zu bytes required, %zu given", op,
                pp.total_bytes, workspace_bytes);
  float* ws = static_cast<float*>(workspace);
  const hipStream_t s = static_cast<hipStream_t>(stream);
  m3::PreOperands po{projected, dt_bias, nullptr, nullptr, ws + pp.o_bh, ws + pp.o_ch,
                     ws + pp.o_dt, ws + pp.o_adt, nullptr, nullptr};
  st = hip_status(op, m3::launch_preprocess_derived(pp.pg, po, s));
  if (st) return st;
  const m3::ScanGeom& g = pp.g;
  const uint32_t o_tr = 2 * pp.I + 2 * pp.M + 2 * g.H;
  m3::ScanOperands o{ws + pp.o_ch, ws + pp.o_bh, projected + pp.I, projected, ws + pp.o_adt, ws + pp.o_dt,
                     projected + o_tr, g.A > 0 ? projected + o_tr + g.H : nullptr, c_bias, b_bias, d,
                     nullptr, nullptr, nullptr, nullptr, out, pp.W, pp.W, pp.W};
  void* scan_ws = m3::plan_workspace_bytes(pp.plan) > 0 ? static_cast<void*>(ws + pp.o_scan) : nullptr;
  return hip_status(op, m3::launch_siso_fwd(g, o, pp.plan, scan_ws, s));
}

size_t m3_mimo_bwd_workspace_bytes(m3_ssm_config cfg) {
  m3::ScanGeom g{};
  if (resolve_scan("m3_mimo_bwd_workspace_bytes", cfg, true, &g) != M3_OK) return 0;
  return m3::mimo_bwd_workspace_floats(g) * sizeof(float);
}

int m3_mimo_bwd(const float* dout, const float* c, const float* b, const float* x, const float* z,
                const float* adt, const float* dt, const float* trap, const float* angle,
                const float* c_bias, const float* b_bias, const float* d, const float* mimo_x,
                const float* mimo_z, const float* mimo_o, const float* norm_weight, m3_ssm_config cfg,
                float* d_c, float* d_b, float* d_x, float* d_z, float* d_adt, float* d_dt,
                float* d_trap, float* d_angle, float* d_c_bias, float* d_b_bias, float* d_d,
                float* d_mimo_x, float* d_mimo_z, float* d_mimo_o, float* d_norm_weight,
                void* workspace, size_t workspace_bytes, void* stream) {
  const char* op = "m3_mimo_bwd";
  clear_error();
  m3::ScanGeom g{};
  int st = resolve_scan(op, cfg, true, &g);
  if (st) return st;
  st = check_ptrs(op, {{"dout", dout}, {"c", c}, {"b", b}, {"x", x}, {"z", z}, {"adt", adt},
                       {"dt", dt}, {"trap", trap}, {"c_bias", c_bias}, {"b_bias", b_bias}, {"d", d},
                       {"mimo_x", mimo_x}, {"mimo_z", mimo_z}, {"mimo_o", mimo_o},
                       {"norm_weight", norm_weight}, {"d_c", d_c}, {"d_b", d_b}, {"d_x", d_x},
                       {"d_z", d_z}, {"d_adt", d_adt}, {"d_dt", d_dt}, {"d_trap", d_trap},
                       {"d_c_bias", d_c_bias}, {"d_b_bias", d_b_bias}, {"d_d", d_d},
                       {"d_mimo_x", d_mimo_x}, {"d_mimo_z", d_mimo_z}, {"d_mimo_o", d_mimo_o},
                       {"d_norm_weight", d_norm_weight}});
  if (st) return st;
  if (g.A > 0 && (angle == nullptr || d_angle == nullptr))
    return fail(M3_ERR_INVALID_ARGUMENT, "%s: operand angle or d_angle is NULL", op);
  if (!m3::mimo_bwd_fits(g))
    return fail(M3_ERR_UNSUPPORTED, "%s: %u heads per group at rank %u with state_size %u exceed the LDS of the "
                "backward kernels", op, g.H / g.G, g.R, g.N);
  const size_t need = m3::mimo_bwd_workspace_floats(g) * sizeof(float);
  if (workspace == nullptr || workspace_bytes < need)
    return fail(M3_ERR_INVALID_ARGUMENT, "%s: workspace of %zu bytes required, %zu given", op, need,
                workspace == nullptr ? (size_t)0 : workspace_bytes);
  m3::ScanOperands o{c, b, x, z, adt, dt, trap, angle, c_bias, b_bias, d,
                     mimo_x, mimo_z, mimo_o, norm_weight, nullptr};
  m3::BwdOperands go{dout, d_c, d_b, d_x, d_z, d_adt, d_dt, d_trap, d_angle, d_c_bias, d_b_bias, d_d,
                     d_mimo_x, d_mimo_z, d_mimo_o, d_norm_weight};
  return hip_status(op, m3::launch_mimo_bwd(g, o, go, workspace, static_cast<hipStream_t>(stream)));
}

size_t m3_siso_fwd_workspace_bytes(m3_ssm_config cfg) {
  m3::ScanGeom g{};
  if (resolve_scan("m3_siso_fwd_workspace_bytes", cfg, false, &g) != M3_OK) return 0;
  return m3::plan_workspace_bytes(m3::plan_siso(g));
}

size_t m3_mimo_fwd_workspace_bytes(m3_ssm_config cfg) {
  m3::ScanGeom g{};
  if (resolve_scan("m3_mimo_fwd_workspace_bytes", cfg, true, &g) != M3_OK) return 0;
  return m3::plan_workspace_bytes(m3::plan_mimo(g));
}

int m3_siso_fwd(const float* c, const float* b, const float* x, const float* z, const float* adt,
                const float* dt, const float* trap, const float* angle, const float* c_bias,
                const float* b_bias, const float* d, m3_ssm_config cfg, float* out, void* workspace,
                size_t workspace_bytes, void* stream) {
  const char* op = "m3_siso_fwd";
  clear_error();
  m3::ScanGeom g{};
  int st = resolve_scan(op, cfg, false, &g);
  if (st) return st;
  st = check_ptrs(op, {{"c", c}, {"b", b}, {"x", x}, {"z", z}, {"adt", adt}, {"dt", dt},
                       {"trap", trap}, {"c_bias", c_bias}, {"b_bias", b_bias}, {"d", d}, {"out", out}});
  if (st) return st;
  if (g.A > 0 && angle == nullptr) return fail(M3_ERR_INVALID_ARGUMENT, "%s: operand angle is NULL", op);
  const m3::ScanPlan plan = m3::plan_siso(g);
  const size_t need = m3::plan_workspace_bytes(plan);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need))
    return fail(M3_ERR_INVALID_ARGUMENT, "%s: workspace of %zu bytes required, %zu given", op, need,
                workspace == nullptr ? (size_t)0 : workspace_bytes);
  m3::ScanOperands o{c, b, x, z, adt, dt, trap, angle, c_bias, b_bias, d,
                     nullptr, nullptr, nullptr, nullptr, out};
  return hip_status(op, m3::launch_siso_fwd(g, o, plan, workspace, static_cast<hipStream_t>(stream)));
}

int m3_mimo_fwd(const float* c, const float* b, const float* x, const float* z, const float* adt,
                const float* dt, const float* trap, const float* angle, const float* c_bias,
                const float* b_bias, const float* d, const float* mimo_x, const float* mimo_z,
                const float* mimo_o, const float* norm_weight, m3_ssm_config cfg, float* out,
                void* workspace, size_t workspace_bytes, void* stream) {
  const char* op = "m3_mimo_fwd";
  clear_error();
  m3::ScanGeom g{};
  int st = resolve_scan(op, cfg, true, &g);
  if (st) return st;
  st = check_ptrs(op, {{"c", c}, {"b", b}, {"x", x}, {"z", z}, {"adt", adt}, {"dt", dt},
                       {"trap", trap}, {"c_bias", c_bias}, {"b_bias", b_bias}, {"d", d},
                       {"mimo_x", mimo_x}, {"mimo_z", mimo_z}, {"mimo_o", mimo_o},
                       {"norm_weight", norm_weight}, {"out", out}});
  if (st) return st;
  if (g.A > 0 && angle == nullptr) return fail(M3_ERR_INVALID_ARGUMENT, "%s: operand angle is NULL", op);
  const m3::ScanPlan plan = m3::plan_mimo(g);
  const size_t need = m3::plan_workspace_bytes(plan);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need))
    return fail(M3_ERR_INVALID_ARGUMENT, "%s: workspace of %zu bytes required, %zu given", op, need,
                workspace == nullptr ? (size_t)0 : workspace_bytes);
  m3::ScanOperands o{c, b, x, z, adt, dt, trap, angle, c_bias, b_bias, d,
                     mimo_x, mimo_z, mimo_o, norm_weight, out};
  return hip_status(op, m3::launch_mimo_fwd(g, o, plan, workspace, static_cast<hipStream_t>(stream)));
}

int m3_siso_step(const float* c, const float* b, const float* x, const float* z, const float* adt,
                 const float* dt, const float* trap, const float* angle, const float* c_bias,
                 const float* b_bias, const float* d, float* ssm_state, float* angle_state,
                 float* k_state, float* v_state, m3_ssm_config cfg, float* out, void* stream) {
  const char* op = "m3_siso_step";
  clear_error();
  m3::ScanGeom g{};
  int st = resolve_scan(op, cfg, false, &g);
  if (st) return st;
  if (cfg.sequence_length != 1)
    return fail(M3_ERR_INVALID_ARGUMENT, "%s: sequence_length is %u; a decode step takes exactly one token", op,
                cfg.sequence_length);
  if (!count_u32({g.B, g.H, g.P, g.N}))
    return fail(M3_ERR_INVALID_ARGUMENT, "%s: state element count exceeds u32", op);
  st = check_ptrs(op, {{"c", c}, {"b", b}, {"x", x}, {"z", z}, {"adt", adt}, {"dt", dt},
                       {"trap", trap}, {"c_bias", c_bias}, {"b_bias", b_bias}, {"d", d},
                       {"ssm_state", ssm_state}, {"k_state", k_state}, {"v_state", v_state},
                       {"out", out}});
  if (st) return st;
  if (g.A > 0 && (angle == nullptr || angle_state == nullptr))
    return fail(M3_ERR_INVALID_ARGUMENT, "%s: operand angle or angle_state is NULL", op);
  m3::ScanOperands o{c, b, x, z, adt, dt, trap, angle, c_bias, b_bias, d,
                     nullptr, nullptr, nullptr, nullptr, out};
  m3::StepStates s{ssm_state, angle_state, k_state, v_state};
  return hip_status(op, m3::launch_siso_step(g, o, s, static_cast<hipStream_t>(stream)));
}

int m3_mimo_step(const float* c, const float* b, const float* x, const float* z, const float* adt,
                 const float* dt, const float* trap, const float* angle, const float* c_bias,
                 const float* b_bias, const float* d, const float* mimo_x, const float* mimo_z,
                 const float* mimo_o, const float* norm_weight, float* ssm_state, float* angle_state,
                 float* k_state, float* v_state, m3_ssm_config cfg, float* out, void* stream) {
  const char* op = "m3_mimo_step";
  clear_error();
  m3::ScanGeom g{};
  int st = resolve_scan(op, cfg, true, &g);
  if (st) return st;
  if (cfg.sequence_length != 1)
    return fail(M3_ERR_INVALID_ARGUMENT, "%s: sequence_length is %u; a decode step takes exactly one token", op,
                cfg.sequence_length);
  if (!count_u32({g.B, g.H, g.P, g.N}) || !count_u32({g.B, g.H, g.R, g.N}) || !count_u32({g.B, g.H, g.R, g.P}))
    return fail(M3_ERR_INVALID_ARGUMENT, "%s: state element count exceeds u32", op);
  st = check_ptrs(op, {{"c", c}, {"b", b}, {"x", x}, {"z", z}, {"adt", adt}, {"dt", dt},
                       {"trap", trap}, {"c_bias", c_bias}, {"b_bias", b_bias}, {"d", d},
                       {"mimo_x", mimo_x}, {"mimo_z", mimo_z}, {"mimo_o", mimo_o},
                       {"norm_weight", norm_weight}, {"ssm_state", ssm_state}, {"k_state", k_state},
                       {"v_state", v_state}, {"out", out}});
  if (st) return st;
  if (g.A > 0 && (angle == nullptr || angle_state == nullptr))
    return fail(M3_ERR_INVALID_ARGUMENT, "%s: operand angle or angle_state is NULL", op);
  m3::ScanOperands o{c, b, x, z, adt, dt, trap, angle, c_bias, b_bias, d,
                     mimo_x, mimo_z, mimo_o, norm_weight, out};
  m3::StepStates s{ssm_state, angle_state, k_state, v_state};
  return hip_status(op, m3::launch_mimo_step(g, o, s, static_cast<hipStream_t>(stream)));
}

}  // extern "C"

// ---- attention layer ---------------------------------------------------------
namespace {

constexpr int64_t kMaxRowBytes = int64_t(8) << 20;  // keeps a tile's byte offsets inside 31 bits

uint32_t dtype_size(uint32_t dtype) { return dtype == M3_F32 ? 4 : 2; }

int resolve_heads(const char* op, uint32_t heads, uint32_t num_groups, uint32_t head_dim, uint32_t dtype, uint32_t* G) {
  *G = num_groups == 0 ? heads : num_groups;
  if (heads == 0) return fail(M3_ERR_INVALID_ARGUMENT, "%s: num_heads is 0; every extent must be at least 1", op);
  if (head_dim == 0) return fail(M3_ERR_INVALID_ARGUMENT, "%s: head_dim is 0; every extent must be at least 1", op);
  if (heads % *G != 0)
    return fail(M3_ERR_INVALID_ARGUMENT, "%s: num_groups %u does not divide num_heads %u", op, *G, heads);
  if (head_dim > 128)
    return fail(M3_ERR_INVALID_ARGUMENT, "%s: head_dim %u is above the limit of 128", op, head_dim);
  if (dtype > M3_F16)
    return fail(M3_ERR_INVALID_ARGUMENT, "%s: dtype %u is not one of float32, bfloat16, float16", op, dtype);
  return M3_OK;
}

struct ViewRule {
  const char* name;
  const m3_view* view;
  uint64_t rows;
  uint32_t heads;
  bool output;
};

bool aligned16(const void* p, std::initializer_list<int64_t> strides, uint32_t size, uint32_t D) {
  if (D % 8 != 0 || (reinterpret_cast<uintptr_t>(p) & 15)) return false;
  for (int64_t s : strides)
    if (s * size % 16 != 0) return false;
  return true;
}

// Whether two of the runs of D elements that start at i a + j b, i < n, j < m, share an element (a, b at least D
// where n, m are above one).  One axis within a step of the other never does; otherwise each multiple of the
// wider stride is held against the multiples of the narrower one beside it.
bool overlap(uint64_t n, int64_t a, uint64_t m, int64_t b, uint32_t D) {
  if (n < 2 || m < 2) return false;
  if (a > b) {
    std::swap(a, b);
    std::swap(n, m);
  }
  typedef __int128 wide;
  if ((wide)(n - 1) * a + D <= b) return false;
  for (uint64_t j = 1; j < m; ++j) {
    if (j > 65536) return true;  // no layout of use comes this far
    const wide at = (wide)j * b, i = at / a, rest = at % a;
    if (i >= (wide)n) break;
    if (rest < D || (i + 1 < (wide)n && a - rest < D)) return true;
  }
  return false;
}

int check_view(const char* op, const ViewRule& r, uint32_t D, uint32_t size) {
  const m3_view& v = *r.view;
  if (r.rows == 0) return M3_OK;
  if (v.data == nullptr) return fail(M3_ERR_INVALID_ARGUMENT, "%s: operand %s is NULL", op, r.name);
  if (reinterpret_cast<uintptr_t>(v.data) % size != 0)
    return fail(M3_ERR_INVALID_ARGUMENT, "%s: operand %s is not aligned to its %u-byte elements", op, r.name, size);
  if (v.row_stride < (int64_t)D)
    return fail(M3_ERR_INVALID_ARGUMENT, "%s: operand %s has row_stride %lld below head_dim %u", op, r.name,
                (long long)v.row_stride, D);
  if (v.row_stride > kMaxRowBytes / size)
    return fail(M3_ERR_UNSUPPORTED, "%s: operand %s has row_stride %lld; rows may stand at most %lld bytes apart", op,
                r.name, (long long)v.row_stride, (long long)kMaxRowBytes);
  if (v.head_stride < 0 || (r.output && r.heads > 1 && v.head_stride < (int64_t)D))
    return fail(M3_ERR_INVALID_ARGUMENT, "%s: operand %s has head_stride %lld; heads must not overlap", op, r.name,
                (long long)v.head_stride);
  if (r.output && overlap(r.rows, v.row_stride, r.heads, v.head_stride, D))
    return fail(M3_ERR_INVALID_ARGUMENT, "%s: operand %s has row_stride %lld and head_stride %lld; its %llu rows of %u "
                "heads must not overlap", op, r.name, (long long)v.row_stride, (long long)v.head_stride,
                (unsigned long long)r.rows, r.heads);
  return M3_OK;
}

int check_views(const char* op, std::initializer_list<ViewRule> rules, uint32_t D, uint32_t size) {
  for (const auto& r : rules) {
    const int st = check_view(op, r, D, size);
    if (st) return st;
  }
  return M3_OK;
}

m3::HeadView in_view(const m3_view& v, uint32_t size, uint32_t D) {
  return {v.data, v.row_stride, v.head_stride, aligned16(v.data, {v.row_stride, v.head_stride}, size, D) ? 1u : 0u};
}
m3::HeadOut out_view(const m3_view& v, uint32_t size, uint32_t D) {
  return {v.data, v.row_stride, v.head_stride, aligned16(v.data, {v.row_stride, v.head_stride}, size, D) ? 1u : 0u};
}

int check_workspace(const char* op, const void* workspace, size_t given, size_t need) {
  if (need > 0 && (workspace == nullptr || given < need))
    return fail(M3_ERR_INVALID_ARGUMENT, "%s: workspace of %zu bytes required, %zu given", op, need,
                workspace == nullptr ? (size_t)0 : given);
  if (need > 0 && (reinterpret_cast<uintptr_t>(workspace) & 15))
    return fail(M3_ERR_INVALID_ARGUMENT, "%s: the workspace is not aligned to 16 bytes", op);
  return M3_OK;
}

int check_launch(const char* op, uint64_t workgroups) {
  if (workgroups > m3::kMaxWorkgroups)
    return fail(M3_ERR_UNSUPPORTED, "%s: %llu workgroups are more than one launch can cover (%llu)", op,
                (unsigned long long)workgroups, (unsigned long long)m3::kMaxWorkgroups);
  return M3_OK;
}

constexpr uint64_t kI31 = 0x7fffffffull;

int resolve_rope(const char* op, const m3_qk_norm_rope_config& cfg, uint32_t rows, m3::RopeGeom* g) {
  uint32_t G;
  const int st = resolve_heads(op, cfg.num_heads, cfg.num_groups, cfg.head_dim, cfg.dtype, &G);
  if (st) return st;
  if (rows == 0) return fail(M3_ERR_INVALID_ARGUMENT, "%s: rows is 0; every extent must be at least 1", op);
  if (2ull * cfg.num_rope_angles > cfg.head_dim)
    return fail(M3_ERR_INVALID_ARGUMENT, "%s: the %u rotary pairs need 2 * num_rope_angles = %llu columns, but "
                "head_dim is %u", op, cfg.num_rope_angles, 2ull * cfg.num_rope_angles, cfg.head_dim);
  if (!std::isfinite(cfg.epsilon)) return fail(M3_ERR_INVALID_ARGUMENT, "%s: epsilon is not a finite number", op);
  if (cfg.epsilon <= 0.f)
    return fail(M3_ERR_INVALID_ARGUMENT, "%s: epsilon is %g; it must be above zero", op, (double)cfg.epsilon);
  if (rows > kI31 || cfg.num_heads > 65536u)
    return fail(M3_ERR_UNSUPPORTED, "%s: more than 2^31 - 1 rows or 65536 heads", op);
  *g = m3::RopeGeom{rows, cfg.num_heads, G, cfg.head_dim, cfg.num_rope_angles, cfg.dtype, cfg.epsilon};
  return M3_OK;
}

int resolve_attn(const char* op, const m3_attn_config& cfg, m3::AttnGeom* g) {
  uint32_t G;
  const struct {
    const char* name;
    uint32_t v;
  } extents[] = {{"batch_size", cfg.batch_size}, {"q_length", cfg.q_length}, {"kv_length", cfg.kv_length}};
  for (const auto& e : extents)
    if (e.v == 0) return fail(M3_ERR_INVALID_ARGUMENT, "%s: %s is 0; every extent must be at least 1", op, e.name);
  const int st = resolve_heads(op, cfg.num_heads, cfg.num_groups, cfg.head_dim, cfg.dtype, &G);
  if (st) return st;
  if (cfg.causal > 1) return fail(M3_ERR_INVALID_ARGUMENT, "%s: flag causal is %u; a flag is 0 or 1", op, cfg.causal);
  if (cfg.window > 0 && !cfg.causal)
    return fail(M3_ERR_INVALID_ARGUMENT, "%s: window %u needs causal attention", op, cfg.window);
  if (!std::isfinite(cfg.scale) || cfg.scale < 0.f)
    return fail(M3_ERR_INVALID_ARGUMENT, "%s: scale is %g; it must be finite and not below zero", op,
                (double)cfg.scale);
  // lengths, windows and the grid run in 31-bit arithmetic
  const uint64_t half = 1ull << 30;
  if (cfg.q_length > half || cfg.kv_length > half || cfg.window > half || cfg.batch_size > half ||
      cfg.num_heads > 65536u || ((uint64_t)cfg.q_length / 32 + 1) * cfg.num_heads * cfg.batch_size > kI31 ||
      ((uint64_t)cfg.kv_length / 32 + 1) * cfg.num_heads * cfg.batch_size > kI31)
    return fail(M3_ERR_UNSUPPORTED, "%s: the lengths, heads and sequences are more than one launch can cover", op);
  *g = m3::AttnGeom{cfg.batch_size, cfg.q_length, cfg.kv_length, cfg.num_heads, G, cfg.head_dim, cfg.causal,
                    cfg.window, cfg.dtype, 0, 0, cfg.scale == 0.f ? 1.f / std::sqrt((float)cfg.head_dim) : cfg.scale};
  return M3_OK;
}

// The rows of both sides; without offsets they follow from the lengths.
int resolve_rows(const char* op, const int32_t* q_offsets, const int32_t* kv_offsets, uint32_t total_q,
                 uint32_t total_kv, m3::AttnGeom* g) {
  const struct {
    const char *name, *len;
    bool cut;
    uint32_t total, length;
  } sides[] = {{"total_q", "q_length", q_offsets != nullptr, total_q, g->Lq},
               {"total_kv", "kv_length", kv_offsets != nullptr, total_kv, g->Lk}};
  for (const auto& s : sides) {
    if (!s.cut && (uint64_t)g->B * s.length != s.total)
      return fail(M3_ERR_INVALID_ARGUMENT, "%s: %s is %u; without offsets it is batch_size * %s = %llu", op, s.name,
                  s.total, s.len, (unsigned long long)g->B * s.length);
    if (s.total > kI31) return fail(M3_ERR_UNSUPPORTED, "%s: %s is above 2^31 - 1", op, s.name);
  }
  g->total_q = total_q;
  g->total_k = total_kv;
  return M3_OK;
}

}  // namespace

extern "C" {

int m3_qk_norm_rope(m3_view q, m3_view k, const int32_t* positions, const float* inv_freq, const float* q_weight,
                    const float* k_weight, uint32_t rows, m3_qk_norm_rope_config cfg, m3_view out_q, m3_view out_k,
                    void* stream) {
  const char* op = "m3_qk_norm_rope";
  clear_error();
  m3::RopeGeom g{};
  int st = resolve_rope(op, cfg, rows, &g);
  if (st) return st;
  const uint32_t size = dtype_size(g.dtype);
  st = check_views(op, {{"q", &q, rows, g.H, false}, {"k", &k, rows, g.G, false}, {"out_q", &out_q, rows, g.H, true},
                        {"out_k", &out_k, rows, g.G, true}}, g.D, size);
  if (st) return st;
  st = check_ptrs(op, {{"positions", positions}, {"q_weight", q_weight}, {"k_weight", k_weight}});
  if (st) return st;
  if (g.A > 0 && inv_freq == nullptr) return fail(M3_ERR_INVALID_ARGUMENT, "%s: operand inv_freq is NULL", op);
  m3::RopeOperands o{};
  o.q = in_view(q, size, g.D);
  o.k = in_view(k, size, g.D);
  o.oq = out_view(out_q, size, g.D);
  o.ok = out_view(out_k, size, g.D);
  o.positions = positions;
  o.inv_freq = inv_freq;
  o.qw = q_weight;
  o.kw = k_weight;
  st = check_launch(op, m3::qk_norm_rope_workgroups(g, o));
  if (st) return st;
  return hip_status(op, m3::launch_qk_norm_rope(g, o, static_cast<hipStream_t>(stream)));
}

size_t m3_qk_norm_rope_bwd_workspace_bytes(m3_qk_norm_rope_config cfg, uint32_t rows) {
  m3::RopeGeom g{};
  if (resolve_rope("m3_qk_norm_rope_bwd_workspace_bytes", cfg, rows, &g) != M3_OK) return 0;
  return m3::qk_norm_rope_bwd_workspace_floats(g) * sizeof(float);
}

int m3_qk_norm_rope_bwd(m3_view g_q, m3_view g_k, m3_view q, m3_view k, const int32_t* positions,
                        const float* inv_freq, const float* q_weight, const float* k_weight, uint32_t rows,
                        m3_qk_norm_rope_config cfg, m3_view d_q, m3_view d_k, float* d_q_weight, float* d_k_weight,
                        void* workspace, size_t workspace_bytes, void* stream) {
  const char* op = "m3_qk_norm_rope_bwd";
  clear_error();
  m3::RopeGeom g{};
  int st = resolve_rope(op, cfg, rows, &g);
  if (st) return st;
  const uint32_t size = dtype_size(g.dtype);
  st = check_views(op, {{"g_q", &g_q, rows, g.H, false}, {"g_k", &g_k, rows, g.G, false}, {"q", &q, rows, g.H, false},
                        {"k", &k, rows, g.G, false}, {"d_q", &d_q, rows, g.H, true}, {"d_k", &d_k, rows, g.G, true}},
                   g.D, size);
  if (st) return st;
  st = check_ptrs(op, {{"positions", positions}, {"q_weight", q_weight}, {"k_weight", k_weight},
                       {"d_q_weight", d_q_weight}, {"d_k_weight", d_k_weight}});
  if (st) return st;
  if (g.A > 0 && inv_freq == nullptr) return fail(M3_ERR_INVALID_ARGUMENT, "%s: operand inv_freq is NULL", op);
  st = check_workspace(op, workspace, workspace_bytes, m3::qk_norm_rope_bwd_workspace_floats(g) * sizeof(float));
  if (st) return st;
  m3::RopeOperands o{};
  o.q = in_view(q, size, g.D);
  o.k = in_view(k, size, g.D);
  o.gq = in_view(g_q, size, g.D);
  o.gk = in_view(g_k, size, g.D);
  o.oq = out_view(d_q, size, g.D);
  o.ok = out_view(d_k, size, g.D);
  o.positions = positions;
  o.inv_freq = inv_freq;
  o.qw = q_weight;
  o.kw = k_weight;
  o.dqw = d_q_weight;
  o.dkw = d_k_weight;
  o.partial = static_cast<float*>(workspace);
  return hip_status(op, m3::launch_qk_norm_rope_bwd(g, o, static_cast<hipStream_t>(stream)));
}

size_t m3_attn_fwd_workspace_bytes(m3_attn_config cfg) {
  m3::AttnGeom g{};
  if (resolve_attn("m3_attn_fwd_workspace_bytes", cfg, &g) != M3_OK) return 0;
  return m3::attn_fwd_workspace_floats(g) * sizeof(float);
}

int m3_attn_fwd(m3_view q, m3_view k, m3_view v, const int32_t* q_offsets, const int32_t* kv_offsets, uint32_t total_q,
                uint32_t total_kv, m3_attn_config cfg, m3_view out, float* lse, void* workspace,
                size_t workspace_bytes, void* stream) {
  const char* op = "m3_attn_fwd";
  clear_error();
  m3::AttnGeom g{};
  int st = resolve_attn(op, cfg, &g);
  if (st) return st;
  st = resolve_rows(op, q_offsets, kv_offsets, total_q, total_kv, &g);
  if (st) return st;
  const uint32_t size = dtype_size(g.dtype);
  st = check_views(op, {{"q", &q, total_q, g.H, false}, {"k", &k, total_kv, g.G, false},
                        {"v", &v, total_kv, g.G, false}, {"out", &out, total_q, g.H, true}}, g.D, size);
  if (st) return st;
  if (total_q > 0 && lse == nullptr) return fail(M3_ERR_INVALID_ARGUMENT, "%s: operand lse is NULL", op);
  st = check_workspace(op, workspace, workspace_bytes, m3::attn_fwd_workspace_floats(g) * sizeof(float));
  if (st) return st;
  if (total_q == 0) return M3_OK;
  st = check_launch(op, m3::attn_fwd_workgroups(g));
  if (st) return st;
  m3::AttnOperands o{};
  o.q = in_view(q, size, g.D);
  o.k = in_view(k, size, g.D);
  o.v = in_view(v, size, g.D);
  o.out = out_view(out, size, g.D);
  o.q_offsets = q_offsets;
  o.kv_offsets = kv_offsets;
  o.lse = lse;
  o.ws = static_cast<float*>(workspace);
  return hip_status(op, m3::launch_attn_fwd(g, o, static_cast<hipStream_t>(stream)));
}

size_t m3_attn_bwd_workspace_bytes(m3_attn_config cfg, uint32_t total_q, uint32_t total_kv) {
  m3::AttnGeom g{};
  if (resolve_attn("m3_attn_bwd_workspace_bytes", cfg, &g) != M3_OK) return 0;
  g.total_q = total_q;
  g.total_k = total_kv;
  return m3::attn_bwd_workspace_floats(g) * sizeof(float);
}

int m3_attn_bwd(m3_view dout, m3_view q, m3_view k, m3_view v, m3_view out, const float* lse, const int32_t* q_offsets,
                const int32_t* kv_offsets, uint32_t total_q, uint32_t total_kv, m3_attn_config cfg, m3_view d_q,
                m3_view d_k, m3_view d_v, void* workspace, size_t workspace_bytes, void* stream) {
  const char* op = "m3_attn_bwd";
  clear_error();
  m3::AttnGeom g{};
  int st = resolve_attn(op, cfg, &g);
  if (st) return st;
  st = resolve_rows(op, q_offsets, kv_offsets, total_q, total_kv, &g);
  if (st) return st;
  const uint32_t size = dtype_size(g.dtype);
  st = check_views(op, {{"dout", &dout, total_q, g.H, false}, {"q", &q, total_q, g.H, false},
                        {"k", &k, total_kv, g.G, false}, {"v", &v, total_kv, g.G, false},
                        {"out", &out, total_q, g.H, false}, {"d_q", &d_q, total_q, g.H, true},
                        {"d_k", &d_k, total_kv, g.G, true}, {"d_v", &d_v, total_kv, g.G, true}}, g.D, size);
  if (st) return st;
  if (total_q > 0 && lse == nullptr) return fail(M3_ERR_INVALID_ARGUMENT, "%s: operand lse is NULL", op);
  st = check_workspace(op, workspace, workspace_bytes, m3::attn_bwd_workspace_floats(g) * sizeof(float));
  if (st) return st;
  st = check_launch(op, m3::attn_bwd_workgroups(g));
  if (st) return st;
  m3::AttnOperands o{};
  o.q = in_view(q, size, g.D);
  o.k = in_view(k, size, g.D);
  o.v = in_view(v, size, g.D);
  o.o = in_view(out, size, g.D);
  o.dout = in_view(dout, size, g.D);
  o.dq = out_view(d_q, size, g.D);
  o.dk = out_view(d_k, size, g.D);
  o.dv = out_view(d_v, size, g.D);
  o.q_offsets = q_offsets;
  o.kv_offsets = kv_offsets;
  o.lse = const_cast<float*>(lse);
  o.ws = static_cast<float*>(workspace);
  return hip_status(op, m3::launch_attn_bwd(g, o, static_cast<hipStream_t>(stream)));
}

}  // extern "C"

namespace {

int resolve_step(const char* op, const m3_attn_config& cfg, m3::AttnGeom* g) {
  const int st = resolve_attn(op, cfg, g);
  if (st) return st;
  if (cfg.q_length != 1)
    return fail(M3_ERR_INVALID_ARGUMENT, "%s: q_length is %u; a decode step takes exactly one token", op, cfg.q_length);
  if (cfg.causal != 1) return fail(M3_ERR_INVALID_ARGUMENT, "%s: a decode step is causal", op);
  return M3_OK;
}

int check_pages(const char* op, const int32_t* block_table, uint32_t num_pages, uint32_t page_size, uint32_t max_pages,
                uint32_t rows, uint32_t kv_length) {
  const struct {
    const char* name;
    uint32_t v;
  } extents[] = {{"num_pages", num_pages}, {"page_size", page_size}, {"max_pages", max_pages}};
  for (const auto& e : extents) {
    if (e.v == 0) return fail(M3_ERR_INVALID_ARGUMENT, "%s: %s is 0; every extent must be at least 1", op, e.name);
    if (e.v > kI31) return fail(M3_ERR_UNSUPPORTED, "%s: %s is above 2^31 - 1", op, e.name);
  }
  if ((uint64_t)max_pages * page_size < kv_length)
    return fail(M3_ERR_INVALID_ARGUMENT, "%s: kv_length %u is above max_pages * page_size = %llu", op, kv_length,
                (unsigned long long)max_pages * page_size);
  if (block_table == nullptr && (max_pages != 1 || num_pages < rows))
    return fail(M3_ERR_INVALID_ARGUMENT, "%s: without a block_table each of the %u rows has one page of its own; "
                "num_pages is %u, max_pages %u", op, rows, num_pages, max_pages);
  return M3_OK;
}

int check_cache(const char* op, const char* name, const m3_cache& c, uint32_t pages, uint32_t page_size, uint32_t G,
                uint32_t D, uint32_t size) {
  if (c.data == nullptr) return fail(M3_ERR_INVALID_ARGUMENT, "%s: operand %s is NULL", op, name);
  if (reinterpret_cast<uintptr_t>(c.data) % size != 0)
    return fail(M3_ERR_INVALID_ARGUMENT, "%s: operand %s is not aligned to its %u-byte elements", op, name, size);
  if ((page_size > 1 && c.row_stride < (int64_t)D) || (G > 1 && c.head_stride < (int64_t)D) ||
      (pages > 1 && c.page_stride < (int64_t)D))
    return fail(M3_ERR_INVALID_ARGUMENT, "%s: operand %s has a stride below head_dim %u; its rows must not overlap", op,
                name, D);
  return M3_OK;
}

int check_cache_apart(const char* op, const char* name, const m3_cache& c, uint32_t pages, uint32_t page_size,
                      uint32_t G, uint32_t D) {
  if (overlap(page_size, c.row_stride, G, c.head_stride, D) || overlap(pages, c.page_stride, G, c.head_stride, D) ||
      overlap(pages, c.page_stride, page_size, c.row_stride, D))
    return fail(M3_ERR_INVALID_ARGUMENT, "%s: operand %s has page_stride %lld, row_stride %lld and head_stride %lld; its "
                "pages, rows and heads must not overlap", op, name, (long long)c.page_stride, (long long)c.row_stride,
                (long long)c.head_stride);
  return M3_OK;
}

m3::StepCache cache_view(const m3_cache& c, uint32_t size, uint32_t D) {
  return {c.data, c.page_stride, c.row_stride, c.head_stride,
          aligned16(c.data, {c.page_stride, c.row_stride, c.head_stride}, size, D) ? 1u : 0u};
}

}  // namespace

extern "C" {

size_t m3_attn_step_workspace_bytes(m3_attn_config cfg) {
  m3::AttnGeom g{};
  if (resolve_step("m3_attn_step_workspace_bytes", cfg, &g) != M3_OK) return 0;
  return m3::attn_step_workspace_floats(g) * sizeof(float);
}

int m3_attn_step(m3_view q, m3_view k, m3_view v, m3_cache k_cache, m3_cache v_cache, const int32_t* lengths,
                 const int32_t* block_table, uint32_t num_pages, uint32_t page_size, uint32_t max_pages,
                 m3_attn_config cfg, m3_view out, void* workspace, size_t workspace_bytes, void* stream) {
  const char* op = "m3_attn_step";
  clear_error();
  m3::AttnGeom g{};
  int st = resolve_step(op, cfg, &g);
  if (st) return st;
  st = check_pages(op, block_table, num_pages, page_size, max_pages, cfg.batch_size, cfg.kv_length);
  if (st) return st;
  const uint32_t size = dtype_size(g.dtype);
  st = check_views(op, {{"q", &q, g.B, g.H, false}, {"k", &k, g.B, g.G, false}, {"v", &v, g.B, g.G, false},
                        {"out", &out, g.B, g.H, true}}, g.D, size);
  if (st) return st;
  st = check_cache(op, "k_cache", k_cache, num_pages, page_size, g.G, g.D, size);
  if (st) return st;
  st = check_cache(op, "v_cache", v_cache, num_pages, page_size, g.G, g.D, size);
  if (st) return st;
  st = check_ptrs(op, {{"lengths", lengths}});
  if (st) return st;
  st = check_workspace(op, workspace, workspace_bytes, m3::attn_step_workspace_floats(g) * sizeof(float));
  if (st) return st;
  st = check_cache_apart(op, "k_cache", k_cache, num_pages, page_size, g.G, g.D);
  if (st) return st;
  st = check_cache_apart(op, "v_cache", v_cache, num_pages, page_size, g.G, g.D);
  if (st) return st;
  st = check_launch(op, m3::attn_step_workgroups(g));
  if (st) return st;
  m3::AttnStepOperands o{in_view(q, size, g.D), in_view(k, size, g.D), in_view(v, size, g.D),
                         cache_view(k_cache, size, g.D), cache_view(v_cache, size, g.D), lengths, block_table,
                         num_pages, page_size, max_pages, out_view(out, size, g.D), static_cast<float*>(workspace)};
  return hip_status(op, m3::launch_attn_step(g, o, static_cast<hipStream_t>(stream)));
}

}  // extern "C"

// ---- 8-bit key / value cache ---------------------------------------------------
namespace {

// A half chunk of 16 rows is read through one resource of less than 2^31 bytes.
constexpr int64_t kMaxCodeStride = int64_t(1) << 26;

int resolve_kv8(const char* op, const m3_kv8_config& cfg, bool step, m3::Kv8Geom* g) {
  const struct {
    const char* name;
    uint32_t v;
  } extents[] = {{"batch_size", cfg.batch_size}, {"q_length", cfg.q_length}, {"kv_length", cfg.kv_length}};
  for (const auto& e : extents)
    if (e.v == 0) return fail(M3_ERR_INVALID_ARGUMENT, "%s: %s is 0; every extent must be at least 1", op, e.name);
  uint32_t G;
  const int st = resolve_heads(op, cfg.num_heads, cfg.num_groups, cfg.head_dim, cfg.dtype, &G);
  if (st) return st;
  if (cfg.block_size != 16 && cfg.block_size != 32 && cfg.block_size != 64 && cfg.block_size != 128)
    return fail(M3_ERR_INVALID_ARGUMENT, "%s: block_size %u is not one of 16, 32, 64, 128", op, cfg.block_size);
  if (!step && (cfg.window != 0 || cfg.sinks != 0))
    return fail(M3_ERR_INVALID_ARGUMENT, "%s: window %u and sinks %u belong to m3_attn_step_kv8; they must be 0 here", op,
                cfg.window, cfg.sinks);
  if (cfg.sinks > 0 && cfg.window == 0)
    return fail(M3_ERR_INVALID_ARGUMENT, "%s: sinks %u need a window; without one every position stays visible", op,
                cfg.sinks);
  if (!std::isfinite(cfg.scale) || cfg.scale < 0.f)
    return fail(M3_ERR_INVALID_ARGUMENT, "%s: scale is %g; it must be finite and not below zero", op,
                (double)cfg.scale);
  const uint64_t half = 1ull << 30;
  if (cfg.batch_size > half || cfg.q_length > half || cfg.kv_length > half || cfg.window > half || cfg.sinks > half ||
      cfg.num_heads > 65536u)
    return fail(M3_ERR_UNSUPPORTED, "%s: the lengths, heads and rows are more than one launch can cover", op);
  if (step && cfg.q_length > 64)
    return fail(M3_ERR_UNSUPPORTED, "%s: q_length is %u; a step takes at most 64 tokens of a row", op, cfg.q_length);
  if (step && (uint64_t)cfg.batch_size * cfg.q_length > kI31)
    return fail(M3_ERR_UNSUPPORTED, "%s: more than 2^31 - 1 tokens", op);
  *g = m3::Kv8Geom{cfg.batch_size, cfg.q_length, cfg.kv_length, cfg.num_heads, G, cfg.head_dim, cfg.block_size,
                   cfg.window, cfg.sinks, cfg.dtype, 0, 0, 0, cfg.batch_size * cfg.q_length,
                   cfg.scale == 0.f ? 1.f / std::sqrt((float)cfg.head_dim) : cfg.scale};
  return M3_OK;
}

int check_kv8_pages(const char* op, const int32_t* block_table, uint32_t num_pages, uint32_t page_size,
                    uint32_t max_pages, m3::Kv8Geom* g) {
  const int st = check_pages(op, block_table, num_pages, page_size, max_pages, g->B, g->capacity);
  if (st) return st;
  if (max_pages > 1 && page_size % g->block != 0)
    return fail(M3_ERR_INVALID_ARGUMENT, "%s: page_size %u is not a multiple of block_size %u", op, page_size, g->block);
  g->num_pages = num_pages;
  g->page_size = page_size;
  g->max_pages = max_pages;
  return M3_OK;
}

// The tokens of a write or read; without offsets they follow from the lengths.
int resolve_tokens(const char* op, const int32_t* offsets, uint32_t total, m3::Kv8Geom* g) {
  if (offsets == nullptr && (uint64_t)g->B * g->T != total)
    return fail(M3_ERR_INVALID_ARGUMENT, "%s: total is %u; without offsets it is batch_size * q_length = %llu", op, total,
                (unsigned long long)g->B * g->T);
  if (total > kI31) return fail(M3_ERR_UNSUPPORTED, "%s: total is above 2^31 - 1", op);
  g->total = total;
  return M3_OK;
}

int check_kv8_cache(const char* op, const char* name, const m3_kv8_cache& c, const m3::Kv8Geom& g) {
  const m3_cache codes{c.codes, c.page_stride, c.row_stride, c.head_stride};
  int st = check_cache(op, name, codes, g.num_pages, g.page_size, g.G, g.D, 1);
  if (st) return st;
  if (c.scales == nullptr) return fail(M3_ERR_INVALID_ARGUMENT, "%s: the scales of operand %s are NULL", op, name);
  if (g.page_size > 1 && c.row_stride > kMaxCodeStride)
    return fail(M3_ERR_UNSUPPORTED, "%s: operand %s has row_stride %lld; rows may stand at most %lld codes apart", op, name,
                (long long)c.row_stride, (long long)kMaxCodeStride);
  return check_cache_apart(op, name, codes, g.num_pages, g.page_size, g.G, g.D);
}

m3::Kv8Cache kv8_view(const m3_kv8_cache& c, const m3::Kv8Geom& g) {
  const bool vec = g.D % 8 == 0 && reinterpret_cast<uintptr_t>(c.codes) % 8 == 0 && c.page_stride % 8 == 0 &&
                   c.row_stride % 8 == 0 && c.head_stride % 8 == 0;
  // the stride of an axis of one element says nothing, and is never multiplied by more than what such an axis has
  return {static_cast<uint8_t*>(c.codes), c.scales, c.page_stride, g.page_size > 1 ? c.row_stride : (int64_t)g.D,
          c.head_stride, vec ? 1u : 0u};
}

}  // namespace

extern "C" {

int m3_kv8_write(m3_view k, m3_view v, const int32_t* offsets, uint32_t total, const int32_t* lengths,
                 m3_kv8_cache k_cache, m3_kv8_cache v_cache, const int32_t* block_table, uint32_t num_pages,
                 uint32_t page_size, uint32_t max_pages, m3_kv8_config cfg, void* stream) {
  const char* op = "m3_kv8_write";
  clear_error();
  m3::Kv8Geom g{};
  int st = resolve_kv8(op, cfg, false, &g);
  if (st) return st;
  st = check_kv8_pages(op, block_table, num_pages, page_size, max_pages, &g);
  if (st) return st;
  st = resolve_tokens(op, offsets, total, &g);
  if (st) return st;
  const uint32_t size = dtype_size(g.dtype);
  st = check_views(op, {{"k", &k, total, g.G, false}, {"v", &v, total, g.G, false}}, g.D, size);
  if (st) return st;
  st = check_ptrs(op, {{"lengths", lengths}});
  if (st) return st;
  st = check_kv8_cache(op, "k_cache", k_cache, g);
  if (st) return st;
  st = check_kv8_cache(op, "v_cache", v_cache, g);
  if (st) return st;
  st = check_launch(op, m3::kv8_write_workgroups(g));
  if (st) return st;
  if (total == 0) return M3_OK;
  m3::Kv8Operands o{};
  o.k = in_view(k, size, g.D);
  o.v = in_view(v, size, g.D);
  o.kc = kv8_view(k_cache, g);
  o.vc = kv8_view(v_cache, g);
  o.lengths = lengths;
  o.offsets = offsets;
  o.table = block_table;
  return hip_status(op, m3::launch_kv8_write(g, o, static_cast<hipStream_t>(stream)));
}

int m3_kv8_read(m3_kv8_cache k_cache, m3_kv8_cache v_cache, const int32_t* starts, const int32_t* offsets,
                uint32_t total, const int32_t* block_table, uint32_t num_pages, uint32_t page_size,
                uint32_t max_pages, m3_kv8_config cfg, m3_view k, m3_view v, void* stream) {
  const char* op = "m3_kv8_read";
  clear_error();
  m3::Kv8Geom g{};
  int st = resolve_kv8(op, cfg, false, &g);
  if (st) return st;
  st = check_kv8_pages(op, block_table, num_pages, page_size, max_pages, &g);
  if (st) return st;
  st = resolve_tokens(op, offsets, total, &g);
  if (st) return st;
  const uint32_t size = dtype_size(g.dtype);
  st = check_views(op, {{"k", &k, total, g.G, true}, {"v", &v, total, g.G, true}}, g.D, size);
  if (st) return st;
  st = check_kv8_cache(op, "k_cache", k_cache, g);
  if (st) return st;
  st = check_kv8_cache(op, "v_cache", v_cache, g);
  if (st) return st;
  st = check_launch(op, m3::kv8_read_workgroups(g));
  if (st) return st;
  if (total == 0) return M3_OK;
  m3::Kv8Operands o{};
  o.kc = kv8_view(k_cache, g);
  o.vc = kv8_view(v_cache, g);
  o.lengths = starts;
  o.offsets = offsets;
  o.table = block_table;
  o.out = out_view(k, size, g.D);
  o.out_v = out_view(v, size, g.D);
  return hip_status(op, m3::launch_kv8_read(g, o, static_cast<hipStream_t>(stream)));
}

size_t m3_attn_step_kv8_workspace_bytes(m3_kv8_config cfg) {
  m3::Kv8Geom g{};
  if (resolve_kv8("m3_attn_step_kv8_workspace_bytes", cfg, true, &g) != M3_OK) return 0;
  return m3::attn_step_kv8_workspace_floats(g) * sizeof(float);
}

int m3_attn_step_kv8(m3_view q, m3_view k, m3_view v, m3_kv8_cache k_cache, m3_kv8_cache v_cache,
                     const int32_t* lengths, const int32_t* block_table, uint32_t num_pages, uint32_t page_size,
                     uint32_t max_pages, m3_kv8_config cfg, m3_view out, void* workspace, size_t workspace_bytes,
                     void* stream) {
  const char* op = "m3_attn_step_kv8";
  clear_error();
  m3::Kv8Geom g{};
  int st = resolve_kv8(op, cfg, true, &g);
  if (st) return st;
  st = check_kv8_pages(op, block_table, num_pages, page_size, max_pages, &g);
  if (st) return st;
  const uint32_t size = dtype_size(g.dtype);
  st = check_views(op, {{"q", &q, g.total, g.H, false}, {"out", &out, g.total, g.H, true}}, g.D, size);
  if (st) return st;
  const bool writes = k.data != nullptr || v.data != nullptr;
  if (writes) {
    st = check_views(op, {{"k", &k, g.total, g.G, false}, {"v", &v, g.total, g.G, false}}, g.D, size);
    if (st) return st;
  }
  st = check_ptrs(op, {{"lengths", lengths}});
  if (st) return st;
  st = check_workspace(op, workspace, workspace_bytes, m3::attn_step_kv8_workspace_floats(g) * sizeof(float));
  if (st) return st;
  st = check_kv8_cache(op, "k_cache", k_cache, g);
  if (st) return st;
  st = check_kv8_cache(op, "v_cache", v_cache, g);
  if (st) return st;
  st = check_launch(op, m3::attn_step_kv8_workgroups(g));
  if (st) return st;
  m3::Kv8Operands o{};
  o.q = in_view(q, size, g.D);
  if (writes) {
    o.k = in_view(k, size, g.D);
    o.v = in_view(v, size, g.D);
  }
  o.kc = kv8_view(k_cache, g);
  o.vc = kv8_view(v_cache, g);
  o.lengths = lengths;
  o.table = block_table;
  o.out = out_view(out, size, g.D);
  o.ws = static_cast<float*>(workspace);
  return hip_status(op, m3::launch_attn_step_kv8(g, o, static_cast<hipStream_t>(stream)));
}

}  // extern "C"

// ---- m3_siso_fwd_noalloc: the scan's workspace in a fixed device array ------
//
// For callers that cannot allocate (code under HIP graph capture, tight
// serving loops): the segment summaries live in `scratch`, a file-scope
// device array that every GPU the library runs on holds until the process
// ends.  Host code never passes the array's name to a kernel (on the host it
// is only a stand-in for the symbol): on the first call on a device, with
// that device current, hipGetSymbolAddress gives that device's own copy,
// and every later call on the device uses the kept pointer.
namespace {

constexpr size_t kScratchBytes = size_t(64) << 20;  // 64 MiB per device
constexpr int kMaxDevices = 64;
__device__ __align__(256) unsigned char scratch[kScratchBytes];
std::once_flag g_scratch_once[kMaxDevices];
void* g_scratch_ptr[kMaxDevices];
hipError_t g_scratch_err[kMaxDevices];

}  // namespace

extern "C" {

int m3_siso_fwd_noalloc(const float* c, const float* b, const float* x, const float* z, const float* adt,
                        const float* dt, const float* trap, const float* angle, const float* c_bias,
                        const float* b_bias, const float* d, m3_ssm_config cfg, float* out, void* stream) {
  const char* op = "m3_siso_fwd_noalloc";
  clear_error();
  m3::ScanGeom g{};
  int st = resolve_scan(op, cfg, false, &g);
  if (st) return st;
  st = check_ptrs(op, {{"c", c}, {"b", b}, {"x", x}, {"z", z}, {"adt", adt}, {"dt", dt},
                       {"trap", trap}, {"c_bias", c_bias}, {"b_bias", b_bias}, {"d", d}, {"out", out}});
  if (st) return st;
  if (g.A > 0 && angle == nullptr) return fail(M3_ERR_INVALID_ARGUMENT, "%s: operand angle is NULL", op);
  const m3::ScanPlan plan = m3::plan_siso(g);
  const size_t need = m3::plan_workspace_bytes(plan);
  if (need > kScratchBytes)
    return fail(M3_ERR_UNSUPPORTED, "%s: this geometry needs %zu bytes of scan workspace; the fixed scratch holds %zu",
                op, need, kScratchBytes);
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return hip_status(op, e);
  if (dev < 0 || dev >= kMaxDevices)
    return fail(M3_ERR_UNSUPPORTED, "%s: device %d is beyond the %d devices the scratch table covers", op, dev,
                kMaxDevices);
  std::call_once(g_scratch_once[dev], [dev] {
    g_scratch_err[dev] = hipGetSymbolAddress(&g_scratch_ptr[dev], HIP_SYMBOL(scratch));
    if (g_scratch_err[dev] != hipSuccess) (void)hipGetLastError();
  });
  if (g_scratch_err[dev] != hipSuccess) return hip_status(op, g_scratch_err[dev]);
  m3::ScanOperands o{c, b, x, z, adt, dt, trap, angle, c_bias, b_bias, d,
                     nullptr, nullptr, nullptr, nullptr, out};
  void* ws = need > 0 ? g_scratch_ptr[dev] : nullptr;
  return hip_status(op, m3::launch_siso_fwd(g, o, plan, ws, static_cast<hipStream_t>(stream)));
}

}  // extern "C"


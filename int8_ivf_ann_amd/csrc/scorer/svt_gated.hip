// svt_gated.hip - the entry points of products with a gate: arguments checked, the type's kernels called (svt_gated.h).
#include "svt_gated.h"

namespace svt {

namespace {

int check_gated(const char *who, int32_t n_rows, int32_t n_in, int32_t n_out, int32_t n_matrices, int32_t dtype,
                int32_t activation, bool by_expert) {
  if (n_rows < 0) return report(SVT_EINVAL, "%s: n_rows %d < 0", who, n_rows);
  if (n_in < 1 || n_in > kGatedMax) return report(SVT_EINVAL, "%s: n_in %d out of [1, %d]", who, n_in, kGatedMax);
  if (n_out < 1 || n_out > kGatedMax) return report(SVT_EINVAL, "%s: n_out %d out of [1, %d]", who, n_out, kGatedMax);
  if (n_matrices < 1 || n_matrices > SVT_MAX_EXPERTS)
    return report(SVT_EINVAL, "%s: n_matrices %d out of [1, %d]", who, n_matrices, SVT_MAX_EXPERTS);
  if (!by_expert && n_matrices != 1)
    return report(SVT_EINVAL, "%s: %d matrices need offsets", who, n_matrices);
  if (!elem_size(dtype)) return report(SVT_EINVAL, "%s: unknown element type %d", who, dtype);
  if (activation < SVT_ACT_NONE || activation > SVT_ACT_GELU)
    return report(SVT_EINVAL, "%s: unknown activation %d", who, activation);
  return SVT_OK;
}

struct Span { const void *at; size_t bytes; };

// whether any of outs overlaps an input or another output
bool any_overlap(const Span *ins, int n_ins, const Span *outs, int n_outs) {
  for (int i = 0; i < n_outs; ++i) {
    for (int j = 0; j < n_ins; ++j)
      if (overlap(outs[i].at, outs[i].bytes, ins[j].at, ins[j].bytes)) return true;
    for (int j = 0; j < i; ++j)
      if (overlap(outs[i].at, outs[i].bytes, outs[j].at, outs[j].bytes)) return true;
  }
  return false;
}

GatedArgs gated_args(int32_t n_rows, int32_t n_in, int32_t n_out, int32_t n_matrices, int elem, const int32_t *offsets) {
  GatedArgs a{};
  a.n_rows = n_rows;
  a.ins = n_in;
  a.outs = n_out;
  a.n_matrices = n_matrices;
  a.offsets = offsets;
  a.splits = 1;
  a.pitch = gated_pitch(n_out, elem);
  a.in_pitch = (int64_t)n_in * elem;
  return a;
}

// whether rows of n_in elements begin at multiples of 4 bytes in all of them (NULL: not there)
bool aligned_rows(int32_t n_in, int elem, const void *x, const void *w_gate, const void *w_up) {
  return (size_t)n_in * elem % 4 == 0 && !misaligned(x, 4) && !misaligned(w_gate, 4) && !misaligned(w_up, 4);
}

const int32_t kSome[1] = {0};   // stands for offsets that are given, where only that counts

}  // namespace

}  // namespace svt

using namespace svt;

extern "C" size_t svt_gated_linear_workspace_size(int32_t n_rows, int32_t n_in, int32_t n_out, int32_t n_matrices,
                                                  int32_t dtype, int32_t by_expert, int32_t aligned) {
  (void)report(SVT_OK, "%s", "");
  if (check_gated("svt_gated_linear_workspace_size", n_rows, n_in, n_out, n_matrices, dtype, SVT_ACT_NONE, by_expert != 0) !=
      SVT_OK)
    return 0;
  const int b = elem_size(dtype);
  const GatedArgs a = gated_args(n_rows, n_in, n_out, n_matrices, b, by_expert ? kSome : nullptr);
  const bool as_is = aligned && aligned_rows(n_in, b, nullptr, nullptr, nullptr);
  if (n_rows == 0 || few_rows(a, !as_is)) return 0;
  const GatedPlan plan = plan_forward(a, b);
  if (!fits(eighths(plan.units * plan.columns))) {
    (void)report(SVT_EINVAL, "svt_gated_linear_workspace_size: too many rows of too many outputs for one call");
    return 0;
  }
  return as_is ? 0 : gated_copies(a, b);
}

extern "C" int svt_gated_linear(int32_t n_rows, int32_t n_in, int32_t n_out, int32_t n_matrices, int32_t dtype,
                                const void *x, const void *w_gate, const void *w_up, const int32_t *offsets,
                                int32_t activation, void *h, void *gate, void *up, void *workspace,
                                size_t workspace_bytes, void *hip_stream) {
  const char *who = "svt_gated_linear";
  (void)report(SVT_OK, "%s", "");
  const int rc = check_gated(who, n_rows, n_in, n_out, n_matrices, dtype, activation, offsets != nullptr);
  if (rc != SVT_OK || n_rows == 0) return rc;
  if (!x || !w_gate || !w_up || !h) return report(SVT_EINVAL, "%s: NULL input or output", who);
  if (!gate != !up) return report(SVT_EINVAL, "%s: gate and up are kept both or neither", who);
  const int b = elem_size(dtype);
  if (misaligned(x, b) || misaligned(w_gate, b) || misaligned(w_up, b) || misaligned(offsets, 4) || misaligned(h, b) ||
      misaligned(gate, b) || misaligned(up, b) || misaligned(workspace, 16))
    return report(SVT_EINVAL, "%s: misaligned input, output or workspace", who);
  GatedArgs a = gated_args(n_rows, n_in, n_out, n_matrices, b, offsets);
  a.act = activation;
  a.x = x;
  a.w_gate = w_gate;
  a.w_up = w_up;
  a.h = h;
  a.gate = gate;
  a.up = up;
  const bool as_is = aligned_rows(n_in, b, x, w_gate, w_up);
  a.few = few_rows(a, !as_is);
  const size_t need = as_is || a.few ? 0 : gated_copies(a, b);
  if (need > 0 && (!workspace || workspace_bytes < need))
    return report(SVT_EINVAL, "%s: workspace of %zu bytes, needs %zu", who, workspace ? workspace_bytes : (size_t)0, need);
  const size_t nx = (size_t)n_rows * n_in * b, nw = (size_t)n_matrices * n_out * n_in * b, nh = (size_t)n_rows * n_out * b;
  const Span ins[4] = {{x, nx}, {w_gate, nw}, {w_up, nw}, {offsets, ((size_t)n_matrices + 1) * 4}};
  const Span outs[4] = {{h, nh}, {gate, nh}, {up, nh}, {workspace, need}};
  if (any_overlap(ins, 4, outs, 4))
    return report(SVT_EINVAL, "%s: an output or the workspace overlaps an input or another output", who);
  const GatedPlan plan = plan_forward(a, b);
  if (!a.few && !fits(eighths(plan.units * plan.columns)))
    return report(SVT_EINVAL, "%s: too many rows of too many outputs for one call", who);
  if (need) {
    a.padded = (char *)workspace;
    a.in_pitch = gated_pitch(n_in, b);
  }
  return with_type(dtype, [&](auto ty) { return gated_forward<decltype(ty)>(who, a, plan, hip_stream); });
}

extern "C" size_t svt_gated_linear_backward_workspace_size(int32_t n_rows, int32_t n_in, int32_t n_out, int32_t n_matrices,
                                                           int32_t dtype, int32_t by_expert, int32_t aligned) {
  const char *who = "svt_gated_linear_backward_workspace_size";
  (void)report(SVT_OK, "%s", "");
  if (check_gated(who, n_rows, n_in, n_out, n_matrices, dtype, SVT_ACT_NONE, by_expert != 0) != SVT_OK) return 0;
  const int b = elem_size(dtype);
  GatedArgs a = gated_args(n_rows, n_in, n_out, n_matrices, b, by_expert ? kSome : nullptr);
  if (n_rows == 0) return 0;
  const GatedPlan plan = plan_backward(a, b);
  if (!fits(gradient_blocks(plan, n_out, true, true, by_expert != 0).all())) {
    (void)report(SVT_EINVAL, "%s: too large a product for one call", who);
    return 0;
  }
  const bool as_is = aligned && aligned_rows(n_in, b, nullptr, nullptr, nullptr);
  return (size_t)(2 * a.n_rows * a.pitch) + (as_is ? 0 : gated_copies(a, b)) +
         (size_t)(dx_parts(a, plan) + dw_parts(a, plan)) * 4;
}

extern "C" int svt_gated_linear_backward(int32_t n_rows, int32_t n_in, int32_t n_out, int32_t n_matrices, int32_t dtype,
                                         const void *dh, const void *x, const void *w_gate, const void *w_up,
                                         const void *gate, const void *up, const int32_t *offsets, int32_t activation,
                                         void *dx, void *dw_gate, void *dw_up, void *workspace, size_t workspace_bytes,
                                         void *hip_stream) {
  const char *who = "svt_gated_linear_backward";
  (void)report(SVT_OK, "%s", "");
  const int rc = check_gated(who, n_rows, n_in, n_out, n_matrices, dtype, activation, offsets != nullptr);
  if (rc != SVT_OK) return rc;
  if (!dw_gate != !dw_up) return report(SVT_EINVAL, "%s: dw_gate and dw_up are given both or neither", who);
  if (!dx && !dw_gate && n_rows > 0) return report(SVT_EINVAL, "%s: NULL outputs", who);
  if (n_rows == 0 && !dw_gate) return SVT_OK;
  if (n_rows > 0 && (!dh || !gate || !up || (dw_gate && !x) || (dx && (!w_gate || !w_up))))
    return report(SVT_EINVAL, "%s: NULL input", who);
  const int b = elem_size(dtype);
  const void *elems[9] = {dh, x, w_gate, w_up, gate, up, dx, dw_gate, dw_up};
  for (const void *p : elems)
    if (misaligned(p, b)) return report(SVT_EINVAL, "%s: misaligned input or output", who);
  if (misaligned(offsets, 4) || misaligned(workspace, 16))
    return report(SVT_EINVAL, "%s: misaligned offsets or workspace", who);
  GatedArgs a = gated_args(n_rows, n_in, n_out, n_matrices, b, offsets);
  a.act = activation;
  a.x = dw_gate ? x : nullptr;   // what is not needed is not copied either
  a.w_gate = dx ? w_gate : nullptr;
  a.w_up = dx ? w_up : nullptr;
  a.gate = const_cast<void *>(gate);
  a.up = const_cast<void *>(up);
  a.dh = dh;
  a.dx = dx;
  a.dw_gate = dw_gate;
  a.dw_up = dw_up;
  const bool as_is = aligned_rows(n_in, b, a.x, a.w_gate, a.w_up);
  const size_t both = (size_t)(2 * a.n_rows * a.pitch), copies = as_is || n_rows == 0 ? 0 : gated_copies(a, b);
  const GatedPlan plan = plan_backward(a, b);
  const int64_t dx_part = dx ? dx_parts(a, plan) : 0, dw_part = dw_gate ? dw_parts(a, plan) : 0;
  const size_t need = both + copies + (size_t)(dx_part + dw_part) * 4;
  if (need > 0 && (!workspace || workspace_bytes < need))
    return report(SVT_EINVAL, "%s: workspace of %zu bytes, needs %zu", who, workspace ? workspace_bytes : (size_t)0, need);
  const size_t nx = (size_t)n_rows * n_in * b, nw = (size_t)n_matrices * n_out * n_in * b, nh = (size_t)n_rows * n_out * b;
  const Span ins[7] = {{dh, nh}, {x, nx}, {w_gate, nw}, {w_up, nw}, {gate, nh}, {up, nh},
                       {offsets, ((size_t)n_matrices + 1) * 4}};
  const Span outs[4] = {{dx, nx}, {dw_gate, nw}, {dw_up, nw}, {workspace, need}};
  if (any_overlap(ins, 7, outs, 4))
    return report(SVT_EINVAL, "%s: an output or the workspace overlaps an input or another output", who);
  if (!fits(gradient_blocks(plan, n_out, dx != nullptr, dw_gate != nullptr, offsets != nullptr).all()))
    return report(SVT_EINVAL, "%s: too large a product for one call", who);
  a.d_both = (char *)workspace;
  if (copies) {
    a.padded = a.d_both + both;
    a.in_pitch = gated_pitch(n_in, b);
  }
  a.partial = (float *)(a.d_both + both + copies);
  a.dw_partial = dx_part;
  return with_type(dtype, [&](auto ty) { return gated_backward<decltype(ty)>(who, a, plan, hip_stream); });
}

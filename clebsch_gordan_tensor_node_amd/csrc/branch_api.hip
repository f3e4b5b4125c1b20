// C entry points of the operators for branching networks (declared in include/cgtp.h):
// argument validation and launches of group normalisation, routing and the gate's gradient.
// Nothing is allocated.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstring>

#include "../../include/cgtp.h"
#include "api_common.hpp"
#include "launch_branch.hpp"

using namespace cgtp;

namespace {

constexpr int64_t kMaxInt32 = 0x7fffffff;
constexpr int64_t kMaxGroupWidth = int64_t(1) << 24;   // the weights' gradients' launch stays below 2^32 threads
constexpr int64_t kMaxSums = int64_t(1) << 37;         // floats of a workspace: past 288 GB

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int elem_size(int type) { return type == CGTP_F32 ? 4 : type == CGTP_BF16 || type == CGTP_F16 ? 2 : 0; }

int check_workspace(const void* workspace, size_t ws_bytes, size_t floats) {
  const size_t need = floats * sizeof(float);
  if (need > 0 && (!workspace || ws_bytes < need))
    return fail(CGTP_ERR_WORKSPACE, "workspace %zu bytes < %zu required", workspace ? ws_bytes : size_t(0), need);
  if (!aligned(workspace, 256)) return fail(CGTP_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  return CGTP_OK;
}

// The sizes of a group normalisation.
int fill_sizes(GroupCall& a, int dtype, int64_t rows, int64_t width, int64_t groups, int64_t samples,
               const int32_t* offsets, int64_t longest) {
  if (!elem_size(dtype)) return fail(CGTP_ERR_INVALID_ARG, "unknown element type %d", dtype);
  if (rows < 0 || samples < 0 || longest < 0) return fail(CGTP_ERR_INVALID_ARG, "negative size");
  if (width < 1) return fail(CGTP_ERR_INVALID_ARG, "a row needs at least one element");
  if (rows > kMaxInt32 || samples > kMaxInt32) return fail(CGTP_ERR_UNSUPPORTED, "more than 2^31 - 1 rows or samples");
  if (width > kMaxGroupWidth) return fail(CGTP_ERR_UNSUPPORTED, "row wider than 2^24");
  if (groups < 1 || groups > width || width % groups)
    return fail(CGTP_ERR_INVALID_ARG, "%lld columns are not a whole number for each of %lld groups", (long long)width,
                (long long)groups);
  if (!offsets && (samples == 0 ? rows > 0 : rows % samples != 0))
    return fail(CGTP_ERR_INVALID_ARG, "%lld rows are not a whole number for each of %lld samples", (long long)rows,
                (long long)samples);
  if (!aligned(offsets, 4)) return fail(CGTP_ERR_INVALID_ARG, "misaligned pointer");
  std::memset(&a, 0, sizeof(a));
  a.rows = rows;
  a.width = width;
  a.groups = groups;
  a.samples = samples;
  a.offsets = offsets;
  a.longest = longest;
  // (tiles + samples) and samples times some rows of sums
  if (double(samples) * double(width) * 6 > double(kMaxSums))
    return fail(CGTP_ERR_UNSUPPORTED, "more than 2^37 sums of samples and columns");
  return CGTP_OK;
}

int fill_group(GroupCall& a, int dtype, const void* x, int64_t ld_x, int weight_dtype, const void* weight,
               const void* bias, int activation) {
  if (weight_dtype != CGTP_F32 && weight_dtype != dtype)
    return fail(CGTP_ERR_INVALID_ARG, "weights are fp32 or of the rows' type");
  if (activation < CGTP_ACT_NONE || activation > CGTP_ACT_GELU)
    return fail(CGTP_ERR_INVALID_ARG, "unknown activation %d", activation);
  if (a.rows > 0 && !x) return fail(CGTP_ERR_INVALID_ARG, "x is NULL");
  if (a.rows > 1 && ld_x < a.width) return fail(CGTP_ERR_INVALID_ARG, "row stride of x below the row's width");
  const size_t ws = size_t(elem_size(weight_dtype));
  if (!aligned(x, size_t(elem_size(dtype))) || !aligned(weight, ws) || !aligned(bias, ws))
    return fail(CGTP_ERR_INVALID_ARG, "misaligned pointer");
  a.x = x;
  a.ld_x = ld_x;
  a.weight = weight;
  a.bias = bias;
  a.act = Act(activation);
  a.weight_f32 = weight_dtype == CGTP_F32;
  return CGTP_OK;
}

int check_route(int dtype, int64_t rows, int n, int k, const void* logits, int64_t ld) {
  const int es = elem_size(dtype);
  if (!es) return fail(CGTP_ERR_INVALID_ARG, "unknown element type %d", dtype);
  if (rows < 0) return fail(CGTP_ERR_INVALID_ARG, "negative size");
  if (rows > kMaxInt32) return fail(CGTP_ERR_UNSUPPORTED, "more than 2^31 - 1 rows");
  if (n < 1 || k < 1 || k > n) return fail(CGTP_ERR_INVALID_ARG, "%d of %d branches: need 1 <= k <= n", k, n);
  if (n > kMaxBranches || k > kMaxChosen)
    return fail(CGTP_ERR_UNSUPPORTED, "%d of %d branches: at most %d of %d", k, n, kMaxChosen, kMaxBranches);
  if (rows > 0 && !logits) return fail(CGTP_ERR_INVALID_ARG, "logits are NULL");
  if (rows > 1 && ld < n) return fail(CGTP_ERR_INVALID_ARG, "row stride of the logits below the row's width");
  if (!aligned(logits, size_t(es))) return fail(CGTP_ERR_INVALID_ARG, "misaligned pointer");
  return CGTP_OK;
}

}  // namespace

extern "C" {

int cgtp_group_norm_workspace_size(int backward, int dtype, int64_t n_rows, int64_t width, int64_t n_groups,
                                   int64_t n_samples, const int32_t* offsets, int64_t longest, size_t* bytes) {
  if (!bytes) return fail(CGTP_ERR_INVALID_ARG, "NULL argument");
  GroupCall a;
  if (int rc = fill_sizes(a, dtype, n_rows, width, n_groups, n_samples, offsets, longest)) return rc;
  *bytes = (group_norm_floats(a, Elem(dtype), backward != 0, backward != 2) * sizeof(float) + 255) / 256 * 256;
  return ok();
}

int cgtp_group_norm_forward(int dtype, int64_t n_rows, int64_t width, int64_t n_groups, int64_t n_samples,
                            const int32_t* offsets, int64_t longest, const void* x, int64_t ld_x, int weight_dtype,
                            const void* weight, const void* bias, int activation, double eps, int zero_outside, void* y,
                            int64_t ld_y, float* stats, void* workspace, size_t ws_bytes, void* stream) {
  GroupCall a;
  if (int rc = fill_sizes(a, dtype, n_rows, width, n_groups, n_samples, offsets, longest)) return rc;
  if (int rc = fill_group(a, dtype, x, ld_x, weight_dtype, weight, bias, activation)) return rc;
  if (!(eps >= 0) || !std::isfinite(eps)) return fail(CGTP_ERR_INVALID_ARG, "eps must be finite and not negative");
  if (n_rows > 0 && !y) return fail(CGTP_ERR_INVALID_ARG, "y is NULL");
  if (n_rows > 1 && ld_y < width) return fail(CGTP_ERR_INVALID_ARG, "row stride of y below the row's width");
  if (!aligned(y, size_t(elem_size(dtype))) || !aligned(stats, 4)) return fail(CGTP_ERR_INVALID_ARG, "misaligned pointer");
  if (int rc = check_workspace(workspace, ws_bytes, group_norm_floats(a, Elem(dtype), false, false))) return rc;
  a.y = y;
  a.ld_y = ld_y;
  a.stats = stats;
  a.eps = float(eps);
  a.zero_outside = zero_outside != 0;
  a.work = static_cast<float*>(workspace);
  CGTP_HIP(launch_group_norm_forward(a, Elem(dtype), static_cast<hipStream_t>(stream)));
  return ok();
}

int cgtp_group_norm_backward(int dtype, int64_t n_rows, int64_t width, int64_t n_groups, int64_t n_samples,
                             const int32_t* offsets, int64_t longest, const void* grad_out, int64_t ld_g,
                             const void* x, int64_t ld_x, const float* stats, int weight_dtype, const void* weight,
                             const void* bias, int activation, void* grad_x, int64_t ld_gx, void* grad_weight,
                             void* grad_bias, void* workspace, size_t ws_bytes, void* stream) {
  GroupCall a;
  if (int rc = fill_sizes(a, dtype, n_rows, width, n_groups, n_samples, offsets, longest)) return rc;
  if (int rc = fill_group(a, dtype, x, ld_x, weight_dtype, weight, bias, activation)) return rc;
  if (n_rows > 0 && (!grad_out || (n_samples > 0 && !stats))) return fail(CGTP_ERR_INVALID_ARG, "NULL argument");
  if (n_rows > 1 && (ld_g < width || (grad_x && ld_gx < width)))
    return fail(CGTP_ERR_INVALID_ARG, "row stride below the row's width");
  const size_t es = size_t(elem_size(dtype)), ws = size_t(elem_size(weight_dtype));
  if (!aligned(grad_out, es) || !aligned(grad_x, es) || !aligned(stats, 4) || !aligned(grad_weight, ws) ||
      !aligned(grad_bias, ws))
    return fail(CGTP_ERR_INVALID_ARG, "misaligned pointer");
  if (!grad_x && !grad_weight && !grad_bias) return ok();
  const bool sums = grad_weight || grad_bias;
  if (int rc = check_workspace(workspace, ws_bytes, group_norm_floats(a, Elem(dtype), true, sums))) return rc;
  a.grad_out = grad_out;
  a.ld_g = ld_g;
  a.stats = const_cast<float*>(stats);
  a.y = grad_x;
  a.ld_y = ld_gx;
  a.grad_weight = grad_weight;
  a.grad_bias = grad_bias;
  a.work = static_cast<float*>(workspace);
  CGTP_HIP(launch_group_norm_backward(a, Elem(dtype), static_cast<hipStream_t>(stream)));
  return ok();
}

int cgtp_route_workspace_size(int64_t n_rows, int n, size_t* bytes) {
  if (!bytes) return fail(CGTP_ERR_INVALID_ARG, "NULL argument");
  if (int rc = check_route(CGTP_F32, n_rows, n, 1, bytes, n)) return rc;
  *bytes = (route_floats(n_rows, n) * sizeof(float) + 255) / 256 * 256;
  return ok();
}

int cgtp_route_forward(int dtype, int64_t n_rows, int n, int k, const void* logits, int64_t ld, const uint8_t* mask,
                       int renormalise, int dense, int32_t* ids, float* gates, int32_t* counts, float* balance,
                       float* slope, void* workspace, size_t ws_bytes, void* stream) {
  if (int rc = check_route(dtype, n_rows, n, k, logits, ld)) return rc;
  if ((n_rows > 0 && (!ids || !gates)) || !counts || !balance || !slope) return fail(CGTP_ERR_INVALID_ARG, "NULL argument");
  if (!aligned(ids, 4) || !aligned(gates, 4) || !aligned(counts, 4) || !aligned(balance, 4) || !aligned(slope, 4))
    return fail(CGTP_ERR_INVALID_ARG, "misaligned pointer");
  if (int rc = check_workspace(workspace, ws_bytes, route_floats(n_rows, n))) return rc;
  RouteCall a;
  std::memset(&a, 0, sizeof(a));
  a.logits = logits;
  a.rows = n_rows;
  a.ld = ld;
  a.n = n;
  a.k = k;
  a.renormalise = renormalise != 0;
  a.dense = dense != 0;
  a.mask = mask;
  a.ids = ids;
  a.gates = gates;
  a.counts = counts;
  a.balance = balance;
  a.slope = slope;
  a.work = static_cast<float*>(workspace);
  CGTP_HIP(launch_route_forward(a, Elem(dtype), static_cast<hipStream_t>(stream)));
  return ok();
}

int cgtp_route_backward(int dtype, int64_t n_rows, int n, int k, const void* logits, int64_t ld, int renormalise,
                        int dense, const int32_t* ids, const float* slope, const float* grad_gates,
                        const float* grad_balance, void* grad_logits, int64_t ld_g, void* stream) {
  if (int rc = check_route(dtype, n_rows, n, k, logits, ld)) return rc;
  if (n_rows > 0 && (!ids || !grad_logits)) return fail(CGTP_ERR_INVALID_ARG, "NULL argument");
  if (grad_balance && !slope) return fail(CGTP_ERR_INVALID_ARG, "slope is NULL");
  if (n_rows > 1 && ld_g < n) return fail(CGTP_ERR_INVALID_ARG, "row stride of the gradient below the row's width");
  if (!aligned(ids, 4) || !aligned(slope, 4) || !aligned(grad_gates, 4) || !aligned(grad_balance, 4) ||
      !aligned(grad_logits, size_t(elem_size(dtype))))
    return fail(CGTP_ERR_INVALID_ARG, "misaligned pointer");
  if (n_rows == 0) return ok();
  RouteCall a;
  std::memset(&a, 0, sizeof(a));
  a.logits = logits;
  a.rows = n_rows;
  a.ld = ld;
  a.n = n;
  a.k = k;
  a.renormalise = renormalise != 0;
  a.dense = dense != 0;
  a.ids = const_cast<int32_t*>(ids);
  a.slope = const_cast<float*>(slope);
  a.grad_gates = grad_gates;
  a.grad_balance = grad_balance;
  a.grad_logits = grad_logits;
  a.ld_g = ld_g;
  CGTP_HIP(launch_route_backward(a, Elem(dtype), static_cast<hipStream_t>(stream)));
  return ok();
}

int cgtp_conv_gate_backward(int64_t n_edges, int64_t w_per_edge, const float* w, const float* grad_w,
                            const uint8_t* mask, const float* gate, float* grad_gate, void* stream) {
  if (n_edges < 0 || w_per_edge < 0) return fail(CGTP_ERR_INVALID_ARG, "negative size");
  if (n_edges > kMaxInt32 || w_per_edge > kMaxInt32) return fail(CGTP_ERR_UNSUPPORTED, "more than 2^31 - 1 edges or weights");
  if (n_edges > 0 && (!gate || !grad_gate || (w_per_edge > 0 && (!w || !grad_w))))
    return fail(CGTP_ERR_INVALID_ARG, "NULL argument");
  if (!aligned(w, 4) || !aligned(grad_w, 4) || !aligned(gate, 4) || !aligned(grad_gate, 4))
    return fail(CGTP_ERR_INVALID_ARG, "misaligned pointer");
  if (n_edges == 0) return ok();
  CGTP_HIP(launch_gate_backward(GateCall{w, grad_w, gate, mask, grad_gate, n_edges, w_per_edge},
                                static_cast<hipStream_t>(stream)));
  return ok();
}

}  // extern "C"

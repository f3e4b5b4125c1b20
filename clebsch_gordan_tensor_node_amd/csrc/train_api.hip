// C entry points of the training operators (declared in include/cgtp.h): argument
// validation and launches of the normalisations, the AdamW step and the gradient norm.
// No allocation happens outside the two create calls.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <new>
#include <string>
#include <vector>

#include "../../include/cgtp.h"
#include "api_common.hpp"
#include "launch_train.hpp"

using namespace cgtp;

struct cgtp_norm_s {
  int64_t features = 0, weights = 0, biases = 0;
  std::vector<NormTerm> terms;
};

struct cgtp_params_s {
  std::vector<int64_t> numel, offset;
  std::vector<int> first_chunk;      // [tensors + 1]
  int64_t state_elems = 0;
  Chunk* d_chunks = nullptr;
  int device = -1;
  bool host_only = true;
};

namespace {

constexpr int64_t kMaxInt32 = 0x7fffffff;
constexpr int64_t kMostElems = int64_t(1) << 37;   // of a tensor and of the set before it: past 288 GB

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int elem_size(int type) { return type == CGTP_F32 ? 4 : type == CGTP_BF16 || type == CGTP_F16 ? 2 : 0; }

// Runs a create call's body; no C++ exception leaves the library.
template <typename F>
int guarded(F&& body) {
  try {
    return body();
  } catch (const std::bad_alloc&) {
    return fail(CGTP_ERR_NO_MEMORY, "out of host memory");
  } catch (...) {
    return fail(CGTP_ERR_NO_MEMORY, "unexpected C++ exception");
  }
}

// ---- normalisation -----------------------------------------------------------------

int fill_norm(NormCall& a, const NormShape& p, int dtype, int64_t rows, const void* x, int64_t ld_x, int weight_dtype,
              const void* weight) {
  const int es = elem_size(dtype);
  if (!es) return fail(CGTP_ERR_INVALID_ARG, "unknown element type %d", dtype);
  if (weight_dtype != CGTP_F32 && weight_dtype != dtype)
    return fail(CGTP_ERR_INVALID_ARG, "weights are fp32 or of the rows' type");
  if (rows < 0) return fail(CGTP_ERR_INVALID_ARG, "negative size");
  if (rows > kMaxInt32) return fail(CGTP_ERR_UNSUPPORTED, "more than 2^31 - 1 rows");
  if (rows > 0 && !x) return fail(CGTP_ERR_INVALID_ARG, "x is NULL");
  if (rows > 1 && ld_x < p.features) return fail(CGTP_ERR_INVALID_ARG, "row stride of x below the row's width");
  if (!aligned(x, size_t(es)) || !aligned(weight, size_t(elem_size(weight_dtype))))
    return fail(CGTP_ERR_INVALID_ARG, "misaligned pointer");
  std::memset(&a, 0, sizeof(a));
  a.x = x;
  a.ld_x = ld_x;
  a.weight = weight;
  a.rows = rows;
  a.weight_f32 = weight_dtype == CGTP_F32;
  return CGTP_OK;
}

int check_width(int64_t width) {
  if (width < 1) return fail(CGTP_ERR_INVALID_ARG, "a row needs at least one element");
  if (width > kMaxInt32 / 2) return fail(CGTP_ERR_UNSUPPORTED, "row wider than 2^30 - 1");
  return CGTP_OK;
}

NormTerm whole_row(int64_t width) { return NormTerm{0, int32_t(width), 1, 0, 0}; }

int norm_forward(const NormShape& p, int dtype, int64_t rows, const void* x, int64_t ld_x, int weight_dtype,
                 const void* weight, const void* bias, double eps, void* y, int64_t ld_y, float* stats, void* stream) {
  NormCall a;
  if (int rc = fill_norm(a, p, dtype, rows, x, ld_x, weight_dtype, weight)) return rc;
  if (!(eps >= 0) || !std::isfinite(eps)) return fail(CGTP_ERR_INVALID_ARG, "eps must be finite and not negative");
  if (rows > 0 && !y) return fail(CGTP_ERR_INVALID_ARG, "y is NULL");
  if (rows > 1 && ld_y < p.features) return fail(CGTP_ERR_INVALID_ARG, "row stride of y below the row's width");
  if (!aligned(y, size_t(elem_size(dtype))) || !aligned(bias, size_t(elem_size(weight_dtype))) || !aligned(stats, 4))
    return fail(CGTP_ERR_INVALID_ARG, "misaligned pointer");
  if (rows == 0) return ok();
  a.bias = bias;
  a.y = y;
  a.ld_y = ld_y;
  a.stats = stats;
  a.eps = float(eps);
  CGTP_HIP(launch_norm_forward(a, p, Elem(dtype), static_cast<hipStream_t>(stream)));
  return ok();
}

int norm_backward_workspace(const NormShape& p, int64_t rows, size_t* bytes) {
  if (!bytes) return fail(CGTP_ERR_INVALID_ARG, "NULL argument");
  if (rows < 0) return fail(CGTP_ERR_INVALID_ARG, "negative size");
  rows = std::min(rows, kMaxInt32);   // more are refused by the call itself
  *bytes = (norm_part_floats(rows, p) * sizeof(float) + 255) / 256 * 256;
  return ok();
}

int norm_backward(const NormShape& p, int dtype, int64_t rows, const void* grad_out, int64_t ld_g, const void* x,
                  int64_t ld_x, const float* stats, int weight_dtype, const void* weight, void* grad_x, int64_t ld_gx,
                  void* grad_weight, void* grad_bias, void* workspace, size_t ws_bytes, void* stream) {
  NormCall a;
  if (int rc = fill_norm(a, p, dtype, rows, x, ld_x, weight_dtype, weight)) return rc;
  const size_t es = size_t(elem_size(dtype)), ws = size_t(elem_size(weight_dtype));
  if (rows > 0 && (!grad_out || !stats)) return fail(CGTP_ERR_INVALID_ARG, "NULL argument");
  if (rows > 1 && (ld_g < p.features || (grad_x && ld_gx < p.features)))
    return fail(CGTP_ERR_INVALID_ARG, "row stride below the row's width");
  if (!aligned(grad_out, es) || !aligned(grad_x, es) || !aligned(stats, 4) || !aligned(grad_weight, ws) ||
      !aligned(grad_bias, ws))
    return fail(CGTP_ERR_INVALID_ARG, "misaligned pointer");
  if (grad_weight || grad_bias) {
    const size_t need = norm_part_floats(rows, p) * sizeof(float);
    if (need > 0 && (!workspace || ws_bytes < need))
      return fail(CGTP_ERR_WORKSPACE, "workspace %zu bytes < %zu required", workspace ? ws_bytes : size_t(0), need);
    if (!aligned(workspace, 256)) return fail(CGTP_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  }
  a.grad_out = grad_out;
  a.ld_g = ld_g;
  a.stats = const_cast<float*>(stats);
  a.y = grad_x;
  a.ld_y = ld_gx;
  a.grad_weight = grad_weight;
  a.grad_bias = grad_bias;
  a.part = static_cast<float*>(workspace);
  CGTP_HIP(launch_norm_backward(a, p, Elem(dtype), static_cast<hipStream_t>(stream)));
  return ok();
}

NormShape shape_of(cgtp_norm_t P) {
  return NormShape{P->features, P->weights, P->biases, P->terms.data(), int(P->terms.size())};
}

}  // namespace

extern "C" {

int cgtp_layer_norm_forward(int dtype, int64_t n_rows, int64_t width, const void* x, int64_t ld_x, int weight_dtype,
                            const void* weight, const void* bias, double eps, void* y, int64_t ld_y, float* stats,
                            void* stream) {
  if (int rc = check_width(width)) return rc;
  const NormTerm t = whole_row(width);
  return norm_forward(NormShape{width, width, width, &t, 1}, dtype, n_rows, x, ld_x, weight_dtype, weight, bias, eps, y,
                      ld_y, stats, stream);
}

int cgtp_layer_norm_backward_workspace_size(int64_t n_rows, int64_t width, size_t* bytes) {
  if (int rc = check_width(width)) return rc;
  const NormTerm t = whole_row(width);
  return norm_backward_workspace(NormShape{width, width, width, &t, 1}, n_rows, bytes);
}

int cgtp_layer_norm_backward(int dtype, int64_t n_rows, int64_t width, const void* grad_out, int64_t ld_g,
                             const void* x, int64_t ld_x, const float* stats, int weight_dtype, const void* weight,
                             void* grad_x, int64_t ld_gx, void* grad_weight, void* grad_bias, void* workspace,
                             size_t ws_bytes, void* stream) {
  if (int rc = check_width(width)) return rc;
  const NormTerm t = whole_row(width);
  return norm_backward(NormShape{width, width, width, &t, 1}, dtype, n_rows, grad_out, ld_g, x, ld_x, stats,
                       weight_dtype, weight, grad_x, ld_gx, grad_weight, grad_bias, workspace, ws_bytes, stream);
}

int cgtp_norm_create(const char* irreps, cgtp_norm_t* out) {
  if (!out) return fail(CGTP_ERR_INVALID_ARG, "out is NULL");
  *out = nullptr;
  return guarded([&]() -> int {
    std::vector<Irrep> ir;
    std::string err;
    if (!parse_irreps(irreps, ir, err)) return fail(CGTP_ERR_PARSE, "%s", err.c_str());
    if (ir.size() > size_t(kMaxNormTerms))
      return fail(CGTP_ERR_UNSUPPORTED, "%zu terms: at most %d", ir.size(), kMaxNormTerms);
    cgtp_norm_s P;
    for (const Irrep& r : ir) {
      if (r.l > 6 || r.mul <= 0)
        return fail(CGTP_ERR_UNSUPPORTED, "irrep %dx%d: need l <= 6 and mul > 0", r.mul, r.l);
      const bool centred = r.l == 0 && r.p == 1;
      const int64_t d = 2 * r.l + 1, len = r.mul * d;
      // up to here the kernels' e / d = (e * inv_d) >> 32 is exact for every d <= 13
      if (P.features + len > int64_t(1) << 29) return fail(CGTP_ERR_UNSUPPORTED, "irreps row wider than 2^29");
      P.terms.push_back(NormTerm{int32_t(P.features), int32_t(len), int32_t(d), int32_t(P.weights),
                                 centred ? int32_t(P.biases) : -1});
      P.features += len;
      P.weights += r.mul;
      if (centred) P.biases += r.mul;
    }
    *out = new cgtp_norm_s(std::move(P));
    return ok();
  });
}

int cgtp_norm_info(cgtp_norm_t P, int64_t* n_features, int64_t* n_weights, int64_t* n_biases, int* n_terms) {
  if (!P) return fail(CGTP_ERR_INVALID_ARG, "plan is NULL");
  if (n_features) *n_features = P->features;
  if (n_weights) *n_weights = P->weights;
  if (n_biases) *n_biases = P->biases;
  if (n_terms) *n_terms = int(P->terms.size());
  return ok();
}

void cgtp_norm_destroy(cgtp_norm_t P) { delete P; }

int cgtp_irreps_norm_forward(cgtp_norm_t P, int dtype, int64_t n_rows, const void* x, int64_t ld_x, int weight_dtype,
                             const void* weight, const void* bias, double eps, void* y, int64_t ld_y, float* stats,
                             void* stream) {
  if (!P) return fail(CGTP_ERR_INVALID_ARG, "plan is NULL");
  return norm_forward(shape_of(P), dtype, n_rows, x, ld_x, weight_dtype, weight, bias, eps, y, ld_y, stats, stream);
}

int cgtp_irreps_norm_backward_workspace_size(cgtp_norm_t P, int64_t n_rows, size_t* bytes) {
  if (!P) return fail(CGTP_ERR_INVALID_ARG, "plan is NULL");
  return norm_backward_workspace(shape_of(P), n_rows, bytes);
}

int cgtp_irreps_norm_backward(cgtp_norm_t P, int dtype, int64_t n_rows, const void* grad_out, int64_t ld_g,
                              const void* x, int64_t ld_x, const float* stats, int weight_dtype, const void* weight,
                              void* grad_x, int64_t ld_gx, void* grad_weight, void* grad_bias, void* workspace,
                              size_t ws_bytes, void* stream) {
  if (!P) return fail(CGTP_ERR_INVALID_ARG, "plan is NULL");
  return norm_backward(shape_of(P), dtype, n_rows, grad_out, ld_g, x, ld_x, stats, weight_dtype, weight, grad_x, ld_gx,
                       grad_weight, grad_bias, workspace, ws_bytes, stream);
}

// ---- optimiser ---------------------------------------------------------------------

int cgtp_params_create(const int64_t* numel, const double* weight_decay, int n_tensors, unsigned flags,
                       cgtp_params_t* out) {
  if (!out) return fail(CGTP_ERR_INVALID_ARG, "out is NULL");
  *out = nullptr;
  if (n_tensors < 0 || (n_tensors > 0 && !numel)) return fail(CGTP_ERR_INVALID_ARG, "bad tensor list");
  if (flags & ~unsigned(CGTP_PLAN_HOST_ONLY)) return fail(CGTP_ERR_INVALID_ARG, "unknown flags 0x%x", flags);
  return guarded([&]() -> int {
    cgtp_params_s P;
    std::vector<Chunk> chunks;
    P.first_chunk.push_back(0);
    for (int t = 0; t < n_tensors; ++t) {
      const double wd = weight_decay ? weight_decay[t] : 0.0;
      if (numel[t] < 0) return fail(CGTP_ERR_INVALID_ARG, "tensor %d has a negative size", t);
      if (!(wd >= 0) || !std::isfinite(wd))
        return fail(CGTP_ERR_INVALID_ARG, "weight decay of tensor %d must be finite and not negative", t);
      if (numel[t] > kMostElems || P.state_elems > kMostElems)
        return fail(CGTP_ERR_UNSUPPORTED, "more than 2^37 elements");
      P.numel.push_back(numel[t]);
      P.offset.push_back(P.state_elems);
      for (int64_t at = 0; at < numel[t]; at += kChunk)
        chunks.push_back(Chunk{t, int32_t(std::min<int64_t>(kChunk, numel[t] - at)), at, P.state_elems + at, wd});
      P.first_chunk.push_back(int(chunks.size()));
      P.state_elems += (numel[t] + kStateBlock - 1) / kStateBlock * kStateBlock;
    }
    P.host_only = (flags & CGTP_PLAN_HOST_ONLY) != 0;
    auto handle = new cgtp_params_s(std::move(P));
    if (!handle->host_only) {
      int rc = CGTP_OK, ndev = 0;
      hipDeviceProp_t prop;
      hipError_t e = hipSuccess;
      if (hipGetDeviceCount(&ndev) != hipSuccess || ndev <= 0)
        rc = fail(CGTP_ERR_NO_DEVICE, "no HIP device");
      else if (hipGetDevice(&handle->device) != hipSuccess ||
               hipGetDeviceProperties(&prop, handle->device) != hipSuccess ||
               std::strncmp(prop.gcnArchName, "gfx950", 6) != 0)
        rc = fail(CGTP_ERR_NO_DEVICE, "current device is not gfx950");
      else if (!chunks.empty()) {
        e = hipMalloc(reinterpret_cast<void**>(&handle->d_chunks), chunks.size() * sizeof(Chunk));
        if (e == hipSuccess)
          e = hipMemcpy(handle->d_chunks, chunks.data(), chunks.size() * sizeof(Chunk), hipMemcpyHostToDevice);
        if (e != hipSuccess) rc = fail(CGTP_ERR_HIP, "tensor list's device set-up: %s", hipGetErrorString(e));
      }
      if (rc != CGTP_OK) {
        if (handle->d_chunks) (void)hipFree(handle->d_chunks);
        delete handle;
        return rc;
      }
    }
    *out = handle;
    return ok();
  });
}

void cgtp_params_destroy(cgtp_params_t P) {
  if (!P) return;
  if (P->d_chunks) {
    int cur = -1;
    (void)hipGetDevice(&cur);
    if (cur != P->device) (void)hipSetDevice(P->device);
    (void)hipFree(P->d_chunks);
    if (cur != P->device && cur >= 0) (void)hipSetDevice(cur);
  }
  delete P;
}

int cgtp_params_info(cgtp_params_t P, int* n_tensors, int64_t* state_elems, int64_t* offsets) {
  if (!P) return fail(CGTP_ERR_INVALID_ARG, "set is NULL");
  if (n_tensors) *n_tensors = int(P->numel.size());
  if (state_elems) *state_elems = P->state_elems;
  if (offsets)
    for (size_t t = 0; t < P->offset.size(); ++t) offsets[t] = P->offset[t];
  return ok();
}

}  // extern "C"

namespace {

int check_set(cgtp_params_t P) {
  if (!P) return fail(CGTP_ERR_INVALID_ARG, "set is NULL");
  if (P->host_only) return fail(CGTP_ERR_INVALID_ARG, "set was created with CGTP_PLAN_HOST_ONLY");
  int dev = -1;
  CGTP_HIP(hipGetDevice(&dev));
  if (dev != P->device)
    return fail(CGTP_ERR_INVALID_ARG, "set was created on device %d, current device is %d", P->device, dev);
  return CGTP_OK;
}

int check_tensors(cgtp_params_t P, int dtype, const void* const* t, const char* what) {
  const int es = elem_size(dtype);
  if (!es) return fail(CGTP_ERR_INVALID_ARG, "unknown element type %d of the %s", dtype, what);
  if (!t && !P->numel.empty()) return fail(CGTP_ERR_INVALID_ARG, "%s is NULL", what);
  for (size_t k = 0; k < P->numel.size(); ++k) {
    if (P->numel[k] && !t[k]) return fail(CGTP_ERR_INVALID_ARG, "%s of tensor %zu is NULL", what, k);
    if (!aligned(t[k], size_t(es))) return fail(CGTP_ERR_INVALID_ARG, "%s of tensor %zu is misaligned", what, k);
  }
  return CGTP_OK;
}

// Calls launch(first tensor, tensors, first chunk, chunks) for ranges of tensors whose
// pointers fit one launch's kernel arguments.
template <typename F>
int for_launches(cgtp_params_t P, F&& launch) {
  const int n = int(P->numel.size());
  for (int t = 0; t < n; t += kTensorsPerLaunch) {
    const int to = std::min(n, t + kTensorsPerLaunch), c0 = P->first_chunk[t], c1 = P->first_chunk[to];
    if (c1 > c0) CGTP_HIP(launch(t, to - t, c0, c1 - c0));
  }
  return ok();
}

// Whether one workgroup takes the whole gradient norm.
bool small_norm(cgtp_params_t P) {
  return P->first_chunk.back() <= kSmallChunks && P->numel.size() <= size_t(kTensorsPerLaunch);
}
// Partial sums of the gradient norm's first pass.
int norm_parts(cgtp_params_t P) {
  if (small_norm(P)) return 0;
  int parts = 0;
  for (size_t t = 0; t < P->numel.size(); t += kTensorsPerLaunch)
    parts += square_blocks(P->first_chunk[std::min(P->numel.size(), t + kTensorsPerLaunch)] - P->first_chunk[t]);
  return parts;
}

int check_betas(double beta1, double beta2) {
  if (!(beta1 >= 0 && beta1 < 1) || !(beta2 >= 0 && beta2 < 1))
    return fail(CGTP_ERR_INVALID_ARG, "betas must be in [0, 1)");
  return CGTP_OK;
}
int check_lr(double lr) {
  if (!(lr >= 0) || !std::isfinite(lr)) return fail(CGTP_ERR_INVALID_ARG, "lr must be finite and not negative");
  return CGTP_OK;
}

// step: counted on the host; scalars (not null): those that cgtp_adamw_scalars wrote, and lr,
// step and the seed are not read.
int adamw_step(cgtp_params_t P, int param_dtype, void* const* params, int grad_dtype, const void* const* grads,
               AdamwArgs& a, bool bits8, double lr, double beta1, double beta2, double eps, int64_t step, uint32_t seed,
               const void* scalars, const float* grad_scale, void* stream) {
  if (int rc = check_tensors(P, param_dtype, params, "params")) return rc;
  if (int rc = check_tensors(P, grad_dtype, grads, "grads")) return rc;
  if (int rc = check_betas(beta1, beta2)) return rc;
  if (!(eps >= 0) || !std::isfinite(eps)) return fail(CGTP_ERR_INVALID_ARG, "eps must be finite and not negative");
  if (!aligned(grad_scale, 4)) return fail(CGTP_ERR_INVALID_ARG, "misaligned grad_scale");
  if (scalars) {
    if (!aligned(scalars, 8)) return fail(CGTP_ERR_INVALID_ARG, "scalars must be 8-byte aligned");
    a.device = static_cast<const AdamwScalars*>(scalars);
  } else {
    if (int rc = check_lr(lr)) return rc;
    if (step < 1) return fail(CGTP_ERR_INVALID_ARG, "step counts from 1");
    a.here.lr = lr;
    a.here.step_size = float(lr / (1 - std::pow(beta1, double(step))));
    a.here.inv_root = float(1 / std::sqrt(1 - std::pow(beta2, double(step))));
    a.here.seed = seed * kSeedFactor;
  }
  a.grad_scale = grad_scale;
  a.b1 = float(beta1);
  a.c1 = float(1 - beta1);
  a.b2 = float(beta2);
  a.c2 = float(1 - beta2);
  a.eps = float(eps);
  const int64_t each = 2 * elem_size(param_dtype) + elem_size(grad_dtype) + (bits8 ? 4 : 16);
  const bool stream_by = P->state_elems * each > kCacheBytes;
  return for_launches(P, [&](int t, int n, int c0, int chunks) {
    a.first_tensor = t;
    std::memcpy(a.param, params + t, size_t(n) * sizeof(void*));
    std::memcpy(a.grad, grads + t, size_t(n) * sizeof(void*));
    for (int from = 0; from < chunks; from += kChunksPerLaunch) {
      a.chunks = P->d_chunks + c0 + from;
      const hipError_t e = launch_adamw(a, std::min(chunks - from, kChunksPerLaunch), Elem(param_dtype),
                                        Elem(grad_dtype), bits8, stream_by, static_cast<hipStream_t>(stream));
      if (e != hipSuccess) return e;
    }
    return hipSuccess;
  });
}

}  // namespace

extern "C" {

int cgtp_adamw_step(cgtp_params_t P, int param_dtype, void* const* params, int grad_dtype, const void* const* grads,
                    float* m, float* v, double lr, double beta1, double beta2, double eps, int64_t step,
                    const void* scalars, const float* grad_scale, void* stream) {
  if (int rc = check_set(P)) return rc;
  if (P->state_elems > 0 && (!m || !v)) return fail(CGTP_ERR_INVALID_ARG, "NULL state");
  if (!aligned(m, 16) || !aligned(v, 16)) return fail(CGTP_ERR_INVALID_ARG, "states must be 16-byte aligned");
  AdamwArgs a{};
  a.m = m;
  a.v = v;
  return adamw_step(P, param_dtype, params, grad_dtype, grads, a, false, lr, beta1, beta2, eps, step, 0, scalars,
                    grad_scale, stream);
}

int cgtp_adamw_step_8bit(cgtp_params_t P, int param_dtype, void* const* params, int grad_dtype,
                         const void* const* grads, uint8_t* m_code, uint8_t* r_code, uint8_t* m_exp, uint8_t* r_exp,
                         double lr, double beta1, double beta2, double eps, int64_t step, uint32_t seed,
                         const void* scalars, const float* grad_scale, void* stream) {
  if (int rc = check_set(P)) return rc;
  if (P->state_elems > 0 && (!m_code || !r_code || !m_exp || !r_exp)) return fail(CGTP_ERR_INVALID_ARG, "NULL state");
  if (!aligned(m_code, 16) || !aligned(r_code, 16)) return fail(CGTP_ERR_INVALID_ARG, "codes must be 16-byte aligned");
  AdamwArgs a{};
  a.m_code = m_code;
  a.r_code = r_code;
  a.m_exp = m_exp;
  a.r_exp = r_exp;
  return adamw_step(P, param_dtype, params, grad_dtype, grads, a, true, lr, beta1, beta2, eps, step, seed, scalars,
                    grad_scale, stream);
}

int cgtp_adamw_scalars(int64_t* step, const float* lr_device, double lr, double beta1, double beta2, uint32_t seed,
                       const float* grad_scale, void* scalars, void* stream) {
  static_assert(sizeof(AdamwScalars) == CGTP_ADAMW_SCALARS_BYTES, "size in cgtp.h");
  if (!step || !scalars) return fail(CGTP_ERR_INVALID_ARG, "NULL argument");
  if (!aligned(step, 8) || !aligned(scalars, 8) || !aligned(lr_device, 4) || !aligned(grad_scale, 4))
    return fail(CGTP_ERR_INVALID_ARG, "misaligned pointer");
  if (!lr_device)
    if (int rc = check_lr(lr)) return rc;
  if (int rc = check_betas(beta1, beta2)) return rc;
  CGTP_HIP(launch_adamw_scalars(step, lr_device, lr, beta1, beta2, seed, grad_scale,
                                static_cast<AdamwScalars*>(scalars), static_cast<hipStream_t>(stream)));
  return ok();
}

int cgtp_adamw_read_8bit(cgtp_params_t P, const uint8_t* m_code, const uint8_t* r_code, const uint8_t* m_exp,
                         const uint8_t* r_exp, void* m, void* r, void* stream) {
  if (int rc = check_set(P)) return rc;
  if (P->state_elems > 0 && (!m_code || !r_code || !m_exp || !r_exp || !m || !r))
    return fail(CGTP_ERR_INVALID_ARG, "NULL argument");
  if (!aligned(m_code, 16) || !aligned(r_code, 16) || !aligned(m, 16) || !aligned(r, 16))
    return fail(CGTP_ERR_INVALID_ARG, "codes and values must be 16-byte aligned");
  CGTP_HIP(launch_decode_states(m_code, r_code, m_exp, r_exp, P->state_elems, m, r, static_cast<hipStream_t>(stream)));
  return ok();
}

int cgtp_grad_norm_workspace_size(cgtp_params_t P, size_t* bytes) {
  if (!P || !bytes) return fail(CGTP_ERR_INVALID_ARG, "NULL argument");
  *bytes = (size_t(norm_parts(P)) * sizeof(double) + 255) / 256 * 256;
  return ok();
}

int cgtp_grad_norm(cgtp_params_t P, int grad_dtype, const void* const* grads, const float* grad_scale, double max_norm,
                   float* out, void* workspace, size_t ws_bytes, void* stream) {
  if (int rc = check_set(P)) return rc;
  if (int rc = check_tensors(P, grad_dtype, grads, "grads")) return rc;
  if (!(max_norm > 0)) return fail(CGTP_ERR_INVALID_ARG, "max_norm must be positive");
  if (!out || !aligned(out, 4) || !aligned(grad_scale, 4)) return fail(CGTP_ERR_INVALID_ARG, "NULL or misaligned pointer");
  const int chunks = P->first_chunk.back(), parts = norm_parts(P);
  const size_t need = size_t(parts) * sizeof(double);
  if (parts > 0 && (!workspace || ws_bytes < need))
    return fail(CGTP_ERR_WORKSPACE, "workspace %zu bytes < %zu required", workspace ? ws_bytes : size_t(0), need);
  if (!aligned(workspace, 256)) return fail(CGTP_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  double* part = static_cast<double*>(workspace);
  GradNormArgs a{};
  if (small_norm(P)) {
    a.chunks = P->d_chunks;
    a.n_chunks = chunks;
    if (!P->numel.empty()) std::memcpy(a.grad, grads, P->numel.size() * sizeof(void*));
    CGTP_HIP(launch_grad_norm_small(a, Elem(grad_dtype), grad_scale, float(max_norm), out,
                                    static_cast<hipStream_t>(stream)));
    return ok();
  }
  int rc = for_launches(P, [&](int t, int n, int c0, int count) {
    a.chunks = P->d_chunks + c0;
    a.part = part;
    part += square_blocks(count);
    a.first_tensor = t;
    a.n_chunks = count;
    std::memcpy(a.grad, grads + t, size_t(n) * sizeof(void*));
    return launch_grad_squares(a, Elem(grad_dtype), static_cast<hipStream_t>(stream));
  });
  if (rc) return rc;
  CGTP_HIP(launch_grad_norm_finish(static_cast<double*>(workspace), parts, grad_scale, float(max_norm), out, static_cast<hipStream_t>(stream)));
  return ok();
}

}  // extern "C"

// Layer normalisation of rows and of irreps rows term by term, forward and backward.
//
// A row's stretch of F values (a NormTerm: the whole row, or one term's [channels][2l+1]
// block) is normalised by itself:
//   mu = sum(x)/F (centred terms; else 0), s2 = sum((x - mu)^2)/F, rstd = 1/sqrt(s2+eps),
//   h = (x - mu) rstd,  y = h w + b.
// Backward, a = g w:  dx = rstd (a - h sum(a h)/F - sum(a)/F), the last only if centred;
//   dw = sum over rows (and a channel's components) of g h, db = sum over rows of g.
// Sums and statistics are fp32 whatever the element type.  s2 is summed from x - mu, not
// from x^2: a row with a large common offset keeps its digits.
#include "elem.hpp"
#include "launch_train.hpp"

namespace cgtp {
namespace {

constexpr int kThreads = 256;

__device__ inline float wave_sum(float v) {
  for (int k = 32; k > 0; k >>= 1) v += __shfl_xor(v, k);
  return v;
}

// Sum over the workgroup, to every thread.
__device__ inline float block_sum(float v, float* lds) {
  v = wave_sum(v);
  __syncthreads();
  if (threadIdx.x % 64 == 0) lds[threadIdx.x / 64] = v;
  __syncthreads();
  float s = 0;
  for (int k = 0; k < kThreads / 64; ++k) s += lds[k];
  return s;
}

// One workgroup per row and term; the row is read again for each sum.
template <typename T>
__global__ __launch_bounds__(kThreads) void norm_fwd_kernel(NormArgs a) {
  __shared__ float lds[kThreads / 64];
  const NormTerm& t = a.term[blockIdx.y];
  const bool centred = t.b_off >= 0;
  const float inv = 1.0f / float(t.len);
  for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + r * a.ld_x + t.off;
    T* y = static_cast<T*>(a.y) + r * a.ld_y + t.off;
    float mu = 0;
    if (centred) {
      float s = 0;
      for (int e = threadIdx.x; e < t.len; e += kThreads) s += to_f32(x[e]);
      mu = block_sum(s, lds) * inv;
    }
    float q = 0;
    for (int e = threadIdx.x; e < t.len; e += kThreads) {
      const float v = to_f32(x[e]) - mu;
      q += v * v;
    }
    const float rstd = 1.0f / sqrtf(block_sum(q, lds) * inv + a.eps);
    for (int e = threadIdx.x; e < t.len; e += kThreads) {
      const int c = e / t.d;
      const float w = a.weight ? load_either<T>(a.weight, a.weight_f32, t.w_off + c) : 1.0f;
      const float b = a.bias && centred ? load_either<T>(a.bias, a.weight_f32, t.b_off + c) : 0.0f;
      y[e] = from_f32<T>((to_f32(x[e]) - mu) * rstd * w + b);
    }
    if (a.stats && threadIdx.x == 0) {
      a.stats[r * a.n_terms + t.index] = mu;
      a.stats[(a.rows + r) * a.n_terms + t.index] = rstd;
    }
  }
}

template <typename T>
__global__ __launch_bounds__(kThreads) void norm_bwd_x_kernel(NormArgs a) {
  __shared__ float lds[kThreads / 64];
  const NormTerm& t = a.term[blockIdx.y];
  const bool centred = t.b_off >= 0;
  const float inv = 1.0f / float(t.len);
  for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + r * a.ld_x + t.off;
    const T* g = static_cast<const T*>(a.grad_out) + r * a.ld_g + t.off;
    T* y = static_cast<T*>(a.y) + r * a.ld_y + t.off;
    const float mu = a.stats[r * a.n_terms + t.index], rstd = a.stats[(a.rows + r) * a.n_terms + t.index];
    float sa = 0, sh = 0;
    for (int e = threadIdx.x; e < t.len; e += kThreads) {
      const float w = a.weight ? load_either<T>(a.weight, a.weight_f32, t.w_off + e / t.d) : 1.0f;
      const float v = to_f32(g[e]) * w;
      sa += v;
      sh += v * ((to_f32(x[e]) - mu) * rstd);
    }
    sa = centred ? block_sum(sa, lds) * inv : 0.0f;
    sh = block_sum(sh, lds) * inv;
    for (int e = threadIdx.x; e < t.len; e += kThreads) {
      const float w = a.weight ? load_either<T>(a.weight, a.weight_f32, t.w_off + e / t.d) : 1.0f;
      const float h = (to_f32(x[e]) - mu) * rstd;
      y[e] = from_f32<T>((to_f32(g[e]) * w - sa - h * sh) * rstd);
    }
  }
}

constexpr int kSlices = 64;   // row slices of the weight's gradient

// One thread per channel and row slice: its sums over the slice's rows.
template <typename T>
__global__ __launch_bounds__(kThreads) void norm_bwd_w_kernel(NormArgs a) {
  const NormTerm& t = a.term[blockIdx.z];
  const bool centred = t.b_off >= 0;
  const int c = blockIdx.x * kThreads + threadIdx.x;
  if (c >= t.len / t.d) return;
  float sw = 0, sb = 0;
  for (int64_t r = blockIdx.y; r < a.rows; r += kSlices) {
    const T* x = static_cast<const T*>(a.x) + r * a.ld_x + t.off;
    const T* g = static_cast<const T*>(a.grad_out) + r * a.ld_g + t.off;
    const float mu = a.stats[r * a.n_terms + t.index], rstd = a.stats[(a.rows + r) * a.n_terms + t.index];
    for (int k = 0; k < t.d; ++k) {
      const float v = to_f32(g[c * t.d + k]);
      sw += v * ((to_f32(x[c * t.d + k]) - mu) * rstd);
      sb += v;
    }
  }
  float* part = a.part + size_t(blockIdx.y) * (a.n_weights + a.n_biases);
  part[t.w_off + c] = sw;
  if (centred) part[a.n_weights + t.b_off + c] = sb;
}

template <typename T>
__global__ __launch_bounds__(kThreads) void norm_bwd_sum_kernel(NormArgs a) {
  const int c = blockIdx.x * kThreads + threadIdx.x, n = a.n_weights + a.n_biases;
  if (c >= n) return;
  float s = 0;
  for (int k = 0; k < kSlices; ++k) s += a.part[size_t(k) * n + c];
  if (c < a.n_weights) {
    if (a.grad_weight) store_either<T>(a.grad_weight, a.weight_f32, c, s);
  } else if (a.grad_bias) {
    store_either<T>(a.grad_bias, a.weight_f32, c - a.n_weights, s);
  }
}

template <typename T>
hipError_t forward(const NormArgs& a, hipStream_t s) {
  if (a.rows > 0) {
    const dim3 grid(unsigned(a.rows < 65536 ? a.rows : 65536), unsigned(a.n_terms));
    hipLaunchKernelGGL(norm_fwd_kernel<T>, grid, dim3(kThreads), 0, s, a);
  }
  return hipGetLastError();
}

template <typename T>
hipError_t backward(const NormArgs& a, hipStream_t s) {
  if (a.rows > 0 && a.y) {
    const dim3 grid(unsigned(a.rows < 65536 ? a.rows : 65536), unsigned(a.n_terms));
    hipLaunchKernelGGL(norm_bwd_x_kernel<T>, grid, dim3(kThreads), 0, s, a);
  }
  if (a.grad_weight || a.grad_bias) {
    int most = 0;
    for (int k = 0; k < a.n_terms; ++k) most = max(most, a.term[k].len / a.term[k].d);
    const dim3 grid(unsigned((most + kThreads - 1) / kThreads), kSlices, unsigned(a.n_terms));
    hipLaunchKernelGGL(norm_bwd_w_kernel<T>, grid, dim3(kThreads), 0, s, a);
    const int n = a.n_weights + a.n_biases;
    hipLaunchKernelGGL(norm_bwd_sum_kernel<T>, dim3(unsigned((n + kThreads - 1) / kThreads)), dim3(kThreads), 0, s, a);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_norm_forward(const NormArgs& a, Elem type, hipStream_t s) {
  return type == Elem::f32 ? forward<float>(a, s) : type == Elem::bf16 ? forward<Bf16>(a, s) : forward<F16>(a, s);
}

size_t norm_part_floats(int64_t rows, int n_weights, int n_biases) {
  (void)rows;
  return size_t(kSlices) * size_t(n_weights + n_biases);
}

hipError_t launch_norm_backward(const NormArgs& a, Elem type, hipStream_t s) {
  return type == Elem::f32 ? backward<float>(a, s) : type == Elem::bf16 ? backward<Bf16>(a, s) : backward<F16>(a, s);
}

}  // namespace cgtp

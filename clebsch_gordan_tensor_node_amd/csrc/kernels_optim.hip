// The AdamW step over many tensors in few launches, with moments in 32 bits or in 8, and
// the gradient norm that clips it.
//
//   g = grad * grad_scale;  p <- p (1 - lr wd);  m <- b1 m + (1 - b1) g;
//   v <- b2 v + (1 - b2) g^2;  p <- p - (lr / (1 - b1^t)) m / (sqrt(v) / sqrt(1 - b2^t) + eps)
// Every step is one fp32 operation, rounded by itself (no contraction, IEEE division and
// square root), in the order written: the result is the same bit for bit wherever it is
// computed, which the 8-bit states' rounding needs to be reproducible.
//
// 8-bit states hold m and r = sqrt(v): the root has half the octaves of v, so 4 exponent
// bits reach as far below a block's largest value as 8 would in v.  A block of 64 elements
// has one exponent byte E, the biased fp32 exponent of its largest magnitude.  A code is
// the top of the fp32 number a 2^(14 - E) (biased exponent 14 at most, one octave of room
// for rounding up): for m a sign, 4 exponent and 3 mantissa bits, for r 4 and 4.  What is
// cut off rounds up with its own probability (16 bits of a hash of element and seed): with
// b2 = 0.999 a step moves r by 1/2000, a code's distance is 1/32, and rounding to nearest
// would never let a state decay.  A positive r keeps at least code 1, so that a lost small
// root cannot leave m over eps.
#include "elem.hpp"
#include "launch_train.hpp"

namespace cgtp {
namespace {

constexpr int kThreads = 256;
constexpr int kFinish = 1024;

__device__ inline uint32_t bits_of(float v) { return __builtin_bit_cast(uint32_t, v); }
__device__ inline float float_of(uint32_t v) { return __builtin_bit_cast(float, v); }

// 32 random bits of state element i.  The odd constants are the fractions of the golden
// ratio and of the square roots of 2 and 3.
__device__ inline uint32_t random_bits(int64_t i, uint32_t seed) {
  uint32_t h = uint32_t(i) * 0x9E3779B9u + uint32_t(uint64_t(i) >> 32) * 0x6A09E667u + seed;
  h ^= h >> 15;
  h *= 0xBB67AE85u;
  return h ^ (h >> 16);
}

constexpr uint32_t kMNan = 0x7f, kRNan = 0xff;   // codes of values that are not finite

__device__ inline float decode_m(uint32_t code, int e) {
  if ((code & 0x7f) == kMNan) return __builtin_nanf("");
  const float a = ldexpf(float_of((code & 0x7f) << 20), max(e, 1) - 14);
  return code & 0x80 ? -a : a;
}
__device__ inline float decode_r(uint32_t code, int e) {
  if (code == kRNan) return __builtin_nanf("");
  return ldexpf(float_of(code << 19), max(e, 1) - 14);
}
__device__ inline uint32_t encode_m(float m, int e, uint32_t u) {
  const float a = fabsf(m);
  const uint32_t c = a < __builtin_inff() ? (bits_of(ldexpf(a, 14 - max(e, 1))) + (u << 4)) >> 20 : kMNan;
  return c | (m < 0 ? 0x80u : 0u);
}
__device__ inline uint32_t encode_r(float r, int e, uint32_t u) {
  if (!(r < __builtin_inff())) return kRNan;
  const uint32_t c = (bits_of(ldexpf(r, 14 - max(e, 1))) + (u << 3)) >> 19;
  return r > 0 && c == 0 ? 1u : c;
}
// A magnitude's biased exponent, 0 where it is not finite (such a value is coded as NaN
// and does not set the block's scale).
__device__ inline int exponent_of(float a) { return a < __builtin_inff() ? int(bits_of(a) >> 23) : 0; }

struct Moments {
  float p, m, v, root;
};
__device__ inline Moments adamw(const AdamwArgs& a, float p, float g, float m, float v, float kept) {
#pragma clang fp contract(off)
  Moments o;
  o.p = p * kept;
  o.m = m * a.b1 + g * a.c1;
  o.v = v * a.b2 + g * g * a.c2;
  o.root = sqrtf(o.v);
  o.p = o.p - o.m * a.step_size / (o.root * a.inv_root + a.eps);
  return o;
}

// A lane's elements: kPasses vectors of 4, the workgroup's lanes after one another.
constexpr int kVec = 4;
constexpr int kPasses = kChunk / (kThreads * kVec);

// Four elements at any element's address; past n they read as 0 and are not written.
template <typename T>
__device__ inline void load4(const T* p, int i, int n, float (&v)[kVec]) {
  T r[kVec];
  if (i + kVec <= n) {
    __builtin_memcpy(r, p + i, sizeof(r));
#pragma unroll
    for (int j = 0; j < kVec; ++j) v[j] = to_f32(r[j]);
  } else {
#pragma unroll
    for (int j = 0; j < kVec; ++j) v[j] = i + j < n ? to_f32(p[i + j]) : 0.0f;
  }
}
template <typename T>
__device__ inline void store4(T* p, int i, int n, const float (&v)[kVec]) {
  T r[kVec];
#pragma unroll
  for (int j = 0; j < kVec; ++j) r[j] = from_f32<T>(v[j]);
  if (i + kVec <= n) {
    __builtin_memcpy(p + i, r, sizeof(r));
  } else {
#pragma unroll
    for (int j = 0; j < kVec; ++j)
      if (i + j < n) p[i + j] = r[j];
  }
}

template <int Ctrl>
__device__ inline int dpp(int v) {
  return __builtin_amdgcn_mov_dpp(v, Ctrl, 0xf, 0xf, true);
}
// Largest of 16 neighbouring lanes: of one block of 64 elements.
__device__ inline int block_max(int v) {
  v = max(v, dpp<0xB1>(v));    // quad_perm 1 0 3 2
  v = max(v, dpp<0x4E>(v));    // quad_perm 2 3 0 1
  v = max(v, dpp<0x141>(v));   // row_half_mirror
  return max(v, dpp<0x140>(v));   // row_mirror
}
static_assert(kStateBlock == 16 * kVec, "a block of states is 16 lanes");

template <typename P, typename G, bool Bits8>
__global__ __launch_bounds__(kThreads) void adamw_kernel(AdamwArgs a) {
  const Chunk c = a.chunks[blockIdx.x];
  const float scale = a.grad_scale ? *a.grad_scale : 1.0f;
  if (scale != scale) return;   // the gradients are not finite: the step is skipped
  P* p = static_cast<P*>(a.param[c.tensor - a.first_tensor]) + c.start;
  const G* g = static_cast<const G*>(a.grad[c.tensor - a.first_tensor]) + c.start;
  const float kept = float(1.0 - a.lr * c.decay);
  const int n = (c.n + kStateBlock - 1) / kStateBlock * kStateBlock;   // states are held in whole blocks
  float pv[kPasses][kVec], gv[kPasses][kVec], mv[kPasses][kVec], vv[kPasses][kVec];
  uint32_t mc[kPasses], rc[kPasses];
  int me[kPasses], re[kPasses];
#pragma unroll
  for (int k = 0; k < kPasses; ++k) {
    const int i = (k * kThreads + int(threadIdx.x)) * kVec;
    if (i < n) {
      const int64_t s = c.state + i;
      load4(p, i, c.n, pv[k]);
      load4(g, i, c.n, gv[k]);
      if constexpr (Bits8) {
        __builtin_memcpy(&mc[k], __builtin_assume_aligned(a.m_code + s, 4), 4);
        __builtin_memcpy(&rc[k], __builtin_assume_aligned(a.r_code + s, 4), 4);
        me[k] = a.m_exp[s / kStateBlock];
        re[k] = a.r_exp[s / kStateBlock];
      } else {
        __builtin_memcpy(mv[k], __builtin_assume_aligned(a.m + s, 16), 16);
        __builtin_memcpy(vv[k], __builtin_assume_aligned(a.v + s, 16), 16);
      }
    }
  }
#pragma unroll
  for (int k = 0; k < kPasses; ++k) {
    const int i = (k * kThreads + int(threadIdx.x)) * kVec;
    if (i < n) {   // the same in the 16 lanes of a block
      const int64_t s = c.state + i;
      Moments o[kVec];
      int em = 0, er = 0;
#pragma unroll
      for (int j = 0; j < kVec; ++j) {
        if constexpr (Bits8) {
          const float r = decode_r(rc[k] >> (8 * j) & 0xff, re[k]);
          o[j] = adamw(a, pv[k][j], gv[k][j] * scale, decode_m(mc[k] >> (8 * j) & 0xff, me[k]), r * r, kept);
          em = max(em, exponent_of(fabsf(o[j].m)));
          er = max(er, exponent_of(o[j].root));
        } else {
          o[j] = adamw(a, pv[k][j], gv[k][j] * scale, mv[k][j], vv[k][j], kept);
          mv[k][j] = o[j].m;
          vv[k][j] = o[j].v;
        }
        pv[k][j] = o[j].p;
      }
      if constexpr (Bits8) {
        em = block_max(em);
        er = block_max(er);
        uint32_t cm = 0, cr = 0;
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
          const uint32_t u = random_bits(s + j, a.seed);
          cm |= encode_m(o[j].m, em, u & 0xffff) << (8 * j);
          cr |= encode_r(o[j].root, er, u >> 16) << (8 * j);
        }
        __builtin_memcpy(__builtin_assume_aligned(a.m_code + s, 4), &cm, 4);
        __builtin_memcpy(__builtin_assume_aligned(a.r_code + s, 4), &cr, 4);
        if (threadIdx.x % 16 == 0) {
          a.m_exp[s / kStateBlock] = uint8_t(em);
          a.r_exp[s / kStateBlock] = uint8_t(er);
        }
      } else {
        __builtin_memcpy(__builtin_assume_aligned(a.m + s, 16), mv[k], 16);
        __builtin_memcpy(__builtin_assume_aligned(a.v + s, 16), vv[k], 16);
      }
      store4(p, i, c.n, pv[k]);
    }
  }
}

__device__ inline double block_sum(double v, double* lds) {
  for (int k = 32; k > 0; k >>= 1) v += __shfl_xor(v, k);
  if (threadIdx.x % 64 == 0) lds[threadIdx.x / 64] = v;
  __syncthreads();
  double s = 0;
  for (unsigned k = 0; k < blockDim.x / 64; ++k) s += lds[k];
  return s;
}

// Squares in fp64: no gradient's square overflows or underflows.
template <typename G>
__global__ __launch_bounds__(kThreads) void grad_squares_kernel(GradNormArgs a) {
  __shared__ double lds[kThreads / 64];
  const Chunk c = a.chunks[blockIdx.x];
  const G* g = static_cast<const G*>(a.grad[c.tensor - a.first_tensor]) + c.start;
  float v[kPasses][kVec];
#pragma unroll
  for (int k = 0; k < kPasses; ++k) load4(g, (k * kThreads + int(threadIdx.x)) * kVec, c.n, v[k]);
  double s = 0;
#pragma unroll
  for (int k = 0; k < kPasses; ++k)
#pragma unroll
    for (int j = 0; j < kVec; ++j) s += double(v[k][j]) * double(v[k][j]);
  s = block_sum(s, lds);
  if (threadIdx.x == 0) a.part[blockIdx.x] = s;
}

__global__ __launch_bounds__(kFinish) void grad_norm_kernel(const double* part, int n, const float* grad_scale,
                                                            float max_norm, float* out) {
  __shared__ double lds[kFinish / 64];
  double s = 0;
#pragma unroll 8
  for (int i = threadIdx.x; i < n; i += kFinish) s += part[i];
  s = block_sum(s, lds);
  if (threadIdx.x == 0) {
    const float scale = grad_scale ? *grad_scale : 1.0f;
    const float norm = float(sqrt(s) * fabs(double(scale)));
    out[0] = norm;
    out[1] = norm < __builtin_inff() ? (norm > max_norm ? scale * (max_norm / norm) : scale) : __builtin_nanf("");
  }
}

// n is a multiple of kStateBlock; 8 elements a lane.
__global__ __launch_bounds__(kThreads) void decode_states_kernel(const uint8_t* m_code, const uint8_t* r_code,
                                                                 const uint8_t* m_exp, const uint8_t* r_exp, int64_t n,
                                                                 Bf16* m, Bf16* r) {
  const int64_t step = int64_t(gridDim.x) * kThreads * 8;
  for (int64_t i = (int64_t(blockIdx.x) * kThreads + threadIdx.x) * 8; i < n; i += step) {
    uint8_t mc[8], rc[8];
    __builtin_memcpy(mc, __builtin_assume_aligned(m_code + i, 8), 8);
    __builtin_memcpy(rc, __builtin_assume_aligned(r_code + i, 8), 8);
    const int me = m_exp[i / kStateBlock], re = r_exp[i / kStateBlock];
    Bf16 mv[8], rv[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      mv[j] = from_f32<Bf16>(decode_m(mc[j], me));
      rv[j] = from_f32<Bf16>(decode_r(rc[j], re));
    }
    __builtin_memcpy(__builtin_assume_aligned(m + i, 16), mv, 16);
    __builtin_memcpy(__builtin_assume_aligned(r + i, 16), rv, 16);
  }
}

template <typename P, typename G>
hipError_t adamw_pg(const AdamwArgs& a, int n, bool bits8, hipStream_t s) {
  if (bits8)
    hipLaunchKernelGGL((adamw_kernel<P, G, true>), dim3(unsigned(n)), dim3(kThreads), 0, s, a);
  else
    hipLaunchKernelGGL((adamw_kernel<P, G, false>), dim3(unsigned(n)), dim3(kThreads), 0, s, a);
  return hipGetLastError();
}
template <typename P>
hipError_t adamw_p(const AdamwArgs& a, int n, Elem grad, bool bits8, hipStream_t s) {
  return grad == Elem::f32 ? adamw_pg<P, float>(a, n, bits8, s)
         : grad == Elem::bf16 ? adamw_pg<P, Bf16>(a, n, bits8, s) : adamw_pg<P, F16>(a, n, bits8, s);
}

}  // namespace

hipError_t launch_adamw(const AdamwArgs& a, int n_chunks, Elem param, Elem grad, bool bits8, hipStream_t s) {
  return param == Elem::f32 ? adamw_p<float>(a, n_chunks, grad, bits8, s)
         : param == Elem::bf16 ? adamw_p<Bf16>(a, n_chunks, grad, bits8, s) : adamw_p<F16>(a, n_chunks, grad, bits8, s);
}

hipError_t launch_grad_squares(const GradNormArgs& a, Elem grad, hipStream_t s) {
  const dim3 grid{unsigned(a.n_chunks)}, block(kThreads);
  if (grad == Elem::f32)
    hipLaunchKernelGGL(grad_squares_kernel<float>, grid, block, 0, s, a);
  else if (grad == Elem::bf16)
    hipLaunchKernelGGL(grad_squares_kernel<Bf16>, grid, block, 0, s, a);
  else
    hipLaunchKernelGGL(grad_squares_kernel<F16>, grid, block, 0, s, a);
  return hipGetLastError();
}

hipError_t launch_grad_norm_finish(const double* part, int n, const float* grad_scale, float max_norm, float* out,
                                   hipStream_t s) {
  hipLaunchKernelGGL(grad_norm_kernel, dim3(1), dim3(kFinish), 0, s, part, n, grad_scale, max_norm, out);
  return hipGetLastError();
}

hipError_t launch_decode_states(const uint8_t* m_code, const uint8_t* r_code, const uint8_t* m_exp,
                                const uint8_t* r_exp, int64_t n, void* m, void* r, hipStream_t s) {
  if (n > 0) {
    const int64_t blocks = (n + kThreads * 8 - 1) / (kThreads * 8);
    hipLaunchKernelGGL(decode_states_kernel, dim3(unsigned(blocks < 8192 ? blocks : 8192)), dim3(kThreads), 0, s,
                       m_code, r_code, m_exp, r_exp, n, static_cast<Bf16*>(m), static_cast<Bf16*>(r));
  }
  return hipGetLastError();
}

}  // namespace cgtp

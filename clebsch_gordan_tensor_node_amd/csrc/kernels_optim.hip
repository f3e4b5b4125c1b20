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

// 32 random bits of state element i: mix(place(i, seed)), with place(i + 1) = place(i) +
// kGolden inside 2^32 elements.  The odd constants are the fractions of the golden ratio
// and of the square roots of 2 and 3.
constexpr uint32_t kGolden = 0x9E3779B9u;
__device__ inline uint32_t place(int64_t i, uint32_t seed) {
  return uint32_t(i) * kGolden + uint32_t(uint64_t(i) >> 32) * 0x6A09E667u + seed;
}
__device__ inline uint32_t mix(uint32_t h) {
  h ^= h >> 15;
  h *= 0xBB67AE85u;
  return h ^ (h >> 16);
}

constexpr uint32_t kMNan = 0x7f, kRNan = 0xff;   // codes of values that are not finite
constexpr uint32_t kInf = 0x7f800000u;

// Values and codes of finite moments (sh = max(E, 1) - 14).
__device__ inline float decode_m(uint32_t code, int sh) {
  return ldexpf(float_of((code & 0x7f) << 20 | (code & 0x80) << 24), sh);
}
__device__ inline float decode_r(uint32_t code, int sh) { return ldexpf(float_of(code << 19), sh); }
__device__ inline uint32_t encode_m(float m, int sh, uint32_t u) {
  return (bits_of(ldexpf(fabsf(m), -sh)) + (u << 4)) >> 20 | bits_of(m) >> 31 << 7;
}
__device__ inline uint32_t encode_r(float r, int sh, uint32_t u) {
  return max((bits_of(ldexpf(r, -sh)) + (u << 3)) >> 19, min(bits_of(r), 1u));
}
// Whether one of four codes is a NaN's: a byte of all ones (m: but for its sign).
__device__ inline bool any_ones(uint32_t v) { return ((~v - 0x01010101u) & v & 0x80808080u) != 0; }
__device__ inline float nan() { return __builtin_nanf(""); }

struct Moments {
  float p, m, v, root;
};
__device__ inline Moments adamw(const AdamwArgs& a, const AdamwScalars& h, float p, float g, float m, float v,
                                float kept) {
#pragma clang fp contract(off)
  Moments o;
  o.p = p * kept;
  o.m = m * a.b1 + g * a.c1;
  o.v = v * a.b2 + g * g * a.c2;
  o.root = sqrtf(o.v);
  o.p = o.p - o.m * h.step_size / (o.root * h.inv_root + a.eps);
  return o;
}

// A lane's elements: kPasses vectors of 4, the workgroup's lanes after one another.
constexpr int kVec = 4;
constexpr int kPasses = kChunk / (kThreads * kVec);

// Four elements at any element's address; past n (unless Full) they read as 0 and are not
// written.  Stream: the access does not keep the line in the caches.
template <typename T>
struct Four {
  typedef uint32_t Bits __attribute__((ext_vector_type(sizeof(T)), aligned(sizeof(T)), may_alias));
  T v[kVec];
};
template <>
struct Four<uint8_t> {
  typedef uint32_t Bits __attribute__((may_alias));
  uint8_t v[kVec];
};
template <bool Stream, typename T>
__device__ inline Four<T> read4(const T* p) {
  typedef typename Four<T>::Bits Bits;
  const Bits* b = reinterpret_cast<const Bits*>(p);
  return __builtin_bit_cast(Four<T>, Stream ? __builtin_nontemporal_load(b) : *b);
}
template <bool Stream, typename T>
__device__ inline void write4(T* p, const Four<T>& v) {
  typedef typename Four<T>::Bits Bits;
  Bits* b = reinterpret_cast<Bits*>(p);
  if constexpr (Stream)
    __builtin_nontemporal_store(__builtin_bit_cast(Bits, v), b);
  else
    *b = __builtin_bit_cast(Bits, v);
}
template <bool Full, bool Stream, typename T>
__device__ inline void load4(const T* p, unsigned i, unsigned n, float (&v)[kVec]) {
  if (Full || i + kVec <= n) {
    const Four<T> r = read4<Stream>(p + i);
#pragma unroll
    for (int j = 0; j < kVec; ++j) v[j] = to_f32(r.v[j]);
  } else {
#pragma unroll
    for (int j = 0; j < kVec; ++j) v[j] = i + j < n ? to_f32(p[i + j]) : 0.0f;
  }
}
template <bool Full, bool Stream, typename T>
__device__ inline void store4(T* p, unsigned i, unsigned n, const float (&v)[kVec]) {
  Four<T> r;
#pragma unroll
  for (int j = 0; j < kVec; ++j) r.v[j] = from_f32<T>(v[j]);
  if (Full || i + kVec <= n) {
    write4<Stream>(p + i, r);
  } else {
#pragma unroll
    for (int j = 0; j < kVec; ++j)
      if (i + j < n) p[i + j] = r.v[j];
  }
}

template <int Ctrl>
__device__ inline uint32_t dpp(uint32_t v) {
  return uint32_t(__builtin_amdgcn_mov_dpp(int(v), Ctrl, 0xf, 0xf, true));
}
// Largest of 16 neighbouring lanes: of one block of 64 elements.
__device__ inline uint32_t block_max(uint32_t v) {
  v = max(v, dpp<0xB1>(v));    // quad_perm 1 0 3 2
  v = max(v, dpp<0x4E>(v));    // quad_perm 2 3 0 1
  v = max(v, dpp<0x141>(v));   // row_half_mirror
  return max(v, dpp<0x140>(v));   // row_mirror
}
static_assert(kStateBlock == 16 * kVec, "a block of states is 16 lanes");

// One chunk.  Full: all kChunk elements are there, nothing is guarded.
template <typename P, typename G, bool Bits8, bool Stream, bool Full>
__device__ inline void adamw_chunk(const AdamwArgs& a, const AdamwScalars& h, const Chunk& c, float scale) {
  P* p = static_cast<P*>(a.param[c.tensor - a.first_tensor]) + c.start;
  const G* g = static_cast<const G*>(a.grad[c.tensor - a.first_tensor]) + c.start;
  float *m = a.m + c.state, *v = a.v + c.state;
  uint8_t *m_code = a.m_code + c.state, *r_code = a.r_code + c.state;
  uint8_t *m_exp = a.m_exp + c.state / kStateBlock, *r_exp = a.r_exp + c.state / kStateBlock;
  const float kept = float(1.0 - h.lr * c.decay);
  const unsigned n = Full ? kChunk : unsigned(c.n), whole = (n + kStateBlock - 1) / kStateBlock * kStateBlock;
  float pv[kPasses][kVec], gv[kPasses][kVec], mv[kPasses][kVec], vv[kPasses][kVec];
  uint32_t mc[kPasses], rc[kPasses];
  int me[kPasses], re[kPasses];
#pragma unroll
  for (int k = 0; k < kPasses; ++k) {
    const unsigned i = (k * kThreads + threadIdx.x) * kVec;
    if (!Full && i >= whole) break;   // states are held in whole blocks
    load4<Full, Stream>(p, i, n, pv[k]);
    load4<Full, Stream>(g, i, n, gv[k]);
    if constexpr (Bits8) {
      mc[k] = __builtin_bit_cast(uint32_t, read4<Stream>(m_code + i));
      rc[k] = __builtin_bit_cast(uint32_t, read4<Stream>(r_code + i));
      me[k] = m_exp[i / kStateBlock];
      re[k] = r_exp[i / kStateBlock];
    } else {
      load4<true, Stream>(m, i, n, mv[k]);
      load4<true, Stream>(v, i, n, vv[k]);
    }
  }
#pragma unroll
  for (int k = 0; k < kPasses; ++k) {
    const unsigned i = (k * kThreads + threadIdx.x) * kVec;
    if (!Full && i >= whole) break;   // the same in the 16 lanes of a block
    if constexpr (Bits8) {
      const int sm = max(me[k], 1) - 14, sr = max(re[k], 1) - 14;
#pragma unroll
      for (int j = 0; j < kVec; ++j) {
        mv[k][j] = decode_m(mc[k] >> (8 * j) & 0xff, sm);
        const float r = decode_r(rc[k] >> (8 * j) & 0xff, sr);
        vv[k][j] = r * r;
      }
      if (any_ones(mc[k] | 0x80808080u) || any_ones(rc[k])) {
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
          if ((mc[k] >> (8 * j) & kMNan) == kMNan) mv[k][j] = nan();
          if ((rc[k] >> (8 * j) & kRNan) == kRNan) vv[k][j] = nan();
        }
      }
    }
    float root[kVec];
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      const Moments o = adamw(a, h, pv[k][j], gv[k][j] * scale, mv[k][j], vv[k][j], kept);
      pv[k][j] = o.p;
      mv[k][j] = o.m;
      vv[k][j] = o.v;
      root[j] = o.root;
    }
    if constexpr (Bits8) {
      // the block's largest magnitudes; where one is not finite, the largest finite ones.  A
      // moment that is not finite is encoded as 0, under the code of NaN: an encoded infinity
      // has more than 8 bits and would reach into the next element's.
      uint32_t tm = 0, tr = 0, nm = 0, nr = 0;
#pragma unroll
      for (int j = 0; j < kVec; ++j) {
        tm = max(tm, bits_of(mv[k][j]) & 0x7fffffffu);
        tr = max(tr, bits_of(root[j]) & 0x7fffffffu);
      }
      tm = block_max(tm);
      tr = block_max(tr);
      const bool bad = tm >= kInf || tr >= kInf;
      if (bad) {
        tm = tr = 0;
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
          if (!(fabsf(mv[k][j]) < float_of(kInf))) {
            nm |= (kMNan | (mv[k][j] < 0 ? 0x80u : 0u)) << (8 * j);
            mv[k][j] = 0;
          }
          if (!(root[j] < float_of(kInf))) {
            nr |= kRNan << (8 * j);
            root[j] = 0;
          }
          tm = max(tm, bits_of(mv[k][j]) & 0x7fffffffu);
          tr = max(tr, bits_of(root[j]));
        }
        tm = block_max(tm);
        tr = block_max(tr);
      }
      const int em = int(tm >> 23), er = int(tr >> 23), sm = max(em, 1) - 14, sr = max(er, 1) - 14;
      const uint32_t h0 = place(c.state + i, h.seed);
      uint32_t cm = nm, cr = nr;
#pragma unroll
      for (int j = 0; j < kVec; ++j) {
        const uint32_t u = mix(h0 + j * kGolden);
        cm |= encode_m(mv[k][j], sm, u & 0xffff) << (8 * j);
        cr |= encode_r(root[j], sr, u >> 16) << (8 * j);
      }
      write4<Stream>(m_code + i, __builtin_bit_cast(Four<uint8_t>, cm));
      write4<Stream>(r_code + i, __builtin_bit_cast(Four<uint8_t>, cr));
      if (threadIdx.x % 16 == 0) {
        m_exp[i / kStateBlock] = uint8_t(em);
        r_exp[i / kStateBlock] = uint8_t(er);
      }
    } else {
      store4<true, Stream>(m, i, n, mv[k]);
      store4<true, Stream>(v, i, n, vv[k]);
    }
    store4<Full, Stream>(p, i, n, pv[k]);
  }
}

// Bound by HBM with 32-bit states: 49.8 M elements, 28 bytes each, 201 us (6.9 TB/s of
// algorithmic bytes, a part of the gradients still cached from their norm).  With 8-bit
// states 37.3 M elements of 16 bytes take 109 us (5.5 TB/s) and some 85 operations each, two
// thirds of the time that the bytes need at that rate: every operation added here costs.
template <typename P, typename G, bool Bits8, bool Stream>
__global__ __launch_bounds__(kThreads) void adamw_kernel(AdamwArgs a) {
  const Chunk c = a.chunks[blockIdx.x];
  const float scale = a.grad_scale ? *a.grad_scale : 1.0f;
  if (scale != scale) return;   // the gradients are not finite: the step is skipped
  const AdamwScalars h = a.device ? *a.device : a.here;
  if (c.n == kChunk)
    adamw_chunk<P, G, Bits8, Stream, true>(a, h, c, scale);
  else
    adamw_chunk<P, G, Bits8, Stream, false>(a, h, c, scale);
}

// One thread, before the step and on its stream: bound by the launch (norm, count and step
// of 24 small tensors replay in 18 us; called, the count adds 5 us to 20).  A kernel of its own,
// so that the step's workgroups read 24 bytes and only one thread raises to powers (in 64
// bits, as the host does: 1 - b^t loses most of its digits at the first steps).
__global__ void adamw_scalars_kernel(int64_t* step, const float* lr_device, double lr, double beta1, double beta2,
                                     uint32_t seed, const float* grad_scale, AdamwScalars* out) {
  if (grad_scale && *grad_scale != *grad_scale) return;   // skipped: not a step
  const int64_t t = ++*step;
  if (lr_device) lr = *lr_device;
  AdamwScalars h;
  h.lr = lr;
  h.step_size = float(lr / (1 - pow(beta1, double(t))));
  h.inv_root = float(1 / sqrt(1 - pow(beta2, double(t))));
  h.seed = (seed + uint32_t(t)) * kSeedFactor;
  h.unused = 0;
  *out = h;
}

__device__ inline double block_sum(double v, double* lds) {
  for (int k = 32; k > 0; k >>= 1) v += __shfl_xor(v, k);
  if (threadIdx.x % 64 == 0) lds[threadIdx.x / 64] = v;
  __syncthreads();
  double s = 0;
  for (unsigned k = 0; k < blockDim.x / 64; ++k) s += lds[k];
  return s;
}

// A lane's part of a chunk, over the lanes of one wave (Lanes = 64) or of a workgroup.
template <int Lanes>
struct Part {
  static constexpr int kReads = kChunk / (Lanes * kVec);
  float v[kReads][kVec];
};
template <int Lanes, typename G>
__device__ inline Part<Lanes> chunk_part(const GradNormArgs& a, int index) {
  Part<Lanes> p;
  const Chunk c = a.chunks[index];
  const G* g = static_cast<const G*>(a.grad[c.tensor - a.first_tensor]) + c.start;
  const unsigned lane = threadIdx.x % Lanes;
  if (c.n == kChunk) {
#pragma unroll
    for (int k = 0; k < p.kReads; ++k) load4<true, false>(g, (k * Lanes + lane) * kVec, kChunk, p.v[k]);
  } else {
#pragma unroll
    for (int k = 0; k < p.kReads; ++k) load4<false, false>(g, (k * Lanes + lane) * kVec, unsigned(c.n), p.v[k]);
  }
  return p;
}
// In fp64: no gradient's square overflows or underflows.
template <int Lanes>
__device__ inline double squares(const Part<Lanes>& p) {
  double s = 0;
#pragma unroll
  for (int k = 0; k < p.kReads; ++k)
#pragma unroll
    for (int j = 0; j < kVec; ++j) s += double(p.v[k][j]) * double(p.v[k][j]);
  return s;
}

// A read of the gradients: 49.8 M fp32 in 33 us (6.0 TB/s), 62 us when lines that a step
// before wrote through the cache had still to be written back.
template <typename G>
__global__ __launch_bounds__(kThreads) void grad_squares_kernel(GradNormArgs a) {
  __shared__ double lds[kThreads / 64];
  double s = 0;
  for (int c = blockIdx.x; c < a.n_chunks; c += int(gridDim.x)) s += squares(chunk_part<kThreads, G>(a, c));
  s = block_sum(s, lds);
  if (threadIdx.x == 0) a.part[blockIdx.x] = s;
}

__device__ inline void write_norm(double sum, const float* grad_scale, float max_norm, float* out) {
  const float scale = grad_scale ? *grad_scale : 1.0f;
  const float norm = float(sqrt(sum) * fabs(double(scale)));
  out[0] = norm;
  out[1] = norm < __builtin_inff() ? (norm > max_norm ? scale * (max_norm / norm) : scale) : nan();
}

__global__ __launch_bounds__(kFinish) void grad_norm_kernel(const double* part, int n, const float* grad_scale,
                                                            float max_norm, float* out) {
  __shared__ double lds[kFinish / 64];
  double s = 0;
#pragma unroll 8
  for (int i = threadIdx.x; i < n; i += kFinish) s += part[i];
  s = block_sum(s, lds);
  if (threadIdx.x == 0) write_norm(s, grad_scale, max_norm, out);
}

// Small sets, in one workgroup and launch: two chunks to each wave, read together.  24
// tensors of 8192 elements at most 5.6 us, and a launch less for the host (3.7 us) than the
// two kernels' 3.1 + 2.0 us.
template <typename G>
__global__ __launch_bounds__(kFinish) void grad_norm_small_kernel(GradNormArgs a, const float* grad_scale,
                                                                  float max_norm, float* out) {
  constexpr int kWaves = kFinish / 64;
  static_assert(kSmallChunks <= 2 * kWaves, "two chunks to a wave");
  __shared__ double lds[kWaves];
  const int c = __builtin_amdgcn_readfirstlane(int(threadIdx.x) / 64);
  Part<64> p = {}, q = {};
  if (c < a.n_chunks) p = chunk_part<64, G>(a, c);
  if (c + kWaves < a.n_chunks) q = chunk_part<64, G>(a, c + kWaves);
  const double s = block_sum(squares(p) + squares(q), lds);
  if (threadIdx.x == 0) write_norm(s, grad_scale, max_norm, out);
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
    const int sm = max(int(m_exp[i / kStateBlock]), 1) - 14, sr = max(int(r_exp[i / kStateBlock]), 1) - 14;
    Bf16 mv[8], rv[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      mv[j] = from_f32<Bf16>((mc[j] & kMNan) == kMNan ? nan() : decode_m(mc[j], sm));
      rv[j] = from_f32<Bf16>(rc[j] == kRNan ? nan() : decode_r(rc[j], sr));
    }
    __builtin_memcpy(__builtin_assume_aligned(m + i, 16), mv, 16);
    __builtin_memcpy(__builtin_assume_aligned(r + i, 16), rv, 16);
  }
}

template <typename P, typename G, bool Bits8>
void adamw_launch(const AdamwArgs& a, int n, bool stream, hipStream_t s) {
  const dim3 grid{unsigned(n)}, block(kThreads);
  if (stream)
    hipLaunchKernelGGL((adamw_kernel<P, G, Bits8, true>), grid, block, 0, s, a);
  else
    hipLaunchKernelGGL((adamw_kernel<P, G, Bits8, false>), grid, block, 0, s, a);
}
template <typename P, typename G>
hipError_t adamw_pg(const AdamwArgs& a, int n, bool bits8, bool stream, hipStream_t s) {
  if (bits8)
    adamw_launch<P, G, true>(a, n, stream, s);
  else
    adamw_launch<P, G, false>(a, n, stream, s);
  return hipGetLastError();
}
template <typename P>
hipError_t adamw_p(const AdamwArgs& a, int n, Elem grad, bool bits8, bool stream, hipStream_t s) {
  return grad == Elem::f32 ? adamw_pg<P, float>(a, n, bits8, stream, s)
         : grad == Elem::bf16 ? adamw_pg<P, Bf16>(a, n, bits8, stream, s) : adamw_pg<P, F16>(a, n, bits8, stream, s);
}

}  // namespace

hipError_t launch_adamw(const AdamwArgs& a, int n_chunks, Elem param, Elem grad, bool bits8, bool stream,
                        hipStream_t s) {
  return param == Elem::f32 ? adamw_p<float>(a, n_chunks, grad, bits8, stream, s)
         : param == Elem::bf16 ? adamw_p<Bf16>(a, n_chunks, grad, bits8, stream, s) : adamw_p<F16>(a, n_chunks, grad, bits8, stream, s);
}

hipError_t launch_adamw_scalars(int64_t* step, const float* lr_device, double lr, double beta1, double beta2,
                                uint32_t seed, const float* grad_scale, AdamwScalars* out, hipStream_t s) {
  hipLaunchKernelGGL(adamw_scalars_kernel, dim3(1), dim3(1), 0, s, step, lr_device, lr, beta1, beta2, seed, grad_scale,
                     out);
  return hipGetLastError();
}

hipError_t launch_grad_squares(const GradNormArgs& a, Elem grad, hipStream_t s) {
  const dim3 grid{unsigned(square_blocks(a.n_chunks))}, block(kThreads);
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

hipError_t launch_grad_norm_small(const GradNormArgs& a, Elem grad, const float* grad_scale, float max_norm, float* out,
                                  hipStream_t s) {
  const dim3 grid(1), block(kFinish);
  if (grad == Elem::f32)
    hipLaunchKernelGGL(grad_norm_small_kernel<float>, grid, block, 0, s, a, grad_scale, max_norm, out);
  else if (grad == Elem::bf16)
    hipLaunchKernelGGL(grad_norm_small_kernel<Bf16>, grid, block, 0, s, a, grad_scale, max_norm, out);
  else
    hipLaunchKernelGGL(grad_norm_small_kernel<F16>, grid, block, 0, s, a, grad_scale, max_norm, out);
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

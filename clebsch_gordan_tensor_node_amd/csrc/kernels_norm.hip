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
//
// Both passes are bound by HBM: 2 (forward) or 3 (backward) elements moved per element for
// 8 to 14 operations.  So a stretch is read once into registers: G lanes hold it, C
// vectors of 16 bytes each (V elements, the next V G elements after one another), and
// both sums and the output come from there.  Rows need no alignment beyond an element's:
// the hardware takes 16-byte accesses at any element's address.  The last vector of a
// stretch that V does not divide is moved back to end with the stretch; the elements that
// it repeats are left out of the sums, and written twice with the same value.
// A workgroup keeps its weights in registers over all its rows (workgroup, then stride).
#include <algorithm>

#include "elem.hpp"
#include "launch_train.hpp"

namespace cgtp {
namespace {

constexpr int kThreads = 256;
constexpr int kWave = 64;

// A term as a launch carries it.
struct TermArgs {
  int32_t off, len, d, w_off, b_off;
  int32_t variant;        // which (V, G, C) handles it
  int32_t n_blocks;       // its workgroups
  uint32_t inv_d;         // ceil(2^32 / d) for d > 1: e / d = (e * inv_d) >> 32 for e < 2^32 / d
  int64_t part;           // backward: its partial sums in `part`: [n_blocks][len] of the weight's
                          // gradient, then (centred terms) as much of the bias's
};
template <int Cap>
struct NormArgs {
  NormCall c;
  int32_t n_terms;
  int32_t direct;             // backward: one workgroup per term, which writes the gradients itself
  int32_t first_block[Cap];   // of each term (INT32_MAX past the last)
  TermArgs term[Cap];
};
constexpr int kCapSmall = 8;

// The variants: a stretch of len elements takes the first whose room it fits.
//   id  V G C             room, 4-byte elements   2-byte elements
enum Variant : int {
  kElem16,    // V = 1, G = 16, C = 1       16                     16   (shorter than a vector)
  kG16C1,     //        G = 16              64                    128
  kG16C2,     //                           128                    256
  kG64C1,     //        G = 64             256                    512
  kG64C2,     //                           512                   1024
  kG64C4,     //                          1024                   2048
  kG64C8,     //                          2048                      -     (forward)
  kG256C2,    //        G = 256           2048                   4096     (backward)
  kG256C4,    //                          4096                   8192
  kG256C8,    //                          8192                      -
  kWide       // any: the row is read again for each sum
};
constexpr int kWideOver = 8192;

// The backward holds five values per element where the forward holds three, and takes at
// most 16 elements per lane as long as a workgroup's lanes reach.
int variant_of(int len, int elem_bytes, bool backward) {
  const int v = 16 / elem_bytes;
  if (len > kWideOver) return kWide;
  if (len < v) return kElem16;
  const int nv = (len + v - 1) / v;
  if (nv <= 16) return kG16C1;
  if (nv <= 32) return kG16C2;
  if (nv <= 64) return kG64C1;
  if (nv <= 128) return kG64C2;
  if (nv <= 256 && !(backward && elem_bytes == 2)) return kG64C4;
  if (nv <= 512 && backward) return kG256C2;
  if (nv <= 512 && elem_bytes == 4) return kG64C8;
  return nv <= 1024 ? kG256C4 : kG256C8;
}
// Stretches that a workgroup of a variant handles at once, and elements per lane.
int groups_of(int variant) { return variant <= kG16C2 ? 16 : variant <= kG64C8 ? 4 : 1; }
int elems_of(int variant, int elem_bytes) {
  const int v = 16 / elem_bytes;
  switch (variant) {
    case kElem16: return 1;
    case kG16C1: case kG64C1: return v;
    case kG16C2: case kG64C2: case kG256C2: return 2 * v;
    case kG64C4: case kG256C4: return 4 * v;
    case kG64C8: case kG256C8: return 8 * v;
    default: return 1;
  }
}

template <typename T, int V>
struct Vec {
  typedef uint32_t Bits __attribute__((ext_vector_type(sizeof(T) * V / 4), aligned(sizeof(T))));
  T v[V];
};
template <>
struct Vec<Bf16, 1> {
  typedef uint16_t Bits;
  Bf16 v[1];
};
template <>
struct Vec<F16, 1> {
  typedef uint16_t Bits;
  F16 v[1];
};
// 16 bytes (or one element) at any element's address.  Stream: the access does not keep
// the line in the caches.
template <bool Stream, typename T, int V>
__device__ inline Vec<T, V> load_vec(const T* p) {
  typedef typename Vec<T, V>::Bits Bits;
  const Bits* b = reinterpret_cast<const Bits*>(p);
  return __builtin_bit_cast(Vec<T, V>, Stream ? __builtin_nontemporal_load(b) : *b);
}
template <bool Stream, typename T, int V>
__device__ inline void store_vec(T* p, const Vec<T, V>& r) {
  typedef typename Vec<T, V>::Bits Bits;
  Bits* b = reinterpret_cast<Bits*>(p);
  if constexpr (Stream)
    __builtin_nontemporal_store(__builtin_bit_cast(Bits, r), b);
  else
    *b = __builtin_bit_cast(Bits, r);
}

template <int Ctrl>
__device__ inline float dpp(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), Ctrl, 0xf, 0xf, true));
}
// Sum over G neighbouring lanes (16 or 64), to each of them.
template <int G>
__device__ inline float lanes_sum(float v) {
  v += dpp<0xB1>(v);    // quad_perm 1 0 3 2
  v += dpp<0x4E>(v);    // quad_perm 2 3 0 1
  v += dpp<0x141>(v);   // row_half_mirror
  v += dpp<0x140>(v);   // row_mirror
  if constexpr (G >= 64) {
    v += __shfl_xor(v, 16);
    v += __shfl_xor(v, 32);
  }
  return v;
}
// The same over a group of G lanes, a whole workgroup for G = 256.  lds: 2 * 8 floats that
// alternate (`turn`), so that one barrier per sum is enough.
template <int G>
__device__ inline float group_sum(float v, float* lds, int& turn) {
  if constexpr (G <= kWave) {
    return lanes_sum<G>(v);
  } else {
    v = lanes_sum<kWave>(v);
    float* l = lds + (turn & 1) * 8;
    turn ^= 1;
    if (threadIdx.x % kWave == 0) l[threadIdx.x / kWave] = v;
    __syncthreads();
    return (l[0] + l[1]) + (l[2] + l[3]);
  }
}
template <int G>
__device__ inline void group_sum2(float& u, float& v, float* lds, int& turn) {
  if constexpr (G <= kWave) {
    u = lanes_sum<G>(u);
    v = lanes_sum<G>(v);
  } else {
    u = lanes_sum<kWave>(u);
    v = lanes_sum<kWave>(v);
    float* l = lds + (turn & 1) * 8;
    turn ^= 1;
    if (threadIdx.x % kWave == 0) {
      l[threadIdx.x / kWave] = u;
      l[4 + threadIdx.x / kWave] = v;
    }
    __syncthreads();
    u = (l[0] + l[1]) + (l[2] + l[3]);
    v = (l[4] + l[5]) + (l[6] + l[7]);
  }
}

// Where a lane's vectors of a stretch lie.
template <int V, int G, int C>
struct Place {
  int lane, len, last;   // last: the chunk that holds the stretch's end (the same in all lanes)
  __device__ Place(int n) : lane(threadIdx.x % G), len(n), last((n - 1) / (V * G)) {}
  __device__ int start(int c) const { return (c * G + lane) * V; }
  __device__ bool has(int c) const { return c < last || (c == last && start(c) < len); }
  __device__ int at(int c) const { return min(start(c), len - V); }   // first element of the vector
  __device__ int skip(int c) const { return start(c) - at(c); }       // of which these belong to the one before
};

template <typename T, int V, int C>
struct Row {
  Vec<T, V> c[C];
};
template <bool Stream, typename T, int V, int G, int C>
__device__ inline Row<T, V, C> read_row(const Place<V, G, C>& p, const T* row) {
  Row<T, V, C> r = {};
#pragma unroll
  for (int c = 0; c < C; ++c)
    if (p.has(c)) r.c[c] = load_vec<Stream, T, V>(row + p.at(c));
  return r;
}
template <typename T, int V, int C>
__device__ inline void widen(const Row<T, V, C>& r, float (&x)[C][V]) {
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int j = 0; j < V; ++j) x[c][j] = to_f32(r.c[c].v[j]);
}
template <bool Stream, typename T, int V, int G, int C>
__device__ inline void store_row(const Place<V, G, C>& p, T* row, const float (&y)[C][V]) {
#pragma unroll
  for (int c = 0; c < C; ++c)
    if (p.has(c)) {
      Vec<T, V> r;
#pragma unroll
      for (int j = 0; j < V; ++j) r.v[j] = from_f32<T>(y[c][j]);
      store_vec<Stream, T, V>(row + p.at(c), r);
    }
}
// Sum of f(c, j) over the lane's own elements.
template <int V, int G, int C, typename F>
__device__ inline float own_sum(const Place<V, G, C>& p, F&& f) {
  float s = 0;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    if (c < p.last) {
#pragma unroll
      for (int j = 0; j < V; ++j) s += f(c, j);
    } else if (c == p.last) {
      const bool has = p.has(c);
      const int skip = p.skip(c);
#pragma unroll
      for (int j = 0; j < V; ++j) s += has && j >= skip ? f(c, j) : 0.0f;
    }
  }
  return s;
}
// The channels' weights (or biases) at the lane's elements; `none` where there are none.
template <typename T, int V, int G, int C>
__device__ inline void load_weights(const Place<V, G, C>& p, const void* w, int f32, int off, const TermArgs& t,
                                    float none, float (&out)[C][V]) {
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int j = 0; j < V; ++j) {
      out[c][j] = none;
      if (w && p.has(c)) {
        const uint32_t e = uint32_t(p.at(c) + j);
        out[c][j] = load_either<T>(w, f32, off + int(t.d == 1 ? e : __umulhi(e, t.inv_d)));
      }
    }
}

template <bool Stream, typename T, int V, int G, int C>
__device__ inline void fwd_rows(const NormCall& a, const TermArgs& t, int n_terms, int index, int block, float* lds) {
  constexpr int kGroups = kThreads / G;
  const Place<V, G, C> p(t.len);
  const bool centred = t.b_off >= 0;
  const float inv = 1.0f / float(t.len);
  float w[C][V], b[C][V], x[C][V];
  load_weights<T>(p, a.weight, a.weight_f32, t.w_off, t, 1.0f, w);
  load_weights<T>(p, centred ? a.bias : nullptr, a.weight_f32, t.b_off, t, 0.0f, b);
  int turn = 0;
  for (int64_t r = int64_t(block) * kGroups + threadIdx.x / G; r < a.rows; r += int64_t(t.n_blocks) * kGroups) {
    widen(read_row<Stream>(p, static_cast<const T*>(a.x) + r * a.ld_x + t.off), x);
    float mu = 0;
    if (centred) mu = group_sum<G>(own_sum(p, [&](int c, int j) { return x[c][j]; }), lds, turn) * inv;
    const float s2 = group_sum<G>(own_sum(p, [&](int c, int j) { return (x[c][j] - mu) * (x[c][j] - mu); }), lds, turn);
    const float rstd = 1.0f / sqrtf(s2 * inv + a.eps);
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int j = 0; j < V; ++j) x[c][j] = (x[c][j] - mu) * rstd * w[c][j] + b[c][j];
    store_row<Stream>(p, static_cast<T*>(a.y) + r * a.ld_y + t.off, x);
    if (a.stats && p.lane == 0) {
      a.stats[r * n_terms + index] = mu;
      a.stats[(a.rows + r) * n_terms + index] = rstd;
    }
  }
}

template <bool Stream, typename T, int V, int G, int C>
__device__ inline void bwd_rows(const NormCall& a, const TermArgs& t, int n_terms, int index, int block, float* lds,
                                bool direct) {
  constexpr int kGroups = kThreads / G;
  const Place<V, G, C> p(t.len);
  const bool centred = t.b_off >= 0;
  const float inv = 1.0f / float(t.len);
  float w[C][V], x[C][V], g[C][V], gw[C][V], gb[C][V];
  load_weights<T>(p, a.weight, a.weight_f32, t.w_off, t, 1.0f, w);
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int j = 0; j < V; ++j) gw[c][j] = gb[c][j] = 0;
  int turn = 0;
  for (int64_t r = int64_t(block) * kGroups + threadIdx.x / G; r < a.rows; r += int64_t(t.n_blocks) * kGroups) {
    widen(read_row<Stream>(p, static_cast<const T*>(a.x) + r * a.ld_x + t.off), x);
    widen(read_row<Stream>(p, static_cast<const T*>(a.grad_out) + r * a.ld_g + t.off), g);
    const float mu = a.stats[r * n_terms + index], rstd = a.stats[(a.rows + r) * n_terms + index];
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int j = 0; j < V; ++j) {
        x[c][j] = (x[c][j] - mu) * rstd;
        gw[c][j] += g[c][j] * x[c][j];
        gb[c][j] += g[c][j];
        g[c][j] *= w[c][j];
      }
    if (!a.y) continue;
    float sa = own_sum(p, [&](int c, int j) { return g[c][j]; });
    float sh = own_sum(p, [&](int c, int j) { return g[c][j] * x[c][j]; });
    group_sum2<G>(sa, sh, lds, turn);
    sa = centred ? sa * inv : 0.0f;
    sh *= inv;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int j = 0; j < V; ++j) g[c][j] = (g[c][j] - sa - x[c][j] * sh) * rstd;
    store_row<Stream>(p, static_cast<T*>(a.y) + r * a.ld_y + t.off, g);
  }
  if (!a.grad_weight && !a.grad_bias) return;
  // the workgroup's sums: its groups' added in LDS, one row of `part`, or the gradients
  float* part = a.part + t.part + int64_t(block) * t.len;
  for (int k = 0; k < (centred ? 2 : 1); ++k, part += int64_t(t.n_blocks) * t.len) {
    __syncthreads();
    float* mine = lds + threadIdx.x / G * t.len;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (p.has(c) && j >= p.skip(c)) mine[p.at(c) + j] = k ? gb[c][j] : gw[c][j];
    __syncthreads();
    void* out = k ? a.grad_bias : a.grad_weight;
    if (direct && !out) continue;
    const int d = direct ? t.d : 1;
    for (int e = threadIdx.x; e < t.len / d; e += kThreads) {
      float s = 0;
      for (int m = 0; m < d; ++m)
        for (int q = 0; q < kGroups; ++q) s += lds[q * t.len + e * d + m];
      if (direct)
        store_either<T>(out, a.weight_f32, (k ? t.b_off : t.w_off) + e, s);
      else
        part[e] = s;
    }
  }
}

// Stretches of any length: one workgroup per row, which is read again for each sum.
template <typename T>
__device__ inline void fwd_wide(const NormCall& a, const TermArgs& t, int n_terms, int index, int block, float* lds) {
  const bool centred = t.b_off >= 0;
  const float inv = 1.0f / float(t.len);
  int turn = 0;
  for (int64_t r = block; r < a.rows; r += t.n_blocks) {
    const T* x = static_cast<const T*>(a.x) + r * a.ld_x + t.off;
    T* y = static_cast<T*>(a.y) + r * a.ld_y + t.off;
    float mu = 0, q = 0;
    if (centred) {
      float s = 0;
      for (int e = threadIdx.x; e < t.len; e += kThreads) s += to_f32(x[e]);
      mu = group_sum<kThreads>(s, lds, turn) * inv;
    }
    for (int e = threadIdx.x; e < t.len; e += kThreads) {
      const float v = to_f32(x[e]) - mu;
      q += v * v;
    }
    const float rstd = 1.0f / sqrtf(group_sum<kThreads>(q, lds, turn) * inv + a.eps);
    for (int e = threadIdx.x; e < t.len; e += kThreads) {
      const int c = t.d == 1 ? e : int(__umulhi(uint32_t(e), t.inv_d));
      const float w = a.weight ? load_either<T>(a.weight, a.weight_f32, t.w_off + c) : 1.0f;
      const float b = a.bias && centred ? load_either<T>(a.bias, a.weight_f32, t.b_off + c) : 0.0f;
      y[e] = from_f32<T>((to_f32(x[e]) - mu) * rstd * w + b);
    }
    if (a.stats && threadIdx.x == 0) {
      a.stats[r * n_terms + index] = mu;
      a.stats[(a.rows + r) * n_terms + index] = rstd;
    }
  }
}
template <typename T>
__device__ inline void bwd_wide(const NormCall& a, const TermArgs& t, int n_terms, int index, int block, float* lds) {
  const bool centred = t.b_off >= 0;
  const float inv = 1.0f / float(t.len);
  int turn = 0;
  for (int64_t r = block; a.y && r < a.rows; r += t.n_blocks) {
    const T* x = static_cast<const T*>(a.x) + r * a.ld_x + t.off;
    const T* g = static_cast<const T*>(a.grad_out) + r * a.ld_g + t.off;
    T* y = static_cast<T*>(a.y) + r * a.ld_y + t.off;
    const float mu = a.stats[r * n_terms + index], rstd = a.stats[(a.rows + r) * n_terms + index];
    auto weight = [&](int e) {
      const int c = t.d == 1 ? e : int(__umulhi(uint32_t(e), t.inv_d));
      return a.weight ? load_either<T>(a.weight, a.weight_f32, t.w_off + c) : 1.0f;
    };
    float sa = 0, sh = 0;
    for (int e = threadIdx.x; e < t.len; e += kThreads) {
      const float v = to_f32(g[e]) * weight(e);
      sa += v;
      sh += v * ((to_f32(x[e]) - mu) * rstd);
    }
    group_sum2<kThreads>(sa, sh, lds, turn);
    sa = centred ? sa * inv : 0.0f;
    sh *= inv;
    for (int e = threadIdx.x; e < t.len; e += kThreads)
      y[e] = from_f32<T>((to_f32(g[e]) * weight(e) - sa - (to_f32(x[e]) - mu) * rstd * sh) * rstd);
  }
  if (!a.grad_weight && !a.grad_bias) return;
  // the sums of the workgroup's rows, column by column
  float* part = a.part + t.part + int64_t(block) * t.len;
  for (int e = threadIdx.x; e < t.len; e += kThreads) {
    float sw = 0, sb = 0;
    for (int64_t r = block; r < a.rows; r += t.n_blocks) {
      const float v = to_f32((static_cast<const T*>(a.grad_out) + r * a.ld_g + t.off)[e]);
      const float mu = a.stats[r * n_terms + index], rstd = a.stats[(a.rows + r) * n_terms + index];
      sw += v * ((to_f32((static_cast<const T*>(a.x) + r * a.ld_x + t.off)[e]) - mu) * rstd);
      sb += v;
    }
    part[e] = sw;
    if (centred) part[int64_t(t.n_blocks) * t.len + e] = sb;
  }
}

// The workgroup's term.
template <int Cap>
__device__ inline int term_of(const NormArgs<Cap>& a) {
  int k = 0;
#pragma unroll
  for (int q = 1; q < Cap; ++q) k += int(blockIdx.x) >= a.first_block[q];
  return __builtin_amdgcn_readfirstlane(k);
}

// One launch for all terms; a kernel holds the variants of up to MaxE elements per lane,
// so that short rows do not pay for long ones' registers.
#define CGTP_NORM_VARIANTS(FN, ...)                                                                          \
  constexpr int V = 16 / int(sizeof(T));                                                                     \
  switch (t.variant) {                                                                                       \
    case kElem16: FN<Stream, T, 1, 16, 1>(a.c, t, a.n_terms, k, block, lds, ##__VA_ARGS__); break;           \
    case kG16C1: FN<Stream, T, V, 16, 1>(a.c, t, a.n_terms, k, block, lds, ##__VA_ARGS__); break;            \
    case kG64C1: FN<Stream, T, V, 64, 1>(a.c, t, a.n_terms, k, block, lds, ##__VA_ARGS__); break;            \
    default:                                                                                                 \
      if constexpr (MaxE >= 2 * V) {                                                                         \
        if (t.variant == kG16C2) FN<Stream, T, V, 16, 2>(a.c, t, a.n_terms, k, block, lds, ##__VA_ARGS__);   \
        if (t.variant == kG64C2) FN<Stream, T, V, 64, 2>(a.c, t, a.n_terms, k, block, lds, ##__VA_ARGS__);   \
        if (t.variant == kG256C2) FN<Stream, T, V, 256, 2>(a.c, t, a.n_terms, k, block, lds, ##__VA_ARGS__); \
      }                                                                                                      \
      if constexpr (MaxE >= 4 * V) {                                                                         \
        if (t.variant == kG64C4) FN<Stream, T, V, 64, 4>(a.c, t, a.n_terms, k, block, lds, ##__VA_ARGS__);   \
        if (t.variant == kG256C4) FN<Stream, T, V, 256, 4>(a.c, t, a.n_terms, k, block, lds, ##__VA_ARGS__); \
      }                                                                                                      \
      if constexpr (MaxE >= 8 * V) {                                                                         \
        if (t.variant == kG64C8) FN<Stream, T, V, 64, 8>(a.c, t, a.n_terms, k, block, lds, ##__VA_ARGS__);   \
        if (t.variant == kG256C8) FN<Stream, T, V, 256, 8>(a.c, t, a.n_terms, k, block, lds, ##__VA_ARGS__); \
      }                                                                                                      \
  }

template <typename T, int MaxE, int Cap, bool Stream>
__global__ __launch_bounds__(kThreads) void norm_fwd_kernel(NormArgs<Cap> a) {
  __shared__ float lds[16];
  const int k = term_of(a);
  const TermArgs& t = a.term[k];
  const int block = int(blockIdx.x) - a.first_block[k];
  if (t.variant == kWide) return fwd_wide<T>(a.c, t, a.n_terms, k, block, lds);
  CGTP_NORM_VARIANTS(fwd_rows)
}

template <typename T, int MaxE, int Cap, bool Stream>
__global__ __launch_bounds__(kThreads) void norm_bwd_kernel(NormArgs<Cap> a) {
  __shared__ float lds[kThreads * MaxE];
  const int k = term_of(a);
  const TermArgs& t = a.term[k];
  const int block = int(blockIdx.x) - a.first_block[k];
  if (t.variant == kWide) return bwd_wide<T>(a.c, t, a.n_terms, k, block, lds);
  CGTP_NORM_VARIANTS(bwd_rows, a.direct)
}

// The weight's and bias's gradients from the workgroups' sums, in a fixed order.  A
// workgroup takes whole channels, at most Tile elements; each slice of Tile of its threads
// adds every n-th partial sum, 16 loads of each kind in flight at once (the kernel is a
// chain of memory latencies, not of bytes), then LDS joins the slices and a channel's
// components.
constexpr int kSumThreads = 1024;
constexpr int kInFlight = 16;

template <typename T, int Cap, int Tile>
__global__ __launch_bounds__(kSumThreads) void norm_sum_kernel(NormArgs<Cap> a) {
  __shared__ float lds[2][kSumThreads / kWave][Tile];
  __shared__ float col[2][Tile];
  const int k = term_of(a);
  const TermArgs& t = a.term[k];
  const bool want_b = t.b_off >= 0 && a.c.grad_bias;
  const int tile = Tile / t.d * t.d, lane = threadIdx.x % Tile;
  const int first = (int(blockIdx.x) - a.first_block[k]) * tile, slices = int(blockDim.x) / Tile;
  float sw = 0, sb = 0;
  if (lane < tile && first + lane < t.len) {
    const float* part = a.c.part + t.part + first + lane;
    const float* part_b = part + int64_t(t.n_blocks) * t.len;
    for (int b0 = threadIdx.x / Tile; b0 < t.n_blocks; b0 += slices * kInFlight) {
      // past the end the last one is read again and left out: loads under a condition wait
      // for one another
      float vw[kInFlight], vb[kInFlight];
#pragma unroll
      for (int q = 0; q < kInFlight; ++q) vw[q] = part[int64_t(min(b0 + q * slices, t.n_blocks - 1)) * t.len];
      if (want_b) {
#pragma unroll
        for (int q = 0; q < kInFlight; ++q) vb[q] = part_b[int64_t(min(b0 + q * slices, t.n_blocks - 1)) * t.len];
#pragma unroll
        for (int q = 0; q < kInFlight; ++q) sb += b0 + q * slices < t.n_blocks ? vb[q] : 0.0f;
      }
#pragma unroll
      for (int q = 0; q < kInFlight; ++q) sw += b0 + q * slices < t.n_blocks ? vw[q] : 0.0f;
    }
  }
#pragma unroll
  for (int x = Tile; x < kWave; x *= 2) {
    sw += __shfl_xor(sw, x);
    sb += __shfl_xor(sb, x);
  }
  if (threadIdx.x % kWave < Tile) {
    lds[0][threadIdx.x / kWave][lane] = sw;
    lds[1][threadIdx.x / kWave][lane] = sb;
  }
  __syncthreads();
  const int q = threadIdx.x / Tile;
  if (q < 2) {
    float v = 0;
    for (unsigned w = 0; w < blockDim.x / kWave; ++w) v += lds[q][w][lane];
    col[q][lane] = v;
  }
  __syncthreads();
  const int ch = first / t.d + lane;
  if (q < 2 && lane < tile / t.d && ch < t.len / t.d) {
    float v = 0;
    for (int m = 0; m < t.d; ++m) v += col[q][lane * t.d + m];
    if (q == 0 && a.c.grad_weight) store_either<T>(a.c.grad_weight, a.c.weight_f32, t.w_off + ch, v);
    if (q == 1 && want_b) store_either<T>(a.c.grad_bias, a.c.weight_f32, t.b_off + ch, v);
  }
}

// Workgroups of a launch, shared among the terms by their length: enough to keep the
// memory busy, which takes more of them where every access goes to HBM, and in the
// backward no more, since each leaves a row of partial sums.  Measured: forward of 114688 x
// 1312 fp32 232, 222 and 219 us with 1024, 2048 and 4096, of 4096 x 5472 (cached) 38, 36
// and 41; backward and sums of 768 x 9088 (cached) 23.3, 23.3, 25.0 and 27.8 us with 512,
// 768, 1024 and 1536, of 32768 x 704 82, 67, 60 and 56.
constexpr int kForwardBlocks = 2048, kForwardBlocksStream = 4096;
constexpr int kBackwardBlocks = 768, kBackwardBlocksStream = 1536;

int64_t share(int64_t total, const NormShape& p, int k) {
  const int64_t s = total * p.terms[k].len / p.features;
  return s > 0 ? s : 1;
}

// Rows that outgrow the last-level cache pass it by, in plans of up to kCapSmall terms.
template <int Cap>
bool streams(const NormCall& c, const NormShape& p, int elem_bytes, int tensors) {
  return Cap == kCapSmall && c.rows * p.features * elem_bytes * tensors > kCacheBytes;
}

// Rows so few that one workgroup per term takes them all, in at most four turns: it then
// writes the weight's and bias's gradients itself.
bool few_rows(int64_t rows, const NormShape& p, int elem_bytes) {
  for (int k = 0; k < p.n_terms; ++k) {
    const int v = variant_of(p.terms[k].len, elem_bytes, true);
    if (v == kWide || rows > 4 * groups_of(v)) return false;
  }
  return true;
}

// Fills a launch's terms with about `total` workgroups; returns their number and the
// largest number of elements per lane.
template <int Cap>
int fill(NormArgs<Cap>& a, const NormCall& c, const NormShape& p, int elem_bytes, bool backward, int64_t total,
         int* max_e) {
  a.c = c;
  a.direct = backward && few_rows(c.rows, p, elem_bytes);
  a.n_terms = p.n_terms;
  int64_t part = 0;
  int at = 0;
  *max_e = 1;
  for (int k = 0; k < Cap; ++k) a.first_block[k] = 0x7fffffff;
  for (int k = 0; k < p.n_terms; ++k) {
    const NormTerm& t = p.terms[k];
    const int v = variant_of(t.len, elem_bytes, backward), g = groups_of(v);
    const int64_t want = (c.rows + g - 1) / g > 0 ? (c.rows + g - 1) / g : 1;
    const int64_t most = a.direct ? 1 : share(total, p, k);
    const int n = int(want < most ? want : most);
    a.term[k] = TermArgs{t.off, t.len, t.d, t.w_off, t.b_off, v, n,
                         t.d > 1 ? uint32_t(((uint64_t(1) << 32) + uint64_t(t.d) - 1) / uint64_t(t.d)) : 0u, part};
    a.first_block[k] = at;
    at += n;
    part += int64_t(n) * t.len * (t.b_off >= 0 ? 2 : 1);
    *max_e = max(*max_e, elems_of(v, elem_bytes));
  }
  return at;
}

template <typename T, int Cap, bool Stream>
void forward(const NormArgs<Cap>& a, int blocks, int max_e, hipStream_t s) {
  const dim3 grid{unsigned(blocks)}, block(kThreads);
  if (max_e <= 8)
    hipLaunchKernelGGL((norm_fwd_kernel<T, 8, Cap, Stream>), grid, block, 0, s, a);
  else if (max_e <= 16)
    hipLaunchKernelGGL((norm_fwd_kernel<T, 16, Cap, Stream>), grid, block, 0, s, a);
  else
    hipLaunchKernelGGL((norm_fwd_kernel<T, 32, Cap, Stream>), grid, block, 0, s, a);
}
template <typename T, int Cap, bool Stream>
void backward(const NormArgs<Cap>& a, int blocks, int max_e, hipStream_t s) {
  const dim3 grid{unsigned(blocks)}, block(kThreads);
  if (max_e <= 8)
    hipLaunchKernelGGL((norm_bwd_kernel<T, 8, Cap, Stream>), grid, block, 0, s, a);
  else if (max_e <= 16)
    hipLaunchKernelGGL((norm_bwd_kernel<T, 16, Cap, Stream>), grid, block, 0, s, a);
  else
    hipLaunchKernelGGL((norm_bwd_kernel<T, 32, Cap, Stream>), grid, block, 0, s, a);
}

template <typename T, int Cap>
hipError_t forward(const NormCall& c, const NormShape& p, hipStream_t s) {
  NormArgs<Cap> a;
  int max_e;
  const bool stream = streams<Cap>(c, p, int(sizeof(T)), 2);
  const int blocks = fill(a, c, p, int(sizeof(T)), false, stream ? kForwardBlocksStream : kForwardBlocks, &max_e);
  if (stream)
    forward<T, Cap, Cap == kCapSmall>(a, blocks, max_e, s);
  else
    forward<T, Cap, false>(a, blocks, max_e, s);
  return hipGetLastError();
}

template <typename T, int Cap>
hipError_t backward(const NormCall& c, const NormShape& p, hipStream_t s) {
  NormArgs<Cap> a;
  int max_e;
  const bool stream = streams<Cap>(c, p, int(sizeof(T)), 3);
  const int blocks = fill(a, c, p, int(sizeof(T)), true, stream ? kBackwardBlocksStream : kBackwardBlocks, &max_e);
  if (stream)
    backward<T, Cap, Cap == kCapSmall>(a, blocks, max_e, s);
  else
    backward<T, Cap, false>(a, blocks, max_e, s);
  if ((c.grad_weight || c.grad_bias) && !a.direct) {
    // Wide tiles read whole lines (a tile that ends inside one has it fetched again by
    // another die's L2), narrow ones spread short stretches over more workgroups: 9088
    // columns took 10.1 us in tiles of 16 and 5.4 in tiles of 64, 481 columns 6.6 and 10.2.
    int tiles = 0, most = 0;
    for (int k = 0; k < p.n_terms; ++k) {
      tiles += p.terms[k].len / 64;
      most = max(most, a.term[k].n_blocks);
    }
    const int wide = tiles >= 16 ? 64 : 16;
    int at = 0;
    for (int k = 0; k < p.n_terms; ++k) {
      const int tile = wide / p.terms[k].d * p.terms[k].d;
      a.first_block[k] = at;
      at += (p.terms[k].len + tile - 1) / tile;
    }
    // as many slices as keep every load in flight, two at least
    const int want = (most + kInFlight - 1) / kInFlight * wide;
    const int threads = want <= 128 ? 128 : want <= 256 ? 256 : want <= 512 ? 512 : kSumThreads;
    if (wide == 64)
      hipLaunchKernelGGL((norm_sum_kernel<T, Cap, 64>), dim3(unsigned(at)), dim3(unsigned(threads)), 0, s, a);
    else
      hipLaunchKernelGGL((norm_sum_kernel<T, Cap, 16>), dim3(unsigned(at)), dim3(unsigned(threads)), 0, s, a);
  }
  return hipGetLastError();
}

template <typename T>
hipError_t run(const NormCall& c, const NormShape& p, bool back, hipStream_t s) {
  if (p.n_terms <= kCapSmall) return back ? backward<T, kCapSmall>(c, p, s) : forward<T, kCapSmall>(c, p, s);
  return back ? backward<T, kMaxNormTerms>(c, p, s) : forward<T, kMaxNormTerms>(c, p, s);
}
hipError_t run(const NormCall& c, const NormShape& p, Elem type, bool back, hipStream_t s) {
  return type == Elem::f32 ? run<float>(c, p, back, s)
         : type == Elem::bf16 ? run<Bf16>(c, p, back, s) : run<F16>(c, p, back, s);
}

}  // namespace

hipError_t launch_norm_forward(const NormCall& c, const NormShape& p, Elem type, hipStream_t s) {
  return run(c, p, type, false, s);
}

size_t norm_part_floats(int64_t rows, const NormShape& p) {
  if (few_rows(rows, p, 2) && few_rows(rows, p, 4)) return 0;
  size_t n = 0;
  for (int k = 0; k < p.n_terms; ++k)
    n += size_t(std::min(std::max<int64_t>(rows, 1), share(kBackwardBlocksStream, p, k))) * size_t(p.terms[k].len) *
         (p.terms[k].b_off >= 0 ? 2 : 1);
  return n;
}

hipError_t launch_norm_backward(const NormCall& c, const NormShape& p, Elem type, hipStream_t s) {
  return run(c, p, type, true, s);
}

}  // namespace cgtp

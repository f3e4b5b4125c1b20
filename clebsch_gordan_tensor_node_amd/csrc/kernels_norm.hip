// Layer normalisation of rows and of irreps rows term by term, forward and backward.
//
// A row's stretch of F values (a NormTerm: the whole row, or one term's [channels][2l+1]
// block) is normalised by itself:
//   mu = sum(x)/F (centred terms; else 0), s2 = sum((x - mu)^2)/F, rstd = 1/sqrt(s2+eps),
//   h = (x - mu) rstd,  y = h w + b.
// Backward, a = g w:  dx = rstd (a - h sum(a h)/F - sum(a)/F), the last only if centred;
//   dw = sum over rows (and a channel's components) of g h, db = sum over rows of g.
// Sums and statistics are fp32 whatever the element type.  s2 is summed from x - mu, not
// from x^2: a row with a large common offset keeps its digits.  mu, an fp32 sum times the
// rounded 1/F, may miss by some ulp; x - mu is summed along with s2 and corrects both.  A
// constant row (60000 in 7 columns: y off by 0.78 without) is its bias then.
//
// Both passes are bound by HBM: 2 (forward) or 3 (backward) elements moved per element for
// 8 to 14 operations.  So a stretch is read once into registers: G lanes hold it, C
// vectors of 16 bytes each (V elements, the next V G elements after one another), and
// both sums and the output come from there.  Rows need no alignment beyond an element's:
// the hardware takes 16-byte accesses at any element's address.  The last vector of a
// stretch that V does not divide is moved back to end with the stretch; the elements that
// it repeats are left out of the sums, and written twice with the same value.
// A workgroup keeps its weights over all its rows (first its own number, then in strides).
// Measured, with 4.75 TB/s for a large device copy: forward of 114688 x 1312 fp32 212 us
// (5.7 TB/s), of 4096 x 5472 in four terms 37 us (4.8); backward with all gradients of 32768
// x 704 in four terms 54 us (5.1), of 114688 x 128 bf16 22 + 5 us for the sums of the
// weight's gradient, which wait for the memory's latency (as do rows of a few lanes).
#include "elem.hpp"
#include "norm_layout.hpp"

namespace cgtp {
namespace {

constexpr int kWave = 64;

// A term as a launch carries it.
struct TermArgs {
  int32_t off, len, d, w_off, b_off;
  int32_t variant;        // which (V, G, C) handles it
  int32_t n_blocks;       // its workgroups
  int32_t n_parts;        // backward: its partial sums
  uint32_t inv_d;         // ceil(2^32 / d) for d > 1: e / d = (e * inv_d) >> 32 for e < 2^29
  int64_t part;           // backward: its partial sums in `part`: [n_parts][len] of the weight's
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

template <typename T, int V>
struct Vec {
  typedef uint32_t Bits __attribute__((ext_vector_type(sizeof(T) * V / 4), aligned(sizeof(T)), may_alias));
  T v[V];
};
template <>
struct Vec<Bf16, 1> {
  typedef uint16_t Bits __attribute__((may_alias));
  Bf16 v[1];
};
template <>
struct Vec<F16, 1> {
  typedef uint16_t Bits __attribute__((may_alias));
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
// Sum over G neighbouring lanes (4 to 64), to each of them.
template <int G>
__device__ inline float lanes_sum(float v) {
  v += dpp<0xB1>(v);                          // quad_perm 1 0 3 2
  v += dpp<0x4E>(v);                          // quad_perm 2 3 0 1
  if constexpr (G >= 8) v += dpp<0x141>(v);   // row_half_mirror
  if constexpr (G >= 16) v += dpp<0x140>(v);  // row_mirror
  if constexpr (G >= 32) v += __shfl_xor(v, 16);
  if constexpr (G >= 64) v += __shfl_xor(v, 32);
  return v;
}
// The same over a group of G lanes, the whole workgroup for G > 64.  lds: two halves of
// 2 * 16 floats that alternate (`turn`), so that one barrier per sum is enough.
constexpr int kSumLds = 64;
template <int G>
__device__ inline void group_sum2(float& u, float& v, float* lds, int& turn) {
  if constexpr (G <= kWave) {
    u = lanes_sum<G>(u);
    v = lanes_sum<G>(v);
  } else {
    constexpr int kWaves = G / kWave;
    u = lanes_sum<kWave>(u);
    v = lanes_sum<kWave>(v);
    float* l = lds + (turn & 1) * 32;
    turn ^= 1;
    if (threadIdx.x % kWave == 0) {
      l[threadIdx.x / kWave] = u;
      l[kWaves + threadIdx.x / kWave] = v;
    }
    __syncthreads();
    u = v = 0;
#pragma unroll
    for (int k = 0; k < kWaves; ++k) {
      u += l[k];
      v += l[kWaves + k];
    }
  }
}
template <int G>
__device__ inline float group_sum(float v, float* lds, int& turn) {
  float none = 0;
  group_sum2<G>(v, none, lds, turn);
  return v;
}

// The mean from a sum, rounded before anything is taken from it: fused into x - mu it would
// leave differences about another mean than the one that about_mean moves.
__device__ inline float mean_of(float sum, float inv) {
#pragma clang fp contract(off)
  return sum * inv;
}
// Moves mu, a rounded mean, by s1, the mean of x - mu, and returns the variance about it, of
// which s2 is the mean of (x - mu)^2.  Where that is not finite, both stay as they are.
__device__ inline float about_mean(float s1, float s2, float& mu) {
  if (!(s2 < __builtin_inff())) return s2;
  mu += s1;
  return fmaxf(s2 - s1 * s1, 0.0f);
}

// Waits for a row's loads here, on every path.  Left to itself the compiler waits where the
// values are used, and, as some paths use none, again before the registers' next load, for
// the row's store too: 100000 x 704 fp32 in four terms 130 us, with this 107, 32768 rows 41
// and 38.  In 16 bits it costs more than it saves (4096 x 5472 30 and 32 us).
template <int V, int C>
__device__ inline void arrived(float (&x)[C][V]) {
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int j = 0; j < V; ++j) asm volatile("" : "+v"(x[c][j]));
}
// Takes `by` off the lane's elements.
template <int V, int C>
__device__ inline void shift(float (&x)[C][V], float by) {
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int j = 0; j < V; ++j) x[c][j] -= by;
}

// Where a lane's vectors of a stretch lie.
template <int V, int G, int C>
struct Place {
  int lane, len, last;   // last: the chunk that holds the stretch's end (the same in all lanes)
  // first: that chunk is known to be the first.  With C = 1 it always is; the backward, which
  // waits for its loads where it tests it, is slower if told so (32768 x 704 fp32 55.5 us, 54.4).
  __device__ Place(int n, bool first) : lane(threadIdx.x % G), len(n), last(first ? 0 : (n - 1) / (V * G)) {}
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
// Adds the lane's own elements to s1, and their squares to s2.
template <int V, int G, int C>
__device__ inline void own_sums(const Place<V, G, C>& p, const float (&x)[C][V], float& s1, float& s2) {
#pragma unroll
  for (int c = 0; c < C; ++c) {
    if (c < p.last) {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        s1 += x[c][j];
        s2 += x[c][j] * x[c][j];
      }
    } else if (c == p.last) {
      const bool has = p.has(c);
      const int skip = p.skip(c);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float v = has && j >= skip ? x[c][j] : 0.0f;
        s1 += v;
        s2 += v * v;
      }
    }
  }
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

template <int B, bool Stream, typename T, int V, int G, int C>
__device__ inline void fwd_rows(const NormCall& a, const TermArgs& t, int n_terms, int index, int block, float* lds) {
  constexpr int kGroups = B / G;
  const Place<V, G, C> p(t.len, C == 1);
  const bool centred = t.b_off >= 0;
  const float inv = 1.0f / float(t.len);
  float w[C][V], b[C][V], x[C][V];
  load_weights<T>(p, a.weight, a.weight_f32, t.w_off, t, 1.0f, w);
  load_weights<T>(p, centred ? a.bias : nullptr, a.weight_f32, t.b_off, t, 0.0f, b);
  int turn = 0;
  for (int64_t r = int64_t(block) * kGroups + threadIdx.x / G; r < a.rows; r += int64_t(t.n_blocks) * kGroups) {
    widen(read_row<Stream>(p, static_cast<const T*>(a.x) + r * a.ld_x + t.off), x);
    if constexpr (sizeof(T) == 4) arrived(x);
    float mu = 0, s1 = 0, s2 = 0;
    if (centred) {
      mu = mean_of(group_sum<G>(own_sum(p, [&](int c, int j) { return x[c][j]; }), lds, turn), inv);
      shift(x, mu);
    }
    own_sums(p, x, s1, s2);
    group_sum2<G>(s1, s2, lds, turn);
    float var = s2 * inv;
    if (centred) {
      const float first = mu;
      var = about_mean(s1 * inv, var, mu);
      shift(x, mu - first);   // x - mu now, of the mean that the stats hold
    }
    const float rstd = 1.0f / sqrtf(var + a.eps);
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int j = 0; j < V; ++j) x[c][j] = x[c][j] * rstd * w[c][j] + b[c][j];
    store_row<Stream>(p, static_cast<T*>(a.y) + r * a.ld_y + t.off, x);
    if (a.stats && p.lane == 0) {
      a.stats[r * n_terms + index] = mu;
      a.stats[(a.rows + r) * n_terms + index] = rstd;
    }
  }
}

// The weights wait in LDS, a vector to each lane's place: they are used once per row, and in
// registers they would leave fewer waves.
template <int B, bool Stream, typename T, int V, int G, int C>
__device__ inline void bwd_rows(const NormCall& a, const TermArgs& t, int n_terms, int index, int block, float* lds,
                                float* sums, bool direct) {
  constexpr int kGroups = B / G;
  const Place<V, G, C> p(t.len, false);
  const bool centred = t.b_off >= 0;
  const float inv = 1.0f / float(t.len);
  float x[C][V], g[C][V], gw[C][V], gb[C][V];
  if (threadIdx.x < G) {
    load_weights<T>(p, a.weight, a.weight_f32, t.w_off, t, 1.0f, x);
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int j = 0; j < V; ++j) lds[p.start(c) + j] = x[c][j];
  }
  __syncthreads();
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
        g[c][j] *= lds[p.start(c) + j];
      }
    if (!a.y) continue;
    float sa = own_sum(p, [&](int c, int j) { return g[c][j]; });
    float sh = own_sum(p, [&](int c, int j) { return g[c][j] * x[c][j]; });
    group_sum2<G>(sa, sh, sums, turn);
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
  for (int k = 0; k < (centred ? 2 : 1); ++k, part += int64_t(t.n_parts) * t.len) {
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
    for (int e = threadIdx.x; e < t.len / d; e += B) {
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

// Stretches of any length, in launches of their own: one workgroup per row, which is read
// again (from the caches, mostly) for each sum.
constexpr int kWideBlock = 1024;
// Calls f(first element, elements) for the thread's vectors.
template <int B, int V, typename F>
__device__ inline void wide_loop(int len, F&& f) {
  for (int e = int(threadIdx.x) * V; e < len; e += B * V) f(e, min(V, len - e));
}
template <int V, typename T>
__device__ inline void read_some(const T* p, int n, float (&v)[V]) {
  if (n == V) {
    const Vec<T, V> r = load_vec<false, T, V>(p);
#pragma unroll
    for (int j = 0; j < V; ++j) v[j] = to_f32(r.v[j]);
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) v[j] = j < n ? to_f32(p[j]) : 0.0f;
  }
}
template <int V, typename T>
__device__ inline void write_some(T* p, int n, const float (&v)[V]) {
  Vec<T, V> r;
#pragma unroll
  for (int j = 0; j < V; ++j) r.v[j] = from_f32<T>(v[j]);
  if (n == V) {
    store_vec<false, T, V>(p, r);
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (j < n) p[j] = r.v[j];
  }
}
// The weights (biases) of the n elements from e on, `none` where there are none.
template <int V, typename T>
__device__ inline void some_weights(const void* w, int f32, int off, const TermArgs& t, int e, int n, float none,
                                    float (&out)[V]) {
  if (w && f32 && t.d == 1 && n == V) {
#pragma unroll
    for (int q = 0; q < V; q += 4) {
      const Vec<float, 4> r = load_vec<false, float, 4>(static_cast<const float*>(w) + off + e + q);
#pragma unroll
      for (int j = 0; j < 4; ++j) out[q + j] = r.v[j];
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < V; ++j) {
    out[j] = none;
    if (w && j < n) out[j] = load_either<T>(w, f32, off + (t.d == 1 ? e + j : int(__umulhi(uint32_t(e + j), t.inv_d))));
  }
}

template <typename T>
__global__ __launch_bounds__(kWideBlock) void norm_fwd_wide_kernel(NormCall a, TermArgs t, int n_terms, int index) {
  __shared__ float sums[kSumLds];
  constexpr int B = kWideBlock;
  constexpr int V = 16 / int(sizeof(T));
  const bool centred = t.b_off >= 0;
  const float inv = 1.0f / float(t.len);
  int turn = 0;
  float v[V];
  for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + r * a.ld_x + t.off;
    T* y = static_cast<T*>(a.y) + r * a.ld_y + t.off;
    float mu = 0, s1 = 0, s2 = 0;
    if (centred) {
      float s = 0;
      wide_loop<B, V>(t.len, [&](int e, int n) {
        read_some<V>(x + e, n, v);
#pragma unroll
        for (int j = 0; j < V; ++j) s += v[j];
      });
      mu = mean_of(group_sum<B>(s, sums, turn), inv);
    }
    wide_loop<B, V>(t.len, [&](int e, int n) {
      read_some<V>(x + e, n, v);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float d = j < n ? v[j] - mu : 0.0f;
        s1 += d;
        s2 += d * d;
      }
    });
    group_sum2<B>(s1, s2, sums, turn);
    const float var = centred ? about_mean(s1 * inv, s2 * inv, mu) : s2 * inv;
    const float rstd = 1.0f / sqrtf(var + a.eps);
    wide_loop<B, V>(t.len, [&](int e, int n) {
      float w[V], b[V];
      read_some<V>(x + e, n, v);
      some_weights<V, T>(a.weight, a.weight_f32, t.w_off, t, e, n, 1.0f, w);
      some_weights<V, T>(centred ? a.bias : nullptr, a.weight_f32, t.b_off, t, e, n, 0.0f, b);
#pragma unroll
      for (int j = 0; j < V; ++j) v[j] = (v[j] - mu) * rstd * w[j] + b[j];
      write_some<V>(y + e, n, v);
    });
    if (a.stats && threadIdx.x == 0) {
      a.stats[r * n_terms + index] = mu;
      a.stats[(a.rows + r) * n_terms + index] = rstd;
    }
  }
}
// dx only: norm_wide_w_kernel adds the weight's gradient.
template <typename T>
__global__ __launch_bounds__(kWideBlock) void norm_bwd_wide_kernel(NormCall a, TermArgs t, int n_terms, int index) {
  __shared__ float sums[kSumLds];
  constexpr int B = kWideBlock;
  constexpr int V = 16 / int(sizeof(T));
  const bool centred = t.b_off >= 0;
  const float inv = 1.0f / float(t.len);
  int turn = 0;
  float xv[V], gv[V];
  for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + r * a.ld_x + t.off;
    const T* g = static_cast<const T*>(a.grad_out) + r * a.ld_g + t.off;
    T* y = static_cast<T*>(a.y) + r * a.ld_y + t.off;
    const float mu = a.stats[r * n_terms + index], rstd = a.stats[(a.rows + r) * n_terms + index];
    auto read = [&](int e, int n) {   // h and a = g w
      float w[V];
      read_some<V>(x + e, n, xv);
      read_some<V>(g + e, n, gv);
      some_weights<V, T>(a.weight, a.weight_f32, t.w_off, t, e, n, 1.0f, w);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        xv[j] = (xv[j] - mu) * rstd;
        gv[j] *= w[j];
      }
    };
    float sa = 0, sh = 0;
    wide_loop<B, V>(t.len, [&](int e, int n) {
      read(e, n);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        sa += j < n ? gv[j] : 0.0f;
        sh += j < n ? gv[j] * xv[j] : 0.0f;
      }
    });
    group_sum2<B>(sa, sh, sums, turn);
    sa = centred ? sa * inv : 0.0f;
    sh *= inv;
    wide_loop<B, V>(t.len, [&](int e, int n) {
      read(e, n);
#pragma unroll
      for (int j = 0; j < V; ++j) gv[j] = (gv[j] - sa - xv[j] * sh) * rstd;
      write_some<V>(y + e, n, gv);
    });
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

// One launch for all terms; a kernel holds the variants of up to E elements per lane, so
// that short rows do not pay for long ones' registers.
#define CGTP_NORM_VARIANTS(FN, ...)                                                                     \
  constexpr int V = 16 / int(sizeof(T));                                                                \
  switch (t.variant) {                                                                                  \
    case kElem8: FN<B, Stream, T, 1, 8, 1>(a.c, t, a.n_terms, k, block, lds, ##__VA_ARGS__); break;     \
    case kG4C1: FN<B, Stream, T, V, 4, 1>(a.c, t, a.n_terms, k, block, lds, ##__VA_ARGS__); break;      \
    case kG8C1: FN<B, Stream, T, V, 8, 1>(a.c, t, a.n_terms, k, block, lds, ##__VA_ARGS__); break;      \
    case kG16C1: FN<B, Stream, T, V, 16, 1>(a.c, t, a.n_terms, k, block, lds, ##__VA_ARGS__); break;    \
    case kG32C1: FN<B, Stream, T, V, 32, 1>(a.c, t, a.n_terms, k, block, lds, ##__VA_ARGS__); break;    \
    case kG64C1: FN<B, Stream, T, V, 64, 1>(a.c, t, a.n_terms, k, block, lds, ##__VA_ARGS__); break;    \
    case kGBC1: FN<B, Stream, T, V, B, 1>(a.c, t, a.n_terms, k, block, lds, ##__VA_ARGS__); break;      \
    default:                                                                                            \
      if constexpr (E >= 2 * V) {                                                                       \
        if (t.variant == kG64C2) FN<B, Stream, T, V, 64, 2>(a.c, t, a.n_terms, k, block, lds, ##__VA_ARGS__); \
        if (t.variant == kGBC2) FN<B, Stream, T, V, B, 2>(a.c, t, a.n_terms, k, block, lds, ##__VA_ARGS__);   \
      }                                                                                                 \
      if constexpr (E >= 4 * V) {                                                                       \
        if (t.variant == kG64C4) FN<B, Stream, T, V, 64, 4>(a.c, t, a.n_terms, k, block, lds, ##__VA_ARGS__); \
        if (t.variant == kGBC4) FN<B, Stream, T, V, B, 4>(a.c, t, a.n_terms, k, block, lds, ##__VA_ARGS__);   \
      }                                                                                                 \
  }

template <typename T, int B, int E, int Cap, bool Stream>
__global__ __launch_bounds__(B) void norm_fwd_kernel(NormArgs<Cap> a) {
  __shared__ float lds[kSumLds];
  const int k = term_of(a);
  const TermArgs& t = a.term[k];
  const int block = int(blockIdx.x) - a.first_block[k];
  CGTP_NORM_VARIANTS(fwd_rows)
}

// 16 elements of 16 bits a lane fit the registers of 4 waves per SIMD without spilling (8138
// x 8192 133 us, 162 with the compiler's 3); 16 of 32 bits do not (1024 columns: 96 us, 86
// with 3).
template <typename T, int B, int E, int Cap, bool Stream>
__global__ __launch_bounds__(B, E > 8 && sizeof(T) == 2 ? 4 : 1) void norm_bwd_kernel(NormArgs<Cap> a) {
  __shared__ __align__(16) float lds[B * E];
  __shared__ float sums[kSumLds];
  const int k = term_of(a);
  const TermArgs& t = a.term[k];
  const int block = int(blockIdx.x) - a.first_block[k];
  CGTP_NORM_VARIANTS(bwd_rows, sums, a.direct)
}

// The partial sums of wide stretches, column by column: a thread's column over every
// kWideSlices-th row.
constexpr int kWideThreads = 256;
template <typename T>
__global__ __launch_bounds__(kWideThreads) void norm_wide_w_kernel(NormCall a, TermArgs t, int n_terms, int index) {
  const int e = int(blockIdx.x) * kWideThreads + int(threadIdx.x);
  if (e >= t.len) return;
  const T* x = static_cast<const T*>(a.x) + t.off + e;
  const T* g = static_cast<const T*>(a.grad_out) + t.off + e;
  float sw = 0, sb = 0;
#pragma unroll 4
  for (int64_t r = blockIdx.y; r < a.rows; r += kWideSlices) {
    const float v = to_f32(g[r * a.ld_g]);
    sw += v * ((to_f32(x[r * a.ld_x]) - a.stats[r * n_terms + index]) * a.stats[(a.rows + r) * n_terms + index]);
    sb += v;
  }
  float* part = a.part + t.part + int64_t(blockIdx.y) * t.len + e;
  part[0] = sw;
  if (t.b_off >= 0) part[int64_t(t.n_parts) * t.len] = sb;
}

// The weight's and bias's gradients from the workgroups' sums, in a fixed order.  A
// workgroup takes whole channels, at most Tile elements; each slice of Tile of its threads
// adds every n-th partial sum, 16 loads of each kind in flight at once (the kernel is a
// chain of memory latencies, not of bytes), then LDS joins the slices and a channel's
// components.
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
    const float* part_b = part + int64_t(t.n_parts) * t.len;
    for (int b0 = threadIdx.x / Tile; b0 < t.n_parts; b0 += slices * kInFlight) {
      // past the end the last one is read again and left out: loads under a condition wait
      // for one another
      float vw[kInFlight], vb[kInFlight];
#pragma unroll
      for (int q = 0; q < kInFlight; ++q) vw[q] = part[int64_t(min(b0 + q * slices, t.n_parts - 1)) * t.len];
      if (want_b) {
#pragma unroll
        for (int q = 0; q < kInFlight; ++q) vb[q] = part_b[int64_t(min(b0 + q * slices, t.n_parts - 1)) * t.len];
#pragma unroll
        for (int q = 0; q < kInFlight; ++q) sb += b0 + q * slices < t.n_parts ? vb[q] : 0.0f;
      }
#pragma unroll
      for (int q = 0; q < kInFlight; ++q) sw += b0 + q * slices < t.n_parts ? vw[q] : 0.0f;
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

// A launch's arguments; returns its workgroups.
template <int Cap>
int fill(NormArgs<Cap>& a, const NormCall& c, const NormShape& p, const Layout& y) {
  a.c = c;
  a.n_terms = p.n_terms;
  a.direct = y.direct;
  int64_t part = 0;
  int at = 0;
  for (int k = 0; k < Cap; ++k) a.first_block[k] = 0x7fffffff;
  for (int k = 0; k < p.n_terms; ++k) {
    const NormTerm& t = p.terms[k];
    a.term[k] = TermArgs{t.off, t.len, t.d, t.w_off, t.b_off, y.variant[k], y.n_blocks[k], y.n_parts[k],
                         t.d > 1 ? uint32_t(((uint64_t(1) << 32) + uint64_t(t.d) - 1) / uint64_t(t.d)) : 0u, part};
    a.first_block[k] = at;
    at += y.n_blocks[k];
    part += int64_t(y.n_parts[k]) * t.len * (t.b_off >= 0 ? 2 : 1);
  }
  return at;
}

// More than 8 elements a lane: the pairs of type and workgroup that elems_of asks for.
template <typename T, int Cap, bool Stream>
void forward(const NormArgs<Cap>& a, int blocks, const Layout& y, hipStream_t s) {
  const dim3 grid{unsigned(blocks)}, block{unsigned(y.block)};
  if (y.max_e > 8) {
    if constexpr (sizeof(T) == 4) {
      if (y.block == 512) {
        hipLaunchKernelGGL((norm_fwd_kernel<T, 512, kMaxE, Cap, Stream>), grid, block, 0, s, a);
        return;
      }
    }
    hipLaunchKernelGGL((norm_fwd_kernel<T, 1024, kMaxE, Cap, Stream>), grid, block, 0, s, a);
    return;
  }
  if (y.block == 256)
    hipLaunchKernelGGL((norm_fwd_kernel<T, 256, 8, Cap, Stream>), grid, block, 0, s, a);
  else if (y.block == 512)
    hipLaunchKernelGGL((norm_fwd_kernel<T, 512, 8, Cap, Stream>), grid, block, 0, s, a);
  else if (y.block == 1024)
    hipLaunchKernelGGL((norm_fwd_kernel<T, 1024, 8, Cap, Stream>), grid, block, 0, s, a);
  else
    hipLaunchKernelGGL((norm_fwd_kernel<T, 128, 8, Cap, Stream>), grid, block, 0, s, a);
}
template <typename T, int Cap, bool Stream>
void backward(const NormArgs<Cap>& a, int blocks, const Layout& y, hipStream_t s) {
  const dim3 grid{unsigned(blocks)}, block{unsigned(y.block)};
  constexpr int kB = sizeof(T) == 4 ? 256 : 512;
  if (y.max_e > 8) {
    if (y.block == kB)
      hipLaunchKernelGGL((norm_bwd_kernel<T, kB, kMaxE, Cap, Stream>), grid, block, 0, s, a);
    else
      hipLaunchKernelGGL((norm_bwd_kernel<T, 1024, kMaxE, Cap, Stream>), grid, block, 0, s, a);
    return;
  }
  if (y.block == 256)
    hipLaunchKernelGGL((norm_bwd_kernel<T, 256, 8, Cap, Stream>), grid, block, 0, s, a);
  else if (y.block == 512)
    hipLaunchKernelGGL((norm_bwd_kernel<T, 512, 8, Cap, Stream>), grid, block, 0, s, a);
  else if (y.block == 1024)
    hipLaunchKernelGGL((norm_bwd_kernel<T, 1024, 8, Cap, Stream>), grid, block, 0, s, a);
  else
    hipLaunchKernelGGL((norm_bwd_kernel<T, 128, 8, Cap, Stream>), grid, block, 0, s, a);
}

unsigned wide_blocks(int64_t rows) { return unsigned(std::min<int64_t>(rows, kForwardBlocks)); }

template <typename T, int Cap>
hipError_t forward(const NormCall& c, const NormShape& p, hipStream_t s) {
  NormArgs<Cap> a;
  const Layout y = lay_out(c.rows, p, int(sizeof(T)), false);
  const int blocks = fill(a, c, p, y);
  for (int k = 0; k < p.n_terms; ++k)
    if (y.variant[k] == kWide)
      hipLaunchKernelGGL(norm_fwd_wide_kernel<T>, dim3(wide_blocks(c.rows)), dim3(kWideBlock), 0, s, c, a.term[k],
                         p.n_terms, k);
  if (blocks == 0) return hipGetLastError();
  if (y.stream)
    forward<T, Cap, Cap == kCapSmall>(a, blocks, y, s);
  else
    forward<T, Cap, false>(a, blocks, y, s);
  return hipGetLastError();
}

template <typename T, int Cap>
hipError_t backward(const NormCall& c, const NormShape& p, hipStream_t s) {
  NormArgs<Cap> a;
  const Layout y = lay_out(c.rows, p, int(sizeof(T)), true);
  const int blocks = fill(a, c, p, y);
  for (int k = 0; k < p.n_terms; ++k)
    if (y.variant[k] == kWide && c.y && c.rows > 0)
      hipLaunchKernelGGL(norm_bwd_wide_kernel<T>, dim3(wide_blocks(c.rows)), dim3(kWideBlock), 0, s, c, a.term[k],
                         p.n_terms, k);
  if (blocks > 0 && y.stream)
    backward<T, Cap, Cap == kCapSmall>(a, blocks, y, s);
  else if (blocks > 0)
    backward<T, Cap, false>(a, blocks, y, s);
  if ((c.grad_weight || c.grad_bias) && !y.direct) {
    for (int k = 0; k < p.n_terms; ++k)
      if (y.variant[k] == kWide) {
        const dim3 grid(unsigned((p.terms[k].len + kWideThreads - 1) / kWideThreads), kWideSlices);
        hipLaunchKernelGGL(norm_wide_w_kernel<T>, grid, dim3(kWideThreads), 0, s, c, a.term[k], p.n_terms, k);
      }
    const SumGrid g = lay_out_sums(p, y);
    int at = 0;
    for (int k = 0; k < p.n_terms; ++k) {
      a.first_block[k] = at;
      at += sum_blocks(p.terms[k], g.tile);
    }
    const dim3 grid{unsigned(g.blocks)}, block{unsigned(g.threads)};
    if (g.tile == 64)
      hipLaunchKernelGGL((norm_sum_kernel<T, Cap, 64>), grid, block, 0, s, a);
    else
      hipLaunchKernelGGL((norm_sum_kernel<T, Cap, 16>), grid, block, 0, s, a);
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
  // whatever the element type
  return size_t(std::max(lay_out(rows, p, 2, true).part, lay_out(rows, p, 4, true).part));
}

hipError_t launch_norm_backward(const NormCall& c, const NormShape& p, Elem type, hipStream_t s) {
  return run(c, p, type, true, s);
}

}  // namespace cgtp

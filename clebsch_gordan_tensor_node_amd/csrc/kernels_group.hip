// Group normalisation of rows, channels last, with an activation: forward and backward.
//
// Over the M values of one sample (a range of rows) and one group (a range of c columns):
//   mu = sum(x)/M, s2 = sum((x - mu)^2)/M, rstd = 1/sqrt(s2 + eps), h = (x - mu) rstd,
//   z = h w + b, y = act(z).
// Backward, d = g act'(z), a = d w:  dx = rstd (a - sum(a)/M - h sum(a h)/M),
//   dw = sum over rows of d h, db = sum over rows of d.
// sum(a) and sum(a h) are the weighted sums of a sample's sums of d and d h per channel, so
// the backward sums d and d h per channel only, once, and all four gradients come from them.
//
// Statistics are fp32, and never a difference of large sums: a thread sums x - K and its square,
// K its first value of the channel.  As K is one of its n values, (K - mean)^2 <= M2, the sum
// of squares about the mean, so that sum (x - K)^2 = M2 + n (K - mean)^2 <= (n + 1) M2: the
// difference that gives M2 loses at most a factor n + 1 of the rounding.  A thread of more than
// kRun = 64 rows (a sample far longer than told; 128 columns from some 2 million rows on) closes
// its sums after each 64: K becomes the mean so far, exactly accounted for, and the squares go to
// a sum of their own.  The factor is 65 at most in the first run and 2 from then on, where the mean
// of m >= 64 rows is K and at most 64 follow: n (K - mean)^2 <= (64 / m) M2.  Of 60000 rows of a
// thread with eight first ones 100 deviations off, rstd is right to 6e-8; in one chain it was to
// 3e-4.  The backward's sums are closed as often, so that their chains are of 64 and n / 64.
// Threads' and workgroups' means and M2 are joined about the first of them, then about the joint
// mean.  A constant sample's mean is exact this way, and y = act(bias).
//
// Columns are a thread's own (four of them), rows are dealt out among a workgroup's
// slices: accesses run along the rows whatever the group's width, and a place may straddle
// groups.  A sample that the registers of one workgroup hold is read once, in one launch.
// Longer ones are cut into tiles of rows whose sums a second launch joins and a third applies,
// reading the rows again.
//
// Both passes move 2 to 3 elements for each that they sum: the caches' and HBM's rate bounds
// them, and in 16 bits the arithmetic of the activations beside it.  Measured, sums, join and
// output in us: forward of 561680 x 128 fp32 in 28 samples 53 + 5 + 93 (5.4 and 6.2 TB/s), of
// 114688 x 128 bf16 in one 9 + 4 + 14; backward of 20060 x 481 fp32 in 48 samples 21 + 6 + 24,
// of 114688 x 128 bf16 with gelu 20 + 6 + 22 (its vector units 75 % busy: two transcendental
// functions of four cycles each beside some 25 operations a value and pass).  418 x 64 in one
// launch of 6.3.  Tried and not kept: loads of the next rows ahead of the sums (45 and 48 us
// for the bf16 backward without and with), and 2, 4 and 8 columns a thread in 16 bits (30, 27
// and 31 us for that forward: eight columns' statistics leave too few waves).
#include <type_traits>

#include "group_layout.hpp"
#include "vec.hpp"

namespace cgtp {
namespace {

// exp(x): 2^t with t = x log2(e) rounded, in fp32 times e^(x - t ln 2), of which 1 and the small
// exponent are enough (some 2 ulp; in 16 bits an error of |x| 2^-24 of it is nothing).  Beyond
// 200 it is 0 or infinity either way.
template <bool Exact>
__device__ inline float exp_of(float x) {
  constexpr float kLog2e = 1.44269504f, kLn2 = 0.693147181f;
  if constexpr (!Exact) return __builtin_amdgcn_exp2f(x * kLog2e);
  x = __builtin_amdgcn_fmed3f(x, -200.0f, 200.0f);
  const float t = x * kLog2e;
  return __builtin_amdgcn_exp2f(t) * (1.0f + fmaf(t, -kLn2, x));
}
// (1 + erf(z / sqrt 2)) / 2 and exp(-z^2 / 2), by q = exp(-z^2 / 2) times a polynomial in t = 1 /
// (1 + p |z|): q where z < 0, else 1 - q.  In 16 bits Abramowitz and Stegun's (Handbook of
// Mathematical Functions, 7.1.26), to 7.5e-8 of 1: nothing beside their rounding.  In 32 bits one of
// degree 9, fitted to the least greatest error of q itself, 3.2e-8.  GELU is off by 1.6e-8 in the
// mean over normal z, by erff 1.5e-8 (which loses all digits of the far negative ones; these keep
// theirs to 1.3e-6), by the shorter polynomial 3.9e-8; the slope by 2.9e-8, 2.0e-8 and 5.4e-8.
// 561680 x 128 fp32 in 28 samples, forward: 151.8 us, with erff 153.9, the shorter 151.0; 24000 x
// 128 in 24: 15.7, 18.2, 15.6; backward of 20060 x 481 in 48: 52.9, 59.3, 52.0.
template <bool Exact>
__device__ inline float normal_cdf(float z, float& density) {
  float t, q;
  if constexpr (Exact) {
    density = exp_of<true>(-0.5f * z * z);
    t = __builtin_amdgcn_rcpf(fmaf(fabsf(z), 0.35f, 1.0f));
    q = fmaf(t, -0.0291652586f, 0.144067422f);
    q = fmaf(t, q, -0.25591585f);
    q = fmaf(t, q, 0.159409285f);
    q = fmaf(t, q, -0.0232754126f);
    q = fmaf(t, q, 0.105579846f);
    q = fmaf(t, q, 0.11981418f);
    q = fmaf(t, q, 0.139864519f);
    q = fmaf(t, q, 0.139621243f);
  } else {
    density = __builtin_amdgcn_exp2f(z * z * (-0.5f * 1.44269504f));
    t = __builtin_amdgcn_rcpf(fmaf(fabsf(z), 0.3275911f * 0.707106781f, 1.0f));
    q = fmaf(t, 0.5f * 1.061405429f, 0.5f * -1.453152027f);
    q = fmaf(t, q, 0.5f * 1.421413741f);
    q = fmaf(t, q, 0.5f * -0.284496736f);
    q = fmaf(t, q, 0.5f * 0.254829592f);
  }
  q *= t * density;
  return z < 0 ? q : 1.0f - q;
}

template <Act A, bool Exact>
__device__ inline float act_value(float z) {
  if constexpr (A == Act::silu) return z * __builtin_amdgcn_rcpf(1.0f + exp_of<Exact>(-z));
  if constexpr (A == Act::gelu) {
    float density;
    return z * normal_cdf<Exact>(z, density);
  }
  return z;
}
template <Act A, bool Exact>
__device__ inline float act_slope(float z) {
  if constexpr (A == Act::silu) {
    const float p = __builtin_amdgcn_rcpf(1.0f + exp_of<Exact>(-z));
    return fmaf(z * p, 1.0f - p, p);
  }
  if constexpr (A == Act::gelu) {
    float density;
    const float p = normal_cdf<Exact>(z, density);
    return fmaf(z * 0.398942280f, density, p);
  }
  return 1.0f;
}
// f with the activation as a constant: one branch for what f does, the same for all lanes.
template <typename F>
__device__ inline void with_act(Act act, F&& f) {
  if (act == Act::silu)
    f(std::integral_constant<Act, Act::silu>{});
  else if (act == Act::gelu)
    f(std::integral_constant<Act, Act::gelu>{});
  else
    f(std::integral_constant<Act, Act::none>{});
}

__device__ inline int sample_begin(const GroupCall& c, const GroupLayout& y, int64_t s) {
  if (!c.offsets) return int(s * y.equal);
  return min(max(c.offsets[s], 0), int(c.rows));
}
// Never before the sample's begin, nor past the rows, whatever the offsets hold.
__device__ inline int sample_end(const GroupCall& c, const GroupLayout& y, int64_t s, int begin) {
  if (!c.offsets) return int((s + 1) * y.equal);
  return min(max(c.offsets[s + 1], begin), int(c.rows));
}
// The first sample that ends behind `row` (samples, if none does): 64 lanes probe at once.
__device__ inline int64_t sample_behind(const GroupCall& c, const GroupLayout& y, int row) {
  if (!c.offsets) return y.equal ? row / y.equal : 0;
  const int64_t lane = threadIdx.x % kWave;
  int64_t lo = 0, n = c.samples;
  while (n > 0) {
    const int64_t step = (n + kWave - 1) / kWave;
    const int64_t at = min((lane + 1) * step, n) - 1;
    const bool before = lane * step < n && c.offsets[lo + at + 1] <= row;
    const int64_t passed = min(__popcll(__ballot(before)) * step, n);
    lo += passed;
    n = step == 1 ? 0 : min(step - 1, n - passed);   // the probed one itself ends behind
  }
  return lo;
}

// The columns of a chunk, and the groups (or the part of one) in it.
struct Chunk {
  int c0, cw;        // first column, columns
  int u0;            // first unit: a group, or a part of one
  int nu, uw;        // units, and the columns of each
};
__device__ inline Chunk chunk_of(const GroupCall& c, const GroupLayout& y, int k) {
  Chunk q;
  if (y.split == 1) {
    q.u0 = k * y.per_chunk;
    q.nu = min(y.per_chunk, int(c.groups) - q.u0);
    q.uw = y.per_group;
    q.c0 = q.u0 * y.per_group;
    q.cw = q.nu * q.uw;
  } else {
    const int g = k / y.split, in = (k - g * y.split) * y.part;
    q.u0 = k;
    q.nu = 1;
    q.c0 = g * y.per_group + in;
    q.cw = q.uw = min(y.part, y.per_group - in);
  }
  return q;
}

// A thread's place: V columns from `at` on, of which [own, end) are its own.  The last place of
// a chunk that V does not divide is moved back to end with the chunk (but not before the row).
template <int V>
struct Place {
  int slice;
  bool in;           // has a place
  int at;            // first column in the row
  int rel;           // the same in the chunk (may be negative)
  int own, end;
  __device__ Place(const Chunk& q, const GroupLayout& y) {
    slice = int(threadIdx.x) / y.lanes;
    const int lane = int(threadIdx.x) - slice * y.lanes;
    const int start = lane * V;
    in = slice < y.slices && start < q.cw;
    rel = min(start, q.cw - V);
    if (q.c0 + rel < 0) rel = -q.c0;
    at = q.c0 + rel;
    own = start - rel;
    end = min(V, q.cw - rel);
  }
  __device__ bool whole() const { return own == 0 && end == V; }
  __device__ bool has(int j) const { return j >= own && j < end; }
};

// stream: past the caches (the same for all lanes).
template <typename T, int V>
__device__ inline void store_own(const Place<V>& p, T* row, const float (&v)[V], int stream) {
  Vec<T, V> r;
#pragma unroll
  for (int j = 0; j < V; ++j) r.v[j] = from_f32<T>(v[j]);
  if (p.whole()) {
    if (stream) {
      // the marks keep the compiler from making one ordinary store of the two
      asm volatile("");
      store_vec<true, T, V>(row + p.at, r);
      asm volatile("");
    } else {
      store_vec<false, T, V>(row + p.at, r);
    }
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (p.has(j)) row[p.at + j] = r.v[j];
  }
}

// Weights (biases) at a place; `none` where there are none.
template <typename T, int V>
__device__ inline void place_weights(const Place<V>& p, const void* w, int f32, float none, float (&out)[V]) {
#pragma unroll
  for (int j = 0; j < V; ++j) out[j] = w && p.in && p.has(j) ? load_either<T>(w, f32, p.at + j) : none;
}

__device__ inline float wave_sum(float v) { return lanes_sum<kWave>(v); }

// ---- statistics --------------------------------------------------------------------

// Rows of a thread whose sums are one chain of additions.
constexpr int kRun = 64;
// A thread's sums of closed runs, in LDS: registers for what few calls have would cost all calls
// waves (4 to 3 of the 16-bit backward).  Places B apart, one for each thread, and nobody else's.
template <int B>
__device__ inline void keep(float* own, int place, float v, bool first) {
  own[place * B] = first ? v : own[place * B] + v;
}

// Sums of x - K and of its square over a thread's rows of a sample.
template <int V>
struct Shifted {
  float k[V], s[V], q[V];
  __device__ void clear() {
#pragma unroll
    for (int j = 0; j < V; ++j) k[j] = s[j] = q[j] = 0;
  }
  __device__ void add(const float (&x)[V]) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const float d = x[j] - k[j];
      s[j] += d;
      q[j] = fmaf(d, d, q[j]);
    }
  }
  // After n rows: K moves by m to their mean, as nearly as it is a number, and with it
  // sum (x - K) to s - n m, sum (x - K)^2 by -m (s + (s - n m)); q goes to the thread's own LDS.
  template <int B>
  __device__ void close(int rows, float* own) {
    const float n = float(rows), inv = 1.0f / n;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const float mean = fmaf(s[j], inv, k[j]), m = mean - k[j], left = fmaf(-n, m, s[j]);
      keep<B>(own, j, fmaf(-m, s[j] + left, q[j]), rows == kRun);
      k[j] = mean;
      s[j] = left;
      q[j] = 0;
    }
  }
  template <int B>
  __device__ void join(const float* own) {
#pragma unroll
    for (int j = 0; j < V; ++j) q[j] += own[j * B];
  }
};

// What a workgroup's threads have of one sample, in LDS: a mean and an M2 for each slice and
// column, or, where no place straddles units, for each slice and place.
struct Entries {
  float* mean;
  float* m2;
  int stride;     // entries of a slice
  int per_unit;   // entries of a slice and unit
  float weight;   // values of an entry per row
  int n;          // rows of the sample here
  float each;     // of which each slice has so many, and the first `more` one more
  int more, slices;
  bool merged;
  __device__ Entries(float* lds, const Chunk& q, const GroupLayout& y, int v, int rows)
      : n(rows), slices(y.slices), merged(q.uw % v == 0) {
    each = float(uint32_t(rows) / uint32_t(slices));
    more = int(uint32_t(rows) % uint32_t(slices));
    stride = merged ? q.cw / v : q.cw;
    per_unit = merged ? q.uw / v : q.uw;
    weight = merged ? float(v) : 1.0f;
    mean = lds;
    m2 = lds + stride * slices;
  }
  __device__ float rows_of(int slice) const { return slice < more ? each + 1 : each; }

  template <int V>
  __device__ void put(const Place<V>& p, const Shifted<V>& t) const {
    if (!p.in) return;
    const float rows = rows_of(p.slice), inv = rows > 0 ? 1.0f / rows : 0.0f;
    float m[V], v[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const float d = t.s[j] * inv;
      m[j] = t.k[j] + d;
      v[j] = t.q[j] - t.s[j] * d;
      v[j] = v[j] < 0 ? 0.0f : v[j];   // NaN stays
    }
    if (merged) {
      float s = 0, u = 0;
#pragma unroll
      for (int j = 0; j < V; ++j) s += m[j] - m[0];
      const float all = m[0] + s * (1.0f / V);
#pragma unroll
      for (int j = 0; j < V; ++j) u += v[j] + rows * (m[j] - all) * (m[j] - all);
      const int at = p.slice * stride + p.rel / V;
      mean[at] = all;
      m2[at] = u;
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (p.has(j)) {
          mean[p.slice * stride + p.rel + j] = m[j];
          m2[p.slice * stride + p.rel + j] = v[j];
        }
    }
  }
  // The mean and M2 of unit u, in each of the G neighbouring lanes that join its entries.
  template <int G>
  __device__ void join(int u, float& mean_out, float& m2_out) const {
    const int total = slices * per_unit, lane = threadIdx.x % G;
    const float first = mean[u * per_unit];   // slice 0 has a row
    float s = 0, v = 0;
    for (int e = lane; e < total; e += G) {
      const int slice = e / per_unit, at = slice * stride + u * per_unit + e - slice * per_unit;
      s += rows_of(slice) * (mean[at] - first);
    }
    const float all = first + lanes_sum<G>(s) / (float(n) * float(per_unit));
    for (int e = lane; e < total; e += G) {
      const int slice = e / per_unit, at = slice * stride + u * per_unit + e - slice * per_unit;
      const float d = mean[at] - all;
      v += m2[at] + rows_of(slice) * weight * d * d;
    }
    mean_out = all;
    m2_out = lanes_sum<G>(v);
  }
  // f(unit, mean, M2, whether the lane is to write) for every unit, by the whole workgroup of B.
  template <int B, typename F>
  __device__ void for_units(const Chunk& q, F&& f) const {
    float mu, ss;
    if (q.nu > B / kWave) {
      for (int u = threadIdx.x / 16; u < q.nu; u += B / 16) {
        join<16>(u, mu, ss);
        f(u, mu, ss, threadIdx.x % 16 == 0);
      }
    } else {
      for (int u = threadIdx.x / kWave; u < q.nu; u += B / kWave) {
        join<kWave>(u, mu, ss);
        f(u, mu, ss, threadIdx.x % kWave == 0);
      }
    }
  }
};

__device__ inline float rstd_of(float m2, float values, float eps) {
  return 1.0f / sqrtf((values > 0 ? m2 / values : 0.0f) + eps);
}

// ---- rows --------------------------------------------------------------------------

// Zeros in the workgroup's columns of rows [from, to).
template <typename T, int V>
__device__ inline void zero_rows(const GroupCall& c, const GroupLayout& y, const Place<V>& p, int64_t from, int64_t to) {
  if (!p.in) return;
  const float none[V] = {};
  for (int64_t r = from + p.slice; r < to; r += y.slices) store_own(p, static_cast<T*>(c.y) + r * c.ld_y, none, y.stream);
}

template <int V>
struct Scales {
  float mean[V], scale[V], shift[V];   // z = (x - mean) scale + shift
};

template <typename T, int V>
__device__ inline void activated(const Vec<T, V>& r, const Scales<V>& k, Act act, float (&z)[V]) {
#pragma unroll
  for (int j = 0; j < V; ++j) z[j] = fmaf(to_f32(r.v[j]) - k.mean[j], k.scale[j], k.shift[j]);
  with_act(act, [&](auto a) {
#pragma unroll
    for (int j = 0; j < V; ++j) z[j] = act_value<a(), sizeof(T) == 4>(z[j]);
  });
}

// The statistics of a place's columns, of sample s.
template <int V>
__device__ inline void place_stats(const GroupCall& c, const int (&group)[V], const float* stats, int64_t s,
                                   float (&mean)[V], float (&rstd)[V]) {
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const float* at = stats + s * c.groups + group[j];
    mean[j] = at[0];
    rstd[j] = at[c.samples * c.groups];
  }
}
// The groups of a place's columns (the first group for columns that it has not).
template <int V>
__device__ inline void place_groups(const GroupLayout& y, const Place<V>& p, int (&group)[V]) {
  if (y.per_group % V == 0 && y.part % V == 0) {   // places do not straddle groups
    const int g = p.in ? p.at / y.per_group : 0;
#pragma unroll
    for (int j = 0; j < V; ++j) group[j] = g;
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) group[j] = p.in && p.has(j) ? (p.at + j) / y.per_group : 0;
  }
}

// What the backward needs at a place: of x - mean its slope d = g act'(z), z = (x - mean) scale
// + shift; h stands as (x - mean) rstd in the sums and means that it is part of.
template <typename T, int V>
__device__ inline void slopes(const Vec<T, V>& x, const Vec<T, V>& g, const Scales<V>& k, Act act, float (&xm)[V],
                              float (&d)[V]) {
#pragma unroll
  for (int j = 0; j < V; ++j) {
    xm[j] = to_f32(x.v[j]) - k.mean[j];
    d[j] = to_f32(g.v[j]);
  }
  with_act(act, [&](auto a) {
#pragma unroll
    for (int j = 0; j < V; ++j) d[j] *= act_slope<a(), sizeof(T) == 4>(fmaf(xm[j], k.scale[j], k.shift[j]));
  });
}
// The backward's constants of a sample: mean, rstd w and b, with w and b given, and rstd.
template <typename T, int V>
struct Back {
  Scales<V> k;
  float rstd[V], w[V];
  __device__ Back(const GroupCall& c, const Place<V>& p) {
    place_weights<T>(p, c.weight, c.weight_f32, 1.0f, w);
    place_weights<T>(p, c.bias, c.weight_f32, 0.0f, k.shift);
  }
  __device__ void sample(const GroupCall& c, const int (&group)[V], int64_t s) {
    place_stats(c, group, c.stats, s, k.mean, rstd);
#pragma unroll
    for (int j = 0; j < V; ++j) k.scale[j] = rstd[j] * w[j];
  }
};
// dx = rstd (d w - ma - h mh), ma and mh the means of a and of a h.
template <typename T, int V>
struct Means {
  float along[V], all[V];   // rstd mh, ma
  __device__ void set(const Back<T, V>& k, const float (&ma)[V], const float (&mh)[V]) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      along[j] = k.rstd[j] * mh[j];
      all[j] = ma[j];
    }
  }
  __device__ void apply(const Back<T, V>& k, Act act, const Vec<T, V>& x, const Vec<T, V>& g, float (&out)[V]) const {
    float xm[V];
    slopes(x, g, k.k, act, xm, out);
#pragma unroll
    for (int j = 0; j < V; ++j) out[j] = fmaf(out[j], k.w[j], -fmaf(xm[j], along[j], all[j])) * k.rstd[j];
  }
};
// A thread's sums of d and d h per column.
template <typename T, int V>
struct Sums {
  float d[V] = {}, h[V] = {};   // h: of d (x - mean), until done
  __device__ void add(const Back<T, V>& k, Act act, const Vec<T, V>& x, const Vec<T, V>& g) {
    float xm[V], v[V];
    slopes(x, g, k.k, act, xm, v);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      d[j] += v[j];
      h[j] = fmaf(v[j], xm[j], h[j]);
    }
  }
  __device__ void done(const Back<T, V>& k) {
#pragma unroll
    for (int j = 0; j < V; ++j) h[j] *= k.rstd[j];
  }
  // A run's sums go to the thread's own LDS, for the next run's to begin at 0.
  template <int B>
  __device__ void close(int rows, float* own) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      keep<B>(own, j, d[j], rows == kRun);
      keep<B>(own, V + j, h[j], rows == kRun);
      d[j] = h[j] = 0;
    }
  }
  template <int B>
  __device__ void join(const float* own) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      d[j] += own[j * B];
      h[j] += own[(V + j) * B];
    }
  }
};

// A thread's sums of d and d h per column, added over the slices in a fixed order: column e's
// are lds[e] and lds[n + e] afterwards, n the returned number.
template <int V>
__device__ inline int column_sums(const Place<V>& p, const Chunk& q, int slices, const float (&sd)[V],
                                  const float (&sh)[V], float* lds) {
  const int n = slices * q.cw;
  if (p.in) {
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (p.has(j)) {
        lds[p.slice * q.cw + p.rel + j] = sd[j];
        lds[n + p.slice * q.cw + p.rel + j] = sh[j];
      }
  }
  __syncthreads();
  // in two steps where there are more threads than columns
  const int threads = int(blockDim.x), sub = min(threads / q.cw, slices);
  if (sub > 1) {
    float a = 0, b = 0;
    const int k = int(threadIdx.x) / q.cw, e = int(threadIdx.x) - k * q.cw;
    if (k < sub)
      for (int i = k; i < slices; i += sub) {
        a += lds[i * q.cw + e];
        b += lds[n + i * q.cw + e];
      }
    __syncthreads();
    if (k < sub) {
      lds[k * q.cw + e] = a;
      lds[n + k * q.cw + e] = b;
    }
    __syncthreads();
  }
  const int rest = sub > 1 ? sub : slices;
  for (int e = threadIdx.x; e < q.cw; e += threads) {
    float a = 0, b = 0;
    for (int i = 0; i < rest; ++i) {
      a += lds[i * q.cw + e];
      b += lds[n + i * q.cw + e];
    }
    lds[e] = a;
    lds[n + e] = b;
  }
  __syncthreads();
  return n;
}

// ---- a whole sample in one workgroup -----------------------------------------------

// Rows outside every sample lie before the first of them and behind the last.
__device__ inline void outside(const GroupCall& c, const GroupLayout& y, int& first, int& last) {
  first = last = int(c.rows);
  if (c.samples == 0) return;
  first = sample_begin(c, y, 0);
  last = max(first, sample_end(c, y, c.samples - 1, sample_begin(c, y, c.samples - 1)));
}
// Zeros in them, by the workgroups behind the samples'.
constexpr int kZeroBlocks = 64;
template <typename T, int V>
__device__ inline void zero_outside(const GroupCall& c, const GroupLayout& y, int64_t block) {
  int first, last;
  outside(c, y, first, last);
  const float none[V] = {};
  for (int k = 0; k < y.chunks; ++k) {
    const Place<V> p(chunk_of(c, y, k), y);
    if (!p.in) continue;
    for (int64_t i = block * y.slices + p.slice; i < first + c.rows - last; i += int64_t(y.slices) * kZeroBlocks)
      store_own(p, static_cast<T*>(c.y) + (i < first ? i : last + i - first) * c.ld_y, none, y.stream);
  }
}

// A sample's rows among the slices: those of the thread, and the most of any.
struct Rows {
  int mine, most;
  template <int V>
  __device__ Rows(const Place<V>& p, int slices, int rows) {
    const uint32_t n = uint32_t(rows), each = n / uint32_t(slices), more = n - each * uint32_t(slices);
    mine = p.in ? int(each + (uint32_t(p.slice) < more)) : 0;
    most = int(each + (more > 0));
  }
};
// A value that the compiler computes where it stands, instead of all rows' addresses and
// conditions ahead, which would take the registers that hold rows.
template <typename T>
__device__ inline T afresh(T v) {
  asm volatile("" : "+v"(v));
  return v;
}
// Rows that a thread reads at once, in tiles; a workgroup that holds rows has few registers left.
constexpr int kInFlight = kTileTurn, kBeside = 2;

// What is done between two runs of kRun rows: nothing, where nothing is summed.
struct NoSums {
  __device__ void operator()(int) const {}
};
// Whether a thread of the workgroup closes a run in `rows` rows.
__device__ inline bool closes(int rows, int slices) { return rows > int64_t(kRun) * slices; }

// Rows lo + slice, + slices ... of [lo, hi): f(vector, whether it is the first) for each, and
// close(rows so far) after each kRun of them that are not the last.
template <typename T, int V, int Q, typename F, typename G = NoSums>
__device__ inline void for_rows(const Place<V>& p, int slices, const T* x, int64_t ld, int lo, int hi, F&& f, G&& close = {}) {
  const int64_t step = int64_t(slices) * ld;
  int left = Rows(p, slices, hi - lo).mine;
  if (left <= 0) return;
  const T* at = x + int64_t(lo + p.slice) * ld + p.at;
  bool first = true;
  int done = 0;
  while (left > 0) {
    Vec<T, V> v[Q];
#pragma unroll
    for (int i = 0; i < Q; ++i) v[i] = load_vec<false, T, V>(at + (i < left ? i : left - 1) * step);
#pragma unroll
    for (int i = 0; i < Q; ++i)
      if (i < left) {
        f(v[i], first);
        first = false;
      }
    at += Q * step;
    left -= Q;
    done += Q;
    if (done % kRun == 0 && left > 0) close(done);
  }
}

// Rows of x and of grad_out together.
template <typename T, int V, int Q, typename F, typename G = NoSums>
__device__ inline void for_row_pairs(const GroupCall& c, const Place<V>& p, int slices, int lo, int hi, F&& f, G&& close = {}) {
  const int64_t sx = int64_t(slices) * c.ld_x, sg = int64_t(slices) * c.ld_g;
  int left = Rows(p, slices, hi - lo).mine;
  if (left <= 0) return;
  const T* x = static_cast<const T*>(c.x) + int64_t(lo + p.slice) * c.ld_x + p.at;
  const T* g = static_cast<const T*>(c.grad_out) + int64_t(lo + p.slice) * c.ld_g + p.at;
  int done = 0;
  while (left > 0) {
    Vec<T, V> vx[Q], vg[Q];
#pragma unroll
    for (int i = 0; i < Q; ++i) {
      vx[i] = load_vec<false, T, V>(x + (i < left ? i : left - 1) * sx);
      vg[i] = load_vec<false, T, V>(g + (i < left ? i : left - 1) * sg);
    }
#pragma unroll
    for (int i = 0; i < Q; ++i)
      if (i < left) f(vx[i], vg[i]);
    x += Q * sx;
    g += Q * sg;
    left -= Q;
    done += Q;
    if (done % kRun == 0 && left > 0) close(done);
  }
}

// A row's vector as it is held: packed, so that the compiler keeps neither its elements nor
// their values in 32 bits until they are used.
template <int Bytes>
struct Words {
  typedef uint32_t Type __attribute__((ext_vector_type(Bytes / 4)));
};
template <>
struct Words<4> {
  typedef uint32_t Type;
};
template <>
struct Words<2> {
  typedef uint16_t Type;
};
template <typename T, int V>
using Held = typename Words<sizeof(T) * V>::Type;
template <typename T, int V>
__device__ inline Held<T, V> hold(const T* p) {
  return __builtin_bit_cast(Held<T, V>, load_vec<false, T, V>(p));
}
template <typename T, int V>
__device__ inline Vec<T, V> unpack(const Held<T, V>& h) {
  return __builtin_bit_cast(Vec<T, V>, h);
}
// An item's sample and chunk.
__device__ inline int64_t sample_of(int64_t item, int chunks, int& chunk) {
  const int64_t s = item >> 32 ? item / chunks : int64_t(uint32_t(item) / uint32_t(chunks));
  chunk = int(item - s * chunks);
  return s;
}

// N rows of a thread are held from the sums to the output; a sample of more has the others read
// again, while the caches may still hold them.
template <typename T, int V, int B, int N>
__global__ __launch_bounds__(B) void group_fwd_kernel(GroupCall c, GroupLayout y, int64_t items) {
  __shared__ __align__(16) float lds[2 * B * V];
  if (int64_t(blockIdx.x) >= items) {
    zero_outside<T, V>(c, y, blockIdx.x - items);
    return;
  }
  for (int64_t item = blockIdx.x; item < c.samples * y.chunks; item += items) {
    int chunk;
    const int64_t s = sample_of(item, y.chunks, chunk);
    const Chunk q = chunk_of(c, y, chunk);
    const Place<V> p(q, y);
    const int begin = sample_begin(c, y, s), end = sample_end(c, y, s, begin), rows = end - begin;
    const Rows own(p, y.slices, rows);
    const T* x = static_cast<const T*>(c.x) + int64_t(begin + p.slice) * c.ld_x + p.at;
    const int64_t step = int64_t(y.slices) * c.ld_x;
    const int rest = begin + N * y.slices;   // the first row that is not held
    Shifted<V> sum;
    sum.clear();
    auto add = [&](const Vec<T, V>& row, bool first) {
      float v[V];
#pragma unroll
      for (int j = 0; j < V; ++j) v[j] = to_f32(row.v[j]);
      if (first) {
#pragma unroll
        for (int j = 0; j < V; ++j) sum.k[j] = v[j];
      }
      sum.add(v);
    };
    if (own.most > N) {
      for_rows<T, V, kBeside>(p, y.slices, static_cast<const T*>(c.x), c.ld_x, rest, end, add,
                              [&](int n) { sum.template close<B>(n, lds + threadIdx.x); });
      if (closes(end - rest, y.slices)) {
        if (own.mine > N + kRun) sum.template join<B>(lds + threadIdx.x);
        __syncthreads();   // before the entries, in the same places
      }
    }
    Held<T, V> held[N];
    const T* at = x;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (i < own.mine) held[i] = hold<T, V>(at);
      at = afresh(at + step);
    }
    const int left = afresh(own.mine);
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i < left) add(unpack<T, V>(held[i]), i == 0 && left <= N);
    float w[V], b[V];
    place_weights<T>(p, c.weight, c.weight_f32, 1.0f, w);
    place_weights<T>(p, c.bias, c.weight_f32, 0.0f, b);
    const Entries e(lds, q, y, V, rows);
    e.put(p, sum);
    __syncthreads();
    if (rows == 0) {
      for (int u = threadIdx.x; c.stats && u < q.nu; u += B) {
        c.stats[s * c.groups + q.u0 + u] = 0;
        c.stats[(c.samples + s) * c.groups + q.u0 + u] = rstd_of(0, 0, c.eps);
      }
      continue;
    }
    e.template for_units<B>(q, [&](int u, float mean, float m2, bool first) {
      if (!first) return;
      const float rstd = rstd_of(m2, float(rows) * float(q.uw), c.eps);
      e.mean[u * e.per_unit] = mean;   // in the place of an entry that only these lanes read
      e.m2[u * e.per_unit] = rstd;
      if (c.stats) {
        c.stats[s * c.groups + q.u0 + u] = mean;
        c.stats[(c.samples + s) * c.groups + q.u0 + u] = rstd;
      }
    });
    __syncthreads();
    int group[V];
    place_groups(y, p, group);
    Scales<V> k;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int u = p.in ? max(group[j] - q.u0, 0) : 0;
      k.mean[j] = e.mean[u * e.per_unit];
      k.scale[j] = e.m2[u * e.per_unit] * w[j];
      k.shift[j] = b[j];
    }
    T* out = static_cast<T*>(c.y) + int64_t(begin + p.slice) * c.ld_y;
    const int64_t step_y = int64_t(y.slices) * c.ld_y;
    const int again = afresh(own.mine);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (i < again) {
        float z[V];
        activated(unpack<T, V>(held[i]), k, c.act, z);
        store_own(p, out, z, y.stream);
      }
      out = afresh(out + step_y);
    }
    if (own.most > N)
      for_rows<T, V, kBeside>(p, y.slices, static_cast<const T*>(c.x), c.ld_x, rest, end, [&](const Vec<T, V>& row, bool) {
        float z[V];
        activated(row, k, c.act, z);
        store_own(p, out, z, y.stream);
        out += step_y;
      });
    __syncthreads();   // before the next sample's entries
  }
}

template <typename T, int V, int B, int N>
__global__ __launch_bounds__(B) void group_bwd_kernel(GroupCall c, GroupLayout y, int64_t items, float* join) {
  __shared__ __align__(16) float lds[2 * B * V];
  if (int64_t(blockIdx.x) >= items) {
    zero_outside<T, V>(c, y, blockIdx.x - items);
    return;
  }
  for (int64_t item = blockIdx.x; item < c.samples * y.chunks; item += items) {
    int chunk;
    const int64_t s = sample_of(item, y.chunks, chunk);
    const Chunk q = chunk_of(c, y, chunk);
    const Place<V> p(q, y);
    const int begin = sample_begin(c, y, s), end = sample_end(c, y, s, begin), rows = end - begin;
    const Rows own(p, y.slices, rows);
    const int rest = begin + N * y.slices;
    const T* x = static_cast<const T*>(c.x) + int64_t(begin + p.slice) * c.ld_x + p.at;
    const T* g = static_cast<const T*>(c.grad_out) + int64_t(begin + p.slice) * c.ld_g + p.at;
    const int64_t step_x = int64_t(y.slices) * c.ld_x, step_g = int64_t(y.slices) * c.ld_g;
    int group[V];
    place_groups(y, p, group);
    Back<T, V> k(c, p);
    if (rows > 0) k.sample(c, group, s);   // without rows there may be no statistics
    Sums<T, V> sum;
    auto add = [&](const Vec<T, V>& vx, const Vec<T, V>& vg) { sum.add(k, c.act, vx, vg); };
    if (own.most > N) {
      for_row_pairs<T, V, kBeside>(c, p, y.slices, rest, end, add,
                                   [&](int n) { sum.template close<B>(n, lds + threadIdx.x); });
      if (closes(end - rest, y.slices)) {
        if (own.mine > N + kRun) sum.template join<B>(lds + threadIdx.x);
        __syncthreads();   // before the columns' sums, in the same places
      }
    }
    Held<T, V> hx[N], hg[N];
    const T *at_x = x, *at_g = g;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (i < own.mine) {
        hx[i] = hold<T, V>(at_x);
        hg[i] = hold<T, V>(at_g);
      }
      at_x = afresh(at_x + step_x);
      at_g = afresh(at_g + step_g);
    }
    const int left = afresh(own.mine);
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i < left) add(unpack<T, V>(hx[i]), unpack<T, V>(hg[i]));
    if (rows > 0) sum.done(k);   // without rows rstd may be infinite
    const int n = column_sums(p, q, y.slices, sum.d, sum.h, lds);
    // the columns' sums, for the weights' gradients
    for (int e = threadIdx.x; e < q.cw; e += B) {
      if (join) {
        join[s * 2 * c.width + q.c0 + e] = lds[e];
        join[(s * 2 + 1) * c.width + q.c0 + e] = lds[n + e];
      } else {
        if (c.grad_bias) store_either<T>(c.grad_bias, c.weight_f32, q.c0 + e, lds[e]);
        if (c.grad_weight) store_either<T>(c.grad_weight, c.weight_f32, q.c0 + e, lds[n + e]);
      }
    }
    if (c.y && rows > 0) {
      __syncthreads();
      // a group's means of a and of a h
      const float inv = 1.0f / (float(rows) * float(q.uw));
      for (int u = threadIdx.x / kWave; u < q.nu; u += B / kWave) {
        float a = 0, b = 0;
        for (int e = threadIdx.x % kWave; e < q.uw; e += kWave) {
          const int at = u * q.uw + e;
          const float w = c.weight ? load_either<T>(c.weight, c.weight_f32, q.c0 + at) : 1.0f;
          a += w * lds[at];
          b += w * lds[n + at];
        }
        a = wave_sum(a) * inv;
        b = wave_sum(b) * inv;
        if (threadIdx.x % kWave == 0) {
          lds[u * q.uw] = a;   // in the place of a column that only this wave reads
          lds[n + u * q.uw] = b;
        }
      }
      __syncthreads();
      float ma[V], mh[V];
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int u = p.in ? max(group[j] - q.u0, 0) : 0;
        ma[j] = lds[u * q.uw];
        mh[j] = lds[n + u * q.uw];
      }
      T* out = static_cast<T*>(c.y) + int64_t(begin + p.slice) * c.ld_y;
      const int64_t step_y = int64_t(y.slices) * c.ld_y;
      Means<T, V> means;
      means.set(k, ma, mh);
      auto apply = [&](const Vec<T, V>& vx, const Vec<T, V>& vg) {
        float d[V];
        means.apply(k, c.act, vx, vg, d);
        store_own(p, out, d, y.stream);
      };
      const int again = afresh(own.mine);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        if (i < again) apply(unpack<T, V>(hx[i]), unpack<T, V>(hg[i]));
        out = afresh(out + step_y);
      }
      if (own.most > N)
        for_row_pairs<T, V, kBeside>(c, p, y.slices, rest, end, [&](const Vec<T, V>& vx, const Vec<T, V>& vg) {
          apply(vx, vg);
          out += step_y;
        });
    }
    __syncthreads();   // before the next sample's sums
  }
}

// ---- tiles -------------------------------------------------------------------------

// A workgroup's tile and chunk.  The second reading comes last first, as what was read last is
// what the 256 MB cache behind the L2s still holds: forward of 561680 x 128 fp32 150 us, 160 in the
// first reading's order, backward 288 and 305; calls that fit it take the same either way.
// Workgroups go to the eight dies (XCDs) by turns, each with an L2 of its own, and a tile keeps its
// place among eight: 0.4 us of 26 for 114688 x 128 bf16 and 0.6 for 96000 x 128 against a plain
// reversal, nothing in 32 bits.  It is not the L2's contents (the second reading fetches past it
// as much as the first), and behind the weights' gradients' workgroups, where their number is no
// multiple of eight, tiles move to other dies at no cost.
struct Tile {
  int tile, chunk, r0, r1;
  __device__ Tile(const GroupCall& c, const GroupLayout& y, int block) {
    tile = int(uint32_t(block) / uint32_t(y.chunks));
    chunk = block - tile * y.chunks;
    r0 = int(int64_t(tile) * y.tile_rows);
    r1 = int(min(int64_t(tile + 1) * y.tile_rows, c.rows));
  }
};
constexpr int kDies = 8;
__device__ inline int from_behind(int block, int blocks) {
  return ((blocks + kDies - 1) / kDies - 1 - block / kDies) * kDies + block % kDies;
}

// Walks through a tile: f(sample, first row, past the last).
template <typename F>
__device__ inline void for_pieces(const GroupCall& c, const GroupLayout& y, const Tile& t, F&& f) {
  for (int64_t s = sample_behind(c, y, t.r0); s < c.samples; ++s) {
    const int begin = sample_begin(c, y, s);
    if (begin >= t.r1) break;
    const int lo = max(begin, t.r0), hi = min(sample_end(c, y, s, begin), t.r1);
    if (lo < hi) f(s, lo, hi);
  }
}

// The pieces' means and M2, [units][tiles + samples][2].
template <typename T, int V>
__global__ __launch_bounds__(kTileBlock) void group_sum_kernel(GroupCall c, GroupLayout y, float* pieces) {
  __shared__ __align__(16) float lds[2 * kTileBlock * V];
  const Tile t(c, y, blockIdx.x);
  const Chunk q = chunk_of(c, y, t.chunk);
  const Place<V> p(q, y);
  const int64_t n_pieces = y.tiles + c.samples;
  for_pieces(c, y, t, [&](int64_t s, int lo, int hi) {
    Shifted<V> sum;
    sum.clear();
    auto add = [&](const Vec<T, V>& r, bool first) {
      float v[V];
#pragma unroll
      for (int j = 0; j < V; ++j) v[j] = to_f32(r.v[j]);
      if (first) {
#pragma unroll
        for (int j = 0; j < V; ++j) sum.k[j] = v[j];
      }
      sum.add(v);
    };
    for_rows<T, V, kInFlight>(p, y.slices, static_cast<const T*>(c.x), c.ld_x, lo, hi, add,
                              [&](int n) { sum.template close<kTileBlock>(n, lds + threadIdx.x); });
    if (closes(hi - lo, y.slices)) {
      if (Rows(p, y.slices, hi - lo).mine > kRun) sum.template join<kTileBlock>(lds + threadIdx.x);
      __syncthreads();
    }
    const Entries e(lds, q, y, V, hi - lo);
    e.put(p, sum);
    __syncthreads();
    e.template for_units<kTileBlock>(q, [&](int u, float mean, float m2, bool first) {
      if (!first) return;
      float* at = pieces + ((q.u0 + u) * n_pieces + t.tile + s) * 2;
      at[0] = mean;
      at[1] = m2;
    });
    __syncthreads();
  });
}

// Sum over a group of G lanes, the workgroup's threads for G = kTileBlock.
template <int G>
__device__ inline float many_sum(float v, float* lds) {
  v = wave_sum(v);
  if constexpr (G > kWave) {
    __syncthreads();
    if (threadIdx.x % kWave == 0) lds[threadIdx.x / kWave] = v;
    __syncthreads();
    v = 0;
#pragma unroll
    for (int i = 0; i < G / kWave; ++i) v += lds[i];
  }
  return v;
}

// G lanes join the pieces of one sample and group.
template <int G>
__global__ __launch_bounds__(kTileBlock) void group_join_kernel(GroupCall c, GroupLayout y, const float* pieces,
                                                                float* stats) {
  __shared__ float lds[kTileBlock / kWave];
  const int lane = threadIdx.x % G;
  const int64_t n_pieces = y.tiles + c.samples;
  for (int64_t k = int64_t(blockIdx.x) * (kTileBlock / G) + threadIdx.x / G; k < c.samples * c.groups;
       k += int64_t(gridDim.x) * (kTileBlock / G)) {
    int g;
    const int64_t s = sample_of(k, int(c.groups), g);
    const int begin = sample_begin(c, y, s), end = sample_end(c, y, s, begin);
    float mean = 0, m2 = 0;
    if (begin < end) {
      const int t0 = begin / y.tile_rows, n = (end - 1) / y.tile_rows - t0 + 1;
      const float values = float(end - begin) * float(y.per_group);
      const float first = pieces[(int64_t(g) * y.split * n_pieces + t0 + s) * 2];
      float a = 0, b = 0;
      for (int part = 0; part < y.split; ++part) {
        const float* at = pieces + ((int64_t(g) * y.split + part) * n_pieces + t0 + s) * 2;
        const float columns = float(min(y.part, y.per_group - part * y.part));
#pragma unroll 4
        for (int t = lane; t < n; t += G) {
          const int64_t r = int64_t(t0 + t) * y.tile_rows;
          a += float(min(r + y.tile_rows, int64_t(end)) - max(r, int64_t(begin))) * columns * (at[2 * t] - first);
        }
      }
      mean = first + many_sum<G>(a, lds) / values;
      for (int part = 0; part < y.split; ++part) {
        const float* at = pieces + ((int64_t(g) * y.split + part) * n_pieces + t0 + s) * 2;
        const float columns = float(min(y.part, y.per_group - part * y.part));
#pragma unroll 4
        for (int t = lane; t < n; t += G) {
          const int64_t r = int64_t(t0 + t) * y.tile_rows;
          const float d = at[2 * t] - mean;
          b += at[2 * t + 1] + float(min(r + y.tile_rows, int64_t(end)) - max(r, int64_t(begin))) * columns * d * d;
        }
      }
      m2 = many_sum<G>(b, lds);
    }
    if (lane == 0) {
      stats[k] = mean;
      stats[c.samples * c.groups + k] = rstd_of(m2, float(end - begin) * float(y.per_group), c.eps);
    }
  }
}

// Zeros of a tile's rows outside every sample.
template <typename T, int V>
__device__ inline void zero_tile(const GroupCall& c, const GroupLayout& y, const Place<V>& p, const Tile& t) {
  int first, last;
  outside(c, y, first, last);
  zero_rows<T>(c, y, p, t.r0, min(t.r1, first));
  zero_rows<T>(c, y, p, max(t.r0, last), t.r1);
}

template <typename T, int V>
__global__ __launch_bounds__(kTileBlock) void group_apply_kernel(GroupCall c, GroupLayout y, const float* stats) {
  const int block = from_behind(blockIdx.x, y.tiles * y.chunks);
  if (block >= y.tiles * y.chunks) return;
  const Tile t(c, y, block);
  const Chunk q = chunk_of(c, y, t.chunk);
  const Place<V> p(q, y);
  int group[V];
  place_groups(y, p, group);
  float w[V], b[V];
  place_weights<T>(p, c.weight, c.weight_f32, 1.0f, w);
  place_weights<T>(p, c.bias, c.weight_f32, 0.0f, b);
  for_pieces(c, y, t, [&](int64_t s, int lo, int hi) {
    Scales<V> k;
    place_stats(c, group, stats, s, k.mean, k.scale);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      k.scale[j] *= w[j];
      k.shift[j] = b[j];
    }
    T* out = static_cast<T*>(c.y) + int64_t(lo + p.slice) * c.ld_y;
    for_rows<T, V, kInFlight>(p, y.slices, static_cast<const T*>(c.x), c.ld_x, lo, hi, [&](const Vec<T, V>& r, bool) {
      float z[V];
      activated(r, k, c.act, z);
      store_own(p, out, z, y.stream);
      out += int64_t(y.slices) * c.ld_y;
    });
  });
  if (c.zero_outside && c.offsets) zero_tile<T>(c, y, p, t);
}

// The pieces' sums of d and d h, [tiles + samples][2][width].
template <typename T, int V>
__global__ __launch_bounds__(kTileBlock) void group_bwd_sum_kernel(GroupCall c, GroupLayout y, float* pieces) {
  __shared__ __align__(16) float lds[2 * kTileBlock * V];
  const Tile t(c, y, blockIdx.x);
  const Chunk q = chunk_of(c, y, t.chunk);
  const Place<V> p(q, y);
  int group[V];
  place_groups(y, p, group);
  Back<T, V> k(c, p);
  for_pieces(c, y, t, [&](int64_t s, int lo, int hi) {
    k.sample(c, group, s);
    Sums<T, V> sum;
    for_row_pairs<T, V, kInFlight / 2>(
        c, p, y.slices, lo, hi, [&](const Vec<T, V>& x, const Vec<T, V>& g) { sum.add(k, c.act, x, g); },
        [&](int n) { sum.template close<kTileBlock>(n, lds + threadIdx.x); });
    if (closes(hi - lo, y.slices)) {
      if (Rows(p, y.slices, hi - lo).mine > kRun) sum.template join<kTileBlock>(lds + threadIdx.x);
      __syncthreads();
    }
    sum.done(k);
    const int n = column_sums(p, q, y.slices, sum.d, sum.h, lds);
    float* at = pieces + (t.tile + s) * 2 * c.width + q.c0;
    for (int e = threadIdx.x; e < q.cw; e += kTileBlock) {
      at[e] = lds[e];
      at[c.width + e] = lds[n + e];
    }
    __syncthreads();
  });
}

// A workgroup of B joins the pieces of one sample and group: the columns' sums, and the means
// of a and a h.
template <typename T, int B>
__global__ __launch_bounds__(B) void group_bwd_join_kernel(GroupCall c, GroupLayout y, const float* pieces, float* join,
                                                           float* coef) {
  __shared__ float lds[2][B];
  const int cg = y.per_group, lanes = min(cg, B), subs = B / lanes;
  const int sub = int(threadIdx.x) / lanes, lane = int(threadIdx.x) - sub * lanes;
  const int64_t ld = 2 * c.width;
  for (int64_t k = blockIdx.x; k < c.samples * c.groups; k += gridDim.x) {
    int g;
    const int64_t s = sample_of(k, int(c.groups), g);
    const int begin = sample_begin(c, y, s), end = sample_end(c, y, s, begin);
    const int t0 = begin / y.tile_rows, n = begin < end ? (end - 1) / y.tile_rows - t0 + 1 : 0;
    float sa = 0, sh = 0;
    for (int c0 = 0; c0 < cg; c0 += lanes) {
      const bool in = sub < subs && c0 + lane < cg;
      const int64_t e = int64_t(g) * cg + c0 + lane;
      float a = 0, b = 0;
      if (in) {
        const float* at = pieces + (t0 + s) * ld + e;
#pragma unroll 8
        for (int t = sub; t < n; t += subs) {
          a += at[t * ld];
          b += at[t * ld + c.width];
        }
      }
      lds[0][threadIdx.x] = a;
      lds[1][threadIdx.x] = b;
      __syncthreads();
      // a tree over the subs, of which there may be any number
      for (int m = subs; m > 1;) {
        const int half = (m + 1) / 2;
        if (sub < m - half) {
          lds[0][threadIdx.x] += lds[0][threadIdx.x + half * lanes];
          lds[1][threadIdx.x] += lds[1][threadIdx.x + half * lanes];
        }
        m = half;
        __syncthreads();
      }
      if (sub == 0 && in) {
        a = lds[0][lane];
        b = lds[1][lane];
        if (join) {
          join[s * ld + e] = a;
          join[s * ld + c.width + e] = b;
        } else {
          if (c.grad_bias) store_either<T>(c.grad_bias, c.weight_f32, e, a);
          if (c.grad_weight) store_either<T>(c.grad_weight, c.weight_f32, e, b);
        }
        const float w = c.weight ? load_either<T>(c.weight, c.weight_f32, e) : 1.0f;
        sa += w * a;
        sh += w * b;
      }
      __syncthreads();
    }
    sa = wave_sum(sa);
    sh = wave_sum(sh);
    if (threadIdx.x % kWave == 0) {
      lds[0][threadIdx.x / kWave] = sa;
      lds[1][threadIdx.x / kWave] = sh;
    }
    __syncthreads();
    if (threadIdx.x < 2) {
      float v = 0;
#pragma unroll
      for (int i = 0; i < B / kWave; ++i) v += lds[threadIdx.x][i];
      coef[k * 2 + threadIdx.x] = begin < end ? v / (float(end - begin) * float(cg)) : 0.0f;
    }
    __syncthreads();
  }
}

// Of many samples, runs of `fold` are summed first, each in the place of its first sample, by a
// thread for each run and column: some 8 sqrt(samples) runs, so that its chain of additions and
// those of sum_params' 64 lanes a column behind it have sqrt(samples) / 8 each.  The backward of
// equal samples with it and without: 5000 (60000 x 64 fp32) 28 and 36 us, 100000 (600000 x 64)
// 235 and 464, 8000 (32000 x 512) 93 and 113; 1200 (14400 x 64) 21 and 19.
constexpr int64_t kFoldFrom = 2048;
int64_t fold_of(const GroupCall& c) {
  return c.samples > kFoldFrom ? int64_t(std::sqrt(double(c.samples)) / 8) : 1;
}
constexpr int kFoldBlock = 256;
__global__ __launch_bounds__(kFoldBlock) void group_fold_kernel(GroupCall c, float* join, int64_t fold) {
  const int64_t ld = 2 * c.width, all = (c.samples + fold - 1) / fold * ld;
  for (int64_t i = int64_t(blockIdx.x) * kFoldBlock + threadIdx.x; i < all; i += int64_t(gridDim.x) * kFoldBlock) {
    const int64_t first = i / ld * fold, last = min(first + fold, c.samples);
    float* at = join + first * ld + i % ld;
    float v = 0;
#pragma unroll 8
    for (int64_t s = 0; s < last - first; ++s) v += at[s * ld];
    *at = v;
  }
}

// The weights' gradients of kParamColumns columns from the (folded) samples' sums, by a workgroup
// of B, in a fixed order.
constexpr int kParamColumns = 16;
template <typename T, int B>
__device__ inline void sum_params(const GroupCall& c, const float* join, int64_t fold, int block) {
  constexpr int kSubs = B / kParamColumns;
  __shared__ float lds[2][B];
  const int sub = threadIdx.x / kParamColumns, lane = threadIdx.x % kParamColumns;
  const int64_t e = int64_t(block) * kParamColumns + lane, ld = 2 * c.width;
  float a = 0, b = 0;
  if (e < c.width) {
#pragma unroll 8
    for (int64_t s = sub * fold; s < c.samples; s += kSubs * fold) {
      a += join[s * ld + e];
      b += join[s * ld + c.width + e];
    }
  }
  lds[0][threadIdx.x] = a;
  lds[1][threadIdx.x] = b;
  for (int half = kSubs / 2; half > 0; half /= 2) {
    __syncthreads();
    if (sub < half) {
      lds[0][threadIdx.x] += lds[0][threadIdx.x + half * kParamColumns];
      lds[1][threadIdx.x] += lds[1][threadIdx.x + half * kParamColumns];
    }
  }
  if (sub == 0 && e < c.width) {
    if (c.grad_bias) store_either<T>(c.grad_bias, c.weight_f32, e, lds[0][lane]);
    if (c.grad_weight) store_either<T>(c.grad_weight, c.weight_f32, e, lds[1][lane]);
  }
}

// The first `params` workgroups sum the weights' gradients, the others have a tile each.
template <typename T, int V>
__global__ __launch_bounds__(kTileBlock) void group_bwd_apply_kernel(GroupCall c, GroupLayout y, const float* coef,
                                                                     const float* join, int64_t fold, int params) {
  if (int(blockIdx.x) < params) {
    sum_params<T, kTileBlock>(c, join, fold, blockIdx.x);
    return;
  }
  const int block = from_behind(blockIdx.x - params, y.tiles * y.chunks);
  if (block >= y.tiles * y.chunks) return;
  const Tile t(c, y, block);
  const Chunk q = chunk_of(c, y, t.chunk);
  const Place<V> p(q, y);
  int group[V];
  place_groups(y, p, group);
  Back<T, V> k(c, p);
  for_pieces(c, y, t, [&](int64_t s, int lo, int hi) {
    k.sample(c, group, s);
    float ma[V], mh[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const float* at = coef + (s * c.groups + group[j]) * 2;
      ma[j] = at[0];
      mh[j] = at[1];
    }
    Means<T, V> means;
    means.set(k, ma, mh);
    T* out = static_cast<T*>(c.y) + int64_t(lo + p.slice) * c.ld_y;
    for_row_pairs<T, V, kInFlight / 2>(c, p, y.slices, lo, hi, [&](const Vec<T, V>& x, const Vec<T, V>& g) {
      float d[V];
      means.apply(k, c.act, x, g, d);
      store_own(p, out, d, y.stream);
      out += int64_t(y.slices) * c.ld_y;
    });
  });
  if (c.offsets) zero_tile<T>(c, y, p, t);
}

// The weights' gradients by themselves, behind whole samples.
constexpr int kParamBlock = 1024;
template <typename T>
__global__ __launch_bounds__(kParamBlock) void group_param_kernel(GroupCall c, const float* join, int64_t fold) {
  sum_params<T, kParamBlock>(c, join, fold, blockIdx.x);
}

// ---- launches ----------------------------------------------------------------------

// Workgroups of one item each, as many as a launch takes.
unsigned blocks_of(int64_t items, int threads) { return unsigned(std::min(items, kGroupGrid / threads - kZeroBlocks)); }

unsigned param_blocks(const GroupCall& c) { return unsigned((c.width + kParamColumns - 1) / kParamColumns); }
void fold(const GroupCall& c, float* join, hipStream_t s) {
  const int64_t f = fold_of(c);
  if (f == 1) return;
  const int64_t threads = (c.samples + f - 1) / f * 2 * c.width;
  hipLaunchKernelGGL(group_fold_kernel, dim3(blocks_of((threads + kFoldBlock - 1) / kFoldBlock, kFoldBlock)), dim3(kFoldBlock),
                     0, s, c, join, f);
}

template <typename T, int V, int B>
void whole(const GroupCall& c, const GroupLayout& y, bool backward, float* join, hipStream_t s) {
  const int64_t items = blocks_of(c.samples * y.chunks, B);
  const bool zeros = c.offsets && c.rows > 0 && (backward ? c.y != nullptr : c.zero_outside != 0);
  const dim3 grid{unsigned(items + (zeros ? kZeroBlocks : 0))}, block{B};
  if (grid.x == 0) return;
  constexpr int kForward = held_most(int(sizeof(T)), false), kBackward = held_most(int(sizeof(T)), true);
  if (!backward) {
    if (y.held == kHeldFew)
      hipLaunchKernelGGL((group_fwd_kernel<T, V, B, kHeldFew>), grid, block, 0, s, c, y, items);
    else
      hipLaunchKernelGGL((group_fwd_kernel<T, V, B, kForward>), grid, block, 0, s, c, y, items);
  } else {
    if (y.held == kHeldFew)
      hipLaunchKernelGGL((group_bwd_kernel<T, V, B, kHeldFew>), grid, block, 0, s, c, y, items, join);
    else
      hipLaunchKernelGGL((group_bwd_kernel<T, V, B, kBackward>), grid, block, 0, s, c, y, items, join);
  }
}

template <typename T, int V>
void tiles(const GroupCall& c, const GroupLayout& y, bool backward, bool sums, float* join, hipStream_t s) {
  const GroupWork at = group_work(c, y, backward, sums);
  float *pieces = c.work + at.pieces, *coef = c.work + at.coef;
  const unsigned blocks = unsigned(y.tiles * y.chunks), back = (blocks + kDies - 1) / kDies * kDies;
  const dim3 block{kTileBlock};
  // lanes for one sample and group: as many as its tiles keep busy
  const int64_t joins = c.samples * c.groups, mean = joins ? y.tiles / c.samples : 0;
  if (!backward) {
    float* stats = c.stats ? c.stats : coef;
    if (blocks) hipLaunchKernelGGL((group_sum_kernel<T, V>), dim3(blocks), block, 0, s, c, y, pieces);
    if (joins && mean > 2 * kWave)
      hipLaunchKernelGGL(group_join_kernel<kTileBlock>, dim3(blocks_of(joins, kTileBlock)), block, 0, s, c, y, pieces, stats);
    else if (joins)
      hipLaunchKernelGGL(group_join_kernel<kWave>, dim3(blocks_of((joins + 3) / 4, kTileBlock)), block, 0, s, c, y, pieces,
                         stats);
    if (blocks) hipLaunchKernelGGL((group_apply_kernel<T, V>), dim3(back), block, 0, s, c, y, stats);
    return;
  }
  if (blocks) hipLaunchKernelGGL((group_bwd_sum_kernel<T, V>), dim3(blocks), block, 0, s, c, y, pieces);
  const int64_t work = mean * y.per_group;   // sums that a workgroup joins
  if (joins && work > 2048)
    hipLaunchKernelGGL((group_bwd_join_kernel<T, 1024>), dim3(blocks_of(joins, 1024)), dim3(1024), 0, s, c, y, pieces, join,
                       coef);
  else if (joins && work > 256)
    hipLaunchKernelGGL((group_bwd_join_kernel<T, 256>), dim3(blocks_of(joins, 256)), dim3(256), 0, s, c, y, pieces, join,
                       coef);
  else if (joins)
    hipLaunchKernelGGL((group_bwd_join_kernel<T, 64>), dim3(blocks_of(joins, 64)), dim3(64), 0, s, c, y, pieces, join, coef);
  const unsigned params = sums ? param_blocks(c) : 0u;
  if (sums) fold(c, join, s);
  if (params + (c.y ? back : 0))
    hipLaunchKernelGGL((group_bwd_apply_kernel<T, V>), dim3(params + (c.y ? back : 0)), block, 0, s, c, y, coef, join,
                       fold_of(c), int(params));
}

template <typename T, int V>
hipError_t run(const GroupCall& c, const GroupLayout& y, bool backward, hipStream_t s) {
  // the sums per sample and channel, unless one sample's are the gradients themselves, which a
  // null join has written (of no sample there are none, and nothing to hold them)
  const bool sums = backward && (c.grad_weight || c.grad_bias) && c.samples != 1;
  float* join = sums ? c.work + group_work(c, y, backward).join : nullptr;
  if (!y.whole) {
    tiles<T, V>(c, y, backward, sums, join, s);
    return hipGetLastError();
  }
  if (y.block == 64)
    whole<T, V, 64>(c, y, backward, join, s);
  else
    whole<T, V, 256>(c, y, backward, join, s);
  if (sums) {
    fold(c, join, s);
    hipLaunchKernelGGL(group_param_kernel<T>, dim3(param_blocks(c)), dim3(kParamBlock), 0, s, c, join, fold_of(c));
  }
  return hipGetLastError();
}

template <typename T>
hipError_t run(const GroupCall& c, bool backward, hipStream_t s) {
  const GroupLayout y = lay_out_group(c, int(sizeof(T)), backward);
  return y.vec == 1 ? run<T, 1>(c, y, backward, s) : run<T, kGroupVec>(c, y, backward, s);
}
hipError_t run(const GroupCall& c, Elem type, bool backward, hipStream_t s) {
  return type == Elem::f32 ? run<float>(c, backward, s)
         : type == Elem::bf16 ? run<Bf16>(c, backward, s) : run<F16>(c, backward, s);
}

}  // namespace

size_t group_norm_floats(const GroupCall& c, Elem type, bool backward, bool sums) {
  return size_t(group_work(c, lay_out_group(c, type == Elem::f32 ? 4 : 2, backward), backward, sums).total);
}

hipError_t launch_group_norm_forward(const GroupCall& c, Elem type, hipStream_t s) { return run(c, type, false, s); }
hipError_t launch_group_norm_backward(const GroupCall& c, Elem type, hipStream_t s) { return run(c, type, true, s); }

}  // namespace cgtp

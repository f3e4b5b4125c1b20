// Routing of rows to branches by their logits, its balance loss, the way back to the
// logits, and the gradient of the convolution's gate.
//
// A row's n logits are held by L neighbouring lanes, E each (n <= L E), lane l those of the
// branches l E to l E + E - 1.  They choose k times the largest of what is left, by a key of
// 32 bits in the logits' order; p = softmax needs the row's maximum, which the first choice
// gives, and a sum.  Each workgroup adds its rows' p and choices per branch, and those sums are
// joined in a fixed order by one last workgroup (up to 64 branches) or several.
//
// Up to 16 branches a row is one lane's, and the two launches' latency bounds the call: 114688
// masked bf16 rows to 2 of 8 branches 7 + 6 us.  131072 fp32 rows to 8 of 256 take 70 + 5 + 5 us
// for 138 MB: the vector units are 95 % busy with 276 operations a row, half of them the eight
// choices (16 each: six steps of a maximum over the wave, the ballot, the keys' move).  A way
// by keys alone, four rows a wave and 72 operations a choice, took 169 us.  Backward: 114688
// rows of 8 branches 5 us, 65536 bf16 rows of 64 12 us.
#include <algorithm>
#include <type_traits>

#include "launch_branch.hpp"
#include "vec.hpp"

namespace cgtp {
namespace {

// ---- lanes -------------------------------------------------------------------------

template <int Ctrl>
__device__ inline uint32_t dpp_u32(uint32_t v) {
  return uint32_t(__builtin_amdgcn_mov_dpp(int(v), Ctrl, 0xf, 0xf, true));
}
// Largest of L neighbouring lanes' values, to each of them: of keys 1 or 4 (the forward's wide
// rows have wave_max), of floats 1, 4, 16 or 64.
template <int L>
__device__ inline uint32_t lanes_max(uint32_t v) {
  static_assert(L == 1 || L == 4, "");
  if constexpr (L == 4) {
    v = max(v, dpp_u32<0xB1>(v));   // quad_perm 1 0 3 2
    v = max(v, dpp_u32<0x4E>(v));   // quad_perm 2 3 0 1
  }
  return v;
}
template <int L>
__device__ inline float lanes_fmax(float v) {
  if constexpr (L >= 4) {
    v = fmaxf(v, dpp<0xB1>(v));
    v = fmaxf(v, dpp<0x4E>(v));
  }
  if constexpr (L >= 16) {
    v = fmaxf(v, dpp<0x141>(v));    // row_half_mirror
    v = fmaxf(v, dpp<0x140>(v));    // row_mirror
  }
  if constexpr (L >= 64) {
    v = fmaxf(v, __shfl_xor(v, 16));
    v = fmaxf(v, __shfl_xor(v, 32));
  }
  return v;
}
// Sum over the lanes of a wave whose numbers leave the same rest by L, to each of them.
template <int L>
__device__ inline float same_sum(float v) {
  if constexpr (L <= 1) v += dpp<0x121>(v);   // row_ror 1, 2, 4, 8
  if constexpr (L <= 2) v += dpp<0x122>(v);
  if constexpr (L <= 4) v += dpp<0x124>(v);
  if constexpr (L <= 8) v += dpp<0x128>(v);
  if constexpr (L <= 16) v += __shfl_xor(v, 16);
  if constexpr (L <= 32) v += __shfl_xor(v, 32);
  return v;
}
template <int L>
__device__ inline float group_sum(float v) {
  if constexpr (L >= 4) v = lanes_sum<L>(v);
  return v;
}

// exp(x), x <= 0, to some 2 ulp: 2^t e^(x - t ln 2) with t = x log2(e) rounded, the second factor
// 1 + its small exponent.  From -200 on it is 0; NaN stays.
__device__ inline float exp_f32(float x) {
  x = x < -200.0f ? -200.0f : x;
  const float t = x * 1.44269504f;
  const float p = __builtin_amdgcn_exp2f(t);
  return fmaf(p, fmaf(t, -0.693147181f, x), p);
}

// Keys in the order of the logits: -infinity is kNone, NaN the largest, -0 is 0.
constexpr uint32_t kNone = 0x007fffffu, kNaN = 0xffffffffu;
__device__ inline uint32_t key_of(float z) {
  if (z != z) return kNaN;
  const uint32_t b = __builtin_bit_cast(uint32_t, z + 0.0f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ inline float of_key(uint32_t k) {
  if (k == kNaN) return __builtin_nanf("");
  return __builtin_bit_cast(float, k & 0x80000000u ? k & 0x7fffffffu : ~k);
}

// A lane's logits of a row; -infinity past the last.
template <int E, typename T>
__device__ inline void read_logits(const T* row, int first, int n, float (&z)[E]) {
  constexpr int V = E < 16 / int(sizeof(T)) ? E : 16 / int(sizeof(T));
  if (first + E <= n) {
#pragma unroll
    for (int q = 0; q < E / V; ++q) {
      const Vec<T, V> r = load_vec<false, T, V>(row + first + q * V);
#pragma unroll
      for (int j = 0; j < V; ++j) z[q * V + j] = to_f32(r.v[j]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < E; ++j) z[j] = first + j < n ? to_f32(row[first + j]) : -__builtin_inff();
  }
}
template <int E, typename T>
__device__ inline void write_logits(T* row, int first, int n, const float (&z)[E]) {
  constexpr int V = E < 16 / int(sizeof(T)) ? E : 16 / int(sizeof(T));
  if (first + E <= n) {
#pragma unroll
    for (int q = 0; q < E / V; ++q) {
      Vec<T, V> r;
#pragma unroll
      for (int j = 0; j < V; ++j) r.v[j] = from_f32<T>(z[q * V + j]);
      store_vec<false, T, V>(row + first + q * V, r);
    }
  } else {
#pragma unroll
    for (int j = 0; j < E; ++j)
      if (first + j < n) row[first + j] = from_f32<T>(z[j]);
  }
}

// ---- forward -----------------------------------------------------------------------

constexpr int kRouteBlock = 256;

// Where the workgroups' sums stand: [blocks][n] of p, [blocks][n] choices, [blocks] rows and
// [blocks] choices of all branches; and the shares of the balance loss of kJoinColumns branches
// each.
struct RouteWork {
  double* shares;
  float* p;
  int32_t* chosen;
  int32_t* rows;
  int32_t* picks;
  int blocks;
};
constexpr int kJoinColumns = 16;
// One workgroup alone has its sums of up to N branches in LDS.
template <int N>
struct RouteOwn {
  float p[N];
  int32_t chosen[N], rows, picks;
  __device__ RouteWork or_of(const RouteWork& w) {
    return w.blocks > 1 ? w : RouteWork{nullptr, p, chosen, &rows, &picks, 1};
  }
};

// Sum over a wave of a double, to every lane.
__device__ inline double wave_sum(double v) {
#pragma unroll
  for (int x = 1; x < kWave; x *= 2) v += __shfl_xor(v, x);
  return v;
}

// Counts, slopes and the balance loss from the workgroups' sums, in a fixed order.  By one
// whole workgroup of B.  Cols branches at once, by B / Cols threads each; lds: 2 (B + 64) doubles.
template <int B, int Cols>
__device__ inline void finish(const RouteCall& c, const RouteWork& w, double* lds) {
  constexpr int kSubs = B / Cols, kWaves = B / kWave;
  const int t = threadIdx.x, sub = t / Cols, lane = t % Cols;
  double* head = lds + 2 * B;   // of each wave: rows, then choices and their p
  int r = 0;
  for (int b = t; b < w.blocks; b += B) r += w.rows[b];
  double rows = wave_sum(double(r));
  if (t % kWave == 0) head[t / kWave] = rows;
  double all = 0, weighted = 0;   // C, and the sum of counts[e] (sum of p[e])
  for (int e0 = 0; e0 < c.n; e0 += Cols) {
    const int e = e0 + lane;
    double p = 0;
    int64_t count = 0;
    if (e < c.n) {
#pragma unroll 8
      for (int b = sub; b < w.blocks; b += kSubs) {
        p += w.p[int64_t(b) * c.n + e];
        count += w.chosen[int64_t(b) * c.n + e];
      }
    }
    double n = double(count);
    // lanes of one wave that have the same branch, then waves
#pragma unroll
    for (int x = Cols; x < kWave; x *= 2) {
      p += __shfl_xor(p, x);
      n += __shfl_xor(n, x);
    }
    __syncthreads();
    if (t % kWave < Cols) {
      lds[2 * t] = p;
      lds[2 * t + 1] = n;
    }
    __syncthreads();
    if (t < Cols && e < c.n) {
      constexpr int kStep = Cols < kWave ? kWave : Cols;   // from one that holds a branch to the next
      p = n = 0;
      for (int i = t; i < B; i += kStep) {
        p += lds[2 * i];
        n += lds[2 * i + 1];
      }
      c.counts[e] = int32_t(n);
      all += n;
      weighted += n * p;
    }
  }
  all = wave_sum(all);
  weighted = wave_sum(weighted);
  if (t % kWave == 0) {
    head[kWaves + t / kWave] = all;
    head[2 * kWaves + t / kWave] = weighted;
  }
  __syncthreads();   // the counts, too
  rows = all = weighted = 0;
#pragma unroll
  for (int i = 0; i < kWaves; ++i) {
    rows += head[i];
    all += head[kWaves + i];
    weighted += head[2 * kWaves + i];
  }
  const double factor = all * rows > 0 ? double(c.n) / (all * rows) : 0.0;
  if (t == 0) c.balance[0] = float(factor > 0 ? factor * weighted : 0.0);
  for (int e = t; e < c.n; e += B) c.slope[e] = float(factor * double(c.counts[e]));
}
// Branches at once, of n.
__host__ __device__ constexpr int columns_of(int n) { return n <= 4 ? 4 : n <= 16 ? 16 : n <= 64 ? 64 : 256; }

// A workgroup's sums from its threads': lanes of a wave that hold the same branches, then
// waves.  lds: B / kWave * L * E floats.
// `sums`: 2 where the choices are counted in n_of, 1 where they are elsewhere.
template <int B, int E, int L>
__device__ inline void write_sums(const RouteCall& c, const RouteWork& w, const float (&p_sum)[E], const int (&n_of)[E],
                                  int n_rows, int n_picks, float* lds, int32_t* lds_rows, int sums) {
  constexpr int kWaves = B / kWave;
  const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave;
  for (int what = 0; what < sums; ++what) {
#pragma unroll
    for (int j = 0; j < E; ++j) {
      const float v = same_sum<L>(what ? float(n_of[j]) : p_sum[j]);   // counts below 2^24: exact
      if (lane < L) lds[wave * L * E + lane * E + j] = v;
    }
    if (what == 0) {
      const float rows = lanes_sum<kWave>(float(n_rows)), picks = lanes_sum<kWave>(float(n_picks));
      if (lane == 0) {
        lds_rows[wave] = int(rows);
        lds_rows[kWaves + wave] = int(picks);
      }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < c.n; e += B) {
      float v = 0;
#pragma unroll
      for (int q = 0; q < kWaves; ++q) v += lds[q * L * E + e];
      if (what)
        w.chosen[int64_t(blockIdx.x) * c.n + e] = int32_t(v);
      else
        w.p[int64_t(blockIdx.x) * c.n + e] = v;
    }
    if (what == 0 && threadIdx.x < 2) {
      int s = 0;
#pragma unroll
      for (int q = 0; q < kWaves; ++q) s += lds_rows[threadIdx.x * kWaves + q];
      (threadIdx.x ? w.picks : w.rows)[blockIdx.x] = s;
    }
    __syncthreads();
  }
}

template <typename T, int E, int L>
__global__ __launch_bounds__(kRouteBlock) void route_fwd_kernel(RouteCall c, RouteWork work) {
  constexpr int kRows = kRouteBlock / L;   // at once
  constexpr int kMost = L * E < kMaxChosen ? L * E : kMaxChosen;
  constexpr int kSums = kRows * L * E, kPicks = kRows * kMost;
  __shared__ __align__(16) float lds[kSums > 2 * kPicks ? kSums : 2 * kPicks];
  __shared__ double room[2 * (kRouteBlock + kWave)];
  __shared__ int32_t lds_rows[2 * kRouteBlock / kWave];
  __shared__ RouteOwn<L * E> own;
  const RouteWork w = own.or_of(work);
  const int lane = threadIdx.x % L, first = lane * E, group = threadIdx.x / L;
  float* picked = lds + group * kMost;                                     // exp(z - top) of the choices
  int32_t* picked_id = reinterpret_cast<int32_t*>(lds) + kPicks + group * kMost;
  float p_sum[E];
  int n_of[E], n_rows = 0;
#pragma unroll
  for (int j = 0; j < E; ++j) p_sum[j] = 0, n_of[j] = 0;
  for (int64_t r = int64_t(blockIdx.x) * kRows + group; r < c.rows; r += int64_t(gridDim.x) * kRows) {
    float z[E];
    uint32_t key[E];
    if (!c.mask || c.mask[r] != 0) {
      read_logits(static_cast<const T*>(c.logits) + r * c.ld, first, c.n, z);
#pragma unroll
      for (int j = 0; j < E; ++j) key[j] = key_of(z[j]);
    } else {
#pragma unroll
      for (int j = 0; j < E; ++j) key[j] = kNone;
    }
    uint32_t chosen = 0;   // of the lane's branches
    bool part = false;
    float top = 0, sum = 0, kept = 0;   // the maximum; sums of exp(z - top), of all and of the chosen
    for (int i = 0; i < c.k; ++i) {
      uint32_t m = key[0];
#pragma unroll
      for (int j = 1; j < E; ++j) m = max(m, key[j]);
      m = lanes_max<L>(m);
      uint32_t at = 0;   // ~ the lowest branch that has it
#pragma unroll
      for (int j = E - 1; j >= 0; --j) at = key[j] == m ? ~uint32_t(first + j) : at;
      at = ~lanes_max<L>(at);
      const bool some = m > kNone;
      if (i == 0 && some) {
        part = true;
        top = of_key(m);
        float s = 0;
#pragma unroll
        for (int j = 0; j < E; ++j) {
          z[j] = exp_f32(z[j] - top);
          s += z[j];
        }
        sum = group_sum<L>(s);
      }
      float e = 0;
      if (some) {
        e = exp_f32(of_key(m) - top);
        kept += e;
#pragma unroll
        for (int j = 0; j < E; ++j)
          if (first + j == int(at)) {
            key[j] = 0;
            chosen |= 1u << j;
          }
      }
      if (lane == 0) {
        picked[i] = e;
        picked_id[i] = some ? int(at) : -1;
      }
    }
    const float inv = __builtin_amdgcn_rcpf(sum), scale = c.renormalise ? __builtin_amdgcn_rcpf(kept) : inv;
#pragma unroll
    for (int j = 0; j < E; ++j) {
      if (part) p_sum[j] += z[j] * inv;
      n_of[j] += chosen >> j & 1;
      if (c.dense && first + j < c.n)
        c.gates[int64_t(first + j) * c.rows + r] = chosen >> j & 1 ? z[j] * scale : 0.0f;
    }
    n_rows += part && lane == 0;
    // the row's lanes read what the first of them, of the same wave, has written
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    for (int i = lane; i < c.k; i += L) {
      const int id = picked_id[i];
      c.ids[r * c.k + i] = id;
      if (!c.dense) c.gates[r * c.k + i] = id < 0 ? 0.0f : picked[i] * scale;
    }
    __builtin_amdgcn_wave_barrier();
  }
  __syncthreads();
  write_sums<kRouteBlock, E, L>(c, w, p_sum, n_of, n_rows, 0, lds, lds_rows, 2);   // (the last step adds the choices itself)
  if (w.blocks == 1) finish<kRouteBlock, columns_of(L * E)>(c, w, room);   // the workgroup sees its own sums
}

// A row to a wave, n > 64.  Each lane sorts its E keys once; then the largest of the lanes'
// first keys is chosen k times, a ballot tells whose it was (of equal ones the lowest lane's,
// which has the lowest branches), and that lane's keys move up by one.  What the whole wave
// finds is held in scalar registers.  Lane i keeps the i-th choice's key and lane, and looks
// its branch up in the end.
constexpr int kLowest = int(0x80000000u);    // below every number's key
template <int Ctrl, int Rows>
__device__ inline int max_dpp(int v) {
  // the lowest number where a lane has no source: the form that fuses into one instruction
  if constexpr (Rows == 0xf) return max(v, __builtin_amdgcn_mov_dpp(v, Ctrl, 0xf, 0xf, true));
  return max(v, __builtin_amdgcn_update_dpp(kLowest, v, Ctrl, Rows, 0xf, false));
}
// To a scalar.
__device__ inline int wave_max(int v) {
  v = max_dpp<0xB1, 0xf>(v);    // quad_perm 1 0 3 2
  v = max_dpp<0x4E, 0xf>(v);    // quad_perm 2 3 0 1
  v = max_dpp<0x141, 0xf>(v);   // row_half_mirror
  v = max_dpp<0x140, 0xf>(v);   // row_mirror
  v = max_dpp<0x142, 0xa>(v);   // row_bcast 15: rows 1 and 3
  v = max_dpp<0x143, 0xc>(v);   // row_bcast 31: rows 2 and 3
  return __builtin_amdgcn_readlane(v, kWave - 1);
}
template <int Ctrl, int Rows>
__device__ inline float add_dpp(float v) {
  const int b = __builtin_bit_cast(int, v);
  if constexpr (Rows == 0xf) return v + dpp<Ctrl>(v);
  return v + __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, b, Ctrl, Rows, 0xf, false));
}
__device__ inline float wave_total(float v) {
  v = add_dpp<0xB1, 0xf>(v);
  v = add_dpp<0x4E, 0xf>(v);
  v = add_dpp<0x141, 0xf>(v);
  v = add_dpp<0x140, 0xf>(v);
  v = add_dpp<0x142, 0xa>(v);   // rows 1 and 3 are pairs of rows
  v = add_dpp<0x143, 0xc>(v);
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), kWave - 1));
}
__device__ inline int wide_key(float z) {
  const int b = __builtin_bit_cast(int, z + 0.0f);
  return b ^ int(uint32_t(b >> 31) >> 1);
}
__device__ inline float of_wide_key(int k) { return __builtin_bit_cast(float, k ^ int(uint32_t(k >> 31) >> 1)); }
constexpr int kMinusInf = int(0x807fffffu);  // -infinity's

// Largest first, by Batcher's odd-even merging network.
template <int E>
__device__ inline void sort_keys(int (&s)[E]) {
#pragma unroll
  for (int p = 1; p < E; p *= 2)
#pragma unroll
    for (int k = p; k >= 1; k /= 2)
#pragma unroll
      for (int j = k % p; j + k < E; j += 2 * k)
#pragma unroll
        for (int i = 0; i < k; ++i)
          if (i + j + k < E && (i + j) / (2 * p) == (i + j + k) / (2 * p)) {
            const int u = s[i + j], v = s[i + j + k];
            s[i + j] = max(u, v);
            s[i + j + k] = min(u, v);
          }
}

// Waves of a workgroup, and of a SIMD: eight of them hide the chain of each one's choices (131072
// rows to 8 of 256: 79 us, 93 with four), where the registers allow.
constexpr int wide_block(int e) { return e <= 8 ? 1024 : 512; }
template <typename T, int E>
__global__ __launch_bounds__(wide_block(E), E <= 4 ? 8 : E <= 8 ? 4 : 2) void route_fwd_wide_kernel(
    RouteCall c, RouteWork work) {
  constexpr int B = wide_block(E), kWaves = B / kWave;
  __shared__ __align__(16) float lds[kWaves * kWave * E];
  __shared__ double room[2 * (B + kWave)];
  __shared__ int32_t lds_rows[2 * kWaves], hist[kWave * E];   // hist: choices of each branch
  __shared__ RouteOwn<kWave * E> own;
  const RouteWork w = own.or_of(work);
  const int lane = threadIdx.x % kWave, first = lane * E;
  float p_sum[E];
  int n_rows = 0, n_picks = 0;
#pragma unroll
  for (int j = 0; j < E; ++j) p_sum[j] = 0;
  for (int e = threadIdx.x; e < c.n; e += B) hist[e] = 0;
  __syncthreads();
  const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x) / kWave);
  // the next row's logits are on their way while a row is routed
  const int64_t r0 = int64_t(blockIdx.x) * kWaves + wave, step = int64_t(gridDim.x) * kWaves;
  float next[E];
  bool next_in = false;
  auto read = [&](int64_t r) {
    next_in = r < c.rows && (!c.mask || c.mask[r] != 0);
    if (next_in) read_logits(static_cast<const T*>(c.logits) + r * c.ld, first, c.n, next);
  };
  read(r0);
  for (int64_t r = r0; r < c.rows; r += step) {
    int id = -1;
    float gate = 0;
    float z[E];
    const bool in = next_in;
#pragma unroll
    for (int j = 0; j < E; ++j) z[j] = next[j];
    read(r + step);
    if (in) {
      int key[E], s[E];
#pragma unroll
      for (int j = 0; j < E; ++j) s[j] = key[j] = wide_key(z[j]);
      sort_keys(s);
      int m = wave_max(s[0]);
      const float top = of_wide_key(m);
      float e[E], sum = 0;
#pragma unroll
      for (int j = 0; j < E; ++j) {
        e[j] = exp_f32(z[j] - top);
        sum += e[j];
      }
      sum = wave_total(sum);
      if (!(sum < __builtin_inff())) {
        // no number on top: NaN above infinity above the others, or all -infinity
#pragma unroll
        for (int j = 0; j < E; ++j) {
          s[j] = key[j] = z[j] != z[j] ? 0x7fffffff : wide_key(z[j]);
          e[j] = sum;   // NaN
        }
        sort_keys(s);
        m = wave_max(s[0]);
      }
      if (m > kMinusInf) {
        int got = kMinusInf, from = 0;   // lane i's: the i-th choice's key and lane
        int found = 0;
        do {
          const int at = __builtin_ctzll(__ballot(s[0] == m));
          const bool mine = __builtin_amdgcn_inverse_ballot_w64(uint64_t(1) << at);
#pragma unroll
          for (int j = 0; j + 1 < E; ++j) {
            const int above = s[j], below = s[j + 1];   // values: of two elements it would select the index
            s[j] = mine ? below : above;
          }
          if (mine) s[E - 1] = kLowest;
          const bool next_one = __builtin_amdgcn_inverse_ballot_w64(uint64_t(1) << found);
          got = next_one ? m : got;
          from = next_one ? at : from;
          if (++found == c.k) break;
          m = wave_max(s[0]);
        } while (m > kMinusInf);
        // a choice's branch is the first of its lane's that has the key, or the one behind where
        // the choice before was of the same lane and key
        const int got_before = __builtin_amdgcn_update_dpp(kLowest, got, 0x138, 0xf, 0xf, false);   // wave_shr 1
        const int from_before = __builtin_amdgcn_update_dpp(-1, from, 0x138, 0xf, 0xf, false);
        int skip = 0;
        if (__ballot(lane < found && got == got_before && from == from_before)) {
          for (int i = 0; i < found; ++i) {
            const int g = __builtin_amdgcn_readlane(got, i), f = __builtin_amdgcn_readlane(from, i);
            skip += i < lane && g == got && f == from;
          }
#pragma unroll
          for (int j = 0; j < E; ++j) {
            const bool same = __builtin_amdgcn_ds_bpermute(from * 4, key[j]) == got;
            if (same && skip-- == 0) id = from * E + j;
          }
        } else {
#pragma unroll
          for (int j = E - 1; j >= 0; --j)
            if (__builtin_amdgcn_ds_bpermute(from * 4, key[j]) == got) id = from * E + j;
        }
        id = lane < found ? id : -1;
        if (lane < found) atomicAdd(hist + id, 1);   // whole numbers: in any order
        const float inv = __builtin_amdgcn_rcpf(sum);
        float mine = exp_f32(of_wide_key(got) - top);
        mine = sum != sum ? sum : mine;   // a NaN key's value is none
        mine = lane < found ? mine : 0.0f;
        const float scale = c.renormalise ? __builtin_amdgcn_rcpf(wave_total(mine)) : inv;
        gate = mine * scale;
#pragma unroll
        for (int j = 0; j < E; ++j) p_sum[j] += e[j] * inv;
        ++n_rows;
        n_picks += found;
      }
    }
    if (lane < c.k) {
      c.ids[r * c.k + lane] = id;
      if (!c.dense) c.gates[r * c.k + lane] = gate;
    }
    if (c.dense) {
      float out[E] = {};
      for (int i = 0; i < c.k; ++i) {
        const int of = __builtin_amdgcn_readlane(id, i);
        const float v = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, gate), i));
#pragma unroll
        for (int j = 0; j < E; ++j) out[j] = first + j == of ? v : out[j];
      }
#pragma unroll
      for (int j = 0; j < E; ++j)
        if (first + j < c.n) c.gates[int64_t(first + j) * c.rows + r] = out[j];
    }
  }
  // rows were counted by every lane
  const int none[E] = {};
  write_sums<B, E, kWave>(c, w, p_sum, none, lane == 0 ? n_rows : 0, lane == 0 ? n_picks : 0, lds, lds_rows, 1);
  for (int e = threadIdx.x; e < c.n; e += B) w.chosen[int64_t(blockIdx.x) * c.n + e] = hist[e];
  if (w.blocks == 1) {
    __syncthreads();
    finish<B, columns_of(kWave * E)>(c, w, room);
  }
}

// n <= 64.
constexpr int kFinishBlock = 1024;
__global__ __launch_bounds__(kFinishBlock) void route_finish_kernel(RouteCall c, RouteWork w) {
  __shared__ double room[2 * (kFinishBlock + kWave)];
  if (c.n <= 4)
    finish<kFinishBlock, 4>(c, w, room);
  else if (c.n <= 16)
    finish<kFinishBlock, 16>(c, w, room);
  else
    finish<kFinishBlock, 64>(c, w, room);
}

// The same in many workgroups, kJoinColumns branches each, where there are many sums: counts,
// slopes and the branches' share of the balance loss, which a last wave adds.
constexpr int kJoinBlock = 1024;
__global__ __launch_bounds__(kJoinBlock) void route_join_kernel(RouteCall c, RouteWork w) {
  constexpr int kWaves = kJoinBlock / kWave, kSubs = kJoinBlock / kJoinColumns;
  __shared__ double head[2][kWaves], lds[2][kWaves][kJoinColumns];
  const int t = threadIdx.x, wave = t / kWave, sub = t / kJoinColumns, lane = t % kJoinColumns;
  const int e = int(blockIdx.x) * kJoinColumns + lane;
  double rows = 0, picks = 0, p = 0, n = 0;
  for (int b = t; b < w.blocks; b += kJoinBlock) {
    rows += w.rows[b];
    picks += w.picks[b];
  }
  if (e < c.n) {
#pragma unroll 8
    for (int b = sub; b < w.blocks; b += kSubs) {
      p += w.p[int64_t(b) * c.n + e];
      n += w.chosen[int64_t(b) * c.n + e];
    }
  }
  rows = wave_sum(rows);
  picks = wave_sum(picks);
#pragma unroll
  for (int x = kJoinColumns; x < kWave; x *= 2) {
    p += __shfl_xor(p, x);
    n += __shfl_xor(n, x);
  }
  if (t % kWave == 0) head[0][wave] = rows, head[1][wave] = picks;
  if (t % kWave < kJoinColumns) lds[0][wave][lane] = p, lds[1][wave][lane] = n;
  __syncthreads();
  if (t >= kWave) return;
  rows = picks = p = n = 0;
#pragma unroll
  for (int i = 0; i < kWaves; ++i) {
    rows += head[0][i];
    picks += head[1][i];
    p += lds[0][i][lane];
    n += lds[1][i][lane];
  }
  const double factor = rows * picks > 0 ? double(c.n) / (rows * picks) : 0.0;
  const bool mine = t < kJoinColumns && e < c.n;
  if (mine) {
    c.counts[e] = int32_t(n);
    c.slope[e] = float(factor * n);
  }
  const double share = wave_sum(mine && factor > 0 ? factor * n * p : 0.0);
  if (t == 0) w.shares[blockIdx.x] = share;
}
__global__ __launch_bounds__(kWave) void route_balance_kernel(RouteCall c, RouteWork w, int shares) {
  const double all = wave_sum(int(threadIdx.x) < shares ? w.shares[threadIdx.x] : 0.0);
  if (threadIdx.x == 0) c.balance[0] = float(all);
}
static_assert(kMaxBranches <= kWave * kJoinColumns, "a wave adds the shares");

// ---- backward ----------------------------------------------------------------------

// Between LDS accesses of one wave's lanes, which the hardware keeps in order.
__device__ inline void wave_in_order() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// The bits of a float that number() does not return.
constexpr uint32_t kNotChosen = 0xffffffffu;
__device__ inline float number(float v) { return v == v ? v : __builtin_nanf(""); }

// dz = p (u - sum(u p)), u the gradient with respect to p: grad_balance slope, and at the
// chosen the gates' gradients.  Renormalised gates q = p / (sum of the chosen p) are a
// softmax of the chosen alone: dz gets q (v - sum(v q)) there instead, v the gates' gradients.
template <typename T, int E, int L>
__global__ __launch_bounds__(kRouteBlock) void route_bwd_kernel(RouteCall c) {
  constexpr int kRows = kRouteBlock / L;
  // where a row has many lanes, the choices' gradients reach their branches' lanes through LDS
  constexpr bool kScatter = L > 1;
  __shared__ __align__(16) uint32_t lds[kScatter ? kRows * L * E : 1];
  const int lane = threadIdx.x % L, first = lane * E;
  float slope[E];
#pragma unroll
  for (int j = 0; j < E; ++j)
    slope[j] = c.grad_balance && first + j < c.n ? c.grad_balance[0] * c.slope[first + j] : 0.0f;
  bool twice = false;   // a branch twice in a row
  auto one_row = [&](int64_t r, auto in_order) {
    T* out = static_cast<T*>(c.grad_logits) + r * c.ld_g;
    const int32_t* ids = c.ids + r * c.k;
    float z[E], d[E];
    if (unsigned(ids[0]) >= unsigned(c.n)) {   // takes no part
#pragma unroll
      for (int j = 0; j < E; ++j) d[j] = 0;
      write_logits(out, first, c.n, d);
      return;
    }
    read_logits(static_cast<const T*>(c.logits) + r * c.ld, first, c.n, z);
    float top = z[0];   // NaN and infinity show in the sum
#pragma unroll
    for (int j = 1; j < E; ++j) top = fmaxf(top, z[j]);
    top = lanes_fmax<L>(top);
    float s = 0, up[E];
    uint32_t chosen = 0;
#pragma unroll
    for (int j = 0; j < E; ++j) {
      z[j] = exp_f32(z[j] - top);
      s += z[j];
      up[j] = 0;
    }
    const float inv = __builtin_amdgcn_rcpf(group_sum<L>(s));
    if constexpr (kScatter) {
      if (c.grad_gates) {
        uint32_t* row = lds + threadIdx.x / L * (L * E);
        auto gate_grad = [&](int id, int i) { return c.grad_gates[c.dense ? int64_t(id) * c.rows + r : r * c.k + i]; };
#pragma unroll
        for (int j = 0; j < E; ++j) row[first + j] = kNotChosen;
        wave_in_order();
        int given = 0, found = 0;   // choices of the wave's rows, and branches that have one
        if constexpr (in_order()) {
          for (int i = 0; lane == 0 && i < c.k; ++i) {
            const int id = ids[i];
            if (unsigned(id) >= unsigned(c.n)) continue;
            const uint32_t b = row[id];
            const float sum = b == kNotChosen ? 0.0f : __builtin_bit_cast(float, b);
            row[id] = __builtin_bit_cast(uint32_t, number(sum + gate_grad(id, i)));
          }
        } else {
          for (int i0 = 0; i0 < c.k; i0 += L) {
            const int i = i0 + lane, id = i < c.k ? ids[i] : -1;
            const bool some = unsigned(id) < unsigned(c.n);
            if (some) row[id] = __builtin_bit_cast(uint32_t, number(gate_grad(id, i) + 0.0f));   // as a sum that begins with 0
            given += __popcll(__ballot(some));
          }
        }
        wave_in_order();
#pragma unroll
        for (int j = 0; j < E; ++j) {
          const uint32_t b = row[first + j];
          const bool in = b != kNotChosen;
          up[j] = in ? __builtin_bit_cast(float, b) : 0.0f;
          chosen |= uint32_t(in) << j;
          found += __popcll(__ballot(in));
        }
        if constexpr (!in_order()) twice |= found != given;
        wave_in_order();
      }
    } else if (c.grad_gates) {
      // four choices' loads at once; past the last it is read again and left out
      for (int i0 = 0; i0 < c.k; i0 += 4) {
        int id[4];
        float v[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) id[q] = ids[min(i0 + q, c.k - 1)];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const bool some = unsigned(id[q]) < unsigned(c.n);
          v[q] = c.grad_gates[c.dense ? int64_t(some ? id[q] : 0) * c.rows + r : r * c.k + min(i0 + q, c.k - 1)];
          if (!some || i0 + q >= c.k) id[q] = -1;
        }
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int j = 0; j < E; ++j)
            if (first + j == id[q]) {
              up[j] += v[q];
              chosen |= 1u << j;
            }
      }
    }
    float dot = 0;
#pragma unroll
    for (int j = 0; j < E; ++j) {
      d[j] = slope[j] + (c.renormalise ? 0.0f : up[j]);
      dot += d[j] * (z[j] * inv);
    }
    dot = group_sum<L>(dot);
#pragma unroll
    for (int j = 0; j < E; ++j) d[j] = z[j] * inv * (d[j] - dot);
    if (c.renormalise && c.grad_gates) {
      float q = 0, v = 0;
#pragma unroll
      for (int j = 0; j < E; ++j) {
        const float e = chosen >> j & 1 ? z[j] : 0.0f;
        q += e;
        v += e * up[j];
      }
      q = 1.0f / group_sum<L>(q);
      v = group_sum<L>(v) * q;
#pragma unroll
      for (int j = 0; j < E; ++j)
        if (chosen >> j & 1) d[j] += z[j] * q * (up[j] - v);
    }
    write_logits(out, first, c.n, d);
  };
  auto rows = [&](auto in_order) {
    uint32_t t = threadIdx.x;
    if constexpr (in_order()) asm volatile("" : "+v"(t));   // computed again, not held meanwhile
    for (int64_t r = int64_t(blockIdx.x) * kRows + t / L; r < c.rows; r += int64_t(gridDim.x) * kRows) one_row(r, in_order);
  };
  rows(std::false_type{});
  // A branch twice in a row, which the forward does not write: the rows again, with gradients added
  // in the choices' order by a row's first lane.  (Done within the loop it made the loop slower:
  // 131072 rows of 256 83 us, 67 so.)
  if constexpr (kScatter)
    if (twice) rows(std::true_type{});
}

// ---- launches ----------------------------------------------------------------------

// The forward's workgroups: one where it would take four turns at most; else no more than fill
// the device.
int route_blocks(int64_t rows, int n) {
  const int at_once = n <= 16 ? kRouteBlock : n <= 64 ? kRouteBlock / 4 : wide_block(n <= 512 ? 8 : 16) / kWave;
  const int64_t turns = (rows + at_once - 1) / at_once;
  return turns <= 4 ? 1 : int(std::min<int64_t>(turns, n <= 64 ? 1024 : n <= 256 ? 512 : 256));
}
RouteWork route_work(const RouteCall& c) {
  RouteWork w;
  w.blocks = route_blocks(c.rows, c.n);
  w.shares = reinterpret_cast<double*>(c.work);
  w.p = c.work + 2 * kWave;
  w.chosen = reinterpret_cast<int32_t*>(w.p + int64_t(w.blocks) * c.n);
  w.rows = w.chosen + int64_t(w.blocks) * c.n;
  w.picks = w.rows + w.blocks;
  return w;
}
// Of up to 64 branches one workgroup joins the sums, 2^16 of them at most; of more, many do.
// Traced, us of the one and of the two launches for many: 448 workgroups' sums of 8 branches 5.9
// and 6.8, 1024 of 32 8.6 and 6.8, 1024 of 64 9.4 and 7 to 9.6 (whole calls 19.0 and 21.9, 21.5 and
// 21.3, 36.1 and 34.3); 512 of 256, by the two, 10.
void finish(const RouteCall& c, const RouteWork& w, hipStream_t s) {
  if (w.blocks == 1) return;
  if (c.n <= 64) {
    hipLaunchKernelGGL(route_finish_kernel, dim3(1), dim3(kFinishBlock), 0, s, c, w);
    return;
  }
  const int shares = (c.n + kJoinColumns - 1) / kJoinColumns;
  hipLaunchKernelGGL(route_join_kernel, dim3(unsigned(shares)), dim3(kJoinBlock), 0, s, c, w);
  hipLaunchKernelGGL(route_balance_kernel, dim3(1), dim3(kWave), 0, s, c, w, shares);
}

template <typename T, int E, int L>
void backward(const RouteCall& c, hipStream_t s) {
  constexpr int64_t kMost = 4096;
  const int64_t blocks = std::min((c.rows * L + kRouteBlock - 1) / kRouteBlock, kMost);
  hipLaunchKernelGGL((route_bwd_kernel<T, E, L>), dim3(unsigned(blocks)), dim3(kRouteBlock), 0, s, c);
}
// E branches a lane and L lanes of a row, in the backward Eb and Lb.
template <typename T, int E, int L, int Eb = E, int Lb = L>
void run(const RouteCall& c, bool back, hipStream_t s) {
  if (back) return backward<T, Eb, Lb>(c, s);
  const RouteWork w = route_work(c);
  hipLaunchKernelGGL((route_fwd_kernel<T, E, L>), dim3(unsigned(w.blocks)), dim3(kRouteBlock), 0, s, c, w);
  finish(c, w, s);
}
// n > 64: a wave to a row in the forward; Eb branches a lane and Lb lanes in the backward.
template <typename T, int E, int Eb, int Lb>
void run_wide(const RouteCall& c, bool back, hipStream_t s) {
  if (back) return backward<T, Eb, Lb>(c, s);
  const RouteWork w = route_work(c);
  hipLaunchKernelGGL((route_fwd_wide_kernel<T, E>), dim3(unsigned(w.blocks)), dim3(wide_block(E)), 0, s, c, w);
  finish(c, w, s);
}
// The backward keeps no sums: four branches a lane take less time than sixteen (131072 rows of 64
// fp32 logits 17 us, 24; of 256 68 us, 93).  One rule for all types: 65536 rows of 64 in bf16 would
// take 10.7 us by sixteen, 11.6 by four.
template <typename T>
hipError_t run(const RouteCall& c, bool backward, hipStream_t s) {
  if (c.n <= 4)
    run<T, 4, 1>(c, backward, s);
  else if (c.n <= 8)
    run<T, 8, 1>(c, backward, s);
  else if (c.n <= 16)
    run<T, 16, 1>(c, backward, s);
  else if (c.n <= 32)
    run<T, 8, 4>(c, backward, s);
  else if (c.n <= 64)
    run<T, 16, 4, 4, 16>(c, backward, s);
  else if (c.n <= 128)
    run_wide<T, 2, 8, 16>(c, backward, s);
  else if (c.n <= 256)
    run_wide<T, 4, 4, 64>(c, backward, s);
  else if (c.n <= 512)
    run_wide<T, 8, 8, 64>(c, backward, s);
  else
    run_wide<T, 16, 16, 64>(c, backward, s);
  return hipGetLastError();
}
hipError_t run(const RouteCall& c, Elem type, bool backward, hipStream_t s) {
  return type == Elem::f32 ? run<float>(c, backward, s)
         : type == Elem::bf16 ? run<Bf16>(c, backward, s) : run<F16>(c, backward, s);
}

// ---- gate --------------------------------------------------------------------------

// An active edge's rows of w and grad_w are read once: bound by HBM.  L lanes take a row, 16
// bytes each, kUnroll loads of each kind in flight.  114688 edges x 1312 weights, half of them
// active: 103 us (5.8 TB/s); 20060 x 2176: 57 us (6.1 TB/s).
constexpr int kGateBlock = 256, kUnroll = 4;
template <int L>
__global__ __launch_bounds__(kGateBlock) void gate_bwd_kernel(GateCall c) {
  constexpr int kRows = kGateBlock / L, V = 4;
  const int lane = threadIdx.x % L;
  for (int64_t e = int64_t(blockIdx.x) * kRows + threadIdx.x / L; e < c.edges; e += int64_t(gridDim.x) * kRows) {
    const float gate = c.mask && c.mask[e] == 0 ? 0.0f : c.gate[e];
    float s[kUnroll] = {};
    if (gate != 0) {
      const float *w = c.w + e * c.width, *g = c.grad_w + e * c.width;
      int64_t at = int64_t(lane) * V;
      for (; at + (kUnroll - 1) * L * V + V <= c.width; at += kUnroll * L * V) {
        Vec<float, V> a[kUnroll], b[kUnroll];
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
          a[i] = load_vec<false, float, V>(w + at + i * L * V);
          b[i] = load_vec<false, float, V>(g + at + i * L * V);
        }
#pragma unroll
        for (int i = 0; i < kUnroll; ++i)
#pragma unroll
          for (int j = 0; j < V; ++j) s[i] = fmaf(a[i].v[j], b[i].v[j], s[i]);
      }
      for (; at < c.width; at += L * V) {
        if (at + V <= c.width) {
          const Vec<float, V> a = load_vec<false, float, V>(w + at), b = load_vec<false, float, V>(g + at);
#pragma unroll
          for (int j = 0; j < V; ++j) s[0] = fmaf(a.v[j], b.v[j], s[0]);
        } else {
          for (int64_t k = at; k < c.width; ++k) s[0] = fmaf(w[k], g[k], s[0]);
        }
      }
    }
    const float dot = lanes_sum<L>((s[0] + s[1]) + (s[2] + s[3]));
    if (lane == 0) c.grad_gate[e] = gate != 0 ? dot / gate : 0.0f;
  }
}

}  // namespace

size_t route_floats(int64_t rows, int n) {
  const size_t blocks = size_t(route_blocks(rows, n));
  return blocks == 1 ? 0 : 2 * kWave + blocks * (2 * size_t(n) + 2);
}
hipError_t launch_route_forward(const RouteCall& c, Elem type, hipStream_t s) { return run(c, type, false, s); }
hipError_t launch_route_backward(const RouteCall& c, Elem type, hipStream_t s) { return run(c, type, true, s); }

hipError_t launch_gate_backward(const GateCall& c, hipStream_t s) {
  const int lanes = c.width <= 128 ? 16 : 64;
  const int64_t blocks = std::min<int64_t>((c.edges * lanes + kGateBlock - 1) / kGateBlock, 1 << 20);
  if (lanes == 16)
    hipLaunchKernelGGL(gate_bwd_kernel<16>, dim3(unsigned(blocks)), dim3(kGateBlock), 0, s, c);
  else
    hipLaunchKernelGGL(gate_bwd_kernel<64>, dim3(unsigned(blocks)), dim3(kGateBlock), 0, s, c);
  return hipGetLastError();
}

}  // namespace cgtp

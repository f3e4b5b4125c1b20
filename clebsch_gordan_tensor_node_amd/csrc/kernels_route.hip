// Routing of rows to branches by their logits, its balance loss, the way back to the
// logits, and the gradient of the convolution's gate.
//
// A row's n logits are held by L neighbouring lanes, E each (n <= L E), lane l those of the
// branches l E to l E + E - 1.  They choose k times the largest of what is left, by a key of
// 32 bits in the logits' order; p = softmax needs the row's maximum, which the first choice
// gives, and a sum.  Each workgroup adds its rows' p and choices per branch, and one last
// workgroup joins those sums in a fixed order.
#include <algorithm>

#include "launch_branch.hpp"
#include "vec.hpp"

namespace cgtp {
namespace {

// ---- lanes -------------------------------------------------------------------------

template <int Ctrl>
__device__ inline uint32_t dpp_u32(uint32_t v) {
  return uint32_t(__builtin_amdgcn_mov_dpp(int(v), Ctrl, 0xf, 0xf, true));
}
// Largest of L neighbouring lanes' values (1, 4, 16 or 64), to each of them.
template <int L>
__device__ inline uint32_t lanes_max(uint32_t v) {
  if constexpr (L >= 4) {
    v = max(v, dpp_u32<0xB1>(v));   // quad_perm 1 0 3 2
    v = max(v, dpp_u32<0x4E>(v));   // quad_perm 2 3 0 1
  }
  if constexpr (L >= 16) {
    v = max(v, dpp_u32<0x141>(v));  // row_half_mirror
    v = max(v, dpp_u32<0x140>(v));  // row_mirror
  }
  if constexpr (L >= 64) {
    v = max(v, uint32_t(__shfl_xor(int(v), 16)));
    v = max(v, uint32_t(__shfl_xor(int(v), 32)));
  }
  return v;
}
template <int L>
__device__ inline float group_sum(float v) {
  if constexpr (L >= 4) v = lanes_sum<L>(v);
  return v;
}

// exp(x), x <= 0, to some 2 ulp: 2^t with t = x log2(e) rounded, times 1 + what that left out.
__device__ inline float exp_f32(float x) {
  constexpr float kLog2e = 1.44269504f, kRest = 1.92596303e-8f, kLn2 = 0.693147181f;
  const float t = x * kLog2e;
  const float rest = fmaf(x, kRest, fmaf(x, kLog2e, -t));
  const float p = __builtin_amdgcn_exp2f(t);
  return p > 0 ? fmaf(p, rest * kLn2, p) : p;   // -infinity leaves NaN in the rest; NaN stays
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

// Where the workgroups' sums stand: [blocks][n] of p, [blocks][n] choices, [blocks] rows.
struct RouteWork {
  float* p;
  int32_t* chosen;
  int32_t* rows;
  int blocks;
};

// Counts, slopes and the balance loss from the workgroups' sums, in a fixed order.  By one
// whole workgroup; lds: 2 * blockDim.x doubles.
__device__ inline void finish(const RouteCall& c, const RouteWork& w, double* lds) {
  const int threads = int(blockDim.x), t = threadIdx.x;
  int r = 0;
  for (int b = t; b < w.blocks; b += threads) r += w.rows[b];
  int* whole = reinterpret_cast<int*>(lds);
  whole[t] = r;
  __syncthreads();
  for (int half = threads / 2; half > 0; half /= 2) {
    if (t < half) whole[t] += whole[t + half];
    __syncthreads();
  }
  const double rows = whole[0];
  __syncthreads();
  // `subs` threads for each of `cols` branches at once
  const int cols = min(threads, c.n <= 4 ? 4 : c.n <= 16 ? 16 : c.n <= 64 ? 64 : c.n <= 256 ? 256 : 1024);
  const int subs = threads / cols, sub = t / cols, lane = t % cols;
  double all = 0, weighted = 0;   // C, and the sum of counts[e] (sum of p[e])
  for (int e0 = 0; e0 < c.n; e0 += cols) {
    const int e = e0 + lane;
    double p = 0, count = 0;
    if (e < c.n) {
#pragma unroll 4
      for (int b = sub; b < w.blocks; b += subs) {
        p += w.p[int64_t(b) * c.n + e];
        count += w.chosen[int64_t(b) * c.n + e];
      }
    }
    lds[2 * t] = p;
    lds[2 * t + 1] = count;
    __syncthreads();
    if (sub == 0 && e < c.n) {
      for (int i = 1; i < subs; ++i) {
        p += lds[2 * (i * cols + lane)];
        count += lds[2 * (i * cols + lane) + 1];
      }
      c.counts[e] = int32_t(count);
      all += count;
      weighted += count * p;
    }
    __syncthreads();
  }
  lds[2 * t] = all;
  lds[2 * t + 1] = weighted;
  __syncthreads();
  for (int half = threads / 2; half > 0; half /= 2) {
    if (t < half) {
      lds[2 * t] += lds[2 * (t + half)];
      lds[2 * t + 1] += lds[2 * (t + half) + 1];
    }
    __syncthreads();
  }
  const double factor = lds[0] * rows > 0 ? double(c.n) / (lds[0] * rows) : 0.0;
  if (t == 0) c.balance[0] = float(factor > 0 ? factor * lds[1] : 0.0);
  for (int e = t; e < c.n; e += threads) c.slope[e] = float(factor * double(c.counts[e]));
}

template <typename T, int E, int L>
__global__ __launch_bounds__(kRouteBlock) void route_fwd_kernel(RouteCall c, RouteWork w) {
  constexpr int kRows = kRouteBlock / L;   // at once
  constexpr int kMost = L * E < kMaxChosen ? L * E : kMaxChosen;
  constexpr int kSums = kRows * L * E, kPicks = kRows * kMost;
  __shared__ __align__(16) float lds[kSums > 2 * kPicks ? kSums : 2 * kPicks];
  __shared__ double room[2 * kRouteBlock];
  __shared__ int32_t lds_rows[kRouteBlock / kWave];
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
    const float inv = 1.0f / sum, scale = c.renormalise ? 1.0f / kept : inv;
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
  // the workgroup's sums: its row groups' in a fixed order
  for (int what = 0; what < 2; ++what) {
#pragma unroll
    for (int j = 0; j < E; ++j) lds[group * L * E + first + j] = what ? float(n_of[j]) : p_sum[j];   // below 2^24: exact
    for (int half = kRows / 2; half > 0; half /= 2) {
      __syncthreads();
      for (int e = threadIdx.x; e < half * L * E; e += kRouteBlock) lds[e] += lds[e + half * L * E];
    }
    __syncthreads();
    for (int e = threadIdx.x; e < c.n; e += kRouteBlock) {
      if (what)
        w.chosen[int64_t(blockIdx.x) * c.n + e] = int32_t(lds[e]);
      else
        w.p[int64_t(blockIdx.x) * c.n + e] = lds[e];
    }
    __syncthreads();
  }
#pragma unroll
  for (int x = 1; x < kWave; x *= 2) n_rows += __shfl_xor(n_rows, x);
  if (threadIdx.x % kWave == 0) lds_rows[threadIdx.x / kWave] = n_rows;
  __syncthreads();
  if (threadIdx.x == 0) {
    int s = 0;
    for (int q = 0; q < kRouteBlock / kWave; ++q) s += lds_rows[q];
    w.rows[blockIdx.x] = s;
  }
  if (w.blocks == 1) {
    __syncthreads();   // the workgroup sees its own sums
    finish(c, w, room);
  }
}

constexpr int kFinishBlock = 1024;
__global__ __launch_bounds__(kFinishBlock) void route_finish_kernel(RouteCall c, RouteWork w) {
  __shared__ double room[2 * kFinishBlock];
  finish(c, w, room);
}

// ---- backward ----------------------------------------------------------------------

// dz = p (u - sum(u p)), u the gradient with respect to p: grad_balance slope, and at the
// chosen the gates' gradients.  Renormalised gates q = p / (sum of the chosen p) are a
// softmax of the chosen alone: dz gets q (v - sum(v q)) there instead, v the gates' gradients.
template <typename T, int E, int L>
__global__ __launch_bounds__(kRouteBlock) void route_bwd_kernel(RouteCall c) {
  constexpr int kRows = kRouteBlock / L;
  const int lane = threadIdx.x % L, first = lane * E;
  float slope[E];
#pragma unroll
  for (int j = 0; j < E; ++j)
    slope[j] = c.grad_balance && first + j < c.n ? c.grad_balance[0] * c.slope[first + j] : 0.0f;
  for (int64_t r = int64_t(blockIdx.x) * kRows + threadIdx.x / L; r < c.rows; r += int64_t(gridDim.x) * kRows) {
    T* out = static_cast<T*>(c.grad_logits) + r * c.ld_g;
    const int32_t* ids = c.ids + r * c.k;
    float z[E], d[E];
    if (unsigned(ids[0]) >= unsigned(c.n)) {   // takes no part
#pragma unroll
      for (int j = 0; j < E; ++j) d[j] = 0;
      write_logits(out, first, c.n, d);
      continue;
    }
    read_logits(static_cast<const T*>(c.logits) + r * c.ld, first, c.n, z);
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < E; ++j) m = max(m, key_of(z[j]));
    const float top = of_key(lanes_max<L>(m));
    float s = 0, up[E];
    uint32_t chosen = 0;
#pragma unroll
    for (int j = 0; j < E; ++j) {
      z[j] = exp_f32(z[j] - top);
      s += z[j];
      up[j] = 0;
    }
    const float inv = 1.0f / group_sum<L>(s);
    if (c.grad_gates) {
      for (int i = 0; i < c.k; ++i) {
        const int id = ids[i];
        if (unsigned(id) >= unsigned(c.n)) continue;
        const float v = c.grad_gates[c.dense ? int64_t(id) * c.rows + r : r * c.k + i];
#pragma unroll
        for (int j = 0; j < E; ++j)
          if (first + j == id) {
            up[j] += v;
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
  }
}

// ---- launches ----------------------------------------------------------------------

// The forward's workgroups: one where they would take four turns at most; else no more than
// leave 2^16 sums of a kind to join (256 at least, 1024 at most).
int route_blocks(int64_t rows, int n) {
  const int lanes = n <= 16 ? 1 : n <= 64 ? 4 : n <= 256 ? 16 : 64;
  const int64_t turns = (rows * lanes + kRouteBlock - 1) / kRouteBlock;
  if (turns <= 4) return 1;
  return int(std::min<int64_t>(turns, std::max(256, std::min(1024, 65536 / n))));
}

template <typename T, int E, int L>
void run(const RouteCall& c, bool backward, hipStream_t s) {
  if (backward) {
    constexpr int64_t kMost = 4096;
    const int64_t blocks = std::min((c.rows * L + kRouteBlock - 1) / kRouteBlock, kMost);
    hipLaunchKernelGGL((route_bwd_kernel<T, E, L>), dim3(unsigned(blocks)), dim3(kRouteBlock), 0, s, c);
    return;
  }
  RouteWork w;
  w.blocks = route_blocks(c.rows, c.n);
  w.p = c.work;
  w.chosen = reinterpret_cast<int32_t*>(c.work + int64_t(w.blocks) * c.n);
  w.rows = w.chosen + int64_t(w.blocks) * c.n;
  hipLaunchKernelGGL((route_fwd_kernel<T, E, L>), dim3(unsigned(w.blocks)), dim3(kRouteBlock), 0, s, c, w);
  if (w.blocks > 1) hipLaunchKernelGGL(route_finish_kernel, dim3(1), dim3(kFinishBlock), 0, s, c, w);
}
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
    run<T, 16, 4>(c, backward, s);
  else if (c.n <= 128)
    run<T, 8, 16>(c, backward, s);
  else if (c.n <= 256)
    run<T, 16, 16>(c, backward, s);
  else if (c.n <= 512)
    run<T, 8, 64>(c, backward, s);
  else
    run<T, 16, 64>(c, backward, s);
  return hipGetLastError();
}
hipError_t run(const RouteCall& c, Elem type, bool backward, hipStream_t s) {
  return type == Elem::f32 ? run<float>(c, backward, s)
         : type == Elem::bf16 ? run<Bf16>(c, backward, s) : run<F16>(c, backward, s);
}

// ---- gate --------------------------------------------------------------------------

// An active edge's rows of w and grad_w are read once: bound by HBM.  L lanes take a row, 16
// bytes each, kUnroll loads of each kind in flight.
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

size_t route_floats(int64_t rows, int n) { return size_t(route_blocks(rows, n)) * (2 * size_t(n) + 1); }
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

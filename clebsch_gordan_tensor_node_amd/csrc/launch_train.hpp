// Argument blocks and host-side launchers of the training operators: layer
// normalisation (of rows, and of irreps term by term), the AdamW step and the gradient
// norm.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace cgtp {

// Element types of the training operators (CGTP_F32, CGTP_BF16, CGTP_F16).
enum class Elem : int { f32 = 0, bf16 = 1, f16 = 2 };

// What the last-level cache holds.  A call that moves more has nothing of it left in the
// caches when it ends: its accesses pass them by (non-temporal), which keeps the lines that
// it writes from being written back during the next kernel.  Measured without and with: a
// clipped AdamW step of 1.4 GB 305 and 240 us, layer norm of 1.2 GB 240 and 212 us; but a
// backward of 84 MB, whose rows the caches hold, 23 and 31 us.
constexpr int64_t kCacheBytes = int64_t(256) << 20;

// ---- normalisation -----------------------------------------------------------------

// One normalised stretch of a row: a term "mul x l p" of an irreps row, or the whole row
// of a layer norm.
struct NormTerm {
  int32_t off;     // first element in a row
  int32_t len;     // elements: channels * d
  int32_t d;       // components that share a channel's weight (2l + 1)
  int32_t w_off;   // first weight
  int32_t b_off;   // first bias; -1: not centred, no bias
};
constexpr int kMaxNormTerms = 64;   // terms of an irreps row (they travel in the kernel arguments)

struct NormShape {
  int64_t features, weights, biases;
  const NormTerm* terms;
  int n_terms;
};

struct NormCall {
  const void* x;
  const void* weight;      // may be null (1)
  const void* bias;        // may be null (0); forward only
  void* y;                 // forward: the output; backward: dL/dx (may be null)
  const void* grad_out;    // backward only
  float* stats;            // [2, rows, terms] mean and rstd: written by the forward (may be
                           // null), read by the backward
  void* grad_weight;       // backward only; may be null
  void* grad_bias;         // backward only; may be null
  float* part;             // backward: partial sums of the weight's and bias's gradients
  int64_t rows;
  int64_t ld_x, ld_y, ld_g;   // elements from row to row
  float eps;
  int weight_f32;          // weight, bias and their gradients are fp32 (else x's type)
};

hipError_t launch_norm_forward(const NormCall& c, const NormShape& p, Elem type, hipStream_t s);
// Floats of partial sums that launch_norm_backward needs in c.part when a weight's or
// bias's gradient is asked for.
size_t norm_part_floats(int64_t rows, const NormShape& p);
hipError_t launch_norm_backward(const NormCall& c, const NormShape& p, Elem type, hipStream_t s);

// ---- optimiser ---------------------------------------------------------------------

constexpr int kStateBlock = 64;          // elements that share an exponent in 8-bit states
// Most elements of one chunk.  A clipped step of 50 M elements with 32-bit states takes 241,
// 238 and 244 us with 4096, 2048 and 1024, one of 37 M with 8-bit states 118, 116 and 120 us.
constexpr int kChunk = 2048;
constexpr int kTensorsPerLaunch = 232;   // tensors whose pointers fit the kernel arguments
constexpr int kChunksPerLaunch = 1 << 22;   // a grid's threads stay below 2^32

// A stretch of one tensor that one workgroup handles.
struct alignas(32) Chunk {
  int32_t tensor;       // index in the set
  int32_t n;            // elements (<= kChunk)
  int64_t start;        // first element in the tensor
  int64_t state;        // its place among the states (a multiple of kStateBlock)
  double decay;         // the tensor's weight decay
};
static_assert(sizeof(Chunk) == 32, "Chunk is 32 bytes");

// What a step's number and rate give.
struct AdamwScalars {
  double lr;
  float step_size, inv_root;     // lr / (1 - b1^t), 1 / sqrt(1 - b2^t)
  uint32_t seed;                 // already multiplied
  uint32_t unused;
};
constexpr uint32_t kSeedFactor = 0x3C6EF373u;

struct AdamwArgs {
  const Chunk* chunks;           // this launch's
  float* m;                      // 32-bit states
  float* v;
  uint8_t *m_code, *r_code;      // 8-bit states: codes and block exponents
  uint8_t *m_exp, *r_exp;
  const float* grad_scale;       // may be null (1)
  const AdamwScalars* device;    // null: `here`
  AdamwScalars here;
  float b1, c1, b2, c2;          // beta and 1 - beta
  float eps;
  int32_t first_tensor;          // of this launch
  void* param[kTensorsPerLaunch];
  const void* grad[kTensorsPerLaunch];
};
static_assert(sizeof(AdamwArgs) <= 4096, "kernel arguments are limited to 4 KiB");

// Advances *step by one, unless *grad_scale (may be null) is NaN, and writes the scalars of
// the step with that number; lr_device (may be null) replaces lr.
hipError_t launch_adamw_scalars(int64_t* step, const float* lr_device, double lr, double beta1, double beta2,
                                uint32_t seed, const float* grad_scale, AdamwScalars* out, hipStream_t s);

struct GradNormArgs {
  const Chunk* chunks;
  double* part;                  // one for each workgroup of the launch
  int32_t first_tensor;
  int32_t n_chunks;
  const void* grad[kTensorsPerLaunch];
};

// stream: params, gradients and states pass by the caches (a step that moves more than
// they hold).
hipError_t launch_adamw(const AdamwArgs& a, int n_chunks, Elem param, Elem grad, bool bits8, bool stream,
                        hipStream_t s);
// Workgroups (and partial sums) of launch_grad_squares over n chunks.
constexpr int kSquareBlocks = 4096;
constexpr int square_blocks(int n) { return n < kSquareBlocks ? n : kSquareBlocks; }
hipError_t launch_grad_squares(const GradNormArgs& a, Elem grad, hipStream_t s);
// out[0] = scale * sqrt(sum of part), out[1] = scale * min(1, max_norm / out[0]), NaN
// where out[0] is not finite; scale = *grad_scale (1 if null).
hipError_t launch_grad_norm_finish(const double* part, int n, const float* grad_scale, float max_norm, float* out,
                                   hipStream_t s);
// Both in one launch of one workgroup, for at most kSmallChunks chunks.
constexpr int kSmallChunks = 32;
hipError_t launch_grad_norm_small(const GradNormArgs& a, Elem grad, const float* grad_scale, float max_norm, float* out,
                                  hipStream_t s);
// Values of n coded states in bf16: m and r = sqrt(v).
hipError_t launch_decode_states(const uint8_t* m_code, const uint8_t* r_code, const uint8_t* m_exp,
                                const uint8_t* r_exp, int64_t n, void* m, void* r, hipStream_t s);

}  // namespace cgtp

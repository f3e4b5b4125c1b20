// Argument blocks and host-side launchers of the operators for branching networks: group
// normalisation with an activation, routing to branches, the gradient of the
// convolution's gate.
#pragma once

#include "launch_train.hpp"

namespace cgtp {

// ---- group normalisation -----------------------------------------------------------

// Activations (CGTP_ACT_NONE, CGTP_ACT_SILU, CGTP_ACT_GELU).
enum class Act : int { none = 0, silu = 1, gelu = 2 };

struct GroupCall {
  const void* x;
  const void* weight;       // may be null (1)
  const void* bias;         // may be null (0)
  const void* grad_out;     // backward only
  void* y;                  // forward: the output; backward: dL/dx (may be null)
  float* stats;             // [2, samples, groups]: written by the forward (may be null), read by the backward
  void* grad_weight;        // backward only; may be null
  void* grad_bias;          // backward only; may be null
  float* work;
  const int32_t* offsets;   // [samples + 1] row bounds; null: samples of rows / samples rows each
  int64_t rows, width, groups, samples;
  int64_t longest;          // rows of the longest sample, as far as the caller knows; 0: unknown
  int64_t ld_x, ld_y, ld_g;
  float eps;
  Act act;
  int weight_f32;           // weight, bias and their gradients are fp32 (else x's type)
  int zero_outside;         // rows outside every sample are written as zeros (else left)
};

// Floats of workspace that a call needs (offsets: whether they are given is looked at); sums:
// whether the backward's weights' gradients are wanted.
size_t group_norm_floats(const GroupCall& c, Elem type, bool backward, bool sums);
hipError_t launch_group_norm_forward(const GroupCall& c, Elem type, hipStream_t s);
hipError_t launch_group_norm_backward(const GroupCall& c, Elem type, hipStream_t s);

// ---- routing -----------------------------------------------------------------------

constexpr int kMaxBranches = 1024, kMaxChosen = 64;

struct RouteCall {
  const void* logits;       // [rows, n], rows ld elements apart
  int64_t rows, ld;
  int n, k;
  int renormalise, dense;
  const uint8_t* mask;      // forward; may be null
  int32_t* ids;             // [rows, k]: written by the forward, read by the backward
  float* gates;             // forward: [rows, k] or dense [n, rows]
  int32_t* counts;          // [n]
  float* balance;           // [1]
  float* slope;             // [n]: written by the forward, read by the backward
  const float* grad_gates;  // backward; may be null
  const float* grad_balance;   // backward; may be null
  void* grad_logits;        // backward: [rows, n], rows ld_g elements apart
  int64_t ld_g;
  float* work;
};

size_t route_floats(int64_t rows, int n);
hipError_t launch_route_forward(const RouteCall& c, Elem type, hipStream_t s);
hipError_t launch_route_backward(const RouteCall& c, Elem type, hipStream_t s);

// ---- gate --------------------------------------------------------------------------

struct GateCall {
  const float* w;           // [edges, width]
  const float* grad_w;
  const float* gate;        // [edges]
  const uint8_t* mask;      // may be null
  float* grad_gate;
  int64_t edges, width;
};

hipError_t launch_gate_backward(const GateCall& c, hipStream_t s);

}  // namespace cgtp

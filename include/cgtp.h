/*
 * cgtp.h -- C ABI of libcgtp.so: the Clebsch-Gordan tensor-product (CGTP)
 * convolution, forward (fp32, and fp64 for l <= 4) and gradients (fp32, l <= 4), for
 * AMD Instinct MI355X (gfx950); and operators that train a network around it (layer and
 * irreps normalisation, AdamW), at the end of this file.
 *
 * What is computed (the pages print no formula; this is the textbook definition that
 * LunaTP's abstract says its kernels preserve):
 *   for every receiver i, every active edge e = (j -> i) of row i, every path
 *   p = (input irrep l1, edge-SH irrep l2 -> l3) and every channel u of the input irrep
 *     out[i, c_p(u), m3] += w[e, c_p(u)] * sum_{m1,m2} C_p[m1,m2,m3] x[j,u,m1] Y_{l2,m2}(r_e)
 *   with r_e = pos[j] - pos[i] + shift_e . cell.
 * Sources: LunaTP ("Enabling Efficient and Scalable Tensor Product for Equivariant
 * MLIPs"), Abstract and Figure 3(a) (node-centric accumulation, one store per node),
 * Table 1 (irreps cases; the uvu multiplicity and path rule are the readings that
 * reproduce its output irreps); BranchIP ("Learning Adaptive Equivariant Computation
 * for Interatomic Potentials"), Method: zero-gated edges are left out of the tensor
 * product and the sparse result equals the dense one; Allegro paragraph: neighbours
 * within a fixed cutoff.
 *
 * Conventions (the pages leave them open; fixed here):
 *   - irreps spec strings "128x0e+64x1o" (mul x l, parity e/o); l <= 6.
 *   - paths: for each input irrep (spec order), each SH irrep (spec order), each
 *     l3 in |l1-l2| .. min(l1+l2, l_out_max): p3 = p1*p2; CGTP_PATHS_PARITY keeps the
 *     path only if p3 == (-1)^l3, CGTP_PATHS_ALL keeps all.  Multiplicity = mul(l1).
 *   - output irreps sorted by (l3, e before o); within one output irrep the path blocks
 *     follow path order.
 *   - real CG: Racah (Condon-Shortley), mapped to real harmonics, real part for even
 *     l1+l2+l3, imaginary part for odd; no path normalisation.
 *   - real SH: component normalisation (Y_0 = 1, sum_m Y_lm^2 = 2l+1), l = 1 is
 *     sqrt(3) (y, z, x); a zero-length edge has Y_0 = 1 and Y_l = 0 for l >= 1.
 * Layouts (fp32 / int, row-major, device memory unless stated):
 *   x   [n_nodes, f_in]   irreps in spec order, each block [mul][2l+1]
 *   out [n_nodes, f_out]  output irreps in sorted order, each block [mul][2l+1]
 *   w   [n_edges, w_per_edge]  column = global output channel index (uvu weights)
 *   pos [n_nodes, 3]; row_ptr int32 [n_nodes+1]; col int32 [n_edges];
 *   shift int8 [n_edges, 3] in {-1,0,1}; mask uint8 [n_edges] (nonzero = active).
 *
 * Ownership: the caller allocates and owns every device buffer, including the
 * workspace; the library never allocates in cgtp_neighbors_build, cgtp_conv_prepare,
 * cgtp_conv_forward or cgtp_edge_sh and keeps no pointer after a call returns.  A plan
 * owns its small device tables and, when its forward takes several kernel launches (plans
 * with paths of l >= 4, or more path groups than one launch carries), up to three HIP
 * streams and four events of its own (all freed by cgtp_plan_destroy).  A plan's tables
 * are immutable after creation; it may be shared by threads and streams (forward calls
 * on one plan take a per-plan lock while they enqueue).
 * Asynchrony: device work is enqueued on `stream` (a hipStream_t; NULL = default
 * stream) and not waited for, except where stated.  Inputs must stay valid until the
 * stream reaches that point.
 * Errors: every int-returning call returns CGTP_OK (0) or a negative code; arguments
 * are validated on the host before any launch; cgtp_last_error() returns a
 * thread-local message for the last failing call.  Contents of device arrays are not
 * validated (a malformed CSR is undefined behaviour).
 */
#ifndef CGTP_H_
#define CGTP_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct cgtp_plan_s* cgtp_plan_t;

enum {
  CGTP_OK = 0,
  CGTP_ERR_INVALID_ARG = -1,  /* null/misaligned pointer, negative size, bad flag */
  CGTP_ERR_PARSE = -2,        /* malformed irreps spec */
  CGTP_ERR_UNSUPPORTED = -3,  /* l > 6, SH multiplicity != 1, no path, too many jobs */
  CGTP_ERR_CAPACITY = -4,     /* edge list longer than the caller's capacity */
  CGTP_ERR_WORKSPACE = -5,    /* workspace smaller than the size query returned */
  CGTP_ERR_HIP = -6,          /* a HIP runtime call failed */
  CGTP_ERR_NO_DEVICE = -7,    /* no usable gfx950 device */
  CGTP_ERR_NO_MEMORY = -8     /* a host allocation of a create call failed */
};

enum { CGTP_PATHS_ALL = 0, CGTP_PATHS_PARITY = 1 };

/* Plan flags.  CGTP_PLAN_HOST_ONLY: build host tables only (no device upload); such a
 * plan answers the query calls but cgtp_conv_* return CGTP_ERR_INVALID_ARG with it.
 * CGTP_PLAN_FP64: the plan's forward runs in fp64 (LunaTP reports its kernels in
 * double precision: Figure 8, Table 11); it is used with cgtp_conv_forward_f64 only,
 * supports l <= 4 (else CGTP_ERR_UNSUPPORTED), and its workspace holds fp64
 * harmonics.  The fp32 forward entry points return CGTP_ERR_INVALID_ARG with an fp64
 * plan and cgtp_conv_forward_f64 with an fp32 plan. */
enum { CGTP_PLAN_HOST_ONLY = 1u, CGTP_PLAN_FP64 = 2u };

/* Parse irreps, enumerate paths, build the real-CG tables and the wave-job schedule,
 * and (unless CGTP_PLAN_HOST_ONLY) upload the job table to the current device.
 * irreps_sh must hold multiplicity-1 irreps.  Source: LunaTP Table 1 (irreps cases)
 * and Figure 3(b) (paths grouped and mapped to SIMD lanes by channel block).
 * Returns CGTP_ERR_PARSE / CGTP_ERR_UNSUPPORTED / CGTP_ERR_NO_DEVICE / CGTP_ERR_HIP. */
int cgtp_plan_create(const char* irreps_in, const char* irreps_sh, int l_out_max,
                     int path_rule, unsigned flags, cgtp_plan_t* out);

/* Sizes of the plan.  Any output pointer may be NULL.  irreps_out receives the
 * output irreps string (NUL-terminated, truncated to irreps_out_cap); for the six
 * irreps cases of LunaTP Table 1 it is the output column of that table. */
int cgtp_plan_info(cgtp_plan_t plan, int64_t* f_in, int64_t* f_out, int64_t* w_per_edge,
                   int* n_paths, int* l_sh_max, char* irreps_out, size_t irreps_out_cap);

/* Host array rows[n_paths * 10]: l1, p1, l2, p2, l3, p3, mul, in_off, out_off, w_off
 * per path (offsets as in the layouts above): the uvu paths whose outputs make up the
 * output irreps of LunaTP Table 1. */
int cgtp_plan_paths(cgtp_plan_t plan, int32_t* rows);

/* Host array dense[(2l1+1)(2l2+1)(2l3+1)] = real CG of path `path`, fp32, index
 * ((m1+l1)(2l2+1) + (m2+l2))(2l3+1) + (m3+l3): the sparse coupling coefficients that
 * LunaTP Figure 3(c) treats as constants of the kernel. */
int cgtp_plan_cg(cgtp_plan_t plan, int path, float* dense);

/* Scheduler summary: number of wave jobs and of distinct kernel variants used. */
int cgtp_plan_schedule(cgtp_plan_t plan, int* n_jobs, int* n_variants);

/* Workspace bytes that cgtp_conv_forward needs for this graph size (alignment 256).
 * Interface bookkeeping: the pages define no such call; it exists because the library
 * allocates nothing. */
int cgtp_workspace_size(cgtp_plan_t plan, int64_t n_nodes, int64_t n_edges, int has_mask,
                        size_t* bytes);

/* Workspace bytes that cgtp_neighbors_build needs. */
int cgtp_neighbors_workspace_size(int64_t n_nodes, const float box[3], float cutoff,
                                  size_t* bytes);

/* Receiver-CSR neighbour list under the minimum image convention of an orthorhombic
 * periodic box (BranchIP, Allegro paragraph: neighbours within a fixed cutoff).
 * Predicate, evaluated in fp64 without contraction, identical bit for bit to any
 * implementation of it:
 *   d = (double)pos_j - (double)pos_i; if d > L/2: d -= L, s = -1; else if d < -L/2:
 *   d += L, s = +1; else s = 0;  r2 = (dx*dx + dy*dy) + dz*dz;
 *   edge iff r2 < (double)cutoff * (double)cutoff and i != j.
 * Rows are sorted by j.  Positions must lie in [0, box).  box (host) and cutoff > 0.
 * Writes row_ptr[n_nodes+1] always; writes col/shift only if the edge count fits
 * edge_capacity, else returns CGTP_ERR_CAPACITY.  *n_edges (host) receives the edge
 * count in both cases.  SYNCHRONISES `stream` (the count is returned to the host). */
int cgtp_neighbors_build(const float* pos, int64_t n_nodes, const float box[3], float cutoff,
                         int32_t* row_ptr, int32_t* col, int8_t* shift, int64_t edge_capacity,
                         int64_t* n_edges, void* workspace, size_t ws_bytes, void* stream);

/* Active-edge CSR and node order (BranchIP sparse evaluation; LunaTP Table 9: nodes in
 * descending degree order).  mask NULL = all edges active.  Outputs (device):
 * act_row_ptr[n_nodes+1]; act_eid[<= n_edges] = ids of active edges in CSR order;
 * order[n_nodes] = nodes by active degree descending, then id ascending.
 * workspace: at least cgtp_workspace_size(plan, n_nodes, n_edges, mask != NULL). */
int cgtp_conv_prepare(cgtp_plan_t plan, const int32_t* row_ptr, const uint8_t* mask,
                      int64_t n_nodes, int64_t n_edges, int32_t* act_row_ptr, int32_t* act_eid,
                      int32_t* order, void* workspace, size_t ws_bytes, void* stream);

/* Real SH of every edge: sh[n_edges, (l_sh_max+1)^2], block l at offset l*l, m = -l..l,
 * of r_e = pos[j] - pos[i] + shift_e . cell (cell host, row-major 3x3, rows are lattice
 * vectors; NULL = open boundaries, shift ignored; shift NULL = zero).  Geometry and
 * harmonics in fp64, stored fp32. */
int cgtp_edge_sh(cgtp_plan_t plan, const float* pos, int64_t n_nodes, const float cell[9],
                 const int32_t* row_ptr, const int32_t* col, const int8_t* shift,
                 int64_t n_edges, float* sh, void* stream);

/* The CGTP convolution forward.  out[n_nodes, f_out] is overwritten (not accumulated);
 * rows with no active edge get exactly 0; w and x_j of inactive edges are never read.
 * Arguments as above; x [n_nodes, f_in], w [n_edges, w_per_edge], mask NULL = all
 * active.  All device pointers 16-byte aligned; x must be smaller than 4 GiB (the
 * kernel addresses it with 32-bit byte offsets), else CGTP_ERR_UNSUPPORTED.
 * Asynchronous on `stream`.  The result is bitwise reproducible from run to run.
 * Launches of different kernel classes write disjoint output columns; when there are
 * several, the call forks the plan's own streams from `stream` after the per-row pass
 * and joins them back into `stream` (events), so work enqueued on `stream` after the
 * call sees the whole output, and the call may be captured into a HIP graph. */
int cgtp_conv_forward(cgtp_plan_t plan, const float* pos, int64_t n_nodes, const float cell[9],
                      const int32_t* row_ptr, const int32_t* col, const int8_t* shift,
                      int64_t n_edges, const float* x, const float* w, const uint8_t* mask,
                      float* out, void* workspace, size_t ws_bytes, void* stream);

/* The forward with BranchIP's continuation gate (BranchIP, Method: each feature is
 * multiplied by its gate f in [0, 1] before the next tensor product, and zero-gated
 * features are omitted — sparse evaluation).  gate: device fp32 [n_edges], 4-byte
 * aligned, NULL = 1.  An edge is active when mask (if any) keeps it and gate[e] != 0;
 * an active edge's message is scaled by gate[e] (the product is linear in the edge's
 * feature), so out[i] = sum over active e of gate[e] * message_e.  w and x_j of
 * inactive edges are never read.  Everything else as cgtp_conv_forward; the workspace
 * size is the same. */
int cgtp_conv_forward_gated(cgtp_plan_t plan, const float* pos, int64_t n_nodes, const float cell[9],
                            const int32_t* row_ptr, const int32_t* col, const int8_t* shift,
                            int64_t n_edges, const float* x, const float* w, const uint8_t* mask,
                            const float* gate, float* out, void* workspace, size_t ws_bytes,
                            void* stream);

/* cgtp_conv_forward_gated (gate may be NULL), and in addition has the caller's HIP events
 * (hipEvent_t) ev_conv_begin / ev_conv_end stamped by the dispatch of the fused
 * convolution kernel itself (at the start of its first launch and the end of its last),
 * so that the caller can time that kernel apart from the prepare and harmonics passes
 * and from launch gaps.  When the launches are spread over the plan's streams the two
 * events are recorded on `stream` just before the fork and just after the join instead.
 * Same kernels, same results. */
int cgtp_conv_forward_timed(cgtp_plan_t plan, const float* pos, int64_t n_nodes, const float cell[9],
                            const int32_t* row_ptr, const int32_t* col, const int8_t* shift,
                            int64_t n_edges, const float* x, const float* w, const uint8_t* mask,
                            const float* gate, float* out, void* workspace, size_t ws_bytes,
                            void* stream, void* ev_conv_begin, void* ev_conv_end);

/* The forward in double precision, for plans created with CGTP_PLAN_FP64 (LunaTP,
 * Figure 8 and Table 11: the kernels are measured in fp64).  Same definition,
 * semantics and integer arguments as cgtp_conv_forward_gated; pos [n_nodes, 3], cell
 * (host, may be NULL), x, w, gate (may be NULL) and out are fp64, x, w and out 16-byte
 * aligned, pos and gate 8-byte aligned; x must be smaller than 4 GiB.  Geometry,
 * harmonics, coefficients and accumulation are fp64.  ev_conv_begin / ev_conv_end
 * (hipEvent_t, may be NULL) are stamped as in cgtp_conv_forward_timed.  The workspace
 * size is cgtp_workspace_size of the same plan. */
int cgtp_conv_forward_f64(cgtp_plan_t plan, const double* pos, int64_t n_nodes, const double cell[9],
                          const int32_t* row_ptr, const int32_t* col, const int8_t* shift,
                          int64_t n_edges, const double* x, const double* w, const uint8_t* mask,
                          const double* gate, double* out, void* workspace, size_t ws_bytes,
                          void* stream, void* ev_conv_begin, void* ev_conv_end);

/* Size of the device scratch array that cgtp_conv_forward_noalloc uses in place of a
 * workspace: 64 MiB per GPU (for fp32 plans with edge harmonics up to l = 3, about
 * 900 000 edges). */
#define CGTP_NOALLOC_SCRATCH_BYTES ((size_t)64 << 20)

/* cgtp_conv_forward_gated without a workspace argument and without any allocation, for
 * callers that cannot allocate device memory: code under HIP graph capture, tight
 * serving loops, harnesses that forbid hipMalloc.  The kernels' scratch (per-row active
 * degrees, node records, the compacted active edges and their harmonics) lives in a
 * device array of CGTP_NOALLOC_SCRATCH_BYTES that the library holds on each GPU it runs
 * on until the process ends; its address is looked up once per device, on the first
 * call.  Graphs whose scratch (cgtp_workspace_size of the same plan and sizes) exceeds
 * the array are refused with CGTP_ERR_WORKSPACE before any launch.  Every call on one
 * GPU shares that GPU's array, and no part of it needs to start at zero: every value a
 * call reads was written by the same call.  Calls that overlap on one GPU (on streams
 * that are not ordered with respect to each other) race on the array; calls in stream
 * order do not.  The caller still allocates x, w, out and the other arguments.  fp32
 * plans only (an fp64 plan gives CGTP_ERR_INVALID_ARG); results are bitwise those of
 * cgtp_conv_forward_gated on the same inputs. */
int cgtp_conv_forward_noalloc(cgtp_plan_t plan, const float* pos, int64_t n_nodes, const float cell[9],
                              const int32_t* row_ptr, const int32_t* col, const int8_t* shift,
                              int64_t n_edges, const float* x, const float* w, const uint8_t* mask,
                              const float* gate, float* out, void* stream);

/* Workspace bytes that cgtp_conv_backward needs for this graph size (alignment 256). */
int cgtp_backward_workspace_size(cgtp_plan_t plan, int64_t n_nodes, int64_t n_edges, size_t* bytes);

/* Gradients of the convolution (the backward pass; LunaTP, Abstract: the derivatives
 * that forces need are within its kernels' scope).  Given grad_out = dL/d out
 * [n_nodes, f_out] for a scalar L of the forward's output, writes (each may be NULL to
 * skip it; each is overwritten):
 *   grad_x [n_nodes, f_in]:   dL/dx;
 *   grad_w [n_edges, w_per_edge]: dL/dw, rows of inactive edges exactly 0;
 *   grad_pos [n_nodes, 3]:    dL/dpos through r_e = pos[j] - pos[i] + shift_e . cell and
 *                             dY/dr (forces are -grad_pos when L is an energy).
 * The mask, gate (BranchIP continuation gate; it scales the message and is not
 * differentiated), cell and shifts are constants; inactive edges contribute nothing
 * and their w and x_j are never read.  fp32 plans whose largest l is 4 or less (else
 * CGTP_ERR_UNSUPPORTED; an fp64 plan gives CGTP_ERR_INVALID_ARG).  Other arguments as
 * cgtp_conv_forward_gated; x, w, grad_out and grad_w 16-byte aligned (the edge pass
 * moves them in 16-byte vectors), the other pointers 4-byte aligned; x smaller than
 * 4 GiB; workspace at least cgtp_backward_workspace_size (256-byte aligned).
 * Asynchronous on `stream`; results are bitwise reproducible (no floating-point
 * atomics). */
int cgtp_conv_backward(cgtp_plan_t plan, const float* pos, int64_t n_nodes, const float cell[9],
                       const int32_t* row_ptr, const int32_t* col, const int8_t* shift,
                       int64_t n_edges, const float* x, const float* w, const uint8_t* mask,
                       const float* gate, const float* grad_out, float* grad_x, float* grad_w,
                       float* grad_pos, void* workspace, size_t ws_bytes, void* stream);

/* ---- Training operators ---------------------------------------------------------
 *
 * What a network around the convolution needs besides it: normalisation of rows (a
 * radial network's hidden rows, per-edge weights) and of irreps features (what goes into
 * and comes out of the convolution), and the optimiser step that applies the gradients.
 * The interface is this library's own; the pages define no such calls (LunaTP, Abstract,
 * names training of whole potentials as the use).  Ownership, asynchrony and errors as
 * above: the library allocates nothing in them and keeps no pointer after a call returns.
 *
 * Element types of rows, parameters and gradients.  Everything is computed in fp32 and
 * rounded to nearest even where it is stored; sums, statistics and 32-bit states are
 * fp32 (the gradient norm fp64) whatever the element type.  Infinities and NaN go where
 * the formulas take them, unless stated. */
enum { CGTP_F32 = 0, CGTP_BF16 = 1, CGTP_F16 = 2 };

/* Layer normalisation of each row x[r, 0..width):
 *   mu = sum(x)/width, s2 = sum((x - mu)^2)/width, rstd = 1/sqrt(s2 + eps),
 *   y = (x - mu) rstd weight + bias
 * x and y are device arrays of type dtype whose rows lie ld_x / ld_y elements apart (>=
 * width) and hold consecutive elements; they need the alignment of one element only.  y may
 * be x itself (ld_y = ld_x): every row is read before it is written, but the backward has no
 * x then.  Rows may not overlap otherwise.  weight and bias [width] (each may be NULL: 1,
 * 0) are of type weight_dtype, CGTP_F32 or dtype.  stats [2, n_rows] fp32 (may be NULL)
 * receives mu and rstd, which the backward reads.  n_rows may be 0; a row of one element
 * gives y = bias.  Asynchronous on `stream`; bitwise reproducible. */
int cgtp_layer_norm_forward(int dtype, int64_t n_rows, int64_t width, const void* x, int64_t ld_x, int weight_dtype,
                            const void* weight, const void* bias, double eps, void* y, int64_t ld_y, float* stats,
                            void* stream);

/* Workspace bytes that cgtp_layer_norm_backward needs when it writes grad_weight or
 * grad_bias. */
int cgtp_layer_norm_backward_workspace_size(int64_t n_rows, int64_t width, size_t* bytes);

/* Gradients of a scalar L of the layer norm's output, given grad_out = dL/dy (rows ld_g
 * elements apart) and the forward's x and stats.  With h = (x - mu) rstd, a = grad_out
 * weight:
 *   grad_x = rstd (a - sum(a)/width - h sum(a h)/width)        rows ld_gx elements apart
 *   grad_weight[c] = sum over rows of grad_out h, grad_bias[c] = sum over rows of grad_out
 * Each output may be NULL to skip it, and is overwritten; it may not overlap an input.
 * grad_weight and grad_bias are of type weight_dtype (with n_rows = 0 they are 0).
 * workspace: 256-byte aligned, not needed (NULL) when both are NULL.  No atomics: bitwise
 * reproducible. */
int cgtp_layer_norm_backward(int dtype, int64_t n_rows, int64_t width, const void* grad_out, int64_t ld_g,
                             const void* x, int64_t ld_x, const float* stats, int weight_dtype, const void* weight,
                             void* grad_x, int64_t ld_gx, void* grad_weight, void* grad_bias, void* workspace,
                             size_t ws_bytes, void* stream);

/* The equivariant layer norm of irreps rows: each term "mul x l p" of `irreps` is
 * normalised by itself.  A 0e term is layer-normalised as above, with a weight and a bias
 * per channel.  Any other term's block [mul][2l+1] has no mean taken off and no bias (both
 * would break equivariance under rotation, or under inversion for 0o): with
 *   s2 = sum(x^2) / (mul (2l+1)), rstd = 1/sqrt(s2 + eps),  y[u, m] = x[u, m] rstd weight[u].
 * The plan holds host memory only and belongs to no device; it may be shared by threads
 * and streams.  At most 64 terms, l <= 6, rows of at most 2^29 values. */
typedef struct cgtp_norm_s* cgtp_norm_t;
int cgtp_norm_create(const char* irreps, cgtp_norm_t* out);

/* Row width, number of weights (all channels, in term order), of biases (channels of the
 * 0e terms, in term order) and of terms.  Any output pointer may be NULL. */
int cgtp_norm_info(cgtp_norm_t plan, int64_t* n_features, int64_t* n_weights, int64_t* n_biases, int* n_terms);
void cgtp_norm_destroy(cgtp_norm_t plan);

/* Forward and backward over rows of n_features elements; arguments as the layer norm's,
 * with weight [n_weights], bias [n_biases] and stats [2, n_rows, n_terms]. */
int cgtp_irreps_norm_forward(cgtp_norm_t plan, int dtype, int64_t n_rows, const void* x, int64_t ld_x,
                             int weight_dtype, const void* weight, const void* bias, double eps, void* y, int64_t ld_y,
                             float* stats, void* stream);
int cgtp_irreps_norm_backward_workspace_size(cgtp_norm_t plan, int64_t n_rows, size_t* bytes);
int cgtp_irreps_norm_backward(cgtp_norm_t plan, int dtype, int64_t n_rows, const void* grad_out, int64_t ld_g,
                              const void* x, int64_t ld_x, const float* stats, int weight_dtype, const void* weight,
                              void* grad_x, int64_t ld_gx, void* grad_weight, void* grad_bias, void* workspace,
                              size_t ws_bytes, void* stream);

/* A set of n_tensors tensors (numel[t] >= 0 elements each, dense) that one optimiser step
 * covers, with a weight decay each (NULL: 0).  It holds their sizes, on the host and in a
 * small table on the current device, and no pointer to them.  Optimiser states of the whole
 * set are flat arrays of state_elems elements: tensor t's begin at offsets[t], a multiple
 * of 64.  flags: 0, or CGTP_PLAN_HOST_ONLY (sizes only, no device).  May be shared by
 * threads and streams; freed by cgtp_params_destroy (NULL is ignored), but not before
 * captured graphs that hold its calls. */
typedef struct cgtp_params_s* cgtp_params_t;
int cgtp_params_create(const int64_t* numel, const double* weight_decay, int n_tensors, unsigned flags,
                       cgtp_params_t* out);
int cgtp_params_info(cgtp_params_t set, int* n_tensors, int64_t* state_elems, int64_t* offsets);
void cgtp_params_destroy(cgtp_params_t set);

/* One AdamW step over the set, in place.  params and grads are host arrays of n_tensors
 * device pointers (read before the call returns; entries of empty tensors may be NULL) of
 * types param_dtype and grad_dtype, aligned to one element; m and v [state_elems] fp32,
 * 16-byte aligned, zero before the first step.  step counts from 1:
 *   g = grad grad_scale[0];  p <- p (1 - lr decay);  m <- beta1 m + (1 - beta1) g;
 *   v <- beta2 v + (1 - beta2) g^2;
 *   p <- p - (lr / (1 - beta1^step)) m / (sqrt(v) / sqrt(1 - beta2^step) + eps)
 * 16-bit parameters are rounded to nearest: a step below half the distance of their values
 * (2^-9 to 2^-8 of a bf16 parameter) leaves them as they are, step after step.  At such rates
 * hold the parameters in fp32 and copy them to 16 bits for the network.
 * grad_scale (device fp32, NULL = 1): the inverse of a loss scale, or the factor that
 * cgtp_grad_norm writes; where it is NaN the whole step is skipped, params and states
 * untouched.  Asynchronous on `stream`; bitwise reproducible.  lr and step travel in the
 * launch, so that a captured graph would repeat the step that it was captured with; with
 * scalars (device, not NULL) both come from cgtp_adamw_scalars instead. */
int cgtp_adamw_step(cgtp_params_t set, int param_dtype, void* const* params, int grad_dtype, const void* const* grads,
                    float* m, float* v, double lr, double beta1, double beta2, double eps, int64_t step,
                    const void* scalars, const float* grad_scale, void* stream);

/* A step counter on the device, for steps in a captured graph: advances step[0] (device, 0
 * before the first step) by one and writes into scalars (device, CGTP_ADAMW_SCALARS_BYTES,
 * 8-byte aligned) what the step with that number takes from lr, the betas and the seed (of
 * the 8-bit states; the step's number is added to it).  lr_device (device, may be NULL)
 * replaces lr, unchecked.  Where grad_scale (may be NULL) is NaN nothing is advanced or written: the
 * step behind it is skipped.  Runs on `stream` before that step, with its betas. */
#define CGTP_ADAMW_SCALARS_BYTES 24
int cgtp_adamw_scalars(int64_t* step, const float* lr_device, double lr, double beta1, double beta2, uint32_t seed,
                       const float* grad_scale, void* scalars, void* stream);

/* The same step with the states in 8 bits: codes of m and of r = sqrt(v) [state_elems each,
 * 16-byte aligned] and one exponent byte per block of 64 elements [state_elems / 64 each];
 * all zero bytes before the first step.  With E a block's exponent byte (the biased fp32
 * exponent of its largest magnitude), a code is the top of the fp32 number |value| 2^(14 -
 * max(E, 1)): for m a sign bit, 4 exponent and 3 mantissa bits, for r 4 exponent and 4
 * mantissa bits.  The rest is rounded up or down at random in proportion, by 16 bits of a
 * hash of the element's place and `seed` (give every step another one; the step number
 * serves), so that moments keep their mean although a step moves them by less than a
 * code's distance; equal seeds give equal results bit for bit.  A positive r is stored as
 * code 1 at least; a moment that is not finite is stored as NaN and does not disturb its
 * block.  p is updated from the moments before they are rounded. */
int cgtp_adamw_step_8bit(cgtp_params_t set, int param_dtype, void* const* params, int grad_dtype,
                         const void* const* grads, uint8_t* m_code, uint8_t* r_code, uint8_t* m_exp, uint8_t* r_exp,
                         double lr, double beta1, double beta2, double eps, int64_t step, uint32_t seed,
                         const void* scalars, const float* grad_scale, void* stream);

/* The values that 8-bit states stand for, m and r [state_elems] in bf16 (which holds them
 * exactly), 16-byte aligned: for checkpoints and inspection. */
int cgtp_adamw_read_8bit(cgtp_params_t set, const uint8_t* m_code, const uint8_t* r_code, const uint8_t* m_exp,
                         const uint8_t* r_exp, void* m, void* r, void* stream);

/* The 2-norm of all gradients of the set and the factor that clips them, on the device:
 *   out[0] = |grad_scale[0]| sqrt(sum of grad^2);
 *   out[1] = grad_scale[0] min(1, max_norm / out[0]), the grad_scale of an AdamW step;
 * NaN where out[0] is not finite, so that the step is skipped.  max_norm > 0 (infinity:
 * no clipping).  Squares and sums in fp64, in a fixed order.  workspace: 256-byte
 * aligned, cgtp_grad_norm_workspace_size bytes. */
int cgtp_grad_norm_workspace_size(cgtp_params_t set, size_t* bytes);
int cgtp_grad_norm(cgtp_params_t set, int grad_dtype, const void* const* grads, const float* grad_scale,
                   double max_norm, float* out, void* workspace, size_t ws_bytes, void* stream);

/* ---- Operators for branching networks --------------------------------------------
 *
 * What a network needs that sends its edges through several branches, each a convolution of
 * its own that takes its edges' gates (cgtp_conv_forward_gated; BranchIP, Method: zero-gated
 * features are omitted): group normalisation with an activation over each structure's rows
 * (the hidden rows that gates and weights come from), the routing that makes the gates, its
 * balance loss, and the way back from the convolution's weight gradient to the gates.  The
 * interface is this library's own.  Types, ownership, asynchrony and errors as for the
 * training operators above. */

/* Activations of cgtp_group_norm_forward: z, z sigmoid(z), z (1 + erf(z / sqrt 2)) / 2. */
enum { CGTP_ACT_NONE = 0, CGTP_ACT_SILU = 1, CGTP_ACT_GELU = 2 };

/* Group normalisation of rows, channels last, with an activation.  The rows of x [n_rows,
 * width] belong to n_samples samples (structures): sample s has rows offsets[s] to
 * offsets[s + 1] - 1, or, where offsets is NULL, n_rows / n_samples of them (which has to be
 * a whole number).  The columns are n_groups groups of width / n_groups (a whole number).
 * Over the M values of one sample and group:
 *   mu = sum(x)/M, s2 = sum((x - mu)^2)/M, rstd = 1/sqrt(s2 + eps),
 *   z = (x - mu) rstd weight + bias,  y = act(z)
 * weight and bias [width] (each may be NULL: 1, 0) are of type weight_dtype, CGTP_F32 or
 * dtype; x and y as cgtp_layer_norm_forward's (rows any stride apart, one element's
 * alignment, y may be x itself).  stats [2, n_samples, n_groups] fp32 (may be NULL) receives
 * mu and rstd, 0 and 1/sqrt(eps) for a sample without rows.  offsets [n_samples + 1] are on
 * the device and ascend; the library reads no row outside 0 to n_rows - 1, whatever they
 * hold.  Rows before offsets[0] and from offsets[n_samples] on belong to no sample: they are
 * not read, and their y is left as it is, or 0 with zero_outside != 0.
 * longest: rows of the longest sample, as far as the caller knows (0: not known).  It chooses
 * between launches, nothing else: a call with another value is as right, and slower where a
 * sample much longer than told falls to one workgroup.
 * workspace: 256-byte aligned, cgtp_group_norm_workspace_size bytes (0: NULL), whose `backward`
 * is 0 for the forward, 1 for the backward, or 2 for a backward of grad_x alone; calls that may
 * run at the same time, replayed graphs among them, need one each.  Rows of at most 2^24
 * values.  No atomics: bitwise reproducible. */
int cgtp_group_norm_workspace_size(int backward, int dtype, int64_t n_rows, int64_t width, int64_t n_groups,
                                   int64_t n_samples, const int32_t* offsets, int64_t longest, size_t* bytes);
int cgtp_group_norm_forward(int dtype, int64_t n_rows, int64_t width, int64_t n_groups, int64_t n_samples,
                            const int32_t* offsets, int64_t longest, const void* x, int64_t ld_x, int weight_dtype,
                            const void* weight, const void* bias, int activation, double eps, int zero_outside, void* y,
                            int64_t ld_y, float* stats, void* workspace, size_t ws_bytes, void* stream);

/* Gradients of a scalar L of that output, given grad_out = dL/dy and the forward's x, stats,
 * weight and bias.  With h = (x - mu) rstd, d = grad_out act'(h weight + bias), a = d weight:
 *   grad_x = rstd (a - sum(a)/M - h sum(a h)/M)               0 for rows outside every sample
 *   grad_weight[c] = sum over rows of d h, grad_bias[c] = sum over rows of d
 * Each output may be NULL to skip it, and is overwritten; it may not overlap an input.
 * grad_weight and grad_bias are of type weight_dtype.  stats of a sample without rows are not
 * read, and may be NULL where n_rows = 0. */
int cgtp_group_norm_backward(int dtype, int64_t n_rows, int64_t width, int64_t n_groups, int64_t n_samples,
                             const int32_t* offsets, int64_t longest, const void* grad_out, int64_t ld_g,
                             const void* x, int64_t ld_x, const float* stats, int weight_dtype, const void* weight,
                             const void* bias, int activation, void* grad_x, int64_t ld_gx, void* grad_weight,
                             void* grad_bias, void* workspace, size_t ws_bytes, void* stream);

/* Routing of rows (edges) to k of n branches by their logits [n_rows, n] (type dtype, rows
 * ld elements apart).  With p = softmax(logits) of a row, the k branches of the largest
 * logits are chosen; equal ones go to the lowest index, NaN counts as larger than every
 * number, and a branch whose logit is -infinity is never chosen.  A row whose mask (may be
 * NULL) is 0, or whose logits are all -infinity, takes no part.  Outputs:
 *   ids [n_rows, k]: the chosen, largest first, -1 where there is none (further);
 *   gates: p of the chosen; with renormalise != 0 divided by their sum.  [n_rows, k] beside
 *     the ids (0 where there is none), or with dense != 0 [n, n_rows], 0 for what a row did
 *     not choose: row b is the gate argument of branch b's convolution (for few branches: of
 *     more than 64 they are written one float at a time, far below the memory's rate);
 *   counts [n]: the rows that chose each branch;
 *   balance [1] and slope [n]: with C the sum of the counts and R the rows that take part,
 *     slope[e] = n counts[e] / (C R), balance = sum over e and rows of slope[e] p[e]: 1 where
 *     choices and probabilities are even, n where one branch has all (0 if R = 0).
 * A row whose logits hold NaN or +infinity has NaN gates and makes balance NaN.
 * 1 <= n <= 1024, 1 <= k <= min(n, 64).  Sums over rows in a fixed order, joined in fp64; no
 * atomics: bitwise reproducible.  workspace: 256-byte aligned, cgtp_route_workspace_size
 * bytes (0: NULL); calls that may run at the same time need one each. */
int cgtp_route_workspace_size(int64_t n_rows, int n, size_t* bytes);
int cgtp_route_forward(int dtype, int64_t n_rows, int n, int k, const void* logits, int64_t ld, const uint8_t* mask,
                       int renormalise, int dense, int32_t* ids, float* gates, int32_t* counts, float* balance,
                       float* slope, void* workspace, size_t ws_bytes, void* stream);

/* The logits' gradient [n_rows, n] (type dtype, rows ld_g elements apart), of a scalar L of
 * the gates and the balance loss: grad_gates = dL/dgates (as the forward's gates are laid
 * out; only the entries of chosen branches are read; NULL: 0), grad_balance [1] =
 * dL/dbalance (NULL: 0).  ids and slope are the forward's: choices and counts are held
 * fixed.  Rows without part receive 0.  Ids outside -1 to n - 1 count as -1; the gradients of a
 * branch that is twice in a row (the forward writes none) are added in the choices' order. */
int cgtp_route_backward(int dtype, int64_t n_rows, int n, int k, const void* logits, int64_t ld, int renormalise,
                        int dense, const int32_t* ids, const float* slope, const float* grad_gates,
                        const float* grad_balance, void* grad_logits, int64_t ld_g, void* stream);

/* The gradient of the convolution with respect to its gate, from the gradient with respect
 * to its weights that cgtp_conv_backward wrote with that gate.  An edge's message is linear
 * in gate[e] w[e], so that
 *   grad_gate[e] = sum over c of w[e, c] grad_w[e, c] / gate[e]
 * and 0 for inactive edges (mask 0, may be NULL, or gate 0), whose w and grad_w are not read.
 * w and grad_w [n_edges, w_per_edge], gate and grad_gate [n_edges], fp32 (grad_w carries the
 * gate: one so small that their product leaves the normal range of fp32 costs digits). */
int cgtp_conv_gate_backward(int64_t n_edges, int64_t w_per_edge, const float* w, const float* grad_w,
                            const uint8_t* mask, const float* gate, float* grad_gate, void* stream);

/* Frees the plan's device tables, streams and events (interface bookkeeping; the pages
 * define no such call).  NULL is ignored. */
void cgtp_plan_destroy(cgtp_plan_t plan);

/* Thread-local message of the last failing call ("" if none).  Interface bookkeeping;
 * the pages define no such call. */
const char* cgtp_last_error(void);

/* Library version string. */
const char* cgtp_version(void);

#ifdef __cplusplus
}
#endif

#endif /* CGTP_H_ */

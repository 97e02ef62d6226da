/*
 * dpg.h -- C ABI of the deterministic BF16 projection GEMM library for AMD
 * MI355X (gfx950).
 *
 * The operations are the dense projection GEMM family and the FP32 router GEMM
 * described on the pages
 *   "plan the 4096 -> 12288 input gradient with the row-half-release program
 *    at T-exact keys" (description: BF16-operand forward, input gradient and
 *    weight gradient; FP32 accumulation; BF16 or FP32 output),
 *   "restore the K1 weight-gradient routes that meet the deterministic
 *    package's absolute FP64 budgets" (description: the weight gradient reduces
 *    over the token count T in 64-token K blocks, with one or two K splits), and
 *   "cache the router entry points' calls by their own tensors" (description:
 *    an FP32 router GEMM with 256 experts computed by BF16x3 emulation, and
 *    deterministic=True as the default).
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * - Every matrix is row-major with a leading dimension `ld*` counted in
 *   elements (ld >= number of columns).  All data pointers are DEVICE pointers
 *   owned by the caller; the library keeps no pointer after a call returns.
 * - `T` is the token count, `N` the output features, `K` the input features
 *   (the pages write a projection as "K -> N", e.g. 4096 -> 12288).
 * - Alignment: every base pointer is 16-byte aligned, every `ld * sizeof(elt)`
 *   is a multiple of 16 bytes, and the contiguous extent of every matrix
 *   (its number of columns) is a multiple of 8 elements.  Otherwise the call
 *   returns DPG_ERR_ALIGNMENT.  T (the row count of X, dY, Y and dX) may be any
 *   value >= 0, including odd counts of 64-token blocks.
 * - Row strides of 2^22 elements or more are supported; such calls run a
 *   slower kernel with 64-bit addressing (the pipelined kernels address a tile
 *   through 32-bit buffer offsets).
 * - Outputs are written only in [rows, cols]; elements of a padded row beyond
 *   `cols` are never touched.  Outputs are overwritten, never read.
 * - An empty output (a zero extent) is a no-op.  An empty reduction (K = 0 for
 *   the forward pass, N = 0 for the input gradient, T = 0 for the weight
 *   gradient) writes zeros.
 * - `deterministic` != 0 (the default of the Python binding) selects the
 *   deterministic plan: the K partition and the in-tile accumulation order are
 *   a fixed function of (pass, T, N, K, output dtype, split_k) alone -- never of
 *   the device, its CU count or the cache state -- so the bits are reproducible
 *   on any MI355X.  deterministic == 0 selects the split-K plan, which may also
 *   use the device's CU count to pick the K split.  `split_k` = 0 lets the
 *   planner choose; 1..64 forces min(split_k, B) K splits in either mode, B
 *   being the number of 64-element blocks of the reduction (K for the forward
 *   pass, N for the input gradient, 64-token blocks of T for the weight
 *   gradient).  S splits partition the blocks evenly: with q = B / S and
 *   r = B % S the first r splits take q + 1 blocks and the others q (split s
 *   starts at block s*q + min(s, r); for S = 2: [0, ceil(B/2)) and the rest).
 *   In BOTH
 *   modes every reduction runs in a fixed order with no atomics, so repeated
 *   calls with the same arguments on one device give bitwise-identical
 *   outputs; different plans may differ from each other in the last bits.
 * - Split partials go to the caller's `workspace`, which must hold at least
 *   dpg_workspace_size(...) bytes for the same shape and flags (it may be NULL
 *   when that size is 0).  The library never allocates and never synchronizes;
 *   all work is enqueued on `stream` (0 = the null stream), so calls may be
 *   captured into a HIP graph.
 * - All validation happens before the first launch: on any error nothing is
 *   launched and nothing is written.  DPG_ERR_HIP reports a failed launch.
 */
#ifndef DPG_H_
#define DPG_H_

#include <stddef.h>
#include <stdint.h>
#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  DPG_OK = 0,
  DPG_ERR_INVALID_ARG = 1, /* negative size, ld < cols, NULL pointer for non-empty data, bad enum */
  DPG_ERR_UNSUPPORTED = 2, /* split_k outside 0..64, a launch beyond the grid limit, or a size beyond an entry point's stated limits */
  DPG_ERR_ALIGNMENT = 3,   /* pointer / ld / contiguous extent not 16-byte compatible */
  DPG_ERR_WORKSPACE = 4,   /* workspace smaller than dpg_workspace_size() */
  DPG_ERR_HIP = 5          /* a kernel launch failed */
} dpg_status;

/* DPG_E4M3 (8-bit floating point, 4 exponent and 3 mantissa bits, no infinities)
 * is a type of optimizer moments only. */
typedef enum { DPG_BF16 = 0, DPG_F32 = 1, DPG_E4M3 = 2 } dpg_dtype;

/* Passes; the short names (DPG_FWD ...) are aliases of the long ones. */
typedef enum {
  DPG_PASS_FORWARD = 0,
  DPG_PASS_DGRAD = 1,
  DPG_PASS_WGRAD = 2,
  DPG_PASS_ROUTER_FORWARD = 3,
  DPG_PASS_ROUTER_DGRAD = 4,
  DPG_PASS_ROUTER_WGRAD = 5,
  DPG_FWD = DPG_PASS_FORWARD,
  DPG_DGRAD = DPG_PASS_DGRAD,
  DPG_WGRAD = DPG_PASS_WGRAD,
  DPG_ROUTER_FWD = DPG_PASS_ROUTER_FORWARD,
  DPG_ROUTER_DGRAD = DPG_PASS_ROUTER_DGRAD,
  DPG_ROUTER_WGRAD = DPG_PASS_ROUTER_WGRAD
} dpg_pass;

/*
 * Forward pass, Y[T,N] = X[T,K] . W[N,K]^T: both operands K-major (the
 * row-half-release page, description, names this the K-major-B form).
 *   x  : BF16 [T, K], row stride ldx     w : BF16 [N, K], row stride ldw
 *   y  : y_dtype (BF16 or FP32) [T, N], row stride ldy
 * FP32 accumulation; BF16 output is rounded to nearest even.
 */
dpg_status dpg_forward(const void* x, int64_t ldx, const void* w, int64_t ldw,
                       void* y, int64_t ldy, dpg_dtype y_dtype,
                       int64_t T, int64_t N, int64_t K, int deterministic, int split_k,
                       void* workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * Input gradient, dX[T,K] = dY[T,N] . W[N,K]: the reduction runs over N, so W
 * is read with its contiguous dimension along the output (the MN-major B form
 * that the row-half-release page adds, description and commit message).
 *   dy : BF16 [T, N], row stride lddy    w : BF16 [N, K], row stride ldw
 *   dx : dx_dtype [T, K], row stride lddx
 */
dpg_status dpg_dgrad(const void* dy, int64_t lddy, const void* w, int64_t ldw,
                     void* dx, int64_t lddx, dpg_dtype dx_dtype,
                     int64_t T, int64_t N, int64_t K, int deterministic, int split_k,
                     void* workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * Weight gradient, dW[N,K] = dY[T,N]^T . X[T,K], reducing over the token count
 * T in 64-token blocks (the K1 weight-gradient page, description; an odd number
 * of 64-token blocks is allowed).  With two K splits, split 0 takes blocks
 * [0, ceil(B/2)) and split 1 the rest, B = ceil(T/64); partials are added in
 * ascending split order.
 *   dy : BF16 [T, N], row stride lddy    x : BF16 [T, K], row stride ldx
 *   dw : dw_dtype [N, K], row stride lddw
 */
dpg_status dpg_wgrad(const void* dy, int64_t lddy, const void* x, int64_t ldx,
                     void* dw, int64_t lddw, dpg_dtype dw_dtype,
                     int64_t T, int64_t N, int64_t K, int deterministic, int split_k,
                     void* workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * Arithmetic of the router passes, a process-wide setting read when a router
 * call is planned (it is part of the plan key).  The router page's ratio table
 * shows plain FP32 library calls beating the BF16x3 emulation at small token
 * counts, and the wgrad page's timeline keeps a router FFMA window; this
 * library has both:
 *   DPG_ROUTER_AUTO   : the planner picks, per shape, BF16x3 on the matrix
 *                       cores or FP32 fused multiply-adds on the vector ALUs
 *                       (the latter only where it measured faster);
 *   DPG_ROUTER_BF16X3 : always BF16x3 (hi*hi + hi*lo + lo*hi per product);
 *   DPG_ROUTER_FP32   : always one FP32 fused multiply-add per product, in
 *                       ascending order of the reduction index within a split.
 * Both kinds meet the FP32 budget; they differ from each other in the last
 * bits.  Each is deterministic in the sense of the conventions above.
 * DPG_ERR_INVALID_ARG for another value.  Thread-safe; calls already planned
 * under the previous setting keep their plans only in the cache entries keyed
 * by that setting.
 */
typedef enum { DPG_ROUTER_AUTO = 0, DPG_ROUTER_BF16X3 = 1, DPG_ROUTER_FP32 = 2 } dpg_router_arith;
dpg_status dpg_set_router_arithmetic(dpg_router_arith arith);
dpg_router_arith dpg_get_router_arithmetic(void);

/*
 * Weight gradient that allocates nothing, for callers that cannot allocate
 * device memory (code under HIP graph capture, tight serving or training
 * loops, harnesses that forbid hipMalloc).  Same arguments, plan and output
 * bits as dpg_wgrad, minus the workspace: the FP32 split partials go to a
 * static device array of the library, DPG_NOALLOC_SCRATCH_BYTES (64 MiB) per
 * GPU, held from the library's first use on that GPU until the process ends.
 * The partial planes are overwritten in full before they are read, so nothing
 * is cleared between calls.  Every call on one GPU shares that GPU's array:
 * calls that may overlap on one GPU (different streams, or different host
 * threads without ordering) race and must not be issued.  A plan whose
 * partials need more than DPG_NOALLOC_SCRATCH_BYTES (dpg_workspace_size above
 * it) returns DPG_ERR_WORKSPACE before any launch; DPG_ERR_HIP if the array's
 * device address cannot be obtained.  Calls no hipMalloc, hipFree or other
 * allocating routine.
 */
#define DPG_NOALLOC_SCRATCH_BYTES (64u << 20)
dpg_status dpg_wgrad_noalloc(const void* dy, int64_t lddy, const void* x, int64_t ldx,
                             void* dw, int64_t lddw, dpg_dtype dw_dtype,
                             int64_t T, int64_t N, int64_t K, int deterministic, int split_k,
                             hipStream_t stream);
/* DPG_NOALLOC_SCRATCH_BYTES as the library was built with it. */
size_t dpg_noalloc_scratch_bytes(void);

/*
 * FP32 router GEMM, E experts (256 on the router page), hidden size H, all
 * operands and outputs FP32 (router page, description and the legend under its
 * ratio table: token-by-hidden activations times a 256-by-hidden weight).  Every product a*b is
 * computed by BF16x3 emulation: hi = bf16_rne(a), lo = bf16_rne(a - hi), and
 * lo_a*hi_b + hi_a*lo_b + hi_a*hi_b accumulate (in that order) in FP32 on the
 * BF16 matrix cores -- or, where dpg_set_router_arithmetic allows it and the
 * plan takes it, by FP32 fused multiply-adds (see below).
 *   forward: y[T,E]  = x[T,H] . w[E,H]^T
 *   dgrad  : dx[T,H] = dy[T,E] . w[E,H]
 *   wgrad  : dw[E,H] = dy[T,E]^T . x[T,H]
 */
dpg_status dpg_router_forward(const float* x, int64_t ldx, const float* w, int64_t ldw,
                              float* y, int64_t ldy, int64_t T, int64_t E, int64_t H,
                              int deterministic, int split_k,
                              void* workspace, size_t workspace_bytes, hipStream_t stream);
dpg_status dpg_router_dgrad(const float* dy, int64_t lddy, const float* w, int64_t ldw,
                            float* dx, int64_t lddx, int64_t T, int64_t E, int64_t H,
                            int deterministic, int split_k,
                            void* workspace, size_t workspace_bytes, hipStream_t stream);
dpg_status dpg_router_wgrad(const float* dy, int64_t lddy, const float* x, int64_t ldx,
                            float* dw, int64_t lddw, int64_t T, int64_t E, int64_t H,
                            int deterministic, int split_k,
                            void* workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * Batched projection GEMMs: `batch` independent problems of one shape in one
 * launch, as the page "[Cake 9/13] dense_gemm: batched projection and FP32
 * router GEMMs" (description) describes for the per-head projections: one
 * batched BF16 GEMM over strided views, forward and both gradients, with a
 * choice of weight layout.
 *   Problem b reads x + b * stride_x (and likewise for every operand; strides in
 *   elements) and writes its output at y + b * stride_y.  An input stride may be
 *   0 (the same matrix for every problem); when batch > 1 the outputs must not
 *   overlap: stacked (stride >= (rows - 1) * ld + cols) or interleaved within
 *   rows (stride >= cols and (batch - 1) * stride + cols <= ld, e.g. per-head
 *   views of a token-major buffer), else DPG_ERR_INVALID_ARG.  Every non-zero stride times the element size is a
 *   multiple of 16 bytes (DPG_ERR_ALIGNMENT).
 *   w_layout DPG_WEIGHT_NK: the weight is W[N, K] as in the single entry points;
 *   DPG_WEIGHT_KN: the weight is stored W[K, N] (row stride ldw >= N), i.e. the
 *   forward is Y = X . W.  For the weight gradient w_layout is the layout of the
 *   output: dW[N, K] = dY^T X, or dW[K, N] = X^T dY (row stride lddw >= N).
 *   Everything else (dtypes, alignment, deterministic, split_k, workspace from
 *   dpg_workspace_size_batched, errors) is as for the single entry points; each
 *   problem's result equals what the single entry point computes for it under
 *   the plan the batched call uses.  batch = 0 is a no-op.
 */
typedef enum { DPG_WEIGHT_NK = 0, DPG_WEIGHT_KN = 1 } dpg_weight_layout;

dpg_status dpg_forward_batched(const void* x, int64_t ldx, int64_t stride_x,
                               const void* w, int64_t ldw, int64_t stride_w, dpg_weight_layout w_layout,
                               void* y, int64_t ldy, int64_t stride_y, dpg_dtype y_dtype,
                               int64_t batch, int64_t T, int64_t N, int64_t K, int deterministic, int split_k,
                               void* workspace, size_t workspace_bytes, hipStream_t stream);

dpg_status dpg_dgrad_batched(const void* dy, int64_t lddy, int64_t stride_dy,
                             const void* w, int64_t ldw, int64_t stride_w, dpg_weight_layout w_layout,
                             void* dx, int64_t lddx, int64_t stride_dx, dpg_dtype dx_dtype,
                             int64_t batch, int64_t T, int64_t N, int64_t K, int deterministic, int split_k,
                             void* workspace, size_t workspace_bytes, hipStream_t stream);

dpg_status dpg_wgrad_batched(const void* dy, int64_t lddy, int64_t stride_dy,
                             const void* x, int64_t ldx, int64_t stride_x,
                             void* dw, int64_t lddw, int64_t stride_dw, dpg_weight_layout w_layout,
                             dpg_dtype dw_dtype, int64_t batch, int64_t T, int64_t N, int64_t K,
                             int deterministic, int split_k,
                             void* workspace, size_t workspace_bytes, hipStream_t stream);

/* Workspace bytes of a batched call (projection passes 0..2 only; (size_t)-1
 * for arguments the call would reject). */
size_t dpg_workspace_size_batched(dpg_pass pass, dpg_weight_layout w_layout, int64_t batch, int64_t T,
                                  int64_t N, int64_t K, dpg_dtype out_dtype, int deterministic, int split_k);

/* Host-only plan description of a batched call (as dpg_plan_describe). */
dpg_status dpg_plan_describe_batched(dpg_pass pass, dpg_weight_layout w_layout, int64_t batch, int64_t T,
                                     int64_t N, int64_t K, dpg_dtype out_dtype, int deterministic, int split_k,
                                     char* buf, size_t buflen);

/*
 * Bytes of workspace the call with these arguments needs (0 when the plan has a
 * single K split): the FP32 partial products of the splits, S planes of the
 * output's rows x columns, which a second kernel adds in ascending split order
 * (the router page's commit message sums the split partials positionally over
 * the split dimension; the K1 weight-gradient page's description names one and
 * two K splits).  For router passes N = E, K = H and out_dtype must be DPG_F32.
 * Returns (size_t)-1 for arguments the matching call would reject.  The size
 * does not depend on the row strides.
 */
size_t dpg_workspace_size(dpg_pass pass, int64_t T, int64_t N, int64_t K, dpg_dtype out_dtype,
                          int deterministic, int split_k);

/*
 * Host-only description of the plan the library would use (kernel variant,
 * tile, raster group, K splits and their K-block partition, workspace) as one
 * line of text in `buf` (truncated to buflen - 1 characters, NUL-terminated):
 * the plan a key maps to, as the row-half-release page's description keys its
 * programs by exact token count and the router page's commit message keys
 * entries by shape, split count and alignment.  Split-K mode is described for
 * 256 CUs.  Row strides of 2^22 elements or more run the same K partition on
 * the generic kernel, which this text does not show.  Makes no HIP call;
 * usable without a GPU.  DPG_ERR_INVALID_ARG for a NULL or empty buffer or
 * arguments no plan covers.
 */
dpg_status dpg_plan_describe(dpg_pass pass, int64_t T, int64_t N, int64_t K, dpg_dtype out_dtype,
                             int deterministic, int split_k, char* buf, size_t buflen);

/*
 * The plan cache (router page, commit message and review: calls are cached by
 * their own arguments, never by data pointers, and the cache is refreshed when
 * the route changes).  It is process-global and mutex-protected, holds at most
 * dpg_plan_cache_capacity() plans (least recently used out first), and its
 * keys carry a generation number.  dpg_clear_plan_cache drops every plan and
 * bumps the generation; it never fails.  dpg_plan_cache_stats writes the
 * number of cached plans and the generation through the non-NULL pointers.
 */
void dpg_clear_plan_cache(void);
void dpg_plan_cache_stats(int64_t* entries, int64_t* generation);
int64_t dpg_plan_cache_capacity(void);

/*
 * Grouped products: the projections of an expert layer.  The rows of the token
 * side are sorted by expert; group e (of E) holds the rows [offsets[e],
 * offsets[e + 1]) and has its own weight matrix at w + e * stride_w.
 *   forward: y[r, N]  = x[r, K] . w[e][N, K]^T           r in group e
 *   dgrad  : dx[r, K] = dy[r, N] . w[e][N, K]
 *   wgrad  : dw[e][N, K] = sum over the group's rows of dy[r, N]^T . x[r, K]
 * BF16 operands, FP32 accumulation, BF16 or FP32 outputs, as for the single
 * entry points.
 *   offsets : int32 [E + 1] on the DEVICE, ascending; offsets[0] is taken as 0.
 *             The sizes need not be known on the host: a call never waits.
 *             Groups may be empty (their weight gradient is zeros).  Offsets
 *             outside [0, R] or descending give unspecified values in the
 *             output, never an access outside the operands.  They must not
 *             change while the call runs: every wave reads them for itself.
 *   R       : rows of the token side.  Rows at offsets[E] and past it belong to
 *             no group: they are not read, and their output rows are zeros.
 *   stride_*: elements between groups' matrices, a multiple of 16 bytes (0: one
 *             weight for all groups).  Weight gradients must not overlap
 *             (stacked, or side by side in wider rows, as for the batched calls).
 * The plan depends on the sizes alone (it is made for 256 CUs whatever the
 * device has), every sum runs in a fixed order and nothing uses atomics: the bits are the same on every
 * call and on every MI355X.  Where there are few output tiles the reduction is
 * split (each group's rows, for wgrad) and the parts are added in order from
 * the workspace: dpg_grouped_workspace_size bytes, 0 where nothing is split.
 * Row strides of x, dy and w below 2^22 elements and of outputs of more than one
 * row below 2^21, R, N, K below 2^31 - 512 and E below 2^24
 * (DPG_ERR_UNSUPPORTED otherwise).  An empty output is a no-op; an empty
 * reduction writes zeros.
 */
size_t dpg_grouped_workspace_size(dpg_pass pass, int64_t E, int64_t R, int64_t N, int64_t K);
/* Host-only description of a grouped call's plan (kernel, tile, K splits, the
 * most units there can be and the grid on 256 CUs, whether the weight gradient
 * takes its groups by size, workspace), as dpg_plan_describe. */
dpg_status dpg_grouped_plan_describe(dpg_pass pass, int64_t E, int64_t R, int64_t N, int64_t K, char* buf,
                                     size_t buflen);
dpg_status dpg_grouped_forward(const void* x, int64_t ldx, const void* w, int64_t ldw, int64_t stride_w, void* y,
                               int64_t ldy, dpg_dtype y_dtype, const int32_t* offsets, int64_t E, int64_t R,
                               int64_t N, int64_t K, void* workspace, size_t workspace_bytes, hipStream_t stream);
dpg_status dpg_grouped_dgrad(const void* dy, int64_t lddy, const void* w, int64_t ldw, int64_t stride_w, void* dx,
                             int64_t lddx, dpg_dtype dx_dtype, const int32_t* offsets, int64_t E, int64_t R,
                             int64_t N, int64_t K, void* workspace, size_t workspace_bytes, hipStream_t stream);
dpg_status dpg_grouped_wgrad(const void* dy, int64_t lddy, const void* x, int64_t ldx, void* dw, int64_t lddw,
                             int64_t stride_dw, dpg_dtype dw_dtype, const int32_t* offsets, int64_t E, int64_t R,
                             int64_t N, int64_t K, void* workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * Routing: the top_k experts of every token, their weights, and the stable
 * order of the (token, slot) pairs by expert.
 *   logits   : FP32 [T, E], row stride ldl (any value >= E)
 *   experts  : int32 [T, top_k], by descending logit, ties to the lowest
 *              expert.  A logit of -infinity masks its expert; a token with
 *              fewer than top_k unmasked experts has -1 in its last slots.
 *   weights  : FP32 [T, top_k]; with renormalize != 0 the softmax over the
 *              chosen experts, else the softmax over all E at the chosen ones;
 *              0 in unused slots.  A NaN logit is never chosen and makes the
 *              token's weights NaN.
 *   offsets  : int32 [E + 1], first row of each expert and, last, the number of
 *              used slots: the grouped products' offsets
 *   rows     : int32 [T * top_k], the flat slot token * top_k + slot at each
 *              row, by (expert, slot); the unused slots follow in order
 *   positions: int32 [T, top_k], the inverse: each slot's row
 * Pointers are 4-byte aligned.  1 <= top_k <= min(E, 32), E <= 512, T * top_k
 * below 2^31 and T at most 33521664 (DPG_ERR_UNSUPPORTED beyond).  Workspace:
 * dpg_route_workspace_size bytes, 16-byte aligned (0 up to 64 tokens, one
 * launch).
 */
size_t dpg_route_workspace_size(int64_t T, int64_t E, int64_t top_k);
dpg_status dpg_route(const float* logits, int64_t ldl, int64_t T, int64_t E, int64_t top_k, int renormalize,
                     int32_t* experts, float* weights, int32_t* offsets, int32_t* rows, int32_t* positions,
                     void* workspace, size_t workspace_bytes, hipStream_t stream);

/* Gradient of the weights by the logits (experts, weights as dpg_route wrote
 * them): dlogits[t, i] = q_i (g_i - sum_j q_j g_j), q the softmax that
 * `renormalize` names and g = dweights at the chosen experts, 0 elsewhere. */
dpg_status dpg_route_dgrad(const float* logits, int64_t ldl, const int32_t* experts, const float* weights,
                           const float* dweights, float* dlogits, int64_t lddl, int64_t T, int64_t E, int64_t top_k,
                           int renormalize, hipStream_t stream);

/*
 * Rows into expert order, and back.  positions [T, top_k] and offsets [E + 1]
 * are dpg_route's; R rows on the sorted side (T * top_k for a whole route).
 *   dispatch: xs[positions[t, j]] = x[t], zeros at rows >= offsets[E]
 *   combine : y[t] = sum_j weights[t, j] ys[positions[t, j]] in FP32, ascending
 *             j, over the slots with positions below offsets[E]; weights NULL
 *             means 1, which is the gradient of dispatch
 *   combine_dgrad: dys[positions[t, j]] = weights[t, j] dy[t] (zeros at rows >=
 *             offsets[E]) and dweights[t, j] = <dy[t], ys[positions[t, j]]> (0
 *             for unused slots), summed in FP32
 * Every row from offsets[E] on is written as zeros, whether a position names it
 * or not (R may exceed T * top_k); a row before it that none names stays as it
 * was.  T = 0 is a no-op: nothing is written.  Matrices follow the conventions at the top (16-byte rows); BF16 or FP32, one
 * type per call except that combine takes one for ys and one for y.  Positions
 * outside [0, R) are left out.  R and T * top_k below 2^31, H and E at most 2^24
 * (DPG_ERR_UNSUPPORTED beyond).
 */
dpg_status dpg_dispatch(const void* x, int64_t ldx, const int32_t* positions, const int32_t* offsets, void* xs,
                        int64_t ldxs, dpg_dtype dtype, int64_t T, int64_t R, int64_t H, int64_t E, int64_t top_k,
                        hipStream_t stream);
dpg_status dpg_combine(const void* ys, int64_t ldys, dpg_dtype ys_dtype, const int32_t* positions,
                       const int32_t* offsets, const float* weights, void* y, int64_t ldy, dpg_dtype y_dtype,
                       int64_t T, int64_t R, int64_t H, int64_t E, int64_t top_k, hipStream_t stream);
dpg_status dpg_combine_dgrad(const void* dy, int64_t lddy, const void* ys, int64_t ldys, const int32_t* positions,
                             const int32_t* offsets, const float* weights, void* dys, int64_t lddys, float* dweights,
                             dpg_dtype dtype, int64_t T, int64_t R, int64_t H, int64_t E, int64_t top_k,
                             hipStream_t stream);

/*
 * One AdamW step over `count` tensors (an array on the HOST), in as few
 * launches as 48 tensors each allow.  Per element, g being the gradient times
 * *grad_scale (a device scalar, NULL: 1), in FP32:
 *   m = beta1 m + (1 - beta1) g          v = beta2 v + (1 - beta2) g^2
 *   p = p (1 - lr weight_decay)
 *       - lr / (1 - beta1^step) m / (sqrt(v / (1 - beta2^step)) + eps)
 * param is FP32 and updated in place; `copy`, if not NULL, receives it rounded
 * to BF16 (the weights the products read).  Gradients are BF16 or FP32, one
 * type per call.  Moments, one type per call:
 *   DPG_F32  : exp_avg holds m, exp_avg_sq holds v
 *   DPG_E4M3 : exp_avg holds m, exp_avg_sq holds sqrt(v), as codes whose values
 *              times the scale of their block of 256 consecutive elements
 *              (avg_scale, sq_scale: ceil(numel / 256) FP32 powers of two) are
 *              the moments.  Storing rounds at random between the neighbouring
 *              codes, from `seed`, the tensor's place in the array and the
 *              element's place alone: the same call gives the same bits, and a
 *              caller changes the seed from step to step.  A positive sqrt(v)
 *              is not rounded to 0.  A moment that is infinite or NaN (a
 *              gradient that is, or whose square is) is stored as NaN and stays
 *              so; its block's scale is that of the other elements, which it
 *              does not change.  Zero codes with any finite scale start.
 * Tensors are contiguous; any element alignment is taken (16-byte aligned ones
 * run wide), up to 2^35 elements each.  step >= 1, 0 <= beta < 1, lr, eps, weight_decay finite and >= 0,
 * else DPG_ERR_INVALID_ARG.  lr and step are host values: a captured call
 * repeats them.
 */
typedef struct {
  float* param;
  const void* grad;
  void* exp_avg;
  void* exp_avg_sq;
  float* avg_scale;
  float* sq_scale;
  void* copy;
  int64_t numel;
} dpg_adamw_tensor;
typedef struct {
  double lr, beta1, beta2, eps, weight_decay;
  int64_t step;
  const float* grad_scale;
  dpg_dtype grad_dtype, state_dtype;
  uint32_t seed;
} dpg_adamw_options;
dpg_status dpg_adamw(const dpg_adamw_tensor* tensors, int64_t count, const dpg_adamw_options* options,
                     hipStream_t stream);

/*
 * Dropout from a counter-based generator (Philox4x32, ten rounds): the mask is a
 * function of seed, step and an element's place in the [T, H] matrix (whatever
 * the strides), so it is never stored, and the same options give it again.
 *   p    : in [0, 1], taken to the nearest multiple of 2^-16; the elements kept
 *          are multiplied by 1 / (1 - p), and what is left out counts as 0
 *          whatever it holds.  p = 1 leaves nothing.
 *   seed : any 64 bits
 *   step : int64 on the DEVICE, 8-byte aligned, or NULL for 0.  A captured call
 *          reads it at each replay: a caller that counts it up on the device
 *          gets another mask each time.
 * Element 8 g + j of the matrix, row after row, takes 16 of the 128 bits of
 * counter (g, step) under the key `seed`: half j % 2 (low first) of word j / 2;
 * it is left out where they are below 65536 p.
 *
 *   y = keep x / (1 - p) [+ residual]
 * residual, of y's type, may be NULL.  y may be x or residual itself (same type
 * and strides).  The gradient by x is the same call on dy without a residual.
 * T and H below 2^31 (DPG_ERR_UNSUPPORTED beyond).
 */
typedef struct {
  double p;
  uint64_t seed;
  const int64_t* step;
} dpg_dropout_options;
dpg_status dpg_dropout(const void* x, int64_t ldx, dpg_dtype x_dtype, const void* residual, int64_t ldr, void* y,
                       int64_t ldy, dpg_dtype y_dtype, int64_t T, int64_t H, const dpg_dropout_options* options,
                       hipStream_t stream);

/*
 * Layer norm over the H columns of each row, FP32 inside:
 *   mean = sum v / H                 rstd = (sum (v - mean)^2 / H + eps)^-1/2
 *   n = (v - mean) rstd              y = n weight + bias
 * of v = x, or (dpg_add_layer_norm) of the sum that a residual block goes on
 * with, v = residual + keep x / (1 - p), which is written to `sum` (of
 * residual's type; it may be residual itself) and normalised as it was before
 * that rounding.
 *   weight, bias : FP32 [H], 16-byte aligned; NULL: ones, zeros
 *   mean, rstd   : FP32 [T], outputs, which the gradient reads
 *   options      : NULL: no dropout
 * Gradients, with u = dy weight:
 *   dv = rstd (u - sum u / H - n sum(u n) / H) + dsum
 *   dweight = sum over the rows of dy n          dbias = sum over the rows of dy
 * dx = dv alone; of a sum, dresidual = dv (of sum's type) and dx = keep dv / (1 -
 * p) (of a type of its own), with the forward call's options and the matrix
 * that it wrote to `sum`.  dsum (of sum's type), the gradient that reaches the
 * sum from elsewhere, may be NULL; dresidual may be dsum itself.  dweight and
 * dbias are FP32 [H], either may be NULL; T = 0 writes zeros to them.  Their
 * sums run in a fixed order through dpg_layer_norm_workspace_size bytes, 16-byte
 * aligned (not needed where both are NULL).  T below 2^31, H at most 16384
 * (DPG_ERR_UNSUPPORTED beyond).
 */
dpg_status dpg_layer_norm(const void* x, int64_t ldx, dpg_dtype x_dtype, const float* weight, const float* bias,
                          void* y, int64_t ldy, dpg_dtype y_dtype, float* mean, float* rstd, int64_t T, int64_t H,
                          double eps, hipStream_t stream);
dpg_status dpg_add_layer_norm(const void* x, int64_t ldx, dpg_dtype x_dtype, const void* residual, int64_t ldr,
                              void* sum, int64_t lds, dpg_dtype sum_dtype, const float* weight, const float* bias,
                              void* y, int64_t ldy, dpg_dtype y_dtype, float* mean, float* rstd, int64_t T, int64_t H,
                              double eps, const dpg_dropout_options* options, hipStream_t stream);
size_t dpg_layer_norm_workspace_size(int64_t T, int64_t H);
dpg_status dpg_layer_norm_dgrad(const void* dy, int64_t lddy, dpg_dtype dy_dtype, const void* x, int64_t ldx,
                                dpg_dtype x_dtype, const float* mean, const float* rstd, const float* weight, void* dx,
                                int64_t lddx, float* dweight, float* dbias, int64_t T, int64_t H, void* workspace,
                                size_t workspace_bytes, hipStream_t stream);
dpg_status dpg_add_layer_norm_dgrad(const void* dy, int64_t lddy, dpg_dtype dy_dtype, const void* sum, int64_t lds,
                                    dpg_dtype sum_dtype, const float* mean, const float* rstd, const float* weight,
                                    const void* dsum, int64_t lddsum, void* dx, int64_t lddx, dpg_dtype dx_dtype,
                                    void* dresidual, int64_t lddr, float* dweight, float* dbias, int64_t T, int64_t H,
                                    const dpg_dropout_options* options, void* workspace, size_t workspace_bytes,
                                    hipStream_t stream);

/*
 * A gated linear recurrence over sequences, channel by channel in FP32:
 *   f = 1 / (1 + e^-gate)     w = 1 - f if `coupled`, else 1
 *   h[t] = f[t] h[t - 1] + w[t] x[t]
 * gate, x, h : [R, D], BF16 or FP32, one type per call; h may be x itself
 * offsets    : NULL: S sequences of R / S rows each, one after the other (S has
 *              to divide R; one row each is a generation step).  Else int32
 *              [S + 1] on the DEVICE, ascending, offsets[0] taken as 0: sequence
 *              s has the rows [offsets[s], offsets[s + 1]).  Sequences may be
 *              empty.  Rows from offsets[S] on are not read, and their rows in
 *              the outputs are zeros.  Offsets outside [0, R] or descending give
 *              unspecified values, never an access outside the operands.
 * state      : FP32 [S, D], h before each sequence's first row; NULL: zeros
 * state_out  : FP32 [S, D], h after its last row (an empty one's is its state);
 *              NULL: not wanted; may be `state` itself
 * carries    : FP32, dpg_recurrence_carries_size bytes, for the gradient; NULL:
 *              not wanted
 * A weight that is exactly 0 leaves its term out whatever the term is, so a
 * gate of -infinity (any below about -87 counts as one) forgets the state, and
 * one of +infinity (any above about 87) with `coupled` passes over the input.  A
 * gate that is NaN makes h NaN from its row on, until a weight of 0.
 *
 * Gradient, from dh [R, D] of h and dstate [S, D] (or NULL: zeros) of state_out,
 * with the forward call's inputs and what it wrote to `carries`:
 *   r[t] = dh[t] + f[t + 1] r[t + 1]      (dstate behind a sequence's last row)
 *   dx[t] = w[t] r[t]
 *   dgate[t] = f[t] (1 - f[t]) r[t] (h[t - 1] - x[t] if `coupled`, else h[t - 1])
 * and into dstate_out (or NULL), not dstate itself, f r of each first row (an
 * empty sequence's is its dstate).
 *
 * A state passes several rows at once by the product of their f in FP32, which
 * below 2^-126 is off by up to 2^-149 for each row: of a large state c, up to
 * |c| 2^-149 a row may be left where rows one by one would leave less.
 * The states between carries are recomputed in FP32.  Sums run in a fixed order
 * that depends on the sizes alone.  Workspace: dpg_recurrence_workspace_size
 * bytes, 16-byte aligned; packed = whether offsets are given.  State matrices
 * and carries are 16-byte aligned.  R at most 2^30, S and D at most 2^24
 * (DPG_ERR_UNSUPPORTED beyond, and for launches of 2^22 workgroups or more).
 */
size_t dpg_recurrence_workspace_size(int64_t S, int64_t R, int64_t D, dpg_dtype dtype, int packed);
size_t dpg_recurrence_carries_size(int64_t S, int64_t R, int64_t D, dpg_dtype dtype, int packed);
dpg_status dpg_recurrence(const void* gate, int64_t ldg, const void* x, int64_t ldx, void* h, int64_t ldh,
                          dpg_dtype dtype, const float* state, float* state_out, float* carries,
                          const int32_t* offsets, int64_t S, int64_t R, int64_t D, int coupled, void* workspace,
                          size_t workspace_bytes, hipStream_t stream);
dpg_status dpg_recurrence_dgrad(const void* dh, int64_t lddh, const void* gate, int64_t ldg, const void* x, int64_t ldx,
                                const float* carries, const float* state, const float* dstate, void* dgate,
                                int64_t lddg, void* dx, int64_t lddx, float* dstate_out, dpg_dtype dtype,
                                const int32_t* offsets, int64_t S, int64_t R, int64_t D, int coupled, void* workspace,
                                size_t workspace_bytes, hipStream_t stream);

/* Static text for a status code ("unknown status" for other values); the
 * error classes follow the validation rules above. */
const char* dpg_status_string(dpg_status status);

/* Library version string (static text naming the target, gfx950). */
const char* dpg_version(void);

#ifdef __cplusplus
}
#endif

#endif /* DPG_H_ */

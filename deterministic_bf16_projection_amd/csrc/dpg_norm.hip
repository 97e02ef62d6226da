// C ABI of layer norm and dropout: validation and launches.  Conventions are
// in include/dpg.h, the kernels in norm_kernels.h and dropout_kernels.h.
#include <hip/hip_runtime.h>
#include <math.h>

#include <algorithm>

#include "api_common.h"
#include "norm_kernels.h"

namespace dpg {
namespace {

bool aligned4(const void* p) { return ((uintptr_t)p & 3u) == 0; }
bool row_type(int dtype) { return dtype == DPG_BF16 || dtype == DPG_F32; }
int elt_size(int dtype) { return dtype == DPG_F32 ? 4 : 2; }
Rows8 rows8(const void* data, int64_t ld) { return Rows8{const_cast<void*>(data), ld}; }

constexpr int64_t kMaxRows = (1ll << 31) - 1;

// Waves of a row and groups of eight columns of a lane.
struct NormLayout {
  int waves, groups;
  int columns() const { return waves * groups * 512; }
};
constexpr NormLayout kNormLayouts[] = {{1, 1}, {1, 2}, {4, 1}, {4, 2}, {4, 3}, {4, 4}, {8, 3}, {8, 4}};
constexpr int64_t kNormColumns = 8 * 4 * 512;

int norm_layout(int64_t H) {
  int i = 0;
  while (kNormLayouts[i].columns() < H) ++i;
  return i;
}

// Workgroups of the gradient: each one's sums for the weight gradient are a row
// of the workspace, so there are no more than fill the CUs, and each has at
// least eight rounds of rows where there are so many.
constexpr int64_t kGradBlocks = 512;
int64_t grad_blocks(int64_t T, int64_t H) {
  const int64_t rounds = (T + norm_rows(kNormLayouts[norm_layout(H)].waves) - 1) / norm_rows(kNormLayouts[norm_layout(H)].waves);
  return std::min(kGradBlocks, (rounds + 7) / 8);
}

template <bool X_BF16, bool ADD>
const void* norm_fn(int layout) {
  static const void* const fns[] = {
      (const void*)&norm_kernel<X_BF16, 1, 1, ADD>, (const void*)&norm_kernel<X_BF16, 1, 2, ADD>,
      (const void*)&norm_kernel<X_BF16, 4, 1, ADD>, (const void*)&norm_kernel<X_BF16, 4, 2, ADD>,
      (const void*)&norm_kernel<X_BF16, 4, 3, ADD>, (const void*)&norm_kernel<X_BF16, 4, 4, ADD>,
      (const void*)&norm_kernel<X_BF16, 8, 3, ADD>, (const void*)&norm_kernel<X_BF16, 8, 4, ADD>};
  return fns[layout];
}
template <bool X_BF16, bool ADD>
const void* norm_dgrad_fn(int layout) {
  static const void* const fns[] = {
      (const void*)&norm_dgrad_kernel<X_BF16, 1, 1, ADD>, (const void*)&norm_dgrad_kernel<X_BF16, 1, 2, ADD>,
      (const void*)&norm_dgrad_kernel<X_BF16, 4, 1, ADD>, (const void*)&norm_dgrad_kernel<X_BF16, 4, 2, ADD>,
      (const void*)&norm_dgrad_kernel<X_BF16, 4, 3, ADD>, (const void*)&norm_dgrad_kernel<X_BF16, 4, 4, ADD>,
      (const void*)&norm_dgrad_kernel<X_BF16, 8, 3, ADD>, (const void*)&norm_dgrad_kernel<X_BF16, 8, 4, ADD>};
  return fns[layout];
}

dpg_status check_norm(int64_t T, int64_t H) {
  if (T < 0 || H < 0) return DPG_ERR_INVALID_ARG;
  if (T > kMaxRows || H > kNormColumns) return DPG_ERR_UNSUPPORTED;
  return DPG_OK;
}

// FP32 vectors of H columns, read 16 bytes at a time
dpg_status check_columns(const void* a, const void* b) {
  return aligned16(a) && aligned16(b) ? DPG_OK : DPG_ERR_ALIGNMENT;
}

// one value a row
dpg_status check_statistics(const void* mean, const void* rstd) {
  if (!mean || !rstd) return DPG_ERR_INVALID_ARG;
  return aligned4(mean) && aligned4(rstd) ? DPG_OK : DPG_ERR_ALIGNMENT;
}

dpg_status drop_params(const dpg_dropout_options* o, DropParams& d) {
  d = DropParams{};
  d.scale = 1.f;
  if (!o) return DPG_OK;
  if (!(o->p >= 0 && o->p <= 1)) return DPG_ERR_INVALID_ARG;
  if (((uintptr_t)o->step & 7u) != 0) return DPG_ERR_ALIGNMENT;
  d.key0 = (unsigned)o->seed;
  d.key1 = (unsigned)(o->seed >> 32);
  d.step = o->step;
  d.bar = (unsigned)floor(o->p * 65536 + 0.5);
  d.scale = d.bar < 65536 ? (float)(65536.0 / (65536 - d.bar)) : 0.f;
  return DPG_OK;
}

dpg_status run_norm(NormParams& p, bool x_bf16, bool add, int64_t T, int64_t H, double eps, hipStream_t stream) {
  p.T = T;
  p.H = (int)H;
  p.inv_h = 1.f / (float)H;
  p.eps = (float)eps;
  const int layout = norm_layout(H);
  const int waves = kNormLayouts[layout].waves;
  const void* fn = x_bf16 ? (add ? norm_fn<true, true>(layout) : norm_fn<true, false>(layout))
                          : (add ? norm_fn<false, true>(layout) : norm_fn<false, false>(layout));
  void* args[] = {&p};
  return launch(fn, std::min<int64_t>((T + norm_rows(waves) - 1) / norm_rows(waves), 2048), norm_threads(waves), 0,
                args, stream);
}

dpg_status run_norm_grad(NormGradParams& p, bool x_bf16, bool add, int64_t T, int64_t H, float* dweight, float* dbias,
                         void* workspace, size_t workspace_bytes, hipStream_t stream) {
  const bool sums = dweight || dbias;
  if (sums && T > 0) {
    const size_t need = dpg_layer_norm_workspace_size(T, H);
    if (!workspace || workspace_bytes < need || !aligned16(workspace)) return DPG_ERR_WORKSPACE;
    p.partial = (float*)workspace;
  }
  p.T = T;
  p.H = (int)H;
  p.inv_h = 1.f / (float)H;
  int blocks = 0;
  if (T > 0) {
    blocks = (int)grad_blocks(T, H);
    const int layout = norm_layout(H);
    const int waves = kNormLayouts[layout].waves;
    const void* fn = x_bf16 ? (add ? norm_dgrad_fn<true, true>(layout) : norm_dgrad_fn<true, false>(layout))
                            : (add ? norm_dgrad_fn<false, true>(layout) : norm_dgrad_fn<false, false>(layout));
    void* args[] = {&p};
    const dpg_status st = launch(fn, blocks, norm_threads(waves), 0, args, stream);
    if (st != DPG_OK) return st;
  }
  if (!sums) return DPG_OK;
  const float* partial = p.partial;
  int h = (int)H;
  void* args[] = {&partial, &blocks, &h, &dweight, &dbias};
  return launch((const void*)&norm_wgrad_kernel, (2 * H + 63) / 64, 1024, 0, args, stream);
}

}  // namespace
}  // namespace dpg

using namespace dpg;

extern "C" {

dpg_status dpg_dropout(const void* x, int64_t ldx, dpg_dtype x_dtype, const void* residual, int64_t ldr, void* y,
                       int64_t ldy, dpg_dtype y_dtype, int64_t T, int64_t H, const dpg_dropout_options* options,
                       hipStream_t stream) {
  if (!row_type((int)x_dtype) || !row_type((int)y_dtype) || !options) return DPG_ERR_INVALID_ARG;
  if (T < 0 || H < 0) return DPG_ERR_INVALID_ARG;
  if (T > kMaxRows || H > kMaxRows) return DPG_ERR_UNSUPPORTED;
  DropoutParams p{};
  dpg_status st = drop_params(options, p.drop);
  if (st != DPG_OK) return st;
  if ((st = check_mat(Mat{x, ldx, T, H, elt_size((int)x_dtype)})) != DPG_OK) return st;
  if ((st = check_mat(Mat{y, ldy, T, H, elt_size((int)y_dtype)})) != DPG_OK) return st;
  if (residual && (st = check_mat(Mat{residual, ldr, T, H, elt_size((int)y_dtype)})) != DPG_OK) return st;
  if (T == 0 || H == 0) return DPG_OK;
  p.T = T;
  p.per_row = (int)(H / 8);
  p.groups = T * (H / 8);
  // rows that follow each other without gaps are one long row, cut where it suits the workgroups
  if (T > 1 ? ldx == H && ldy == H && (!residual || ldr == H) : true) {
    constexpr int kGroups = 2048;
    p.per_row = kGroups;
    p.T = (p.groups + kGroups - 1) / kGroups;
    ldx = ldy = ldr = 8 * kGroups;
  }
  p.x = rows8(x, ldx);
  p.y = rows8(y, ldy);
  p.residual = rows8(residual, ldr);
  p.lanes_log2 = 3;
  while (p.lanes_log2 < 8 && (1 << p.lanes_log2) < std::min<int64_t>(p.per_row, p.groups)) ++p.lanes_log2;
  const bool a = x_dtype == DPG_BF16, b = y_dtype == DPG_BF16;
  const void* fn =
      residual ? (a ? (b ? (const void*)&dropout_kernel<true, true, true> : (const void*)&dropout_kernel<true, false, true>)
                    : (b ? (const void*)&dropout_kernel<false, true, true> : (const void*)&dropout_kernel<false, false, true>))
               : (a ? (b ? (const void*)&dropout_kernel<true, true, false> : (const void*)&dropout_kernel<true, false, false>)
                    : (b ? (const void*)&dropout_kernel<false, true, false> : (const void*)&dropout_kernel<false, false, false>));
  const int64_t each = 256 >> p.lanes_log2;
  void* args[] = {&p};
  return launch(fn, std::min<int64_t>((p.T + each - 1) / each, 1 << 22), 256, 0, args, stream);
}

dpg_status dpg_layer_norm(const void* x, int64_t ldx, dpg_dtype x_dtype, const float* weight, const float* bias,
                          void* y, int64_t ldy, dpg_dtype y_dtype, float* mean, float* rstd, int64_t T, int64_t H,
                          double eps, hipStream_t stream) {
  if (!row_type((int)x_dtype) || !row_type((int)y_dtype) || !(eps >= 0) || !isfinite(eps)) return DPG_ERR_INVALID_ARG;
  dpg_status st = check_norm(T, H);
  if (st != DPG_OK) return st;
  if ((st = check_mat(Mat{x, ldx, T, H, elt_size((int)x_dtype)})) != DPG_OK) return st;
  if ((st = check_mat(Mat{y, ldy, T, H, elt_size((int)y_dtype)})) != DPG_OK) return st;
  if ((st = check_columns(weight, bias)) != DPG_OK) return st;
  if (T == 0 || H == 0) return DPG_OK;
  if ((st = check_statistics(mean, rstd)) != DPG_OK) return st;
  NormParams p{};
  p.x = rows8(x, ldx);
  p.y = rows8(y, ldy);
  p.weight = weight;
  p.bias = bias;
  p.mean = mean;
  p.rstd = rstd;
  p.y_bf16 = y_dtype == DPG_BF16;
  return run_norm(p, x_dtype == DPG_BF16, false, T, H, eps, stream);
}

dpg_status dpg_add_layer_norm(const void* x, int64_t ldx, dpg_dtype x_dtype, const void* residual, int64_t ldr,
                              void* sum, int64_t lds, dpg_dtype sum_dtype, const float* weight, const float* bias,
                              void* y, int64_t ldy, dpg_dtype y_dtype, float* mean, float* rstd, int64_t T, int64_t H,
                              double eps, const dpg_dropout_options* options, hipStream_t stream) {
  if (!row_type((int)x_dtype) || !row_type((int)sum_dtype) || !row_type((int)y_dtype) || !(eps >= 0) || !isfinite(eps))
    return DPG_ERR_INVALID_ARG;
  dpg_status st = check_norm(T, H);
  if (st != DPG_OK) return st;
  NormParams p{};
  if ((st = drop_params(options, p.drop)) != DPG_OK) return st;
  if ((st = check_mat(Mat{x, ldx, T, H, elt_size((int)x_dtype)})) != DPG_OK) return st;
  if ((st = check_mat(Mat{residual, ldr, T, H, elt_size((int)sum_dtype)})) != DPG_OK) return st;
  if ((st = check_mat(Mat{sum, lds, T, H, elt_size((int)sum_dtype)})) != DPG_OK) return st;
  if ((st = check_mat(Mat{y, ldy, T, H, elt_size((int)y_dtype)})) != DPG_OK) return st;
  if ((st = check_columns(weight, bias)) != DPG_OK) return st;
  if (T == 0 || H == 0) return DPG_OK;
  if ((st = check_statistics(mean, rstd)) != DPG_OK) return st;
  p.x = rows8(residual, ldr);
  p.branch = rows8(x, ldx);
  p.sum = rows8(sum, lds);
  p.y = rows8(y, ldy);
  p.weight = weight;
  p.bias = bias;
  p.mean = mean;
  p.rstd = rstd;
  p.y_bf16 = y_dtype == DPG_BF16;
  p.branch_bf16 = x_dtype == DPG_BF16;
  return run_norm(p, sum_dtype == DPG_BF16, true, T, H, eps, stream);
}

size_t dpg_layer_norm_workspace_size(int64_t T, int64_t H) {
  if (check_norm(T, H) != DPG_OK) return (size_t)-1;
  return T > 0 && H > 0 ? (size_t)grad_blocks(T, H) * 2 * (size_t)H * sizeof(float) : 0;
}

dpg_status dpg_layer_norm_dgrad(const void* dy, int64_t lddy, dpg_dtype dy_dtype, const void* x, int64_t ldx,
                                dpg_dtype x_dtype, const float* mean, const float* rstd, const float* weight, void* dx,
                                int64_t lddx, float* dweight, float* dbias, int64_t T, int64_t H, void* workspace,
                                size_t workspace_bytes, hipStream_t stream) {
  if (!row_type((int)dy_dtype) || !row_type((int)x_dtype)) return DPG_ERR_INVALID_ARG;
  dpg_status st = check_norm(T, H);
  if (st != DPG_OK) return st;
  const int xe = elt_size((int)x_dtype);
  if ((st = check_mat(Mat{dy, lddy, T, H, elt_size((int)dy_dtype)})) != DPG_OK) return st;
  if ((st = check_mat(Mat{x, ldx, T, H, xe})) != DPG_OK) return st;
  if ((st = check_mat(Mat{dx, lddx, T, H, xe})) != DPG_OK) return st;
  if (!aligned4(dweight) || !aligned4(dbias) || !aligned16(weight)) return DPG_ERR_ALIGNMENT;
  if (H == 0) return DPG_OK;
  if (H % 8 != 0) return DPG_ERR_ALIGNMENT;
  if (T > 0 && (st = check_statistics(mean, rstd)) != DPG_OK) return st;
  NormGradParams p{};
  p.dy = rows8(dy, lddy);
  p.x = rows8(x, ldx);
  p.dx = rows8(dx, lddx);
  p.mean = mean;
  p.rstd = rstd;
  p.weight = weight;
  p.dy_bf16 = dy_dtype == DPG_BF16;
  return run_norm_grad(p, x_dtype == DPG_BF16, false, T, H, dweight, dbias, workspace, workspace_bytes, stream);
}

dpg_status dpg_add_layer_norm_dgrad(const void* dy, int64_t lddy, dpg_dtype dy_dtype, const void* sum, int64_t lds,
                                    dpg_dtype sum_dtype, const float* mean, const float* rstd, const float* weight,
                                    const void* dsum, int64_t lddsum, void* dx, int64_t lddx, dpg_dtype dx_dtype,
                                    void* dresidual, int64_t lddr, float* dweight, float* dbias, int64_t T, int64_t H,
                                    const dpg_dropout_options* options, void* workspace, size_t workspace_bytes,
                                    hipStream_t stream) {
  if (!row_type((int)dy_dtype) || !row_type((int)sum_dtype) || !row_type((int)dx_dtype)) return DPG_ERR_INVALID_ARG;
  dpg_status st = check_norm(T, H);
  if (st != DPG_OK) return st;
  NormGradParams p{};
  if ((st = drop_params(options, p.drop)) != DPG_OK) return st;
  const int se = elt_size((int)sum_dtype);
  if ((st = check_mat(Mat{dy, lddy, T, H, elt_size((int)dy_dtype)})) != DPG_OK) return st;
  if ((st = check_mat(Mat{sum, lds, T, H, se})) != DPG_OK) return st;
  if (dsum && (st = check_mat(Mat{dsum, lddsum, T, H, se})) != DPG_OK) return st;
  if ((st = check_mat(Mat{dx, lddx, T, H, elt_size((int)dx_dtype)})) != DPG_OK) return st;
  if ((st = check_mat(Mat{dresidual, lddr, T, H, se})) != DPG_OK) return st;
  if (!aligned4(dweight) || !aligned4(dbias) || !aligned16(weight)) return DPG_ERR_ALIGNMENT;
  if (H == 0) return DPG_OK;
  if (H % 8 != 0) return DPG_ERR_ALIGNMENT;
  if (T > 0 && (st = check_statistics(mean, rstd)) != DPG_OK) return st;
  p.dy = rows8(dy, lddy);
  p.x = rows8(sum, lds);
  p.dsum = rows8(dsum, lddsum);
  p.dx = rows8(dx, lddx);
  p.dresidual = rows8(dresidual, lddr);
  p.mean = mean;
  p.rstd = rstd;
  p.weight = weight;
  p.dy_bf16 = dy_dtype == DPG_BF16;
  p.dx_bf16 = dx_dtype == DPG_BF16;
  return run_norm_grad(p, sum_dtype == DPG_BF16, true, T, H, dweight, dbias, workspace, workspace_bytes, stream);
}

}  // extern "C"

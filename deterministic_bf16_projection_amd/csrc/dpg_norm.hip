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

constexpr int64_t kNormColumns = kNormWaves * 1024;
struct NormLayout {
  int chunks, waves, sets;  // groups of eight columns of a lane; waves of a row; rows of a workgroup at once
  int lanes;                // of a row in a wave: below 64, several rows share the wave
  int threads() const { return lanes < 64 ? lanes * sets : 64 * waves * sets; }
};
// Rows of up to 256 columns leave a wave half empty or more: 64 / lanes rows to a
// wave (65536 rows of 64 columns, BF16: forward 19 us with a wave each, 7 so;
// gradient 27 and 14).
int norm_lanes(int64_t H) { return H <= 64 ? 8 : H <= 128 ? 16 : H <= 256 ? 32 : 64; }
// Forward.  Few rows, and sums: up to two groups to a lane, weights in
// registers, so that a row's latency is spread over waves.  Many rows: as few
// waves to a row as hold it with eight groups to a lane, so that none waits for
// others (16384 rows of 4096 columns, BF16: one wave 47.8 us, four 52, eight 62;
// sums of 8192 rows, FP32 and BF16: two waves 81 us, four 78).  Near the border,
// BF16, us, many rows' cut and few rows': 1024 rows of 4096 columns 7.3 and 6.5, of
// 16384 columns 21.3 and 20.7; 2048 rows of 8192 columns 19.0 and 16.3, of 16384
// 34 and 46; 4096 rows of 4096 columns 14.2 and 14.6, of 8192 31.4 and 32.0.
constexpr int64_t kNormManyRows = 1024;
NormLayout norm_layout(int64_t T, int64_t H, bool add) {
  NormLayout l;
  if (T < kNormManyRows || H <= 1024 || add)
    l.chunks = H <= 512 ? 1 : 2;
  else
    l.chunks = H <= 2048 ? 4 : 8;
  l.waves = (int)((H + 512 * l.chunks - 1) / (512 * l.chunks));
  // workgroups of enough waves for eight to a CU with their weights in LDS
  l.sets = std::max(1, (norm_shares_weights(l.chunks) && H > 4096 ? 8 : 4) / l.waves);
  l.lanes = norm_lanes(H);
  l.sets *= 64 / l.lanes;
  return l;
}
// workgroups that go through all rows: 2 to 8 to a CU
int64_t norm_grid(const NormLayout& l) { return norm_shares_weights(l.chunks) ? 512 : 2048; }
// Gradient: one group to a lane as long as sixteen waves hold the row (16384 rows
// of 4096 columns 79 us; two groups with eight or twelve waves 82 to 84), and as
// many rows at once as sixteen waves hold, since each workgroup's sums for the
// weight gradient are a row of the workspace.
NormLayout grad_layout(int64_t H) {
  NormLayout l;
  l.chunks = H <= kNormWaves * 512 ? 1 : 2;
  l.waves = (int)((H + 512 * l.chunks - 1) / (512 * l.chunks));
  l.lanes = norm_lanes(H);
  l.sets = kNormWaves / l.waves * (64 / l.lanes);
  return l;
}
// One workgroup to a CU, and at least two rows of each set where there are so many.
constexpr int64_t kGradBlocks = 256;
int64_t grad_blocks(int64_t T, int64_t H) {
  const int64_t each = 2 * grad_layout(H).sets;
  return std::min(kGradBlocks, (T + each - 1) / each);
}

template <bool X, bool Y, int C, bool SMALL>
const void* norm_fn(bool add, bool branch) {
  if constexpr (!norm_shares_weights(C)) {  // sums have up to two groups to a lane
    if (add) return branch ? (const void*)&norm_kernel<X, Y, C, true, true, SMALL> : (const void*)&norm_kernel<X, Y, C, true, false, SMALL>;
  }
  return (const void*)&norm_kernel<X, Y, C, false, X, SMALL>;
}
template <int C, bool SMALL>
const void* norm_fn(bool x, bool y, bool add, bool branch) {
  return x ? (y ? norm_fn<true, true, C, SMALL>(add, branch) : norm_fn<true, false, C, SMALL>(add, branch))
           : (y ? norm_fn<false, true, C, SMALL>(add, branch) : norm_fn<false, false, C, SMALL>(add, branch));
}
const void* norm_fn(const NormLayout& l, bool x, bool y, bool add, bool branch) {
  if (l.lanes < 64) return norm_fn<1, true>(x, y, add, branch);
  switch (l.chunks) {
    case 1: return norm_fn<1, false>(x, y, add, branch);
    case 2: return norm_fn<2, false>(x, y, add, branch);
    case 4: return norm_fn<4, false>(x, y, add, branch);
    default: return norm_fn<8, false>(x, y, add, branch);
  }
}
template <bool X, bool DY, int C, bool SMALL>
const void* norm_dgrad_fn(bool add) {
  return add ? (const void*)&norm_dgrad_kernel<X, DY, C, true, SMALL> : (const void*)&norm_dgrad_kernel<X, DY, C, false, SMALL>;
}
template <bool X, bool DY>
const void* norm_dgrad_fn(const NormLayout& l, bool add) {
  if (l.lanes < 64) return norm_dgrad_fn<X, DY, 1, true>(add);
  return l.chunks == 1 ? norm_dgrad_fn<X, DY, 1, false>(add) : norm_dgrad_fn<X, DY, 2, false>(add);
}
template <bool X, bool Y>
const void* dropout_fn(bool add, bool past) {
  if (add) return past ? (const void*)&dropout_kernel<X, Y, true, true> : (const void*)&dropout_kernel<X, Y, true, false>;
  return past ? (const void*)&dropout_kernel<X, Y, false, true> : (const void*)&dropout_kernel<X, Y, false, false>;
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

dpg_status run_norm(NormParams& p, bool x_bf16, bool y_bf16, bool add, bool branch_bf16, int64_t T, int64_t H,
                    double eps, hipStream_t stream) {
  const NormLayout l = norm_layout(T, H, add);
  p.T = T;
  p.H = (int)H;
  p.waves = l.waves;
  p.groups = l.sets;
  p.lanes = l.lanes;
  p.inv_h = 1.f / (float)H;
  p.eps = (float)eps;
  const void* fn = norm_fn(l, x_bf16, y_bf16, add, branch_bf16);
  const size_t lds = norm_shares_weights(l.chunks) ? (size_t)H * 2 * sizeof(float) : 0;
  void* args[] = {&p};
  return launch(fn, std::min<int64_t>((T + l.sets - 1) / l.sets, norm_grid(l)), l.threads(), lds, args, stream);
}

dpg_status run_norm_grad(NormGradParams& p, bool x_bf16, bool dy_bf16, bool add, int64_t T, int64_t H, float* dweight,
                         float* dbias, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  const bool sums = dweight || dbias;
  if (sums && T > 0) {
    const size_t need = dpg_layer_norm_workspace_size(T, H);
    if (!workspace || workspace_bytes < need || !aligned16(workspace)) return DPG_ERR_WORKSPACE;
    p.partial = (float*)workspace;
  }
  const NormLayout l = grad_layout(H);
  p.T = T;
  p.H = (int)H;
  p.waves = l.waves;
  p.groups = l.sets;
  p.lanes = l.lanes;
  int blocks = 0;
  if (T > 0) {
    blocks = (int)grad_blocks(T, H);
    const void* fn = x_bf16 ? (dy_bf16 ? norm_dgrad_fn<true, true>(l, add) : norm_dgrad_fn<true, false>(l, add))
                            : (dy_bf16 ? norm_dgrad_fn<false, true>(l, add) : norm_dgrad_fn<false, false>(l, add));
    const size_t lds = sums && l.sets > 1 ? (size_t)l.sets * H * sizeof(float) : 0;
    void* args[] = {&p};
    const dpg_status st = launch(fn, blocks, l.threads(), lds, args, stream);
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
  // outputs that do not fit the XCDs' 32 MB of L2 go past it, and so do their inputs
  const bool past = T * H >= (int64_t)(32 << 20) / elt_size((int)y_dtype);
  p.T = T;
  p.per_row = (int)(H / 8);
  p.groups = T * (H / 8);
  // rows that follow each other without gaps are one long row, cut where it suits the workgroups
  if (T > 1 ? ldx == H && ldy == H && (!residual || ldr == H) : true) {
    constexpr int kGroups = 512;
    p.per_row = kGroups;
    p.T = (p.groups + kGroups - 1) / kGroups;
    ldx = ldy = ldr = 8 * kGroups;
  }
  p.x = rows8(x, ldx);
  p.y = rows8(y, ldy);
  p.residual = rows8(residual, ldr);
  p.lanes_log2 = 3;
  while (p.lanes_log2 < 8 && (1 << p.lanes_log2) < std::min<int64_t>(p.per_row, p.groups)) ++p.lanes_log2;
  const bool add = residual != nullptr;
  const void* fn = x_dtype == DPG_BF16
                       ? (y_dtype == DPG_BF16 ? dropout_fn<true, true>(add, past) : dropout_fn<true, false>(add, past))
                       : (y_dtype == DPG_BF16 ? dropout_fn<false, true>(add, past) : dropout_fn<false, false>(add, past));
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
  return run_norm(p, x_dtype == DPG_BF16, y_dtype == DPG_BF16, false, false, T, H, eps, stream);
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
  return run_norm(p, sum_dtype == DPG_BF16, y_dtype == DPG_BF16, true, x_dtype == DPG_BF16, T, H, eps, stream);
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
  return run_norm_grad(p, x_dtype == DPG_BF16, dy_dtype == DPG_BF16, false, T, H, dweight, dbias, workspace, workspace_bytes, stream);
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
  p.dx_bf16 = dx_dtype == DPG_BF16;
  return run_norm_grad(p, sum_dtype == DPG_BF16, dy_dtype == DPG_BF16, true, T, H, dweight, dbias, workspace, workspace_bytes, stream);
}

}  // extern "C"

// C ABI of the grouped products (rows sorted by expert, one weight matrix per
// expert): validation and launches.  Conventions are in include/dpg.h, the
// unit stream in grouped_units.h, the kernels in gemm_fast.h.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "api_common.h"
#include "gemm_fast.h"

namespace dpg {
namespace {

typedef void (*GroupedFn)(GroupedParams);

template <int BM, int BN, int WM_, int WN_, int LAYOUT>
struct GroupedRow {
  static constexpr GroupedFn fns[2] = {
      &gemm_fast_kernel<BM, BN, WM_, WN_, LAYOUT != LAYOUT_WGRAD, LAYOUT == LAYOUT_FWD, OUT_BF16, false, false, true>,
      &gemm_fast_kernel<BM, BN, WM_, WN_, LAYOUT != LAYOUT_WGRAD, LAYOUT == LAYOUT_FWD, OUT_F32, false, false, true>};
};

struct GroupedTile {
  int bm, bn, threads, per_cu;
};
constexpr GroupedTile kGroupedTiles[] = {{256, 256, 512, 1}, {128, 128, 256, 2}};

GroupedFn lookup_grouped_kernel(int tile, int layout, int out) {
  static const GroupedFn table[2][3][2] = {
      {{GroupedRow<256, 256, 2, 4, 0>::fns[0], GroupedRow<256, 256, 2, 4, 0>::fns[1]},
       {GroupedRow<256, 256, 2, 4, 1>::fns[0], GroupedRow<256, 256, 2, 4, 1>::fns[1]},
       {GroupedRow<256, 256, 2, 4, 2>::fns[0], GroupedRow<256, 256, 2, 4, 2>::fns[1]}},
      {{GroupedRow<128, 128, 2, 2, 0>::fns[0], GroupedRow<128, 128, 2, 2, 0>::fns[1]},
       {GroupedRow<128, 128, 2, 2, 1>::fns[0], GroupedRow<128, 128, 2, 2, 1>::fns[1]},
       {GroupedRow<128, 128, 2, 2, 2>::fns[0], GroupedRow<128, 128, 2, 2, 2>::fns[1]}}};
  return table[tile][layout][out];
}

// 256x256 tiles where the average group fills them, 128x128 otherwise.
int grouped_tile(int layout, int64_t R, int64_t E, int64_t M, int64_t N) {
  if (layout == LAYOUT_WGRAD) return M >= 256 && N >= 256 ? 0 : 1;
  return R >= 192 * E && N >= 256 ? 0 : 1;
}

// One grouped pass.  (a, b) are (x, w), (dy, w) and (dy, x); `stride` is the
// element stride between the groups' weights (weight gradient: outputs).
dpg_status run_grouped(int layout, const void* a, int64_t lda, const void* b, int64_t ldb, void* c, int64_t ldc,
                       int64_t stride, int out, const int32_t* offsets, int64_t E, int64_t R, int64_t N, int64_t K,
                       hipStream_t stream) {
  if (out != DPG_BF16 && out != DPG_F32) return DPG_ERR_INVALID_ARG;
  if (E < 0 || R < 0 || N < 0 || K < 0 || stride < 0) return DPG_ERR_INVALID_ARG;
  const int out_elt = out == DPG_F32 ? 4 : 2;
  const bool wgrad = layout == LAYOUT_WGRAD;
  const int64_t weights = E > 0 ? N : 0;  // no groups: no weight is touched
  const Mat ma = {a, lda, R, layout == LAYOUT_FWD ? K : N, 2};
  const Mat mb = wgrad ? Mat{b, ldb, R, K, 2} : Mat{b, ldb, weights, K, 2};
  const Mat mc = wgrad ? Mat{c, ldc, weights, K, out_elt} : Mat{c, ldc, R, layout == LAYOUT_FWD ? N : K, out_elt};
  // an empty output is a no-op whatever the operands are
  const bool empty = mc.rows == 0 || mc.cols == 0;
  dpg_status st;
  if ((st = check_mat(ma)) != DPG_OK) return st;
  if ((st = check_mat(mb)) != DPG_OK) return st;
  if ((st = check_mat(mc)) != DPG_OK) return st;
  const Mat& mw = wgrad ? mc : mb;
  if (E > 1 && mw.rows > 0 && mw.cols > 0) {
    if (stride * mw.elt % 16 != 0) return DPG_ERR_ALIGNMENT;
    // the groups' weight gradients may not overlap: stacked, or side by side in wider rows
    const bool stacked = stride >= (mw.rows - 1) * mw.ld + mw.cols;
    const bool beside = stride >= mw.cols && (E - 1) * stride + mw.cols <= mw.ld;
    if (wgrad && !stacked && !beside) return DPG_ERR_INVALID_ARG;
  }
  if (empty) return DPG_OK;
  if (E > 0 && (!offsets || ((uintptr_t)offsets & 3u))) return offsets ? DPG_ERR_ALIGNMENT : DPG_ERR_INVALID_ARG;
  // a tile is addressed through 32-bit buffer offsets, rows and units through 32-bit indexes
  if (std::max(lda, ldb) >= (1 << 22)) return DPG_ERR_UNSUPPORTED;
  if (R >= (1ll << 31) - 512 || N >= (1ll << 31) - 512 || K >= (1ll << 31) - 512 || E >= (1ll << 24))
    return DPG_ERR_UNSUPPORTED;

  GroupedParams p{};
  p.a = a;
  p.b = b;
  p.c = c;
  p.lda = lda;
  p.ldb = ldb;
  p.ldc = ldc;
  p.M = (int)(wgrad ? N : R);
  p.N = (int)(layout == LAYOUT_FWD ? N : K);
  p.K = (int)(layout == LAYOUT_FWD ? K : N);  // weight gradient: each group's rows
  p.splits = 1;
  p.batch = 1;
  p.batch_b = stride;
  p.batch_c = stride;
  p.offsets = offsets;
  p.groups = (int)E;
  p.rows = (int)R;
  const int tile = grouped_tile(layout, R, E, p.M, p.N);
  const GroupedTile& t = kGroupedTiles[tile];
  p.tiles_m = (p.M + t.bm - 1) / t.bm;
  p.tiles_n = (p.N + t.bn - 1) / t.bn;
  p.kt_total = std::max(1, (p.K + 63) / 64);
  p.group_m = 4;
  // the most units there can be: every group with rows may end in a part of a
  // tile, and so may the rows past the last group
  const int64_t tiles_m = wgrad ? E * p.tiles_m : R / t.bm + std::min<int64_t>(E + 1, R);
  const int64_t units = tiles_m * p.tiles_n;
  if (units >= (1ll << 31) - (1 << 20)) return DPG_ERR_UNSUPPORTED;
  const int64_t grid = std::min<int64_t>(units, (int64_t)device_cus() * t.per_cu);
  void* args[] = {&p};
  return launch((const void*)lookup_grouped_kernel(tile, layout, out), grid, t.threads, 0, args, stream);
}

}  // namespace
}  // namespace dpg

using namespace dpg;

extern "C" {

dpg_status dpg_grouped_forward(const void* x, int64_t ldx, const void* w, int64_t ldw, int64_t stride_w, void* y,
                               int64_t ldy, dpg_dtype y_dtype, const int32_t* offsets, int64_t E, int64_t R,
                               int64_t N, int64_t K, hipStream_t stream) {
  return run_grouped(LAYOUT_FWD, x, ldx, w, ldw, y, ldy, stride_w, (int)y_dtype, offsets, E, R, N, K, stream);
}

dpg_status dpg_grouped_dgrad(const void* dy, int64_t lddy, const void* w, int64_t ldw, int64_t stride_w, void* dx,
                             int64_t lddx, dpg_dtype dx_dtype, const int32_t* offsets, int64_t E, int64_t R,
                             int64_t N, int64_t K, hipStream_t stream) {
  return run_grouped(LAYOUT_DGRAD, dy, lddy, w, ldw, dx, lddx, stride_w, (int)dx_dtype, offsets, E, R, N, K, stream);
}

dpg_status dpg_grouped_wgrad(const void* dy, int64_t lddy, const void* x, int64_t ldx, void* dw, int64_t lddw,
                             int64_t stride_dw, dpg_dtype dw_dtype, const int32_t* offsets, int64_t E, int64_t R,
                             int64_t N, int64_t K, hipStream_t stream) {
  return run_grouped(LAYOUT_WGRAD, dy, lddy, x, ldx, dw, lddw, stride_dw, (int)dw_dtype, offsets, E, R, N, K,
                     stream);
}

}  // extern "C"

// C ABI of the grouped products (rows sorted by expert, one weight matrix per
// expert): validation and launches.  Conventions are in include/dpg.h, the
// unit stream in grouped_units.h, the kernels in gemm_fast.h.
#include <hip/hip_runtime.h>

#include <stdio.h>

#include <algorithm>
#include <cmath>

#include "api_common.h"
#include "gemm_fast.h"
#include "grouped_skinny.h"

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

// The variants: the large kernel's two tiles, then the few-row kernels (forward:
// 16 rows by 16 columns or 32 by 32, input gradient: 16 by 128).
enum Variant { TILE_256, TILE_128, ROWS_16X16, ROWS_32X32, ROWS_16X128 };
constexpr GroupedTile kGroupedTiles[] = {
    {256, 256, 512, 1}, {128, 128, 256, 2}, {16, 16, 512, 2}, {32, 32, 512, 2}, {16, 128, 512, 2}};

template <int OUT>
GroupedFn lookup_skinny_kernel(int variant) {
  return variant == ROWS_16X16   ? &grouped_rows16_kernel<OUT>
         : variant == ROWS_32X32 ? &grouped_skinny_kernel<false, 2, 2, 3, OUT>
                                 : &grouped_skinny_kernel<true, 1, 8, 1, OUT>;
}

GroupedFn lookup_grouped_kernel(int variant, int layout, int out) {
  if (variant >= ROWS_16X16)
    return out == DPG_F32 ? lookup_skinny_kernel<OUT_F32>(variant) : lookup_skinny_kernel<OUT_BF16>(variant);
  static const GroupedFn table[2][3][2] = {
      {{GroupedRow<256, 256, 2, 4, 0>::fns[0], GroupedRow<256, 256, 2, 4, 0>::fns[1]},
       {GroupedRow<256, 256, 2, 4, 1>::fns[0], GroupedRow<256, 256, 2, 4, 1>::fns[1]},
       {GroupedRow<256, 256, 2, 4, 2>::fns[0], GroupedRow<256, 256, 2, 4, 2>::fns[1]}},
      {{GroupedRow<128, 128, 2, 2, 0>::fns[0], GroupedRow<128, 128, 2, 2, 0>::fns[1]},
       {GroupedRow<128, 128, 2, 2, 1>::fns[0], GroupedRow<128, 128, 2, 2, 1>::fns[1]},
       {GroupedRow<128, 128, 2, 2, 2>::fns[0], GroupedRow<128, 128, 2, 2, 2>::fns[1]}}};
  return table[variant][layout][out];
}

struct GroupedPlan {
  int variant, splits;
};

// The plan with the least estimated time, from the sizes alone (a CU count of
// 256 whatever the device, so that the bits do not depend on it).  The
// estimates are fitted to some 700 timings of 130 sizes on an MI355X (64 to
// 2048 by 128 to 4096, 1 to 256 groups, 1 to 65536 rows, each with every variant
// and several splits).  In us:
//   tiles: a unit takes its steps of 64 (about 1 while few units run; more when
//     they share the chip) and its epilogue; splitting adds a launch and the
//     traffic of its planes.  For example a weight gradient of 30000 rows into
//     512 x 512: 438 in 128-tiles, 40 with 16 splits; a forward of 1024 rows
//     and 8 groups, 1024 x 4096: 66 and 33 with 4.
//   few rows: each CU moves 38 GB/s (forward) or 72 (input gradient) through
//     its unit's fragments, or the memory its weights.  A forward of 8 rows in
//     8 of 256 groups, 512 x 4096: 8.6, in 128-tiles 66; of 256 rows in 64
//     groups, 1024 x 4096: 90, 121 and in 32-row units 107; of 1024 rows 167,
//     126 and 148.
// A weight gradient's longest group is taken to hold 1.3 times the mean.
GroupedPlan grouped_plan(int layout, int64_t E, int64_t R, int64_t N, int64_t K) {
  GroupedPlan best = {TILE_128, 1};
  if (E == 0 || R == 0 || N == 0 || K == 0) return best;
  constexpr double kCus = kDetCus, kStart = 4.6;  // us
  const bool wgrad = layout == LAYOUT_WGRAD;
  const double groups =  // with rows: as many as R random ones reach
      std::max(1.0, (double)E * (1 - std::exp(-(double)R / (double)E)));
  const double cols = (double)(layout == LAYOUT_FWD ? N : K), weights = groups * (double)N * (double)K * 2;
  const double reduced = wgrad ? 1.3 * (double)R / (double)E : (double)(layout == LAYOUT_FWD ? K : N);
  const double outputs = wgrad ? (double)E * (double)N * (double)K : (double)R * cols;
  // row tiles: one a group, or `ends` parts of one more than the rows fill
  const auto row_tiles = [&](double bm, double ends) {
    const double filled = std::ceil((double)R / bm);
    return (double)R / groups > bm / 4 ? std::max(filled, (double)R / bm + ends * groups) : std::max(groups, filled);
  };
  // bytes of weights per us from memory: the tiles, and the few-row kernels
  // while most groups are one unit high
  static constexpr double kTileRate[2][2] = {{4.45e6, 4.6e6}, {4.6e6, 5.7e6}};
  const bool low = (double)R / groups <= 8;
  const double rows_rate[3] = {low ? 6.0e6 : 5.0e6, 5.1e6, low ? 6.1e6 : 5.2e6};
  static constexpr double kStepAlone[3][2] = {{1.0, 0.64}, {1.11, 0.78}, {0.81, 0.67}};
  static constexpr double kStepFull[3][2] = {{1.61, 1.09}, {1.04, 0.97}, {1.65, 1.17}};
  static constexpr double kEpilogue[2] = {5.0, 2.9};
  double least = 0;
  for (int v = TILE_256; v <= TILE_128; ++v) {
    const GroupedTile& t = kGroupedTiles[v];
    const double slots = kCus * t.per_cu;
    const double tiles = wgrad ? (double)E * std::ceil((double)N / t.bm) * std::ceil((double)K / t.bn)
                               : row_tiles(t.bm, 0.5) * std::ceil(cols / t.bn);
    const double steps = std::ceil(reduced / 64);
    for (int s = 1; s <= 16; ++s) {
      if (s > 1 && (s > steps || s * outputs * 4 > (double)(1ll << 30))) break;
      const double rounds = tiles * s / slots, load = std::min(1.0, rounds);
      const double step = kStepAlone[layout][v] + (kStepFull[layout][v] - kStepAlone[layout][v]) * load;
      double us = kStart + (rounds < 3 ? std::max(1.0, std::ceil(rounds)) : rounds + 0.5) *
                               (std::ceil(steps / s) * step + kEpilogue[v]);
      if (!wgrad) us = std::max(us, kStart + weights / kTileRate[layout][v]);
      if (s > 1) us += 1.8 + (s + 1) * outputs * 4 / 4.55e6;
      if (least == 0 || us < least) {
        least = us;
        best = {v, s};
      }
    }
  }
  for (int v = ROWS_16X16; v <= ROWS_16X128 && !wgrad; ++v) {
    if ((v == ROWS_16X128) != (layout == LAYOUT_DGRAD)) continue;
    const GroupedTile& t = kGroupedTiles[v];
    const double tiles = row_tiles(t.bm, v == ROWS_32X32 ? 1.0 : 0.7);
    const double rows = std::min((double)t.bm, std::ceil((double)R / tiles));
    const double bytes = reduced * 2 * (rows + t.bn) + 26e3, rate = layout == LAYOUT_FWD ? 38e3 : 72e3;
    const double us = kStart + std::max(std::max(tiles * std::ceil(cols / t.bn) / kCus, 1.0) * bytes / rate,
                                        weights / rows_rate[v - ROWS_16X16]);
    if (us < least) {
      least = us;
      best = {v, 1};
    }
  }
  return best;
}

size_t grouped_workspace(int layout, const GroupedPlan& plan, int64_t E, int64_t R, int64_t N, int64_t K) {
  if (plan.splits == 1) return 0;
  const int64_t elements = layout == LAYOUT_FWD ? R * N : layout == LAYOUT_DGRAD ? R * K : E * N * K;
  return (size_t)plan.splits * (size_t)elements * sizeof(float);
}

bool within_limits(int64_t E, int64_t R, int64_t N, int64_t K) {
  return std::max(R, std::max(N, K)) < (1ll << 31) - 512 && E < (1ll << 24);
}

// The most units there can be: every group with rows may end in a part of a
// tile, and so may the rows past the last group.
int64_t grouped_units(int layout, const GroupedPlan& plan, int64_t E, int64_t R, int64_t N, int64_t K) {
  const GroupedTile& t = kGroupedTiles[plan.variant];
  const bool wgrad = layout == LAYOUT_WGRAD;
  const int64_t cols = layout == LAYOUT_FWD ? N : K;
  const int64_t tiles_m = wgrad ? E * ((N + t.bm - 1) / t.bm) : R / t.bm + std::min<int64_t>(E + 1, R);
  return tiles_m * ((cols + t.bn - 1) / t.bn) * plan.splits;
}

// The weight gradient's groups by descending size: worth its microsecond where
// a workgroup takes several groups' units.
bool grouped_ordered(int layout, int64_t E, int64_t units, int64_t grid) {
  return layout == LAYOUT_WGRAD && E <= kOrderGroups && E > 1 && units > grid;
}

// One grouped pass.  (a, b) are (x, w), (dy, w) and (dy, x); `stride` is the
// element stride between the groups' weights (weight gradient: outputs).
dpg_status run_grouped(int layout, const void* a, int64_t lda, const void* b, int64_t ldb, void* c, int64_t ldc,
                       int64_t stride, int out, const int32_t* offsets, int64_t E, int64_t R, int64_t N, int64_t K,
                       void* workspace, size_t workspace_bytes, hipStream_t stream) {
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
  if (std::max(lda, ldb) >= (1 << 22) || (mc.rows > 1 && ldc >= (1 << 21))) return DPG_ERR_UNSUPPORTED;
  if (!within_limits(E, R, N, K)) return DPG_ERR_UNSUPPORTED;

  GroupedParams p{};
  p.a = a;
  p.b = b;
  p.c = c;
  p.lda = lda;
  p.ldb = ldb;
  // of one row the stride finds no element, whatever it is; the tiles' 32-bit
  // offsets of the rows past it have to lie past it (256 rows by 2^20 columns
  // by 4 bytes: below 2^31), however many columns there are
  const int64_t one_row = std::min<int64_t>(mc.cols, 1 << 20);
  p.ldc = mc.rows > 1 ? ldc : one_row;
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
  const GroupedPlan plan = grouped_plan(layout, E, R, N, K);
  const GroupedTile& t = kGroupedTiles[plan.variant];
  p.tiles_m = (p.M + t.bm - 1) / t.bm;
  p.tiles_n = (p.N + t.bn - 1) / t.bn;
  p.kt_total = std::max(1, (p.K + 63) / 64);
  p.group_m = 4;
  p.splits = plan.splits;
  const int64_t units = grouped_units(layout, plan, E, R, N, K);
  if (units >= (1ll << 31) - (1 << 20)) return DPG_ERR_UNSUPPORTED;
  const int64_t grid = std::min<int64_t>(units, (int64_t)device_cus() * t.per_cu);
  p.ordered = grouped_ordered(layout, E, units, grid);
  // Outputs in whole 64-byte pieces go past the caches whatever their size; that
  // pays with the kernel that reads them next counted too.  Through the caches /
  // past them, us: up projection, activation and down projection with 4 MB of
  // outputs each 38.1 / 37.7, 16 MB 94.5 / 92.3, 32 and 64 MB 207 / 181, 128 and
  // 512 MB 1210 / 1196; down projection and combination 8 MB 26.1 / 25.4, 128 MB
  // 164 / 160; the worst found, input gradient of 64 MB and combination, 94.4 / 97.0.
  const auto in64 = [](int64_t bytes) { return (bytes & 63) == 0; };
  p.stream = p.splits == 1 && in64((int64_t)(uintptr_t)c) && in64(ldc * out_elt) && (!wgrad || in64(stride * out_elt));
  void* args[] = {&p};
  if (p.splits == 1)
    return launch((const void*)lookup_grouped_kernel(plan.variant, layout, out), grid, t.threads, 0, args, stream);
  // the splits' sums go to planes of the workspace: [splits][R][cols], or
  // [E][splits][N][K] of the weight gradient
  if (!workspace || workspace_bytes < grouped_workspace(layout, plan, E, R, N, K) || !aligned16(workspace))
    return DPG_ERR_WORKSPACE;
  p.c = workspace;
  p.ldc = mc.rows > 1 ? mc.cols : one_row;
  p.split_stride = (int64_t)p.M * p.N;
  p.batch_c = p.split_stride * p.splits;
  st = launch((const void*)lookup_grouped_kernel(plan.variant, layout, DPG_F32), grid, t.threads, 0, args, stream);
  if (st != DPG_OK) return st;
  const float* ws = (const float*)workspace;
  int64_t batch = wgrad ? E : 1;
  const int gx = (p.N / 4 + 255) / 256;
  const int gy = (int)std::max<int64_t>(1, std::min<int64_t>(batch * p.M, std::max(1, 2048 / gx)));
  void* rargs[] = {&ws, &p.splits, &p.split_stride, &p.M, &p.N, &c, &ldc, &batch, &stride};
  const hipError_t e = hipLaunchKernel(out == DPG_F32 ? (const void*)&splitk_reduce_kernel<OUT_F32>
                                                      : (const void*)&splitk_reduce_kernel<OUT_BF16>,
                                       dim3(gx, gy), dim3(256), rargs, 0, stream);
  return e == hipSuccess ? DPG_OK : DPG_ERR_HIP;
}

}  // namespace
}  // namespace dpg

using namespace dpg;

extern "C" {

size_t dpg_grouped_workspace_size(dpg_pass pass, int64_t E, int64_t R, int64_t N, int64_t K) {
  const int layout = (int)pass;
  if (layout < LAYOUT_FWD || layout > LAYOUT_WGRAD || E < 0 || R < 0 || N < 0 || K < 0) return (size_t)-1;
  return grouped_workspace(layout, grouped_plan(layout, E, R, N, K), E, R, N, K);
}

dpg_status dpg_grouped_plan_describe(dpg_pass pass, int64_t E, int64_t R, int64_t N, int64_t K, char* buf,
                                     size_t buflen) {
  static const char* kPass[] = {"forward", "dgrad", "wgrad"};
  const int layout = (int)pass;
  if (!buf || buflen == 0) return DPG_ERR_INVALID_ARG;
  if (layout < LAYOUT_FWD || layout > LAYOUT_WGRAD || E < 0 || R < 0 || N < 0 || K < 0) return DPG_ERR_INVALID_ARG;
  // (so that the units fit 64 bits)
  if (!within_limits(E, R, N, K) || (double)E * (double)N * (double)K >= 0x1p62) return DPG_ERR_UNSUPPORTED;
  const GroupedPlan plan = grouped_plan(layout, E, R, N, K);
  const GroupedTile& t = kGroupedTiles[plan.variant];
  const int64_t units = grouped_units(layout, plan, E, R, N, K);
  const int64_t grid = std::min<int64_t>(units, (int64_t)kDetCus * t.per_cu);
  snprintf(buf, buflen, "pass=%s kind=grouped kernel=%s tile=%dx%d threads=%d splits=%d units=%lld grid=%lld ordered=%d "
           "workspace=%zu", kPass[layout], plan.variant >= ROWS_16X16 ? "few_rows" : "pipelined", t.bm, t.bn, t.threads,
           plan.splits, (long long)units, (long long)grid, (int)grouped_ordered(layout, E, units, grid),
           grouped_workspace(layout, plan, E, R, N, K));
  return DPG_OK;
}

dpg_status dpg_grouped_forward(const void* x, int64_t ldx, const void* w, int64_t ldw, int64_t stride_w, void* y,
                               int64_t ldy, dpg_dtype y_dtype, const int32_t* offsets, int64_t E, int64_t R,
                               int64_t N, int64_t K, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  return run_grouped(LAYOUT_FWD, x, ldx, w, ldw, y, ldy, stride_w, (int)y_dtype, offsets, E, R, N, K, workspace,
                     workspace_bytes, stream);
}

dpg_status dpg_grouped_dgrad(const void* dy, int64_t lddy, const void* w, int64_t ldw, int64_t stride_w, void* dx,
                             int64_t lddx, dpg_dtype dx_dtype, const int32_t* offsets, int64_t E, int64_t R,
                             int64_t N, int64_t K, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  return run_grouped(LAYOUT_DGRAD, dy, lddy, w, ldw, dx, lddx, stride_w, (int)dx_dtype, offsets, E, R, N, K, workspace,
                     workspace_bytes, stream);
}

dpg_status dpg_grouped_wgrad(const void* dy, int64_t lddy, const void* x, int64_t ldx, void* dw, int64_t lddw,
                             int64_t stride_dw, dpg_dtype dw_dtype, const int32_t* offsets, int64_t E, int64_t R,
                             int64_t N, int64_t K, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  return run_grouped(LAYOUT_WGRAD, dy, lddy, x, ldx, dw, lddw, stride_dw, (int)dw_dtype, offsets, E, R, N, K,
                     workspace, workspace_bytes, stream);
}

}  // extern "C"

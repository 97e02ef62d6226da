// C ABI of the routing: validation and launches.  Conventions are in
// include/dpg.h, the kernels in route_kernels.h.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "api_common.h"
#include "route_kernels.h"

namespace dpg {
namespace {

// Tokens of one block of the choice: 64 (four per wave), more where the
// counts of the blocks would pass 512 rows; all of them in one block up to 64.
constexpr int kTokensPerBlock = 64, kMaxBlocks = 512;

struct RouteGrid {
  int tokens_per_block, blocks;
};

RouteGrid route_grid(int64_t T) {
  RouteGrid g;
  g.tokens_per_block = kTokensPerBlock;
  if (T > (int64_t)kTokensPerBlock * kMaxBlocks)
    g.tokens_per_block = (int)((T + kMaxBlocks * kRouteWaves - 1) / (kMaxBlocks * kRouteWaves)) * kRouteWaves;
  g.blocks = (int)((T + g.tokens_per_block - 1) / g.tokens_per_block);
  return g;
}

dpg_status check_route(int64_t T, int64_t E, int64_t top_k) {
  if (T < 0 || E < 1 || top_k < 1 || top_k > E) return DPG_ERR_INVALID_ARG;
  if (E > kRouteMaxExperts || top_k > kRouteMaxTopK || T > ((1ll << 31) - 1) / top_k) return DPG_ERR_UNSUPPORTED;
  return DPG_OK;
}

bool aligned4(const void* p) { return ((uintptr_t)p & 3u) == 0; }

// registers of logits per lane: 64, 128, 256 or 512 experts
int expert_regs(int64_t E) { return E <= 64 ? 0 : E <= 128 ? 1 : E <= 256 ? 2 : 3; }

typedef void (*ChooseFn)(RouteParams);
typedef void (*RouteGradFn)(const float*, int64_t, const int32_t*, const float*, const float*, float*, int64_t,
                            int64_t, int, int, int);
typedef void (*RowsFn)(RowsParams);

// Threads of one token in the row kernels: one for 16 bytes of its row, at
// least 8 (a 128-byte line) and at most 256.
int row_lanes_log2(int64_t chunks) {
  int n = 3;
  while (n < 8 && (1 << n) < chunks) ++n;
  return n;
}

dpg_status check_rows(const void* positions, const void* offsets, int64_t T, int64_t R, int64_t H, int64_t E,
                      int64_t top_k) {
  if (T < 0 || R < 0 || H < 0 || E < 0 || top_k < 1) return DPG_ERR_INVALID_ARG;
  if (T > 0 && top_k > ((1ll << 31) - 1) / T) return DPG_ERR_UNSUPPORTED;
  if (R >= (1ll << 31) || H > (1 << 24) || E > (1 << 24) || T >= (1ll << 31)) return DPG_ERR_UNSUPPORTED;
  if (T > 0 && (!positions || !offsets)) return DPG_ERR_INVALID_ARG;
  if (!aligned4(positions) || !aligned4(offsets)) return DPG_ERR_ALIGNMENT;
  return DPG_OK;
}

int elt_size(int dtype) { return dtype == DPG_F32 ? 4 : 2; }
bool row_dtype(int dtype) { return dtype == DPG_BF16 || dtype == DPG_F32; }

}  // namespace
}  // namespace dpg

using namespace dpg;

extern "C" {

size_t dpg_route_workspace_size(int64_t T, int64_t E, int64_t top_k) {
  if (check_route(T, E, top_k) != DPG_OK) return (size_t)-1;
  const RouteGrid g = route_grid(T);
  return g.blocks > 1 ? (size_t)g.blocks * (size_t)(E + 1) * sizeof(int32_t) : 0;
}

dpg_status dpg_route(const float* logits, int64_t ldl, int64_t T, int64_t E, int64_t top_k, int renormalize,
                     int32_t* experts, float* weights, int32_t* offsets, int32_t* rows, int32_t* positions,
                     void* workspace, size_t workspace_bytes, hipStream_t stream) {
  dpg_status st = check_route(T, E, top_k);
  if (st != DPG_OK) return st;
  if (!offsets) return DPG_ERR_INVALID_ARG;
  if (T > 0 && (!logits || ldl < E || !experts || !weights || !rows || !positions)) return DPG_ERR_INVALID_ARG;
  if (!aligned4(logits) || !aligned4(experts) || !aligned4(weights) || !aligned4(offsets) || !aligned4(rows) ||
      !aligned4(positions))
    return DPG_ERR_ALIGNMENT;
  const RouteGrid g = route_grid(T);
  const size_t need = dpg_route_workspace_size(T, E, top_k);
  if (need > 0 && (!workspace || workspace_bytes < need || !aligned4(workspace))) return DPG_ERR_WORKSPACE;

  RouteParams p{};
  p.logits = logits;
  p.ldl = ldl;
  p.T = T;
  p.E = (int)E;
  p.k = (int)top_k;
  p.renorm = renormalize != 0;
  p.tokens_per_block = g.tokens_per_block;
  p.blocks = g.blocks;
  p.experts = experts;
  p.weights = weights;
  p.offsets = offsets;
  p.rows = rows;
  p.positions = positions;
  p.hist = (int32_t*)workspace;
  static const ChooseFn choose_one[4] = {&route_choose_kernel<1, true>, &route_choose_kernel<2, true>,
                                         &route_choose_kernel<4, true>, &route_choose_kernel<8, true>};
  static const ChooseFn choose_many[4] = {&route_choose_kernel<1, false>, &route_choose_kernel<2, false>,
                                          &route_choose_kernel<4, false>, &route_choose_kernel<8, false>};
  const int keys = p.E + 1;
  void* args[] = {&p};
  if (g.blocks <= 1)  // T = 0 too: the offsets become zeros
    return launch((const void*)choose_one[expert_regs(E)], 1, kRouteThreads,
                  (size_t)(2 + kRouteWaves) * keys * sizeof(int), args, stream);
  st = launch((const void*)choose_many[expert_regs(E)], g.blocks, kRouteThreads, keys * sizeof(int), args, stream);
  if (st != DPG_OK) return st;
  return launch((const void*)&route_order_kernel, g.blocks, kRouteThreads,
                (size_t)(3 + kRouteWaves) * keys * sizeof(int), args, stream);
}

dpg_status dpg_route_dgrad(const float* logits, int64_t ldl, const int32_t* experts, const float* weights,
                           const float* dweights, float* dlogits, int64_t lddl, int64_t T, int64_t E, int64_t top_k,
                           int renormalize, hipStream_t stream) {
  const dpg_status st = check_route(T, E, top_k);
  if (st != DPG_OK) return st;
  if (T == 0) return DPG_OK;
  if (!logits || !experts || !weights || !dweights || !dlogits || ldl < E || lddl < E) return DPG_ERR_INVALID_ARG;
  if (!aligned4(logits) || !aligned4(experts) || !aligned4(weights) || !aligned4(dweights) || !aligned4(dlogits))
    return DPG_ERR_ALIGNMENT;
  static const RouteGradFn fns[4] = {&route_dgrad_kernel<1>, &route_dgrad_kernel<2>, &route_dgrad_kernel<4>,
                                     &route_dgrad_kernel<8>};
  int e = (int)E, k = (int)top_k, renorm = renormalize != 0;
  void* args[] = {&logits, &ldl, &experts, &weights, &dweights, &dlogits, &lddl, &T, &e, &k, &renorm};
  return launch((const void*)fns[expert_regs(E)], (T + 3) / 4, 256, 0, args, stream);
}

dpg_status dpg_dispatch(const void* x, int64_t ldx, const int32_t* positions, const int32_t* offsets, void* xs,
                        int64_t ldxs, dpg_dtype dtype, int64_t T, int64_t R, int64_t H, int64_t E, int64_t top_k,
                        hipStream_t stream) {
  if (!row_dtype((int)dtype)) return DPG_ERR_INVALID_ARG;
  dpg_status st = check_rows(positions, offsets, T, R, H, E, top_k);
  if (st != DPG_OK) return st;
  const int elt = elt_size((int)dtype);
  if ((st = check_mat(Mat{x, ldx, T, H, elt})) != DPG_OK) return st;
  if ((st = check_mat(Mat{xs, ldxs, R, H, elt})) != DPG_OK) return st;
  if (T == 0 || R == 0 || H == 0) return DPG_OK;
  RowsParams p{};
  p.a = x;
  p.out = xs;
  p.positions = positions;
  p.routed = offsets + E;
  p.lda = ldx;
  p.ldo = ldxs;
  p.T = T;
  p.R = R;
  p.H = (int)H;
  p.k = (int)top_k;
  p.lanes_log2 = row_lanes_log2(H * elt / 16);
  void* args[] = {&p};
  const RowsFn fn = elt == 2 ? &dispatch_kernel<2> : &dispatch_kernel<4>;
  return launch((const void*)fn, ((T << p.lanes_log2) + 255) / 256, 256, 0, args, stream);
}

dpg_status dpg_combine(const void* ys, int64_t ldys, dpg_dtype ys_dtype, const int32_t* positions,
                       const int32_t* offsets, const float* weights, void* y, int64_t ldy, dpg_dtype y_dtype,
                       int64_t T, int64_t R, int64_t H, int64_t E, int64_t top_k, hipStream_t stream) {
  if (!row_dtype((int)ys_dtype) || !row_dtype((int)y_dtype)) return DPG_ERR_INVALID_ARG;
  dpg_status st = check_rows(positions, offsets, T, R, H, E, top_k);
  if (st != DPG_OK) return st;
  if ((st = check_mat(Mat{ys, ldys, R, H, elt_size((int)ys_dtype)})) != DPG_OK) return st;
  if ((st = check_mat(Mat{y, ldy, T, H, elt_size((int)y_dtype)})) != DPG_OK) return st;
  if (!aligned4(weights)) return DPG_ERR_ALIGNMENT;
  if (T == 0 || H == 0) return DPG_OK;
  RowsParams p{};
  p.b = ys;
  p.out = y;
  p.positions = positions;
  p.routed = offsets + E;
  p.weights = weights;
  p.ldb = ldys;
  p.ldo = ldy;
  p.T = T;
  p.R = R;
  p.H = (int)H;
  p.k = (int)top_k;
  p.lanes_log2 = row_lanes_log2(H / 8);
  void* args[] = {&p};
  const bool in4 = ys_dtype == DPG_F32, out4 = y_dtype == DPG_F32;
  const RowsFn fn = in4 ? (out4 ? &combine_kernel<4, 4> : &combine_kernel<4, 2>)
                        : (out4 ? &combine_kernel<2, 4> : &combine_kernel<2, 2>);
  return launch((const void*)fn, ((T << p.lanes_log2) + 255) / 256, 256, 0, args, stream);
}

dpg_status dpg_combine_dgrad(const void* dy, int64_t lddy, const void* ys, int64_t ldys, const int32_t* positions,
                             const int32_t* offsets, const float* weights, void* dys, int64_t lddys, float* dweights,
                             dpg_dtype dtype, int64_t T, int64_t R, int64_t H, int64_t E, int64_t top_k,
                             hipStream_t stream) {
  if (!row_dtype((int)dtype)) return DPG_ERR_INVALID_ARG;
  dpg_status st = check_rows(positions, offsets, T, R, H, E, top_k);
  if (st != DPG_OK) return st;
  const int elt = elt_size((int)dtype);
  if ((st = check_mat(Mat{dy, lddy, T, H, elt})) != DPG_OK) return st;
  if ((st = check_mat(Mat{ys, ldys, R, H, elt})) != DPG_OK) return st;
  if ((st = check_mat(Mat{dys, lddys, R, H, elt})) != DPG_OK) return st;
  if (T == 0) return DPG_OK;
  if (!weights || !dweights) return DPG_ERR_INVALID_ARG;
  if (!aligned4(weights) || !aligned4(dweights)) return DPG_ERR_ALIGNMENT;
  RowsParams p{};
  p.a = dy;
  p.b = ys;
  p.out = dys;
  p.dweights = dweights;
  p.positions = positions;
  p.routed = offsets + E;
  p.weights = weights;
  p.lda = lddy;
  p.ldb = ldys;
  p.ldo = lddys;
  p.T = T;
  p.R = R;
  p.H = (int)H;
  p.k = (int)top_k;
  void* args[] = {&p};
  const RowsFn fn = elt == 2 ? &combine_dgrad_kernel<2> : &combine_dgrad_kernel<4>;
  return launch((const void*)fn, (T + 3) / 4, 256, 0, args, stream);
}

}  // extern "C"

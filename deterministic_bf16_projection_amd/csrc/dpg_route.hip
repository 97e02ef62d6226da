// C ABI of the routing: validation and launches.  Conventions are in
// include/dpg.h, the kernels in route_kernels.h.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "api_common.h"
#include "route_kernels.h"

namespace dpg {
namespace {

// Tokens of one block of the choice: 64, one round of its waves, more where
// there would be over 512 blocks.  Up to 64 tokens are one block.
constexpr int kMaxBlocks = 512;
// a block's counts are kept in 16 bits
constexpr int64_t kMaxTokens = (int64_t)kMaxBlocks * (65535 / kRouteRound) * kRouteRound;

// Up to kWideTokens, blocks of 16 tokens, one wave a token: with dispatch and
// combination, 419 tokens of 403 experts 30.7 -> 25.6 us, 1000 of 256 30.0 ->
// 26.6, 201 of 64 level.
constexpr int64_t kWideTokens = 1024;

struct RouteGrid {
  int tokens_per_block, blocks;
  int hist_ld() const { return (blocks + 7) & ~7; }  // rows of 16 bytes
};

RouteGrid route_grid(int64_t T) {
  RouteGrid g;
  const int64_t per_round = (int64_t)kMaxBlocks * kRouteRound;
  g.tokens_per_block = (int)(std::max<int64_t>(1, (T + per_round - 1) / per_round) * kRouteRound);
  if (T > kRouteRound && T <= kWideTokens) g.tokens_per_block = 16;
  g.blocks = (int)((T + g.tokens_per_block - 1) / g.tokens_per_block);
  return g;
}

dpg_status check_route(int64_t T, int64_t E, int64_t top_k) {
  if (T < 0 || E < 1 || top_k < 1 || top_k > E) return DPG_ERR_INVALID_ARG;
  if (E > kRouteMaxExperts || top_k > kRouteMaxTopK || T > ((1ll << 31) - 1) / top_k || T > kMaxTokens)
    return DPG_ERR_UNSUPPORTED;
  return DPG_OK;
}

bool aligned4(const void* p) { return ((uintptr_t)p & 3u) == 0; }

// registers of logits per lane of 16 (choice) or 64 (gradient): 64, 128, 256 or 512 experts
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

// Workgroups for n tokens or slots, `each` of them to one: a launch takes fewer
// than 2^32 threads, so the kernels go round beyond 2^22 workgroups.
int64_t row_grid(int64_t n, int64_t each) { return std::min<int64_t>((n + each - 1) / each, 1 << 22); }

// Sorted rows that do not fit the XCDs' 32 MB of L2 go past it, which leaves
// it to the token side: routing of 16384 tokens, 8 slots of 4096 columns, forward
// and backward, 1247 us without and 1174 with.  Smaller ones stay for the
// product that reads them next, and so do rows that are no multiples of 64
// bytes, whose lines would be moved in pieces.
bool stream_rows(const void* rows, int64_t ld, int64_t R, int64_t H, int elt) {
  return R * H >= (int64_t)(32 << 20) / elt && (((uintptr_t)rows | (uint64_t)(ld * elt) | (uint64_t)(H * elt)) & 63) == 0;
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
  return g.blocks > 1 ? (size_t)g.hist_ld() * (size_t)E * sizeof(uint16_t) : 0;
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
  if (need > 0 && (!workspace || workspace_bytes < need || !aligned16(workspace))) return DPG_ERR_WORKSPACE;

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
  p.hist_ld = g.hist_ld();
  p.hist = (uint16_t*)workspace;
  // one wave a token up to 16 tokens, rows of 16 lanes beyond
  static const ChooseFn wide[4] = {&route_choose_kernel<64, 1, true>, &route_choose_kernel<64, 2, true>,
                                   &route_choose_kernel<64, 4, true>, &route_choose_kernel<64, 8, true>};
  static const ChooseFn one[4] = {&route_choose_kernel<16, 4, true>, &route_choose_kernel<16, 8, true>,
                                  &route_choose_kernel<16, 16, true>, &route_choose_kernel<16, 32, true>};
  static const ChooseFn many[4] = {&route_choose_kernel<16, 4, false>, &route_choose_kernel<16, 8, false>,
                                   &route_choose_kernel<16, 16, false>, &route_choose_kernel<16, 32, false>};
  const int keys = p.E + 1;
  void* args[] = {&p};
  if (g.blocks <= 1) {  // T = 0 too: the offsets become zeros
    const int threads = T <= 4 ? 256 : kRouteThreads;
    return launch((const void*)(T <= 16 ? wide : one)[expert_regs(E)], 1, threads,
                  (size_t)((2 + threads / 64) * keys + T * top_k) * sizeof(int), args, stream);
  }
  static const ChooseFn many_wide[4] = {&route_choose_kernel<64, 1, false>, &route_choose_kernel<64, 2, false>,
                                        &route_choose_kernel<64, 4, false>, &route_choose_kernel<64, 8, false>};
  st = launch((const void*)(T <= kWideTokens ? many_wide : many)[expert_regs(E)], g.blocks, kRouteThreads, keys * sizeof(int), args, stream);
  if (st != DPG_OK) return st;
  return launch((const void*)&route_order_kernel, g.blocks, kRouteThreads,
                (size_t)(3 + kRouteThreads / 64) * keys * sizeof(int), args, stream);
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
  return launch((const void*)fns[expert_regs(E)], row_grid(T, 4), 256, 0, args, stream);
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
  const bool past = stream_rows(xs, ldxs, R, H, elt);
  const RowsFn fn = elt == 2 ? (past ? &dispatch_kernel<2, true> : &dispatch_kernel<2, false>)
                             : (past ? &dispatch_kernel<4, true> : &dispatch_kernel<4, false>);
  // rows past the slots' share the tokens' threads: top_k of them to a token
  return launch((const void*)fn, row_grid(std::max(T, (R + top_k - 1) / top_k), 256 >> p.lanes_log2), 256, 0, args,
                stream);
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
  static const RowsFn fns[2][2][2] = {
      {{&combine_kernel<2, 2, false>, &combine_kernel<2, 2, true>},
       {&combine_kernel<2, 4, false>, &combine_kernel<2, 4, true>}},
      {{&combine_kernel<4, 2, false>, &combine_kernel<4, 2, true>},
       {&combine_kernel<4, 4, false>, &combine_kernel<4, 4, true>}}};
  const RowsFn fn = fns[ys_dtype == DPG_F32][y_dtype == DPG_F32][stream_rows(ys, ldys, R, H, elt_size((int)ys_dtype))];
  return launch((const void*)fn, row_grid(T, 256 >> p.lanes_log2), 256, 0, args, stream);
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
  const bool past = stream_rows(ys, ldys, R, H, elt) && stream_rows(dys, lddys, R, H, elt);
  const RowsFn fn = elt == 2 ? (past ? &combine_dgrad_kernel<2, true> : &combine_dgrad_kernel<2, false>)
                             : (past ? &combine_dgrad_kernel<4, true> : &combine_dgrad_kernel<4, false>);
  return launch((const void*)fn, row_grid(std::max(T * top_k, R), 4), 256, 0, args, stream);
}

}  // extern "C"

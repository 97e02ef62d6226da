// C ABI of the gated recurrence: validation, the cut into axes and spans, and
// launches.  Conventions are in include/dpg.h, the kernels in
// recurrence_kernels.h.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "api_common.h"
#include "recurrence_kernels.h"

namespace dpg {
namespace {

constexpr int64_t kRecMaxRows = 1 << 30;  // places behind the last row are counted in 32 bits too
constexpr int64_t kRecMaxOther = 1 << 24;  // sequences, channels
// Workgroups that fill the device: one to each of 256 CUs.
constexpr int64_t kRecFull = 256;

bool row_type(int dtype) { return dtype == DPG_BF16 || dtype == DPG_F32; }
Rows8 rows8(const void* data, int64_t ld) { return Rows8{const_cast<void*>(data), ld}; }
size_t padded(size_t bytes) { return (bytes + 15) & ~(size_t)15; }

// Matrices that do not fit the XCDs' 32 MB of L2 go past it: copies in the order
// of a training batch's forward pass take 148 to 157 us through it, 146 past it.
bool past_caches(int64_t R, int64_t D, int elt) { return R * D >= (int64_t)(32 << 20) / elt; }

struct RecPlan {
  int64_t length;                 // of a sequence, 0 where they are packed
  int64_t axis_rows, axes, tiles, spans, span_tiles, blocks;
  size_t seq_bytes, summary_bytes, copy_bytes, carry_bytes;
  size_t workspace() const { return seq_bytes + summary_bytes + copy_bytes; }
};

// S sequences in R rows of D channels; R > 0.
dpg_status rec_plan(int64_t S, int64_t R, int64_t D, bool packed, RecPlan& g) {
  const int64_t tile = kRecTileRows;
  g = RecPlan{};
  if (packed) {
    g.axis_rows = R;
    g.axes = 1;
  } else {
    g.length = R / S;
    g.axis_rows = g.length * std::max<int64_t>(1, tile / g.length);
    g.axes = (R + g.axis_rows - 1) / g.axis_rows;
  }
  g.tiles = (g.axis_rows + tile - 1) / tile;
  g.blocks = (D + kRecChannels - 1) / kRecChannels;
  const int64_t have = g.axes * g.blocks;
  g.spans = 1;
  // One sequence of 512 rows, 4096 channels (32 workgroups): whole 16.4 us, in
  // spans of one tile 12.8.  From 129 workgroups on, spans would double the
  // passes over the inputs to gain less than a second workgroup a CU.  At the border,
  // 4096 rows, BF16, us forward and gradient: 128 workgroups, in two spans 111 and 155,
  // whole 122 and 223; 144 workgroups, 154 and 261, whole 127 and 231.  A workgroup
  // goes through the spans before its own one by one: 32768 rows of 128 channels, 256
  // spans, 78 us (whole: 840).
  if (have * 2 <= kRecFull && g.tiles > 2)
    g.spans = std::min(kRecFull / have, g.tiles);
  g.span_tiles = (g.tiles + g.spans - 1) / g.spans;
  g.spans = (g.tiles + g.span_tiles - 1) / g.span_tiles;
  if (g.axes * g.spans * g.blocks >= (1ll << 22)) return DPG_ERR_UNSUPPORTED;
  g.seq_bytes = packed ? padded((size_t)R * sizeof(int32_t)) : 0;
  if (g.spans > 1) {
    g.summary_bytes = padded((size_t)(g.axes * g.spans * 2 * D) * sizeof(float));
    g.copy_bytes = padded((size_t)(S * D) * sizeof(float));
  }
  g.carry_bytes = (size_t)(g.axes * 2 * g.tiles * D) * sizeof(float);
  return DPG_OK;
}

dpg_status check_sizes(int64_t S, int64_t R, int64_t D, int dtype, bool packed) {
  if (S < 0 || R < 0 || D < 0 || !row_type(dtype)) return DPG_ERR_INVALID_ARG;
  if (!packed && (S == 0 ? R != 0 : R % S != 0)) return DPG_ERR_INVALID_ARG;
  if (R > kRecMaxRows || S > kRecMaxOther || D > kRecMaxOther) return DPG_ERR_UNSUPPORTED;
  return DPG_OK;
}

// FP32 [S, D] or null
dpg_status check_states(const void* a, const void* b) {
  return aligned16(a) && aligned16(b) ? DPG_OK : DPG_ERR_ALIGNMENT;
}

const void* forward_fn(bool bf16, bool coupled, bool nt) {
  static const void* const fns[2][2][2] = {
      {{(const void*)&recurrence_kernel<false, false, false>, (const void*)&recurrence_kernel<false, false, true>},
       {(const void*)&recurrence_kernel<false, true, false>, (const void*)&recurrence_kernel<false, true, true>}},
      {{(const void*)&recurrence_kernel<true, false, false>, (const void*)&recurrence_kernel<true, false, true>},
       {(const void*)&recurrence_kernel<true, true, false>, (const void*)&recurrence_kernel<true, true, true>}}};
  return fns[bf16][coupled][nt];
}
const void* forward_span_fn(bool bf16, bool coupled) {
  return bf16 ? (coupled ? (const void*)&recurrence_span_kernel<true, true> : (const void*)&recurrence_span_kernel<true, false>)
              : (coupled ? (const void*)&recurrence_span_kernel<false, true> : (const void*)&recurrence_span_kernel<false, false>);
}
const void* step_fn(bool bf16, bool coupled) {
  return bf16 ? (coupled ? (const void*)&recurrence_step_kernel<true, true> : (const void*)&recurrence_step_kernel<true, false>)
              : (coupled ? (const void*)&recurrence_step_kernel<false, true> : (const void*)&recurrence_step_kernel<false, false>);
}
const void* dgrad_fn(bool bf16, bool coupled, bool nt) {
  static const void* const fns[2][2][2] = {
      {{(const void*)&recurrence_dgrad_kernel<false, false, false>, (const void*)&recurrence_dgrad_kernel<false, false, true>},
       {(const void*)&recurrence_dgrad_kernel<false, true, false>, (const void*)&recurrence_dgrad_kernel<false, true, true>}},
      {{(const void*)&recurrence_dgrad_kernel<true, false, false>, (const void*)&recurrence_dgrad_kernel<true, false, true>},
       {(const void*)&recurrence_dgrad_kernel<true, true, false>, (const void*)&recurrence_dgrad_kernel<true, true, true>}}};
  return fns[bf16][coupled][nt];
}
const void* dgrad_span_fn(bool bf16) {
  return bf16 ? (const void*)&recurrence_dgrad_span_kernel<true> : (const void*)&recurrence_dgrad_span_kernel<false>;
}

// Rows' sequences, and what passes through sequences without rows.
dpg_status run_rows(const int32_t* offsets, int64_t S, int64_t R, int32_t* seq, const float* from, float* to, int64_t D,
                    hipStream_t stream) {
  int row_blocks = seq ? (int)((R + 255) / 256) : 0, s = (int)S, r = (int)R, d = (int)D;
  const int64_t grid = row_blocks + (to ? std::min<int64_t>(S, 4096) : 0);
  if (grid == 0) return DPG_OK;
  void* args[] = {&offsets, &s, &r, &row_blocks, &seq, &from, &to, &d};
  return launch((const void*)&recurrence_rows_kernel, grid, 256, 0, args, stream);
}

void fill(RecParams& p, const RecPlan& g, int64_t R, int64_t D, void* workspace) {
  char* ws = (char*)workspace;
  p.seq = g.seq_bytes ? (int32_t*)ws : nullptr;
  p.summary = g.summary_bytes ? (float*)(ws + g.seq_bytes) : nullptr;
  p.R = (int)R;
  p.D = (int)D;
  p.length = (int)g.length;
  p.axis_rows = (int)g.axis_rows;
  p.tiles = (int)g.tiles;
  p.span_tiles = (int)g.span_tiles;
  p.spans = (int)g.spans;
  p.blocks = (int)g.blocks;
}

}  // namespace
}  // namespace dpg

using namespace dpg;

extern "C" {

size_t dpg_recurrence_workspace_size(int64_t S, int64_t R, int64_t D, dpg_dtype dtype, int packed) {
  if (check_sizes(S, R, D, (int)dtype, packed != 0) != DPG_OK) return (size_t)-1;
  if (R == 0 || D == 0) return 0;
  RecPlan g;
  return rec_plan(S, R, D, packed != 0, g) == DPG_OK ? g.workspace() : (size_t)-1;
}

size_t dpg_recurrence_carries_size(int64_t S, int64_t R, int64_t D, dpg_dtype dtype, int packed) {
  if (check_sizes(S, R, D, (int)dtype, packed != 0) != DPG_OK) return (size_t)-1;
  if (R == 0 || D == 0) return 0;
  RecPlan g;
  return rec_plan(S, R, D, packed != 0, g) == DPG_OK ? g.carry_bytes : (size_t)-1;
}

dpg_status dpg_recurrence(const void* gate, int64_t ldg, const void* x, int64_t ldx, void* h, int64_t ldh,
                          dpg_dtype dtype, const float* state, float* state_out, float* carries,
                          const int32_t* offsets, int64_t S, int64_t R, int64_t D, int coupled, void* workspace,
                          size_t workspace_bytes, hipStream_t stream) {
  const bool packed = offsets != nullptr, bf16 = dtype == DPG_BF16;
  dpg_status st = check_sizes(S, R, D, (int)dtype, packed);
  if (st != DPG_OK) return st;
  const int elt = bf16 ? 2 : 4;
  if ((st = check_mat(Mat{gate, ldg, R, D, elt})) != DPG_OK) return st;
  if ((st = check_mat(Mat{x, ldx, R, D, elt})) != DPG_OK) return st;
  if ((st = check_mat(Mat{h, ldh, R, D, elt})) != DPG_OK) return st;
  if ((st = check_states(state, state_out)) != DPG_OK) return st;
  if (!aligned16(carries) || ((uintptr_t)offsets & 3u) != 0 || D % 8 != 0) return DPG_ERR_ALIGNMENT;
  if (D == 0) return DPG_OK;
  if (R == 0) return state_out == state ? DPG_OK : run_rows(nullptr, S, 0, nullptr, state, state_out, D, stream);
  RecPlan g;
  if ((st = rec_plan(S, R, D, packed, g)) != DPG_OK) return st;
  if (g.workspace() > 0 && (!workspace || workspace_bytes < g.workspace() || !aligned16(workspace)))
    return DPG_ERR_WORKSPACE;
  RecParams p{};
  fill(p, g, R, D, workspace);
  p.gate = rows8(gate, ldg);
  p.x = rows8(x, ldx);
  p.h = rows8(h, ldh);
  p.state = state;
  p.state_out = state_out;
  p.carries = carries;
  if (packed && (st = run_rows(offsets, S, R, const_cast<int32_t*>(p.seq), state, state_out == state ? nullptr : state_out,
                               D, stream)) != DPG_OK)
    return st;
  void* args[] = {&p};
  // Sequences of one row: 32 of them, 4096 channels, 7.9 us by tiles, 6.3
  // row by row (both mostly the call).  The gradient finds the states itself where every row is a first
  // one, so that the carries need no values.
  if (!packed && S == R)
    return launch(step_fn(bf16, coupled != 0), std::min<int64_t>((R * (D / 8) + 255) / 256, 1 << 16), 256, 0, args, stream);
  if (g.spans > 1) {
    if (state && state == state_out) {
      // a sequence's last span may write its state before the first has read it
      const f32x4* from = (const f32x4*)state;
      f32x4* to = (f32x4*)((char*)workspace + g.seq_bytes + g.summary_bytes);
      int64_t n = S * D / 4;
      void* copy_args[] = {&from, &to, &n};
      st = launch((const void*)&recurrence_copy_kernel, std::min<int64_t>((n + 255) / 256, 2048), 256, 0, copy_args, stream);
      if (st != DPG_OK) return st;
      p.state = (const float*)to;
    }
    st = launch(forward_span_fn(bf16, coupled != 0), g.axes * g.spans * g.blocks, kRecThreads, 0, args, stream);
    if (st != DPG_OK) return st;
  }
  return launch(forward_fn(bf16, coupled != 0, past_caches(R, D, elt)), g.axes * g.spans * g.blocks, kRecThreads, 0, args, stream);
}

dpg_status dpg_recurrence_dgrad(const void* dh, int64_t lddh, const void* gate, int64_t ldg, const void* x, int64_t ldx,
                                const float* carries, const float* state, const float* dstate, void* dgate,
                                int64_t lddg, void* dx, int64_t lddx, float* dstate_out, dpg_dtype dtype,
                                const int32_t* offsets, int64_t S, int64_t R, int64_t D, int coupled, void* workspace,
                                size_t workspace_bytes, hipStream_t stream) {
  const bool packed = offsets != nullptr, bf16 = dtype == DPG_BF16;
  dpg_status st = check_sizes(S, R, D, (int)dtype, packed);
  if (st != DPG_OK) return st;
  const int elt = bf16 ? 2 : 4;
  if ((st = check_mat(Mat{dh, lddh, R, D, elt})) != DPG_OK) return st;
  if ((st = check_mat(Mat{gate, ldg, R, D, elt})) != DPG_OK) return st;
  if ((st = check_mat(Mat{x, ldx, R, D, elt})) != DPG_OK) return st;
  if ((st = check_mat(Mat{dgate, lddg, R, D, elt})) != DPG_OK) return st;
  if ((st = check_mat(Mat{dx, lddx, R, D, elt})) != DPG_OK) return st;
  if ((st = check_states(state, dstate)) != DPG_OK) return st;
  if (!aligned16(carries) || !aligned16(dstate_out) || ((uintptr_t)offsets & 3u) != 0 || D % 8 != 0)
    return DPG_ERR_ALIGNMENT;
  if (dstate_out && dstate_out == dstate) return DPG_ERR_INVALID_ARG;
  if (D == 0) return DPG_OK;
  if (R == 0) return run_rows(nullptr, S, 0, nullptr, dstate, dstate_out, D, stream);
  if (!carries) return DPG_ERR_INVALID_ARG;
  RecPlan g;
  if ((st = rec_plan(S, R, D, packed, g)) != DPG_OK) return st;
  if (g.workspace() > 0 && (!workspace || workspace_bytes < g.workspace() || !aligned16(workspace)))
    return DPG_ERR_WORKSPACE;
  RecParams p{};
  fill(p, g, R, D, workspace);
  p.dh = rows8(dh, lddh);
  p.gate = rows8(gate, ldg);
  p.x = rows8(x, ldx);
  p.dgate = rows8(dgate, lddg);
  p.dx = rows8(dx, lddx);
  p.carries = const_cast<float*>(carries);
  p.state = state;
  p.dstate = dstate;
  p.dstate_out = dstate_out;
  if (packed && (st = run_rows(offsets, S, R, const_cast<int32_t*>(p.seq), dstate, dstate_out, D, stream)) != DPG_OK)
    return st;
  void* args[] = {&p};
  if (g.spans > 1) {
    st = launch(dgrad_span_fn(bf16), g.axes * g.spans * g.blocks, kRecThreads, 0, args, stream);
    if (st != DPG_OK) return st;
  }
  return launch(dgrad_fn(bf16, coupled != 0, past_caches(R, D, elt)), g.axes * g.spans * g.blocks, kRecGradThreads,
                0, args, stream);
}

}  // extern "C"

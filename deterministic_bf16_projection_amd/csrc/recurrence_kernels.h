// A gated linear recurrence over the rows of sequences, and its gradient.  Per
// channel, with f = 1 / (1 + e^-gate) and w = 1 - f (coupled) or 1:
//   h_t = f_t h_(t-1) + w_t x_t
//   r_t = dh_t + q_(t+1),  q_t = f_t r_t        (q after the last row: dstate)
//   dx_t = w_t r_t         dgate_t = f_t (1 - f_t) r_t (h_(t-1) - x_t, or h_(t-1))
// A weight that is exactly zero leaves its term out, whatever the term is: a
// gate of -infinity forgets any state, and one of +infinity (coupled) passes
// over any input.
//
// Composition.  A run of rows maps the state before it to c -> A c + H, A the
// product of its f and H its result from zero; two runs compose to (A1 A2, A2
// H1 + H2).  A workgroup owns 64 channels and goes through its rows by tiles:
// sixteen lanes hold 64 channels of a run of U rows, sixteen runs make a tile.
// Each run's (A, H) meets the others' in LDS, every lane finds the state
// before its run, and then each row's, from values that stayed in registers:
// the rows are read once.  A is zero only if some f is: products that
// underflow are held at the smallest number, so that an infinite state stays
// infinite.
//
// Rows are grouped in axes, each a whole sequence or several short ones; a
// sequence's first row takes f = 0 there and the initial state into its input.
// Where there are too few axes and channels to fill the device, an axis is cut
// into spans: a first launch finds each span's (A, H), and the second starts a
// span from the composition of those before it, for 5 passes over memory
// instead of 3.  All of it depends on sizes alone, and every sum runs in a
// fixed order.
//
// The forward pass can keep the FP32 state before each tile (1/64 of h's size
// in BF16); the gradient recomputes the states in between from them, exactly
// as they were, instead of reading rounded ones.
#pragma once
#include <type_traits>

#include "rows8.h"

namespace dpg {

constexpr int kRecChannels = 64;
constexpr int kRecRuns = 16;   // of a tile
__host__ __device__ constexpr int rec_run_rows(bool bf16) { return bf16 ? 8 : 4; }
__host__ __device__ constexpr int rec_tile_rows(bool bf16) { return kRecRuns * rec_run_rows(bf16); }

struct RecParams {
  Rows8 gate, x, h, dh, dgate, dx;
  const float* state;      // [S, D] before the first rows, or null: zeros
  float* state_out;        // [S, D] after the last rows, or null
  const float* dstate;     // [S, D] gradient of the latter, or null: zeros
  float* dstate_out;       // [S, D] gradient of the former, or null
  float* carries;          // [axes * tiles, D]
  float* summary;          // [axes * spans, 2, D]: A, then H or Q
  const int32_t* seq;      // packed: each row's sequence, -1 behind the last
  int R, D, length;        // length: of every sequence, where they are not packed
  int axis_rows, tiles;    // of an axis
  int span_tiles, spans;
  int blocks;              // of 64 channels
};

// ----------------------------------------------------------- four values --
template <bool BF16>
using Raw4 = std::conditional_t<BF16, u32x2, f32x4>;

template <bool BF16>
__device__ __forceinline__ Raw4<BF16> load4(const Rows8& m, int64_t row, int channel) {
  if constexpr (BF16)
    return *(const u32x2*)((const unsigned short*)m.data + row * m.ld + channel);
  else
    return *(const f32x4*)((const float*)m.data + row * m.ld + channel);
}
__device__ __forceinline__ f32x4 unpack4(const u32x2& r) {
  return f32x4{bf16_value(r[0] & 0xffffu), __builtin_bit_cast(float, r[0] & 0xffff0000u), bf16_value(r[1] & 0xffffu),
               __builtin_bit_cast(float, r[1] & 0xffff0000u)};
}
__device__ __forceinline__ f32x4 unpack4(const f32x4& r) { return r; }
template <bool BF16>
__device__ __forceinline__ void store4(const Rows8& m, int64_t row, int channel, const f32x4& v) {
  if constexpr (BF16)
    *(u32x2*)((unsigned short*)m.data + row * m.ld + channel) = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
  else
    *(f32x4*)((float*)m.data + row * m.ld + channel) = v;
}

// f and 1 - f, each to its own relative accuracy.  The exponential and the
// reciprocal of the hardware (one unit in the last place) serve BF16 inputs;
// FP32 ones get the exponent's rounding error back (it is up to |gate| 2^-24 of
// the result) and a Newton step.
template <bool BF16>
__device__ __forceinline__ void gate_weights(float g, float& f, float& rest) {
  const float a = -fabsf(g), t = a * 1.44269504f;
  float e = __builtin_amdgcn_exp2f(t);
  if (!BF16) {
    const float lost = fmaf(a, 1.44269504f, -t) + a * 1.92596299e-8f;  // of a log2(e) as a sum of two numbers
    e = fabsf(g) < 200.f ? fmaf(e, lost * 0.693147181f, e) : e;
  }
  const float d = 1.f + e;
  float inverse = __builtin_amdgcn_rcpf(d);
  if (!BF16) inverse = fmaf(fmaf(-d, inverse, 1.f), inverse, inverse);
  const float small = e * inverse;
  f = g >= 0.f ? inverse : small;
  rest = g >= 0.f ? small : inverse;
}

// a b, 0 where the weight a is
__device__ __forceinline__ float weighted(float a, float b) { return a == 0.f ? 0.f : a * b; }
__device__ __forceinline__ float carry_on(float a, float c, float b) { return a == 0.f ? b : fmaf(a, c, b); }
// 0 exactly where either is, else at least the smallest positive number
__device__ __forceinline__ float product_of(float a, float b) {
  return fmaxf(a * b, fminf(fminf(a, b), 0x1p-149f));
}

// ---------------------------------------------------------------- places --
struct RecPlace {
  int lane16, run;        // place in the tile
  int channel, safe;      // first of the lane's four channels, and one to load from
  bool live;              // the channels exist
  int begin, end;         // rows of the axis
  int first, last;        // tiles of the span
  int64_t tile0, span0;   // of the axis
  int span;
};
template <bool BF16>
__device__ __forceinline__ RecPlace rec_place(const RecParams& p) {
  constexpr int TR = rec_tile_rows(BF16);
  RecPlace q;
  const int id = blockIdx.x, rest = id / p.blocks, axis = rest / p.spans;
  q.span = rest - axis * p.spans;
  q.lane16 = threadIdx.x & 15;
  q.run = threadIdx.x >> 4;
  q.channel = (id - rest * p.blocks) * kRecChannels + 4 * q.lane16;
  q.live = q.channel < p.D;
  q.safe = min(q.channel, p.D - 4);
  q.begin = axis * p.axis_rows;
  q.end = min(p.R - q.begin, p.axis_rows) + q.begin;
  q.first = q.span * p.span_tiles;
  q.last = min(q.first + p.span_tiles, (q.end - q.begin + TR - 1) / TR);
  q.tile0 = (int64_t)axis * p.tiles;
  q.span0 = (int64_t)axis * p.spans;
  return q;
}

// What is special about a run's rows: bit u for row u.  The sixteen lanes of a
// run agree.
struct RecEdges {
  unsigned live, start, last;
  int seq;     // sequence of the first row (not packed)
  bool plain;  // of the whole wave: all rows live, none starts or ends a sequence
};
// packed: lane l of a run holds the sequence of row l - 1; rows outside the
// axis have -2
template <int U>
__device__ __forceinline__ int rec_fetch_seq(const RecParams& p, const RecPlace& q, int row) {
  const int r = row - 1 + q.lane16;
  return p.seq && r >= 0 && r < q.end && q.lane16 < U + 2 ? p.seq[r] : -2;
}
template <int U>
__device__ __forceinline__ RecEdges rec_edges(const RecParams& p, const RecPlace& q, int row, int sq) {
  RecEdges e{0, 0, 0, 0, false};
  const int n = min(max(q.end - row, 0), U);
  if (p.seq) {
    const int before = __builtin_amdgcn_update_dpp(-2, sq, 0x111, 0xf, 0xf, false);  // lane l - 1 of the sixteen
    const int shift = threadIdx.x & 48;
    const unsigned full = (1u << U) - 1;
    const unsigned differ = (unsigned)(__ballot(sq != before) >> shift) & 0xffffu;
    e.live = (unsigned)(__ballot(sq >= 0) >> (shift + 1)) & full;
    e.start = (differ >> 1) & e.live;
    e.last = (differ >> 2) & e.live;
  } else {
    e.live = (1u << n) - 1;
    e.seq = row / p.length;
    int at = row - e.seq * p.length;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      e.start |= at == 0 ? 1u << u : 0;
      ++at;
      e.last |= at == p.length ? 1u << u : 0;
      at = at == p.length ? 0 : at;
    }
    e.start &= e.live;
    e.last &= e.live;
  }
  e.plain = __ballot(e.live != (1u << U) - 1 || (e.start | e.last) != 0) == 0;
  return e;
}
__device__ __forceinline__ int64_t rec_sequence(const RecParams& p, const RecEdges& e, int row, int u) {
  return p.seq ? p.seq[row + u] : e.seq + __builtin_popcount(e.start & ((2u << u) - 1) & ~1u);
}
__device__ __forceinline__ f32x4 rec_state(const float* state, const RecParams& p, const RecEdges& e,
                                           const RecPlace& q, int row, int u) {
  if (!state) return f32x4{0.f, 0.f, 0.f, 0.f};
  return *(const f32x4*)(state + rec_sequence(p, e, row, u) * p.D + q.safe);
}

// ------------------------------------------------------- rows of one run --
// f and b = w x of a run's rows; where the run is not plain, rows without a
// sequence get zeros, and a first row f = 0 and the initial state in b.
template <bool BF16, bool COUPLED, int U>
__device__ __forceinline__ void rec_inputs(const RecParams& p, const RecPlace& q, const RecEdges& e, int row,
                                           const Raw4<BF16> (&gate)[U], const Raw4<BF16> (&x)[U], f32x4 (&f)[U],
                                           f32x4 (&b)[U]) {
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const f32x4 g = unpack4(gate[u]), v = unpack4(x[u]);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float fk, rest;
      gate_weights<BF16>(g[k], fk, rest);
      f[u][k] = fk;
      b[u][k] = COUPLED ? weighted(rest, v[k]) : v[k];
    }
  }
  if (e.plain) return;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const bool live = e.live >> u & 1, start = e.start >> u & 1;
    if (start && p.state) {
      const f32x4 c = rec_state(p.state, p, e, q, row, u);
#pragma unroll
      for (int k = 0; k < 4; ++k) b[u][k] = carry_on(f[u][k], c[k], b[u][k]);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      f[u][k] = live && !start ? f[u][k] : 0.f;
      b[u][k] = live ? b[u][k] : 0.f;
    }
  }
}

template <int U>
__device__ __forceinline__ void rec_compose(const f32x4 (&f)[U], const f32x4 (&b)[U], f32x4& A, f32x4& H) {
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      A[k] = product_of(A[k], f[u][k]);
      H[k] = carry_on(f[u][k], H[k], b[u][k]);
    }
}

// --------------------------------------------------------------- forward --
template <bool BF16, bool COUPLED>
__global__ void __launch_bounds__(256) recurrence_kernel(RecParams p) {
  constexpr int U = rec_run_rows(BF16), TR = rec_tile_rows(BF16);
  __shared__ f32x4 products[2][kRecRuns][16], results[2][kRecRuns][16];
  const RecPlace q = rec_place<BF16>(p);
  if (q.first >= q.last) return;
  f32x4 carry = {0.f, 0.f, 0.f, 0.f};
  for (int s = 0; s < q.span; ++s) {
    const float* at = p.summary + (q.span0 + s) * 2 * p.D + q.safe;
    const f32x4 A = *(const f32x4*)at, H = *(const f32x4*)(at + p.D);
#pragma unroll
    for (int k = 0; k < 4; ++k) carry[k] = carry_on(A[k], carry[k], H[k]);
  }
  Raw4<BF16> gate[U], x[U];
  int sq = -2;
  const auto first_row = [&](int tile) { return q.begin + tile * TR + q.run * U; };
  const auto fetch = [&](int tile) {
    const int row = first_row(tile);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = min(row + u, q.end - 1);
      gate[u] = load4<BF16>(p.gate, r, q.safe);
      x[u] = load4<BF16>(p.x, r, q.safe);
    }
    sq = rec_fetch_seq<U>(p, q, row);
  };
  fetch(q.first);
  for (int tile = q.first; tile < q.last; ++tile) {
    const int row = first_row(tile), turn = tile & 1;
    const RecEdges e = rec_edges<U>(p, q, row, sq);
    f32x4 f[U], b[U];
    rec_inputs<BF16, COUPLED, U>(p, q, e, row, gate, x, f, b);
    if (tile + 1 < q.last) fetch(tile + 1);
    f32x4 A = {1.f, 1.f, 1.f, 1.f}, H = {0.f, 0.f, 0.f, 0.f};
    rec_compose<U>(f, b, A, H);
    // two places in LDS by turns: one barrier a tile
    products[turn][q.run][q.lane16] = A;
    results[turn][q.run][q.lane16] = H;
    if (p.carries && q.run == 0 && q.live) *(f32x4*)(p.carries + (q.tile0 + tile) * p.D + q.channel) = carry;
    __syncthreads();
    f32x4 h = carry;
#pragma unroll
    for (int s = 0; s < kRecRuns; ++s) {
      const f32x4 As = products[turn][s][q.lane16], Hs = results[turn][s][q.lane16];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        h[k] = s == q.run ? carry[k] : h[k];
        carry[k] = carry_on(As[k], carry[k], Hs[k]);
      }
    }
    const int n = min(max(q.end - row, 0), U);
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int k = 0; k < 4; ++k) h[k] = carry_on(f[u][k], h[k], b[u][k]);
      if (u < n && q.live) store4<BF16>(p.h, row + u, q.channel, h);
      if (!e.plain && p.state_out && (e.last >> u & 1) && q.live)
        *(f32x4*)(p.state_out + rec_sequence(p, e, row, u) * p.D + q.channel) = h;
    }
  }
}

// (A, H) of each span but an axis's last, whose rows' end nothing follows.  No
// order is needed until the end, so that each run takes U span_tiles rows in
// one piece.
template <bool BF16, bool COUPLED>
__global__ void __launch_bounds__(256) recurrence_span_kernel(RecParams p) {
  constexpr int U = rec_run_rows(BF16), TR = rec_tile_rows(BF16);
  __shared__ f32x4 products[kRecRuns][16], results[kRecRuns][16];
  const RecPlace q = rec_place<BF16>(p);
  if (q.first >= q.last || q.span == p.spans - 1) return;
  const int row0 = q.begin + q.first * TR + q.run * p.span_tiles * U;
  f32x4 A = {1.f, 1.f, 1.f, 1.f}, H = {0.f, 0.f, 0.f, 0.f};
  Raw4<BF16> gate[U], x[U];
  int sq = -2;
  const auto fetch = [&](int row) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = min(row + u, q.end - 1);
      gate[u] = load4<BF16>(p.gate, r, q.safe);
      x[u] = load4<BF16>(p.x, r, q.safe);
    }
    sq = rec_fetch_seq<U>(p, q, row);
  };
  fetch(row0);
  for (int i = 0; i < p.span_tiles; ++i) {
    const int row = row0 + i * U;
    const RecEdges e = rec_edges<U>(p, q, row, sq);
    f32x4 f[U], b[U];
    rec_inputs<BF16, COUPLED, U>(p, q, e, row, gate, x, f, b);
    if (i + 1 < p.span_tiles) fetch(row + U);
    rec_compose<U>(f, b, A, H);
  }
  products[q.run][q.lane16] = A;
  results[q.run][q.lane16] = H;
  __syncthreads();
  if (q.run != 0 || !q.live) return;
#pragma unroll
  for (int s = 1; s < kRecRuns; ++s)
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float a = products[s][q.lane16][k];
      A[k] = product_of(A[k], a);
      H[k] = carry_on(a, H[k], results[s][q.lane16][k]);
    }
  float* at = p.summary + (q.span0 + q.span) * 2 * p.D + q.channel;
  *(f32x4*)at = A;
  *(f32x4*)(at + p.D) = H;
}

// -------------------------------------------------------------- gradient --
// f and 1 - f of a run's rows, zeros at those without a sequence.
template <bool BF16, int U>
__device__ __forceinline__ void rec_weights(const RecEdges& e, const Raw4<BF16> (&gate)[U], f32x4 (&f)[U],
                                            f32x4 (&rest)[U]) {
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const f32x4 g = unpack4(gate[u]);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float fk, rk;
      gate_weights<BF16>(g[k], fk, rk);
      f[u][k] = fk;
      rest[u][k] = rk;
    }
  }
  if (e.plain) return;
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      f[u][k] = e.live >> u & 1 ? f[u][k] : 0.f;
      rest[u][k] = e.live >> u & 1 ? rest[u][k] : 0.f;
    }
}

// dh of row u, with dstate at a last row
template <bool BF16, bool PLAIN>
__device__ __forceinline__ f32x4 rec_dh(const RecParams& p, const RecPlace& q, const RecEdges& e, int row, int u,
                                        const Raw4<BF16>& raw) {
  f32x4 d = unpack4(raw);
  if (PLAIN) return d;
  if ((e.last >> u & 1) && p.dstate) {
    const f32x4 more = rec_state(p.dstate, p, e, q, row, u);
#pragma unroll
    for (int k = 0; k < 4; ++k) d[k] += more[k];
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) d[k] = e.live >> u & 1 ? d[k] : 0.f;
  return d;
}

// A run backwards takes c, what reaches it from the rows after it, to A c + Q;
// A is the same product as forward.
template <bool BF16, bool PLAIN, int U>
__device__ __forceinline__ void rec_compose_back(const RecParams& p, const RecPlace& q, const RecEdges& e, int row,
                                                 const f32x4 (&f)[U], const Raw4<BF16> (&grad)[U], f32x4& A, f32x4& Q) {
#pragma unroll
  for (int u = U - 1; u >= 0; --u) {
    const f32x4 dh = rec_dh<BF16, PLAIN>(p, q, e, row, u, grad[u]);
    const bool stop = !PLAIN && (e.start >> u & 1);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float fk = stop ? 0.f : f[u][k];
      A[k] = product_of(A[k], fk);
      Q[k] = weighted(fk, dh[k] + Q[k]);
    }
  }
}

// The run's states from h, the one before it: before[u] is the state that row
// u starts from.  Returns the last row's.  Rows without a sequence, which no
// other follows, may give anything.
template <bool BF16, bool COUPLED, bool PLAIN, int U>
__device__ __forceinline__ f32x4 rec_states(const RecParams& p, const RecPlace& q, const RecEdges& e, int row,
                                            const f32x4 (&f)[U], const f32x4 (&rest)[U], const Raw4<BF16> (&x)[U],
                                            f32x4 h, f32x4 (&before)[U]) {
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const f32x4 v = unpack4(x[u]);
    if (!PLAIN && (e.start >> u & 1)) h = rec_state(p.state, p, e, q, row, u);
    before[u] = h;
#pragma unroll
    for (int k = 0; k < 4; ++k) h[k] = carry_on(f[u][k], h[k], COUPLED ? weighted(rest[u][k], v[k]) : v[k]);
  }
  return h;
}

template <bool BF16, bool COUPLED, bool PLAIN, int U>
__device__ __forceinline__ void rec_finish(const RecParams& p, const RecPlace& q, const RecEdges& e, int row,
                                           const f32x4 (&f)[U], const f32x4 (&rest)[U], const Raw4<BF16> (&x)[U],
                                           const Raw4<BF16> (&grad)[U], const f32x4& h, f32x4 c) {
  f32x4 before[U];
  rec_states<BF16, COUPLED, PLAIN, U>(p, q, e, row, f, rest, x, h, before);
  const int n = min(max(q.end - row, 0), U);
#pragma unroll
  for (int u = U - 1; u >= 0; --u) {
    const f32x4 v = unpack4(x[u]), dh = rec_dh<BF16, PLAIN>(p, q, e, row, u, grad[u]);
    f32x4 dx, dg;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float g = dh[k] + c[k];
      dx[k] = COUPLED ? weighted(rest[u][k], g) : g;
      dg[k] = weighted(f[u][k] * rest[u][k], g * (COUPLED ? before[u][k] - v[k] : before[u][k]));
      c[k] = weighted(f[u][k], g);
    }
    if (q.live && (PLAIN || u < n)) {
      store4<BF16>(p.dx, row + u, q.channel, dx);
      store4<BF16>(p.dgate, row + u, q.channel, dg);
    }
    if (!PLAIN && (e.start >> u & 1)) {
      if (p.dstate_out && q.live) *(f32x4*)(p.dstate_out + rec_sequence(p, e, row, u) * p.D + q.channel) = c;
      c = f32x4{0.f, 0.f, 0.f, 0.f};
    }
  }
}

template <bool BF16, bool COUPLED>
__global__ void __launch_bounds__(256) recurrence_dgrad_kernel(RecParams p) {
  constexpr int U = rec_run_rows(BF16), TR = rec_tile_rows(BF16);
  __shared__ f32x4 products[2][kRecRuns][16], results[2][kRecRuns][16], gradients[2][kRecRuns][16];
  const RecPlace q = rec_place<BF16>(p);
  if (q.first >= q.last) return;
  f32x4 back = {0.f, 0.f, 0.f, 0.f};  // what reaches the tile from the rows after it
  for (int s = p.spans - 1; s > q.span; --s) {
    const float* at = p.summary + (q.span0 + s) * 2 * p.D + q.safe;
    const f32x4 A = *(const f32x4*)at, Q = *(const f32x4*)(at + p.D);
#pragma unroll
    for (int k = 0; k < 4; ++k) back[k] = carry_on(A[k], back[k], Q[k]);
  }
  Raw4<BF16> gate[U], x[U], grad[U];
  f32x4 carry;
  int sq = -2;
  const auto first_row = [&](int tile) { return q.begin + tile * TR + q.run * U; };
  const auto fetch = [&](int tile) {
    const int row = first_row(tile);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = min(row + u, q.end - 1);
      gate[u] = load4<BF16>(p.gate, r, q.safe);
      x[u] = load4<BF16>(p.x, r, q.safe);
      grad[u] = load4<BF16>(p.dh, r, q.safe);
    }
    carry = *(const f32x4*)(p.carries + (q.tile0 + tile) * p.D + q.safe);
    sq = rec_fetch_seq<U>(p, q, row);
  };
  fetch(q.last - 1);
  for (int tile = q.last - 1; tile >= q.first; --tile) {
    const int row = first_row(tile), turn = tile & 1;
    const RecEdges e = rec_edges<U>(p, q, row, sq);
    f32x4 f[U], rest[U], unused[U];
    Raw4<BF16> v[U], dh[U];
    rec_weights<BF16, U>(e, gate, f, rest);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      v[u] = x[u];
      dh[u] = grad[u];
    }
    f32x4 h = carry;
    if (tile > q.first) fetch(tile - 1);
    f32x4 A = {1.f, 1.f, 1.f, 1.f}, Q = {0.f, 0.f, 0.f, 0.f}, H = {0.f, 0.f, 0.f, 0.f};
    if (e.plain) {
      rec_compose_back<BF16, true, U>(p, q, e, row, f, dh, A, Q);
      H = rec_states<BF16, COUPLED, true, U>(p, q, e, row, f, rest, v, H, unused);
    } else {
      rec_compose_back<BF16, false, U>(p, q, e, row, f, dh, A, Q);
      H = rec_states<BF16, COUPLED, false, U>(p, q, e, row, f, rest, v, H, unused);
    }
    products[turn][q.run][q.lane16] = A;
    results[turn][q.run][q.lane16] = H;
    gradients[turn][q.run][q.lane16] = Q;
    __syncthreads();
#pragma unroll
    for (int s = 0; s < kRecRuns - 1; ++s) {
      const f32x4 As = products[turn][s][q.lane16], Hs = results[turn][s][q.lane16];
#pragma unroll
      for (int k = 0; k < 4; ++k) h[k] = s < q.run ? carry_on(As[k], h[k], Hs[k]) : h[k];
    }
    f32x4 c = back;
#pragma unroll
    for (int s = kRecRuns - 1; s >= 0; --s) {
      const f32x4 As = products[turn][s][q.lane16], Qs = gradients[turn][s][q.lane16];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        c[k] = s == q.run ? back[k] : c[k];
        back[k] = carry_on(As[k], back[k], Qs[k]);
      }
    }
    if (e.plain)
      rec_finish<BF16, COUPLED, true, U>(p, q, e, row, f, rest, v, dh, h, c);
    else
      rec_finish<BF16, COUPLED, false, U>(p, q, e, row, f, rest, v, dh, h, c);
  }
}

// (A, Q) of each span but an axis's first.
template <bool BF16>
__global__ void __launch_bounds__(256) recurrence_dgrad_span_kernel(RecParams p) {
  constexpr int U = rec_run_rows(BF16), TR = rec_tile_rows(BF16);
  __shared__ f32x4 products[kRecRuns][16], gradients[kRecRuns][16];
  const RecPlace q = rec_place<BF16>(p);
  if (q.first >= q.last || q.span == 0) return;
  const int row0 = q.begin + q.first * TR + q.run * p.span_tiles * U;
  f32x4 A = {1.f, 1.f, 1.f, 1.f}, Q = {0.f, 0.f, 0.f, 0.f};
  Raw4<BF16> gate[U], grad[U];
  int sq = -2;
  const auto fetch = [&](int row) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = min(row + u, q.end - 1);
      gate[u] = load4<BF16>(p.gate, r, q.safe);
      grad[u] = load4<BF16>(p.dh, r, q.safe);
    }
    sq = rec_fetch_seq<U>(p, q, row);
  };
  fetch(row0 + (p.span_tiles - 1) * U);
  for (int i = p.span_tiles - 1; i >= 0; --i) {
    const int row = row0 + i * U;
    const RecEdges e = rec_edges<U>(p, q, row, sq);
    f32x4 f[U], rest[U];
    Raw4<BF16> dh[U];
    rec_weights<BF16, U>(e, gate, f, rest);
#pragma unroll
    for (int u = 0; u < U; ++u) dh[u] = grad[u];
    if (i > 0) fetch(row - U);
    if (e.plain)
      rec_compose_back<BF16, true, U>(p, q, e, row, f, dh, A, Q);
    else
      rec_compose_back<BF16, false, U>(p, q, e, row, f, dh, A, Q);
  }
  products[q.run][q.lane16] = A;
  gradients[q.run][q.lane16] = Q;
  __syncthreads();
  if (q.run != kRecRuns - 1 || !q.live) return;
#pragma unroll
  for (int s = kRecRuns - 2; s >= 0; --s)
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float a = products[s][q.lane16][k];
      A[k] = product_of(A[k], a);
      Q[k] = carry_on(a, Q[k], gradients[s][q.lane16][k]);
    }
  float* at = p.summary + (q.span0 + q.span) * 2 * p.D + q.channel;
  *(f32x4*)at = A;
  *(f32x4*)(at + p.D) = Q;
}

// ---------------------------------------------------------- packed rows --
// Each row's sequence, by bisection of the offsets; and for sequences without
// rows, what comes in goes out (from, to: [S, D], null: zeros, nothing).
// offsets null: no sequence has rows.
__global__ void __launch_bounds__(256) recurrence_rows_kernel(const int32_t* offsets, int S, int R, int row_blocks,
                                                              int32_t* seq, const float* from, float* to, int D) {
  if ((int)blockIdx.x < row_blocks) {
    const int r = blockIdx.x * 256 + threadIdx.x;
    if (r >= R) return;
    int lo = 0, hi = S;  // the first sequence that ends behind row r
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (offsets[mid + 1] > r)
        hi = mid;
      else
        lo = mid + 1;
    }
    seq[r] = lo < S ? lo : -1;
    return;
  }
  if (!to) return;
  const int blocks = gridDim.x - row_blocks;
  for (int s = blockIdx.x - row_blocks; s < S; s += blocks) {
    if (offsets && offsets[s + 1] > (s ? offsets[s] : 0)) continue;
    for (int i = 4 * threadIdx.x; i < D; i += 1024)
      *(f32x4*)(to + (int64_t)s * D + i) =
          from ? *(const f32x4*)(from + (int64_t)s * D + i) : f32x4{0.f, 0.f, 0.f, 0.f};
  }
}

__global__ void __launch_bounds__(256) recurrence_copy_kernel(const f32x4* from, f32x4* to, int64_t n) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) to[i] = from[i];
}

}  // namespace dpg

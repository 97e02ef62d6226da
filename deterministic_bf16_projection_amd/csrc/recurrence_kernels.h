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
// half a wave holds 64 channels of a run of eight rows, sixteen runs make a
// tile.  The halves compose their runs, the waves meet in LDS, every lane finds
// the state before its run, and then each row's, from values that stayed in
// registers: the rows are read once.  A is zero only if some f is: products that
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
// in BF16); the gradient recomputes the states in between from them instead of
// reading rounded ones.
#pragma once
#include <type_traits>

#include "rows8.h"

namespace dpg {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

constexpr int kRecChannels = 64;
constexpr int kRecWaves = 8;
constexpr int kRecThreads = 64 * kRecWaves;
constexpr int kRecRuns = 2 * kRecWaves;  // of a tile
constexpr int kRecRunRows = 8;
constexpr int kRecTileRows = kRecRuns * kRecRunRows;

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

// ------------------------------------------------------------ two values --
template <bool BF16>
using Raw2 = std::conditional_t<BF16, unsigned, f32x2>;

__device__ __forceinline__ f32x2 unpack2(unsigned r) {
  return f32x2{__builtin_bit_cast(float, r << 16), __builtin_bit_cast(float, r & 0xffff0000u)};
}
__device__ __forceinline__ f32x2 unpack2(const f32x2& r) { return r; }
template <bool BF16>
__device__ __forceinline__ Raw2<BF16> pack2(const f32x2& v) {
  if constexpr (BF16)
    return __builtin_bit_cast(unsigned, __builtin_convertvector(v, bf16x2));
  else
    return v;
}

// a b, and 0 where either is 0, whatever the other is: a weight of 0 leaves its
// term out.  One instruction of the hardware, for which there is no builtin.
__device__ float mul_zero_wins(float a, float b) __asm("llvm.amdgcn.fmul.legacy");
__device__ __forceinline__ float weighted(float a, float b) { return mul_zero_wins(a, b); }
__device__ __forceinline__ float carry_on(float a, float c, float b) { return weighted(a, c) + b; }
// a product of weights: 0 exactly where the least of them is, else at least the
// smallest normal number
__device__ __forceinline__ float held(float product, float least) {
  return fmaxf(product, fminf(least, 0x1p-126f));
}

// f and 1 - f, each to its own relative accuracy.  With e = exp(-gate), f = 1 /
// (1 + e) and 1 - f = e f, which is infinity times 0 for the lowest gates: the
// minimum with 1 makes that 1.  For BF16 inputs the exponential and the
// reciprocal of the hardware (one unit in the last place) do.  FP32 ones take
// the smaller weight from exp(-|gate|), whose exponent gets its rounding error
// back (up to |gate| 2^-24 of the result), and a Newton step.
template <bool BF16>
__device__ __forceinline__ void gate_weights(float g, float& f, float& rest) {
  if (BF16) {
    const float e = __builtin_amdgcn_exp2f(g * -1.44269504f);
    f = __builtin_amdgcn_rcpf(1.f + e);
    rest = fminf(e * f, 1.f);
    return;
  }
  const float a = -fabsf(g), t = a * 1.44269504f;
  float e = __builtin_amdgcn_exp2f(t);
  const float lost = fmaf(a, 1.44269504f, -t) + a * 1.92596299e-8f;  // of a log2(e) as a sum of two numbers
  e = fabsf(g) < 200.f ? fmaf(e, lost * 0.693147181f, e) : e;
  const float d = 1.f + e;
  float inverse = __builtin_amdgcn_rcpf(d);
  inverse = fmaf(fmaf(-d, inverse, 1.f), inverse, inverse);
  const float small = e * inverse;
  f = g >= 0.f ? inverse : small;
  rest = g >= 0.f ? small : inverse;
}

// ---------------------------------------------------------------- places --
struct RecPlace {
  int lane, run, wave;    // of the run's 32 lanes; place in the tile
  int channel, safe;      // first of the lane's two channels, and one to load from
  bool live;              // the channels exist
  int begin, end;         // rows of the axis
  int first, last;        // tiles of the span
  int span;
  int64_t tile0, span0;   // of the axis
};
__device__ __forceinline__ RecPlace rec_place(const RecParams& p) {
  constexpr int TR = kRecTileRows;
  RecPlace q;
  const int id = blockIdx.x, rest = id / p.blocks, axis = rest / p.spans;
  q.span = rest - axis * p.spans;
  q.lane = threadIdx.x & 31;
  q.run = threadIdx.x >> 5;
  q.wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  q.channel = (id - rest * p.blocks) * kRecChannels + 2 * q.lane;
  q.live = q.channel < p.D;
  q.safe = min(q.channel, p.D - 2);
  q.begin = axis * p.axis_rows;
  q.end = min(p.R - q.begin, p.axis_rows) + q.begin;
  q.first = q.span * p.span_tiles;
  q.last = min(q.first + p.span_tiles, (q.end - q.begin + TR - 1) / TR);
  q.tile0 = (int64_t)axis * p.tiles;
  q.span0 = (int64_t)axis * p.spans;
  return q;
}

// One matrix as a lane sees it.  A block of rows (a tile, or a step of a span)
// starts at a row that is the same for the workgroup and lies in a scalar
// register; the lane's own offset from there stays the same from block to block.
template <bool BF16>
struct RecRows {
  const char* data;
  int64_t pitch;     // bytes of a row
  unsigned lane;     // bytes from the block's first row and column 0 to the lane's
  unsigned column;   // bytes of the lane's column
  __device__ __forceinline__ RecRows(const Rows8& m, int lane_row, int channel) {
    constexpr int E = BF16 ? 2 : 4;
    data = (const char*)m.data;
    pitch = m.ld * E;
    column = (unsigned)(channel * E);
    lane = (unsigned)lane_row * (unsigned)pitch + column;
  }
  __device__ __forceinline__ Raw2<BF16> load(int64_t row, int u) const {
    return *(const Raw2<BF16>*)(data + (row + u) * pitch + lane);
  }
  // row + r
  __device__ __forceinline__ Raw2<BF16> load_row(int64_t row, int r) const {
    return *(const Raw2<BF16>*)(data + row * pitch + ((unsigned)r * (unsigned)pitch + column));
  }
  __device__ __forceinline__ void store(int64_t row, int u, const Raw2<BF16>& v) const {
    *(Raw2<BF16>*)(const_cast<char*>(data) + (row + u) * pitch + lane) = v;
  }
};

// The same for the long runs of a span, which may lie more than 4 GB apart: a
// pointer for each lane.
template <bool BF16>
struct RecRun {
  const char* data;  // the run's first row
  int64_t pitch;
  __device__ __forceinline__ RecRun(const Rows8& m, int row, int channel) {
    constexpr int E = BF16 ? 2 : 4;
    pitch = m.ld * E;
    data = (const char*)m.data + row * pitch + channel * E;
  }
  __device__ __forceinline__ Raw2<BF16> load(int64_t r) const { return *(const Raw2<BF16>*)(data + r * pitch); }
};

// What is special about a run's rows: bit u for row u.  The lanes of a run
// agree.
struct RecEdges {
  unsigned live, start, last;
  int seq;     // sequence of the first row (not packed)
};
// packed: lane l of a run holds the sequences of rows l - 1 and l; rows outside
// the axis have -2
struct RecSeq {
  int before, at;
};
template <int U>
__device__ __forceinline__ RecSeq rec_fetch_seq(const RecParams& p, const RecPlace& q, int row) {
  const int r = row + q.lane;
  RecSeq s;
  s.before = q.lane <= U && r >= 1 && r <= q.end ? p.seq[r - 1] : -2;
  s.at = q.lane <= U && r < q.end ? p.seq[r] : -2;
  return s;
}
template <int U>
__device__ __forceinline__ RecEdges rec_edges(const RecParams& p, const RecPlace& q, int row, const RecSeq& sq) {
  RecEdges e{0, 0, 0, 0};
  const unsigned full = (1u << U) - 1;
  if (p.seq) {
    const int shift = threadIdx.x & 32;
    const unsigned differ = (unsigned)(__ballot(sq.at != sq.before) >> shift);
    e.live = (unsigned)(__ballot(sq.at >= 0) >> shift) & full;
    e.start = differ & e.live;
    e.last = (differ >> 1) & e.live;
  } else {
    const int n = min(max(q.end - row, 0), U);
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
  return e;
}
// Whether rows [row, row + n) of an axis that is one sequence of equal ones
// are all inside it and neither its first nor its last: known without a look at
// each.
__device__ __forceinline__ bool rec_inside(const RecParams& p, const RecPlace& q, int row, int n) {
  return !p.seq && p.length == p.axis_rows && row > q.begin && row + n < q.end;
}
__device__ __forceinline__ bool rec_ordinary(const RecEdges& e, int U) {
  return __ballot(e.live != (1u << U) - 1 || (e.start | e.last) != 0) == 0;
}
__device__ __forceinline__ int64_t rec_sequence(const RecParams& p, const RecEdges& e, int row, int u) {
  return p.seq ? p.seq[row + u] : e.seq + __builtin_popcount(e.start & ((2u << u) - 1) & ~1u);
}
__device__ __forceinline__ f32x2 rec_state(const float* state, const RecParams& p, const RecEdges& e,
                                           const RecPlace& q, int row, int u) {
  if (!state) return f32x2{0.f, 0.f};
  return *(const f32x2*)(state + rec_sequence(p, e, row, u) * p.D + q.safe);
}
__device__ __forceinline__ void rec_put_state(float* state, const RecParams& p, const RecEdges& e, const RecPlace& q,
                                              int row, int u, const f32x2& v) {
  if (state && q.live) *(f32x2*)(state + rec_sequence(p, e, row, u) * p.D + q.channel) = v;
}

// N matrices' rows of one run, loaded a block ahead of their use.
template <bool BF16, int N, int U>
struct RecFetch {
  Raw2<BF16> raw[N][U];
  RecSeq sq;
  // the tile from `row` on, of which the lane has the rows from lane_row on
  __device__ __forceinline__ void tile(const RecParams& p, const RecPlace& q, const RecRows<BF16>* const (&m)[N],
                                       int row, int lane_row) {
    if (row + kRecRuns * U <= q.end) {
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < N; ++i) raw[i][u] = m[i]->load(row, u);
    } else {
      // rows behind the axis are read from its last one
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int r = min(lane_row + u, q.end - 1 - row);
#pragma unroll
        for (int i = 0; i < N; ++i) raw[i][u] = m[i]->load_row(row, r);
      }
    }
    if (p.seq) sq = rec_fetch_seq<U>(p, q, row + lane_row);
  }
  // rows [at, at + U) of the run that starts at run_row
  __device__ __forceinline__ void run(const RecParams& p, const RecPlace& q, const RecRun<BF16>* const (&m)[N],
                                      int run_row, int at, bool whole) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t r = whole ? at + u : min(at + u, q.end - 1 - min(run_row, q.end - 1));
#pragma unroll
      for (int i = 0; i < N; ++i) raw[i][u] = m[i]->load(r);
    }
    if (p.seq) sq = rec_fetch_seq<U>(p, q, run_row + at);
  }
};

// --------------------------------------------------------------- forward --
// f and b = w x of a run's rows.  Where the run is not plain, rows without a
// sequence get zeros, and a first row f = 0 and the initial state in b.
template <bool BF16, bool COUPLED, bool PLAIN, int U>
__device__ __forceinline__ void rec_inputs(const RecParams& p, const RecPlace& q, const RecEdges& e, int row,
                                           const Raw2<BF16> (&gate)[U], const Raw2<BF16> (&x)[U], f32x2 (&f)[U],
                                           f32x2 (&b)[U]) {
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const f32x2 g = unpack2(gate[u]), v = unpack2(x[u]);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float fk, rest;
      gate_weights<BF16>(g[k], fk, rest);
      f[u][k] = fk;
      b[u][k] = COUPLED ? weighted(rest, v[k]) : v[k];
    }
  }
  if (PLAIN) return;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const bool live = e.live >> u & 1, start = e.start >> u & 1;
    if (start) {
      const f32x2 c = rec_state(p.state, p, e, q, row, u);
#pragma unroll
      for (int k = 0; k < 2; ++k) b[u][k] = carry_on(f[u][k], c[k], b[u][k]);
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      f[u][k] = live && !start ? f[u][k] : 0.f;
      b[u][k] = live ? b[u][k] : 0.f;
    }
  }
}

// (A, H) of a run after (A, H) of what precedes it
template <int U>
__device__ __forceinline__ void rec_compose(const f32x2 (&f)[U], const f32x2 (&b)[U], f32x2& A, f32x2& H) {
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    float least = A[k];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      A[k] *= f[u][k];
      least = fminf(least, f[u][k]);
      H[k] = carry_on(f[u][k], H[k], b[u][k]);
    }
    A[k] = held(A[k], least);
  }
}

// Both halves' values of a wave, in all lanes: of run 2 w, and of run 2 w + 1.
struct RecHalves {
  f32x2 first, second;
};
__device__ __forceinline__ RecHalves rec_halves(const f32x2& v) {
  RecHalves h;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    // (a bit cast of a vector's element itself would take the first one's)
    const float value = v[k];
    const unsigned bits = __builtin_bit_cast(unsigned, value);
    const auto both = __builtin_amdgcn_permlane32_swap(bits, bits, false, false);
    const unsigned lower = both[0], upper = both[1];
    h.first[k] = __builtin_bit_cast(float, lower);
    h.second[k] = __builtin_bit_cast(float, upper);
  }
  return h;
}
__device__ __forceinline__ f32x2 rec_carry(const f32x2& A, const f32x2& c, const f32x2& H) {
  return f32x2{carry_on(A[0], c[0], H[0]), carry_on(A[1], c[1], H[1])};
}
__device__ __forceinline__ f32x2 rec_product(const f32x2& A, const f32x2& B) {
  return f32x2{held(A[0] * B[0], fminf(A[0], B[0])), held(A[1] * B[1], fminf(A[1], B[1]))};
}

// The rows of a tile, one matrix's: all of them exist, or those before q.end.
template <bool BF16, int U>
__device__ __forceinline__ void rec_store(const RecPlace& q, const RecRows<BF16>& m, int row0, int row, bool whole,
                                          const Raw2<BF16> (&v)[U]) {
  if (!q.live) return;
  if (whole) {
#pragma unroll
    for (int u = 0; u < U; ++u) m.store(row0, u, v[u]);
  } else {
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (row + u < q.end) m.store(row0, u, v[u]);
  }
}

template <bool BF16, bool COUPLED>
__global__ void __launch_bounds__(kRecThreads) recurrence_kernel(RecParams p) {
  constexpr int U = kRecRunRows, TR = kRecTileRows;
  __shared__ f32x2 products[2][kRecWaves][32], results[2][kRecWaves][32];
  const RecPlace q = rec_place(p);
  if (q.first >= q.last) return;
  f32x2 carry = {0.f, 0.f};
  for (int s = 0; s < q.span; ++s) {
    const float* at = p.summary + (q.span0 + s) * 2 * p.D + q.safe;
    carry = rec_carry(*(const f32x2*)at, carry, *(const f32x2*)(at + p.D));
  }
  const int lane_row = q.run * U;
  const bool second = q.run & 1;
  const RecRows<BF16> gates(p.gate, lane_row, q.safe), xs(p.x, lane_row, q.safe), out(p.h, lane_row, q.channel);
  const RecRows<BF16>* const in[2] = {&gates, &xs};
  RecFetch<BF16, 2, U> next;
  Raw2<BF16> done[U];
  next.tile(p, q, in, q.begin + q.first * TR, lane_row);
  for (int tile = q.first; tile < q.last; ++tile) {
    const int row0 = q.begin + tile * TR, row = row0 + lane_row, turn = tile & 1;
    const bool inside = rec_inside(p, q, row0, TR);
    RecEdges e{};
    if (!inside) e = rec_edges<U>(p, q, row, next.sq);
    const bool plain = inside || rec_ordinary(e, U);
    f32x2 f[U], b[U];
    if (plain)
      rec_inputs<BF16, COUPLED, true, U>(p, q, e, row, next.raw[0], next.raw[1], f, b);
    else
      rec_inputs<BF16, COUPLED, false, U>(p, q, e, row, next.raw[0], next.raw[1], f, b);
    // Memory operations are waited for in the order of their issue: stores that
    // came after the next tile's loads would have to end before those are used.
    // So a tile's results are stored one tile later, before the loads.
    if (tile > q.first) rec_store<BF16, U>(q, out, row0 - TR, row - TR, true, done);
    if (p.carries && q.run == 0 && q.live) *(f32x2*)(p.carries + (q.tile0 + tile) * p.D + q.channel) = carry;
    if (tile + 1 < q.last) next.tile(p, q, in, row0 + TR, lane_row);
    f32x2 A = {1.f, 1.f}, H = {0.f, 0.f};
    rec_compose<U>(f, b, A, H);
    const RecHalves As = rec_halves(A), Hs = rec_halves(H);
    // two places in LDS by turns: one barrier a tile
    if (second)
      products[turn][q.wave][q.lane] = rec_product(As.first, As.second);
    else
      results[turn][q.wave][q.lane] = rec_carry(As.second, Hs.first, Hs.second);
    __syncthreads();
    f32x2 h = carry;
#pragma unroll
    for (int s = 0; s < kRecWaves; ++s) {
      if (s == q.wave) h = carry;
      carry = rec_carry(products[turn][s][q.lane], carry, results[turn][s][q.lane]);
    }
    const f32x2 over = rec_carry(As.first, h, Hs.first);
#pragma unroll
    for (int k = 0; k < 2; ++k) h[k] = second ? over[k] : h[k];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      h = rec_carry(f[u], h, b[u]);
      done[u] = pack2<BF16>(h);
      if (!plain && (e.last >> u & 1)) rec_put_state(p.state_out, p, e, q, row, u, h);
    }
  }
  const int row0 = q.begin + (q.last - 1) * TR;
  rec_store<BF16, U>(q, out, row0, row0 + lane_row, false, done);
}

// (A, H) of each span but an axis's last, whose rows' end nothing follows.  No
// order is needed until the end, so that each run takes U span_tiles rows in
// one piece.
template <bool BF16, bool COUPLED>
__global__ void __launch_bounds__(kRecThreads) recurrence_span_kernel(RecParams p) {
  constexpr int U = kRecRunRows, TR = kRecTileRows;
  __shared__ f32x2 products[kRecRuns][32], results[kRecRuns][32];
  const RecPlace q = rec_place(p);
  if (q.first >= q.last || q.span == p.spans - 1) return;
  // every row of a span that is not its axis's last exists
  const int run_row = q.begin + q.first * TR + q.run * p.span_tiles * U;
  const RecRun<BF16> gates(p.gate, run_row, q.safe), xs(p.x, run_row, q.safe);
  const RecRun<BF16>* const in[2] = {&gates, &xs};
  const bool inside = rec_inside(p, q, q.begin + q.first * TR, p.span_tiles * TR);
  f32x2 A = {1.f, 1.f}, H = {0.f, 0.f};
  RecFetch<BF16, 2, U> next;
  next.run(p, q, in, run_row, 0, true);
  for (int at = 0; at < p.span_tiles * U; at += U) {
    const int row = run_row + at;
    RecEdges e{};
    if (!inside) e = rec_edges<U>(p, q, row, next.sq);
    f32x2 f[U], b[U];
    if (inside || rec_ordinary(e, U))
      rec_inputs<BF16, COUPLED, true, U>(p, q, e, row, next.raw[0], next.raw[1], f, b);
    else
      rec_inputs<BF16, COUPLED, false, U>(p, q, e, row, next.raw[0], next.raw[1], f, b);
    if (at + U < p.span_tiles * U) next.run(p, q, in, run_row, at + U, true);
    rec_compose<U>(f, b, A, H);
  }
  products[q.run][q.lane] = A;
  results[q.run][q.lane] = H;
  __syncthreads();
  if (q.run != 0 || !q.live) return;
#pragma unroll
  for (int s = 1; s < kRecRuns; ++s)
  {
    H = rec_carry(products[s][q.lane], H, results[s][q.lane]);
    A = rec_product(A, products[s][q.lane]);
  }
  float* at = p.summary + (q.span0 + q.span) * 2 * p.D + q.channel;
  *(f32x2*)at = A;
  *(f32x2*)(at + p.D) = H;
}

// -------------------------------------------------------------- gradient --
// f and 1 - f of a run's rows, zeros at those without a sequence.
template <bool BF16, bool PLAIN, int U>
__device__ __forceinline__ void rec_weights(const RecEdges& e, const Raw2<BF16> (&gate)[U], f32x2 (&f)[U],
                                            f32x2 (&rest)[U]) {
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const f32x2 g = unpack2(gate[u]);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float fk, rk;
      gate_weights<BF16>(g[k], fk, rk);
      f[u][k] = PLAIN || (e.live >> u & 1) ? fk : 0.f;
      rest[u][k] = PLAIN || (e.live >> u & 1) ? rk : 0.f;
    }
  }
}

// dh of row u, with dstate at a last row
template <bool BF16, bool PLAIN>
__device__ __forceinline__ f32x2 rec_dh(const RecParams& p, const RecPlace& q, const RecEdges& e, int row, int u,
                                        const Raw2<BF16>& raw) {
  f32x2 d = unpack2(raw);
  if (PLAIN) return d;
  if (e.last >> u & 1) {
    const f32x2 more = rec_state(p.dstate, p, e, q, row, u);
#pragma unroll
    for (int k = 0; k < 2; ++k) d[k] += more[k];
  }
#pragma unroll
  for (int k = 0; k < 2; ++k) d[k] = e.live >> u & 1 ? d[k] : 0.f;
  return d;
}

// A run backwards takes c, what reaches it from the rows after it, to A c + Q;
// A is the same product as forward.
template <bool BF16, bool PLAIN, int U>
__device__ __forceinline__ void rec_compose_back(const RecParams& p, const RecPlace& q, const RecEdges& e, int row,
                                                 const f32x2 (&f)[U], const Raw2<BF16> (&grad)[U], f32x2& A, f32x2& Q) {
  f32x2 least = A;
#pragma unroll
  for (int u = U - 1; u >= 0; --u) {
    const f32x2 dh = rec_dh<BF16, PLAIN>(p, q, e, row, u, grad[u]);
    const bool stop = !PLAIN && (e.start >> u & 1);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float fk = stop ? 0.f : f[u][k];
      A[k] *= fk;
      least[k] = fminf(least[k], fk);
      Q[k] = weighted(fk, dh[k] + Q[k]);
    }
  }
#pragma unroll
  for (int k = 0; k < 2; ++k) A[k] = held(A[k], least[k]);
}

// The run's states from h, the one before it: before[u] is the state that row
// u starts from.  Returns the last row's.  Rows without a sequence, which no
// other follows, may give anything.
template <bool BF16, bool COUPLED, bool PLAIN, int U>
__device__ __forceinline__ f32x2 rec_states(const RecParams& p, const RecPlace& q, const RecEdges& e, int row,
                                            const f32x2 (&f)[U], const f32x2 (&rest)[U], const Raw2<BF16> (&x)[U],
                                            f32x2 h, f32x2 (&before)[U]) {
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const f32x2 v = unpack2(x[u]);
    if (!PLAIN && (e.start >> u & 1)) h = rec_state(p.state, p, e, q, row, u);
    before[u] = h;
#pragma unroll
    for (int k = 0; k < 2; ++k) h[k] = carry_on(f[u][k], h[k], COUPLED ? weighted(rest[u][k], v[k]) : v[k]);
  }
  return h;
}

template <bool BF16, bool COUPLED, bool PLAIN, int U>
__device__ __forceinline__ void rec_finish(const RecParams& p, const RecPlace& q, const RecEdges& e, int row,
                                           const f32x2 (&f)[U], const f32x2 (&rest)[U], const Raw2<BF16> (&x)[U],
                                           const Raw2<BF16> (&grad)[U], const f32x2& h, f32x2 c, Raw2<BF16> (&dgate)[U],
                                           Raw2<BF16> (&dx)[U]) {
  f32x2 before[U];
  rec_states<BF16, COUPLED, PLAIN, U>(p, q, e, row, f, rest, x, h, before);
#pragma unroll
  for (int u = U - 1; u >= 0; --u) {
    const f32x2 v = unpack2(x[u]), dh = rec_dh<BF16, PLAIN>(p, q, e, row, u, grad[u]);
    f32x2 out_x, out_g;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float g = dh[k] + c[k];
      out_x[k] = COUPLED ? weighted(rest[u][k], g) : g;
      out_g[k] = weighted(f[u][k] * rest[u][k], g * (COUPLED ? before[u][k] - v[k] : before[u][k]));
      c[k] = weighted(f[u][k], g);
    }
    dx[u] = pack2<BF16>(out_x);
    dgate[u] = pack2<BF16>(out_g);
    if (!PLAIN && (e.start >> u & 1)) {
      rec_put_state(p.dstate_out, p, e, q, row, u, c);
      c = f32x2{0.f, 0.f};
    }
  }
}

template <bool BF16, bool COUPLED>
__global__ void __launch_bounds__(kRecThreads) recurrence_dgrad_kernel(RecParams p) {
  constexpr int U = kRecRunRows, TR = kRecTileRows;
  __shared__ f32x2 products[2][kRecWaves][32], results[2][kRecWaves][32], gradients[2][kRecWaves][32];
  const RecPlace q = rec_place(p);
  if (q.first >= q.last) return;
  f32x2 back = {0.f, 0.f};  // what reaches the tile from the rows after it
  for (int s = p.spans - 1; s > q.span; --s) {
    const float* at = p.summary + (q.span0 + s) * 2 * p.D + q.safe;
    back = rec_carry(*(const f32x2*)at, back, *(const f32x2*)(at + p.D));
  }
  const int lane_row = q.run * U;
  const bool second = q.run & 1;
  const RecRows<BF16> gates(p.gate, lane_row, q.safe), xs(p.x, lane_row, q.safe), dhs(p.dh, lane_row, q.safe);
  const RecRows<BF16> dgate(p.dgate, lane_row, q.channel), dx(p.dx, lane_row, q.channel);
  const RecRows<BF16>* const in[3] = {&gates, &xs, &dhs};
  const auto carried = [&](int tile) { return *(const f32x2*)(p.carries + (q.tile0 + tile) * p.D + q.safe); };
  RecFetch<BF16, 3, U> next;
  Raw2<BF16> done_g[U], done_x[U];
  next.tile(p, q, in, q.begin + (q.last - 1) * TR, lane_row);
  f32x2 carry = carried(q.last - 1);
  for (int tile = q.last - 1; tile >= q.first; --tile) {
    const int row0 = q.begin + tile * TR, row = row0 + lane_row, turn = tile & 1;
    const bool inside = rec_inside(p, q, row0, TR);
    RecEdges e{};
    if (!inside) e = rec_edges<U>(p, q, row, next.sq);
    const bool plain = inside || rec_ordinary(e, U);
    f32x2 f[U], rest[U], unused[U];
    Raw2<BF16> v[U], dh[U];
    if (plain)
      rec_weights<BF16, true, U>(e, next.raw[0], f, rest);
    else
      rec_weights<BF16, false, U>(e, next.raw[0], f, rest);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      v[u] = next.raw[1][u];
      dh[u] = next.raw[2][u];
    }
    f32x2 h = carry;
    // one tile late, before the next loads, as in the forward pass
    if (tile + 1 < q.last) {
      const bool whole = row0 + 2 * TR <= q.end;
      rec_store<BF16, U>(q, dgate, row0 + TR, row + TR, whole, done_g);
      rec_store<BF16, U>(q, dx, row0 + TR, row + TR, whole, done_x);
    }
    if (tile > q.first) {
      next.tile(p, q, in, row0 - TR, lane_row);
      carry = carried(tile - 1);
    }
    f32x2 A = {1.f, 1.f}, Q = {0.f, 0.f}, H = {0.f, 0.f};
    if (plain) {
      rec_compose_back<BF16, true, U>(p, q, e, row, f, dh, A, Q);
      H = rec_states<BF16, COUPLED, true, U>(p, q, e, row, f, rest, v, H, unused);
    } else {
      rec_compose_back<BF16, false, U>(p, q, e, row, f, dh, A, Q);
      H = rec_states<BF16, COUPLED, false, U>(p, q, e, row, f, rest, v, H, unused);
    }
    const RecHalves As = rec_halves(A), Hs = rec_halves(H), Qs = rec_halves(Q);
    if (second) {
      products[turn][q.wave][q.lane] = rec_product(As.first, As.second);
    } else {
      results[turn][q.wave][q.lane] = rec_carry(As.second, Hs.first, Hs.second);
      gradients[turn][q.wave][q.lane] = rec_carry(As.first, Qs.second, Qs.first);
    }
    __syncthreads();
    f32x2 c = back;
#pragma unroll
    for (int s = 0; s < kRecWaves - 1; ++s)
      if (s < q.wave) h = rec_carry(products[turn][s][q.lane], h, results[turn][s][q.lane]);
#pragma unroll
    for (int s = kRecWaves - 1; s >= 0; --s) {
      if (s == q.wave) c = back;
      back = rec_carry(products[turn][s][q.lane], back, gradients[turn][s][q.lane]);
    }
    const f32x2 over = rec_carry(As.first, h, Hs.first), under = rec_carry(As.second, c, Qs.second);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      h[k] = second ? over[k] : h[k];
      c[k] = second ? c[k] : under[k];
    }
    if (plain)
      rec_finish<BF16, COUPLED, true, U>(p, q, e, row, f, rest, v, dh, h, c, done_g, done_x);
    else
      rec_finish<BF16, COUPLED, false, U>(p, q, e, row, f, rest, v, dh, h, c, done_g, done_x);
  }
  const int row0 = q.begin + q.first * TR;
  rec_store<BF16, U>(q, dgate, row0, row0 + lane_row, false, done_g);
  rec_store<BF16, U>(q, dx, row0, row0 + lane_row, false, done_x);
}

// (A, Q) of each span but an axis's first.
template <bool BF16>
__global__ void __launch_bounds__(kRecThreads) recurrence_dgrad_span_kernel(RecParams p) {
  constexpr int U = kRecRunRows, TR = kRecTileRows;
  __shared__ f32x2 products[kRecRuns][32], gradients[kRecRuns][32];
  const RecPlace q = rec_place(p);
  if (q.first >= q.last || q.span == 0) return;
  const int run_row = q.begin + q.first * TR + q.run * p.span_tiles * U, safe_row = min(run_row, q.end - 1);
  const RecRun<BF16> gates(p.gate, safe_row, q.safe), dhs(p.dh, safe_row, q.safe);
  const RecRun<BF16>* const in[2] = {&gates, &dhs};
  const bool whole = q.begin + (q.first + p.span_tiles) * TR <= q.end;
  const bool inside = rec_inside(p, q, q.begin + q.first * TR, p.span_tiles * TR);
  f32x2 A = {1.f, 1.f}, Q = {0.f, 0.f};
  RecFetch<BF16, 2, U> next;
  next.run(p, q, in, run_row, (p.span_tiles - 1) * U, whole);
  for (int at = (p.span_tiles - 1) * U; at >= 0; at -= U) {
    const int row = run_row + at;
    RecEdges e{};
    if (!inside) e = rec_edges<U>(p, q, row, next.sq);
    const bool plain = inside || rec_ordinary(e, U);
    f32x2 f[U], rest[U];
    Raw2<BF16> dh[U];
    if (plain)
      rec_weights<BF16, true, U>(e, next.raw[0], f, rest);
    else
      rec_weights<BF16, false, U>(e, next.raw[0], f, rest);
#pragma unroll
    for (int u = 0; u < U; ++u) dh[u] = next.raw[1][u];
    if (at > 0) next.run(p, q, in, run_row, at - U, whole);
    if (plain)
      rec_compose_back<BF16, true, U>(p, q, e, row, f, dh, A, Q);
    else
      rec_compose_back<BF16, false, U>(p, q, e, row, f, dh, A, Q);
  }
  products[q.run][q.lane] = A;
  gradients[q.run][q.lane] = Q;
  __syncthreads();
  if (q.run != kRecRuns - 1 || !q.live) return;
#pragma unroll
  for (int s = kRecRuns - 2; s >= 0; --s)
  {
    Q = rec_carry(products[s][q.lane], Q, gradients[s][q.lane]);
    A = rec_product(A, products[s][q.lane]);
  }
  float* at = p.summary + (q.span0 + q.span) * 2 * p.D + q.channel;
  *(f32x2*)at = A;
  *(f32x2*)(at + p.D) = Q;
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

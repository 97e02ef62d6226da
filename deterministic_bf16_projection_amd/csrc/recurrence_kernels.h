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
// H1 + H2).  A workgroup owns 128 channels, two to a lane, and goes through its
// rows by tiles: each of its waves composes a run of eight rows, the waves'
// (A, H) meet in LDS, every wave finds the state before its run, and then each
// row's, from values that stayed in registers: the rows are read once.  A is
// zero only if some f is: products that underflow are held at the smallest
// number, 2^-149, so that an infinite state stays infinite.  Below the normal
// numbers each multiplication of A is off by up to that: a finite state c that
// passes whole runs, by |c| 2^-149 for every row of them.
//
// Rows are grouped in axes, each a whole sequence or several short ones; a
// sequence's first row takes f = 0 there and the initial state into its input.
// Where there are too few axes and channels to fill the device, an axis is cut
// into spans: a first launch finds each span's (A, H), and the second starts a
// span from the composition of those before it, for 5 passes over memory
// instead of 3.  All of it depends on sizes alone, and every sum runs in a
// fixed order.
//
// The forward pass can keep the FP32 state before every 64 rows (1/32 of h's
// size in BF16); the gradient recomputes the states in between from them
// instead of reading rounded ones: 3 reads and 2 writes, not 4 and 2.
//
// Bound by memory, in this order of access: a kernel that only copies so, rows of
// 256 bytes walked by one workgroup each, reaches 5.5 TB/s with two reads and a
// write and 5.3 with three and two (rows of 128 bytes, two reads and a write:
// 4.5).  8 sequences of 4096 rows, 4096 channels, BF16: forward 155 us (5.2
// TB/s), gradient 254 us (5.3).  One sequence of 65536 rows, 2048 channels: 239 us
// for its two launches (5.6 TB/s of their five passes).  What it came from:
// forward 204 us and gradient 477 without a store a tile late and scalar row
// addresses, 180 and 307 with them; 159 with runs of 256-byte rows; gradient 313
// with one copy of the work for runs with and without edges, 252 with two.
#pragma once
#include <type_traits>

#include "rows8.h"

namespace dpg {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

constexpr int kRecChannels = 128;
// Runs of a tile (waves), and rows of a run: forward and in the launches over
// spans, and of the gradient, whose registers allow two waves to a SIMD
// (forward with eight waves too: 157 us where sixteen take 155).
constexpr int kRecWaves = 16, kRecRows = 8;
constexpr int kRecGradWaves = 8, kRecGradRows = 8;
constexpr int kRecThreads = 64 * kRecWaves, kRecGradThreads = 64 * kRecGradWaves;
constexpr int kRecTileRows = kRecWaves * kRecRows;
constexpr int kRecCarryRows = kRecGradWaves * kRecGradRows;
static_assert(kRecTileRows == 2 * kRecCarryRows, "two carries to a forward tile");

struct RecParams {
  Rows8 gate, x, h, dh, dgate, dx;
  const float* state;      // [S, D] before the first rows, or null: zeros
  float* state_out;        // [S, D] after the last rows, or null
  const float* dstate;     // [S, D] gradient of the latter, or null: zeros
  float* dstate_out;       // [S, D] gradient of the former, or null
  float* carries;          // [axes * 2 tiles, D]
  float* summary;          // [axes * spans, 2, D]: A, then H or Q
  const int32_t* seq;      // packed: each row's sequence, -1 behind the last
  int R, D, length;        // length: of every sequence, where they are not packed
  int axis_rows, tiles;    // of an axis
  int span_tiles, spans;
  int blocks;              // of 128 channels
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
// v, and NaN where the weight f (0 to 1) is, which a term of 0 would hide in
// weighted() and the minimum in 1 - f
__device__ __forceinline__ float or_nan(float f, float v) { return fmaf(f, 0.f, v); }
// a product of weights: 0 exactly where the least of them is, else at least 2^-149,
// the smallest number above 0, which is no more than a product's own rounding
__device__ __forceinline__ float held(float product, float least) { return fmaxf(product, fminf(least, 0x1p-149f)); }
// two runs, the first's values first
__device__ __forceinline__ f32x2 rec_carry(const f32x2& A, const f32x2& c, const f32x2& H) {
  return f32x2{carry_on(A[0], c[0], H[0]), carry_on(A[1], c[1], H[1])};
}
__device__ __forceinline__ f32x2 rec_product(const f32x2& A, const f32x2& B) {
  return f32x2{held(A[0] * B[0], fminf(A[0], B[0])), held(A[1] * B[1], fminf(A[1], B[1]))};
}

// f and 1 - f, each to its own relative accuracy.  With e = exp(-gate), f = 1 /
// (1 + e) and 1 - f = e f.  For BF16 inputs the exponential and the reciprocal of
// the hardware (one unit in the last place) do.  That reciprocal gives 0 for
// denormal numbers, so f is 0 from e = 2^126 on (gates below about -87.3), where
// e f is 0, or infinity times 0: 1 - f is 1 there (a compare and a select more: 408
// us for the training batch that took 406).  FP32 ones take
// the smaller weight from exp(-|gate|), whose exponent gets its rounding error
// back (up to |gate| 2^-24 of the result), and a Newton step.
template <bool BF16>
__device__ __forceinline__ void gate_weights(float g, float& f, float& rest) {
  if (BF16) {
    const float e = __builtin_amdgcn_exp2f(g * -1.44269504f);
    f = __builtin_amdgcn_rcpf(1.f + e);
    rest = f > 0.f ? __builtin_amdgcn_fmed3f(e * f, 0.f, 1.f) : 1.f;
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
// Everything but the channels is the same for a wave and lies in scalar
// registers.
struct RecPlace {
  int lane, wave;
  int channel, safe;      // first of the lane's two channels, and one to load from
  bool live;              // the channels exist
  int begin, end;         // rows of the axis
  int first, last;        // tiles of the span
  int span;
  int64_t carry0, span0;  // of the axis
};
__device__ __forceinline__ RecPlace rec_place(const RecParams& p) {
  RecPlace q;
  const int id = blockIdx.x, rest = id / p.blocks, axis = rest / p.spans;
  q.span = rest - axis * p.spans;
  q.lane = threadIdx.x & 63;
  q.wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  q.channel = (id - rest * p.blocks) * kRecChannels + 2 * q.lane;
  q.live = q.channel < p.D;
  q.safe = min(q.channel, p.D - 2);
  q.begin = axis * p.axis_rows;
  q.end = min(p.R - q.begin, p.axis_rows) + q.begin;
  q.first = q.span * p.span_tiles;
  q.last = min(q.first + p.span_tiles, (q.end - q.begin + kRecTileRows - 1) / kRecTileRows);
  q.carry0 = (int64_t)axis * 2 * p.tiles;
  q.span0 = (int64_t)axis * p.spans;
  return q;
}

// One matrix as a lane sees it: a row's address lies in scalar registers, to
// which an access adds the lane's offset by itself.  The empty statements keep
// the compiler from adding both up in vector registers (of the offset it would
// otherwise make 64 bits before the loop).  NT: past the caches.
template <bool BF16, bool NT>
struct RecRows {
  typedef __attribute__((address_space(1))) char* Bytes;
  typedef __attribute__((address_space(1))) Raw2<BF16>* Values;
  uint64_t data;
  int64_t pitch;     // bytes of a row
  unsigned lane;     // byte of the lane's first channel
  __device__ __forceinline__ RecRows(const Rows8& m, int channel)
      : data((uint64_t)m.data), pitch(m.ld * (BF16 ? 2 : 4)), lane((unsigned)channel * (BF16 ? 2u : 4u)) {}

  // U rows from `row` on; those behind the axis are its last one
  template <int U>
  __device__ __forceinline__ void load(const RecPlace& q, int row, Raw2<BF16> (&v)[U]) const {
    unsigned offset = lane;
    uint64_t base = data + min(row, q.end - 1) * pitch;
    const auto get = [&](int u) {
      asm volatile("" : "+s"(base), "+v"(offset));
      const Values at = (Values)((Bytes)base + offset);
      v[u] = NT ? __builtin_nontemporal_load(at) : *at;
    };
    if (row + U <= q.end) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        get(u);
        base += pitch;
      }
    } else {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        get(u);
        base += row + u + 1 < q.end ? pitch : 0;
      }
      asm volatile("" ::: "memory");  // not one set of loads for both branches
    }
  }
  // those of U rows that exist
  template <int U>
  __device__ __forceinline__ void store(const RecPlace& q, int row, const Raw2<BF16> (&v)[U]) const {
    if (!q.live) return;
    unsigned offset = lane;
    uint64_t base = data + row * pitch;
    const auto put = [&](int u) {
      asm volatile("" : "+s"(base), "+v"(offset));
      const Values at = (Values)((Bytes)base + offset);
      if (NT)
        __builtin_nontemporal_store(v[u], at);
      else
        *at = v[u];
      base += pitch;
    };
    if (row + U <= q.end) {
#pragma unroll
      for (int u = 0; u < U; ++u) put(u);
    } else {
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (row + u < q.end) put(u);
      asm volatile("" ::: "memory");
    }
  }
};

// U rows of N matrices, loaded ahead of their use.
template <bool BF16, bool NT, int N, int U>
struct RecFetch {
  Raw2<BF16> raw[N][U];
  int before, at;  // packed: lane l holds the sequences of rows l - 1 and l; rows outside the axis have -2
  __device__ __forceinline__ void operator()(const RecParams& p, const RecPlace& q, const RecRows<BF16, NT>* const (&m)[N],
                                             int row) {
#pragma unroll
    for (int i = 0; i < N; ++i) m[i]->load(q, row, raw[i]);
    if (p.seq) {
      const int r = row + q.lane;
      before = q.lane <= U && r >= 1 && r <= q.end ? p.seq[r - 1] : -2;
      at = q.lane <= U && r < q.end ? p.seq[r] : -2;
    }
  }
};

// What is special about a run's rows: bit u for row u.
struct RecEdges {
  unsigned live, start, last;
  int seq;     // sequence of the first row (not packed)
  bool plain;  // all rows live, none starts or ends a sequence
};
// Work that depends on a run's edges, with a copy for plain runs, in which the
// compiler leaves the questions out.
template <int U, class F>
__device__ __forceinline__ void rec_by_edges(const RecEdges& e, const F& work) {
  if (e.plain)
    work(RecEdges{(1u << U) - 1, 0, 0, 0, true});
  else
    work(e);
}
template <int U>
__device__ __forceinline__ RecEdges rec_edges(const RecParams& p, const RecPlace& q, int row, int before, int at) {
  RecEdges e{0, 0, 0, 0, false};
  constexpr unsigned full = (1u << U) - 1;
  if (p.seq) {
    const unsigned differ = (unsigned)__ballot(at != before);
    e.live = (unsigned)__ballot(at >= 0) & full;
    e.start = differ & e.live;
    e.last = (differ >> 1) & e.live;
  } else if (p.length == p.axis_rows && row > q.begin && row + U < q.end) {
    e.live = full;  // an axis is a sequence, and these rows are inside
  } else {
    const int n = min(max(q.end - row, 0), U);
    e.live = (1u << n) - 1;
    e.seq = row / p.length;
    int place = row - e.seq * p.length;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      e.start |= place == 0 ? 1u << u : 0;
      ++place;
      e.last |= place == p.length ? 1u << u : 0;
      place = place == p.length ? 0 : place;
    }
    e.start &= e.live;
    e.last &= e.live;
  }
  e.plain = e.live == full && (e.start | e.last) == 0;
  return e;
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

// --------------------------------------------------------------- forward --
// f and b = w x of a run's rows.  Where the run is not plain, rows without a
// sequence get zeros, and a first row f = 0 and the initial state in b.
template <bool BF16, bool COUPLED, int U>
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
      b[u][k] = or_nan(fk, COUPLED ? weighted(rest, v[k]) : v[k]);
    }
  }
  if (e.plain) return;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const f32x2 zero = {0.f, 0.f};
    if (e.start >> u & 1) {
      if (p.state) b[u] = rec_carry(f[u], rec_state(p.state, p, e, q, row, u), b[u]);
      f[u] = zero;
    }
    if (!(e.live >> u & 1)) f[u] = b[u] = zero;
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

template <bool BF16, bool COUPLED, bool NT>
__global__ void __launch_bounds__(kRecThreads) recurrence_kernel(RecParams p) {
  constexpr int U = kRecRows, TR = kRecTileRows;
  __shared__ f32x2 products[2][kRecWaves][64], results[2][kRecWaves][64];
  const RecPlace q = rec_place(p);
  if (q.first >= q.last) return;
  f32x2 carry = {0.f, 0.f};
  for (int s = 0; s < q.span; ++s) {
    const float* at = p.summary + (q.span0 + s) * 2 * p.D + q.safe;
    carry = rec_carry(*(const f32x2*)at, carry, *(const f32x2*)(at + p.D));
  }
  const RecRows<BF16, NT> gates(p.gate, q.safe), xs(p.x, q.safe), out(p.h, q.channel);
  const RecRows<BF16, NT>* const in[2] = {&gates, &xs};
  RecFetch<BF16, NT, 2, U> next;
  Raw2<BF16> done[U];
  f32x2 start = carry;  // the state before the run of the tile before
  int row = q.begin + q.first * TR + q.wave * U;
  next(p, q, in, row);
  for (int tile = q.first; tile < q.last; ++tile, row += TR) {
    const int turn = tile & 1;
    const RecEdges e = rec_edges<U>(p, q, row, next.before, next.at);
    f32x2 f[U], b[U];
    rec_by_edges<U>(e, [&](const RecEdges& g) {
      rec_inputs<BF16, COUPLED, U>(p, q, g, row, next.raw[0], next.raw[1], f, b);
    });
    // Memory operations are waited for in the order of their issue: stores that
    // came after the next tile's loads would have to end before those are used.
    // So a tile's results are stored one tile later, before the loads.
    const auto put = [&](int t, int r) {
      out.store(q, r, done);
      if (p.carries && q.wave % (kRecWaves / 2) == 0 && q.live)
        *(f32x2*)(p.carries + (q.carry0 + 2 * t + q.wave / (kRecWaves / 2)) * p.D + q.channel) = start;
    };
    if (tile > q.first) put(tile - 1, row - TR);
    if (tile + 1 < q.last) next(p, q, in, row + TR);
    f32x2 A = {1.f, 1.f}, H = {0.f, 0.f};
    rec_compose<U>(f, b, A, H);
    // two places in LDS by turns: one barrier a tile
    products[turn][q.wave][q.lane] = A;
    results[turn][q.wave][q.lane] = H;
    __syncthreads();
    f32x2 h = carry;
#pragma unroll
    for (int s = 0; s < kRecWaves; ++s) {
      if (s == q.wave) h = carry;
      carry = rec_carry(products[turn][s][q.lane], carry, results[turn][s][q.lane]);
    }
    start = h;
    rec_by_edges<U>(e, [&](const RecEdges& g) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        h = rec_carry(f[u], h, b[u]);
        done[u] = pack2<BF16>(h);
        if (g.last >> u & 1) rec_put_state(p.state_out, p, g, q, row, u, h);
      }
    });
    if (tile + 1 == q.last) put(tile, row);
  }
}

// (A, H) of each span but an axis's last, whose rows' end nothing follows.  No
// order is needed until the end, so that each wave takes U span_tiles rows in
// one piece.
template <bool BF16, bool COUPLED>
__global__ void __launch_bounds__(kRecThreads) recurrence_span_kernel(RecParams p) {
  constexpr int U = kRecRows;
  __shared__ f32x2 products[kRecWaves][64], results[kRecWaves][64];
  const RecPlace q = rec_place(p);
  if (q.first >= q.last || q.span == p.spans - 1) return;
  const RecRows<BF16, false> gates(p.gate, q.safe), xs(p.x, q.safe);
  const RecRows<BF16, false>* const in[2] = {&gates, &xs};
  f32x2 A = {1.f, 1.f}, H = {0.f, 0.f};
  RecFetch<BF16, false, 2, U> next;
  int row = q.begin + q.first * kRecTileRows + q.wave * p.span_tiles * U;
  const int end = row + p.span_tiles * U;
  next(p, q, in, row);
  for (; row < end; row += U) {
    const RecEdges e = rec_edges<U>(p, q, row, next.before, next.at);
    f32x2 f[U], b[U];
    rec_by_edges<U>(e, [&](const RecEdges& g) {
      rec_inputs<BF16, COUPLED, U>(p, q, g, row, next.raw[0], next.raw[1], f, b);
    });
    if (row + U < end) next(p, q, in, row + U);
    rec_compose<U>(f, b, A, H);
  }
  products[q.wave][q.lane] = A;
  results[q.wave][q.lane] = H;
  __syncthreads();
  if (q.wave != 0 || !q.live) return;
#pragma unroll
  for (int s = 1; s < kRecWaves; ++s) {
    H = rec_carry(products[s][q.lane], H, results[s][q.lane]);
    A = rec_product(A, products[s][q.lane]);
  }
  float* at = p.summary + (q.span0 + q.span) * 2 * p.D + q.channel;
  *(f32x2*)at = A;
  *(f32x2*)(at + p.D) = H;
}

// Sequences of one row each, a generation step: nothing to compose, eight
// channels to a thread and one row after the other.
template <bool BF16, bool COUPLED>
__global__ void __launch_bounds__(256) recurrence_step_kernel(RecParams p) {
  const int groups = p.D >> 3;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < (int64_t)p.R * groups; i += (int64_t)gridDim.x * 256) {
    const int64_t row = i / groups;
    const int group = (int)(i - row * groups);
    float g[8], x[8], h[8];
    const Raw8<BF16> gates = load8<BF16>(p.gate, row, group), xs = load8<BF16>(p.x, row, group);
    f32x4 c[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
    const int64_t at = row * p.D + 8 * group;
    if (p.state) {
      c[0] = *(const f32x4*)(p.state + at);
      c[1] = *(const f32x4*)(p.state + at + 4);
    }
    unpack8(gates, g);
    unpack8(xs, x);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float f, rest;
      gate_weights<BF16>(g[j], f, rest);
      h[j] = carry_on(f, c[j >> 2][j & 3], or_nan(f, COUPLED ? weighted(rest, x[j]) : x[j]));
    }
    store8<BF16>(p.h, row, group, h);
    if (p.state_out) {
      *(f32x4*)(p.state_out + at) = f32x4{h[0], h[1], h[2], h[3]};
      *(f32x4*)(p.state_out + at + 4) = f32x4{h[4], h[5], h[6], h[7]};
    }
  }
}

// -------------------------------------------------------------- gradient --
// f and 1 - f of a run's rows, zeros at those without a sequence.
template <bool BF16, int U>
__device__ __forceinline__ void rec_weights(const RecEdges& e, const Raw2<BF16> (&gate)[U], f32x2 (&f)[U],
                                            f32x2 (&rest)[U]) {
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const f32x2 g = unpack2(gate[u]);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float fk, rk;
      gate_weights<BF16>(g[k], fk, rk);
      f[u][k] = fk;
      rest[u][k] = rk;
    }
  }
  if (e.plain) return;
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (!(e.live >> u & 1)) f[u] = rest[u] = f32x2{0.f, 0.f};
}

// dh of row u, with dstate at a last row
template <bool BF16>
__device__ __forceinline__ f32x2 rec_dh(const RecParams& p, const RecPlace& q, const RecEdges& e, int row, int u,
                                        const Raw2<BF16>& raw) {
  f32x2 d = unpack2(raw);
  if (e.plain) return d;
  if (e.last >> u & 1) {
    const f32x2 more = rec_state(p.dstate, p, e, q, row, u);
    d = f32x2{d[0] + more[0], d[1] + more[1]};
  }
  if (!(e.live >> u & 1)) d = f32x2{0.f, 0.f};
  return d;
}

// A run backwards takes c, what reaches it from the rows after it, to A c + Q;
// A is the same product as forward.
template <bool BF16, int U>
__device__ __forceinline__ void rec_compose_back(const RecParams& p, const RecPlace& q, const RecEdges& e, int row,
                                                 const f32x2 (&f)[U], const Raw2<BF16> (&grad)[U], f32x2& A, f32x2& Q) {
  f32x2 least = A;
#pragma unroll
  for (int u = U - 1; u >= 0; --u) {
    const f32x2 dh = rec_dh<BF16>(p, q, e, row, u, grad[u]);
    f32x2 fu = f[u];
    if (e.start >> u & 1) fu = f32x2{0.f, 0.f};
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      A[k] *= fu[k];
      least[k] = fminf(least[k], fu[k]);
      Q[k] = weighted(fu[k], or_nan(fu[k], dh[k] + Q[k]));
    }
  }
#pragma unroll
  for (int k = 0; k < 2; ++k) A[k] = held(A[k], least[k]);
}

// The run's states from h, the one before it: before[u] is the state that row
// u starts from.  Returns the last row's.  Rows without a sequence, which no
// other follows, may give anything.
template <bool BF16, bool COUPLED, int U>
__device__ __forceinline__ f32x2 rec_states(const RecParams& p, const RecPlace& q, const RecEdges& e, int row,
                                            const f32x2 (&f)[U], const f32x2 (&rest)[U], const Raw2<BF16> (&x)[U],
                                            f32x2 h, f32x2 (&before)[U]) {
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const f32x2 v = unpack2(x[u]);
    if (e.start >> u & 1) h = rec_state(p.state, p, e, q, row, u);
    before[u] = h;
#pragma unroll
    for (int k = 0; k < 2; ++k) h[k] = carry_on(f[u][k], h[k], or_nan(f[u][k], COUPLED ? weighted(rest[u][k], v[k]) : v[k]));
  }
  return h;
}

template <bool BF16, bool COUPLED, bool NT>
__global__ void __launch_bounds__(kRecGradThreads, 2) recurrence_dgrad_kernel(RecParams p) {
  constexpr int U = kRecGradRows, TR = kRecCarryRows;
  __shared__ f32x2 products[2][kRecGradWaves][64], results[2][kRecGradWaves][64], gradients[2][kRecGradWaves][64];
  const RecPlace q = rec_place(p);
  if (q.first >= q.last) return;
  f32x2 back = {0.f, 0.f};  // what reaches the tile from the rows after it
  for (int s = p.spans - 1; s > q.span; --s) {
    const float* at = p.summary + (q.span0 + s) * 2 * p.D + q.safe;
    back = rec_carry(*(const f32x2*)at, back, *(const f32x2*)(at + p.D));
  }
  const RecRows<BF16, NT> gates(p.gate, q.safe), xs(p.x, q.safe), dhs(p.dh, q.safe);
  const RecRows<BF16, NT> dgate(p.dgate, q.channel), dx(p.dx, q.channel);
  const RecRows<BF16, NT>* const in[3] = {&gates, &xs, &dhs};
  const auto carried = [&](int tile) { return *(const f32x2*)(p.carries + (q.carry0 + tile) * p.D + q.safe); };
  const int first = 2 * q.first, last = min(2 * q.last, (q.end - q.begin + TR - 1) / TR);  // tiles of 64 rows
  RecFetch<BF16, NT, 3, U> next;
  Raw2<BF16> done_g[U], done_x[U];
  int row = q.begin + (last - 1) * TR + q.wave * U;
  next(p, q, in, row);
  f32x2 carry = carried(last - 1);
  for (int tile = last - 1; tile >= first; --tile, row -= TR) {
    const int turn = tile & 1;
    const RecEdges e = rec_edges<U>(p, q, row, next.before, next.at);
    f32x2 f[U], rest[U], before[U];
    Raw2<BF16> v[U], dh[U];
    rec_by_edges<U>(e, [&](const RecEdges& g) { rec_weights<BF16, U>(g, next.raw[0], f, rest); });
#pragma unroll
    for (int u = 0; u < U; ++u) {
      v[u] = next.raw[1][u];
      dh[u] = next.raw[2][u];
    }
    f32x2 h = carry;
    // one tile late, before the next loads, as in the forward pass
    const auto put = [&](int r) {
      dgate.store(q, r, done_g);
      dx.store(q, r, done_x);
    };
    if (tile + 1 < last) put(row + TR);
    if (tile > first) {
      next(p, q, in, row - TR);
      carry = carried(tile - 1);
    }
    f32x2 A = {1.f, 1.f}, Q = {0.f, 0.f}, H = {0.f, 0.f};
    rec_by_edges<U>(e, [&](const RecEdges& g) {
      rec_compose_back<BF16, U>(p, q, g, row, f, dh, A, Q);
      H = rec_states<BF16, COUPLED, U>(p, q, g, row, f, rest, v, H, before);
    });
    products[turn][q.wave][q.lane] = A;
    results[turn][q.wave][q.lane] = H;
    gradients[turn][q.wave][q.lane] = Q;
    __syncthreads();
    f32x2 c = back;
#pragma unroll
    for (int s = 0; s < kRecGradWaves - 1; ++s)
      if (s < q.wave) h = rec_carry(products[turn][s][q.lane], h, results[turn][s][q.lane]);
#pragma unroll
    for (int s = kRecGradWaves - 1; s >= 0; --s) {
      if (s == q.wave) c = back;
      back = rec_carry(products[turn][s][q.lane], back, gradients[turn][s][q.lane]);
    }
    rec_by_edges<U>(e, [&](const RecEdges& g) {
      rec_states<BF16, COUPLED, U>(p, q, g, row, f, rest, v, h, before);
#pragma unroll
      for (int u = U - 1; u >= 0; --u) {
        const f32x2 xu = unpack2(v[u]), du = rec_dh<BF16>(p, q, g, row, u, dh[u]);
        f32x2 out_x, out_g;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float plain = du[k] + c[k], r = or_nan(f[u][k], plain);
          out_x[k] = COUPLED ? weighted(rest[u][k], r) : plain;
          out_g[k] = weighted(f[u][k] * rest[u][k], r * (COUPLED ? before[u][k] - xu[k] : before[u][k]));
          c[k] = weighted(f[u][k], r);
        }
        done_x[u] = pack2<BF16>(out_x);
        done_g[u] = pack2<BF16>(out_g);
        if (g.start >> u & 1) {
          rec_put_state(p.dstate_out, p, g, q, row, u, c);
          c = f32x2{0.f, 0.f};
        }
      }
    });
    if (tile == first) put(row);
  }
}

// (A, Q) of each span but an axis's first.
template <bool BF16>
__global__ void __launch_bounds__(kRecThreads) recurrence_dgrad_span_kernel(RecParams p) {
  constexpr int U = kRecRows;
  __shared__ f32x2 products[kRecWaves][64], gradients[kRecWaves][64];
  const RecPlace q = rec_place(p);
  if (q.first >= q.last || q.span == 0) return;
  const RecRows<BF16, false> gates(p.gate, q.safe), dhs(p.dh, q.safe);
  const RecRows<BF16, false>* const in[2] = {&gates, &dhs};
  f32x2 A = {1.f, 1.f}, Q = {0.f, 0.f};
  RecFetch<BF16, false, 2, U> next;
  const int begin = q.begin + q.first * kRecTileRows + q.wave * p.span_tiles * U;
  int row = begin + (p.span_tiles - 1) * U;
  next(p, q, in, row);
  for (; row >= begin; row -= U) {
    const RecEdges e = rec_edges<U>(p, q, row, next.before, next.at);
    f32x2 f[U], rest[U];
    Raw2<BF16> dh[U];
    rec_by_edges<U>(e, [&](const RecEdges& g) { rec_weights<BF16, U>(g, next.raw[0], f, rest); });
#pragma unroll
    for (int u = 0; u < U; ++u) dh[u] = next.raw[1][u];
    if (row > begin) next(p, q, in, row - U);
    rec_by_edges<U>(e, [&](const RecEdges& g) { rec_compose_back<BF16, U>(p, q, g, row, f, dh, A, Q); });
  }
  products[q.wave][q.lane] = A;
  gradients[q.wave][q.lane] = Q;
  __syncthreads();
  if (q.wave != kRecWaves - 1 || !q.live) return;
#pragma unroll
  for (int s = kRecWaves - 2; s >= 0; --s) {
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

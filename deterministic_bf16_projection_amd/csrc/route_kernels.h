// Routing kernels: the choice of experts, the stable order of the chosen
// (token, slot) pairs by expert, rows moved into that order and back, and the
// gradients.
#pragma once
#include "device_common.h"

namespace dpg {

constexpr int kRouteThreads = 1024;
constexpr int kRouteMaxExperts = 512;
constexpr int kRouteMaxTopK = 32;
constexpr int kRouteRound = 64;          // tokens of a block that are chosen for at once

// -------------------------------------------------------------- choice --
struct RouteParams {
  const float* logits;
  int64_t ldl;
  int64_t T;
  int E, k, renorm;
  int tokens_per_block;  // blocks of consecutive tokens: 16, or a multiple of kRouteRound
  int blocks, hist_ld;
  int32_t* experts;      // [T, k]
  float* weights;        // [T, k]
  int32_t* offsets;      // [E + 1]
  int32_t* rows;         // [T k]
  int32_t* positions;    // [T, k]
  uint16_t* hist;        // [E, hist_ld]: counts of the blocks
};

// One token by LANES lanes: a row of 16, four tokens to a wave, or the whole
// wave.  The logits sit in registers, lane l holding the experts l, LANES + l,
// ...; each of the k rounds takes the maximum over the lanes and, among equal
// ones, the lowest expert.  Only a logit of -infinity masks an expert; a NaN is
// never chosen but makes the token's weights NaN.  Lane l returns the choices
// l and (rows of 16) 16 + l.
//
// Many tokens are bound by the rounds' instructions, of which four tokens in a
// wave share most (16384 tokens of 256 experts, 8 chosen: 20 us with a token
// to a wave, 15 with rows).  A few tokens wait for their dependent steps,
// which are fewer with 64 lanes (one token, order included: 6.1 us, 7.5 with a
// row; 4.2 since few slots are ordered without counts).
template <int LANES, int NR>
__device__ __forceinline__ void choose(const RouteParams& p, int64_t t, bool live, int lane, int (&expert)[2],
                                       float (&weight)[2]) {
  constexpr bool ROW = LANES == 16;
  static_assert(ROW || LANES == 64, "a row or a wave");
  const auto lanes_max = [](float x) { return ROW ? row_max(x) : wave_max(x); };
  const auto lanes_sum = [](float x) { return ROW ? row_sum(x) : wave_sum(x); };
  const float kMasked = -__builtin_inff();
  const int sub = lane & (LANES - 1);
  float v[NR];
  bool nan = false;
#pragma unroll
  for (int r = 0; r < NR; ++r) {
    const int i = r * LANES + sub;
    const float x = live && i < p.E ? p.logits[t * p.ldl + i] : kMasked;
    nan |= x != x;
    v[r] = x != x ? kMasked : x;
  }
  const uint64_t nans = __ballot(nan);
  const bool any_nan = ROW ? ((nans >> (lane & 48)) & 0xffff) != 0 : nans != 0;
  float local = v[0];
#pragma unroll
  for (int r = 1; r < NR; ++r) local = fmaxf(local, v[r]);
  const float top = lanes_max(local);
  float total = 0.f;
  if (!p.renorm) {
#pragma unroll
    for (int r = 0; r < NR; ++r) total += top > kMasked ? expf(v[r] - top) : 0.f;
    total = lanes_sum(total);
  }
  float mine[2] = {kMasked, kMasked};
  expert[0] = expert[1] = -1;
  float m = top;
#pragma unroll
  for (int half = 0; half < (ROW ? 2 : 1); ++half) {
    for (int j = LANES * half; j < min(p.k, LANES * half + LANES); ++j) {
      if (__ballot(m > kMasked) == 0) break;  // all the wave's tokens are out of experts
      unsigned at = 0xffffu;
      if constexpr (ROW) {
#pragma unroll
        for (int r = NR - 1; r >= 0; --r) at = v[r] == m ? (unsigned)(r * 16 + sub) : at;
        at = row_min(at);
      } else {
#pragma unroll
        for (int r = NR - 1; r >= 0; --r) {
          const uint64_t eq = __ballot(v[r] == m);
          if (eq) at = (unsigned)(r * 64 + __builtin_ctzll(eq));
        }
      }
      if (sub == (j & (LANES - 1)) && m > kMasked) {
        expert[half] = (int)at;
        mine[half] = m;
      }
      const unsigned d = at - (unsigned)sub;
#pragma unroll
      for (int r = 0; r < NR; ++r) v[r] = d == (unsigned)(r * LANES) ? kMasked : v[r];
      local = v[0];
#pragma unroll
      for (int r = 1; r < NR; ++r) local = fmaxf(local, v[r]);
      m = lanes_max(local);
    }
  }
  const float e0 = expert[0] >= 0 ? expf(mine[0] - top) : 0.f, e1 = expert[1] >= 0 ? expf(mine[1] - top) : 0.f;
  if (p.renorm) total = lanes_sum(e0 + e1);
  weight[0] = expert[0] < 0 ? 0.f : any_nan ? __builtin_nanf("") : e0 / total;
  weight[1] = expert[1] < 0 ? 0.f : any_nan ? __builtin_nanf("") : e1 / total;
}

// --------------------------------------------------------- stable order --
// Slots (token * k + slot) of one block, ranked by (expert, slot): `start[e]`
// is the place of the block's first slot of expert e (experts in ascending
// order, unused slots last as expert E).  Each wave owns a run of consecutive
// slots; the counts per (wave, expert) in LDS, summed over the waves before,
// give every wave its own running places, and inside a wave the lanes with
// equal experts are found with one ballot per bit.  Integer counts: no order
// matters, the result is the same every time.  `experts` are the block's
// (unused: negative), in LDS or in memory.
__device__ __forceinline__ void scatter_block(const RouteParams& p, int64_t slot0, int slots, const int* experts,
                                              const int* start, int* counts /* waves x (E + 1) */, int tid) {
  const int keys = p.E + 1;
  const int threads = blockDim.x, waves = threads >> 6;
  const int lane = tid & 63, wave = tid >> 6;
  const int per_wave = ((slots + waves - 1) / waves + 63) & ~63;
  const int s0 = wave * per_wave, s1 = min(slots, s0 + per_wave);
  for (int i = tid; i < waves * keys; i += threads) counts[i] = 0;
  __syncthreads();
  for (int s = s0 + lane; s < s1; s += 64) {
    const int e = experts[s];
    atomicAdd(&counts[wave * keys + (e < 0 ? p.E : e)], 1);
  }
  __syncthreads();
  for (int key = tid; key < keys; key += threads) {
    int at = start[key];
    for (int w = 0; w < waves; ++w) {
      const int n = counts[w * keys + key];
      counts[w * keys + key] = at;
      at += n;
    }
  }
  __syncthreads();
  const int bits = 32 - __builtin_clz(keys);
  for (int base = s0; base < s1; base += 64) {
    const int s = base + lane;
    const bool live = s < s1;
    int key = p.E;
    if (live) {
      const int e = experts[s];
      key = e < 0 ? p.E : e;
    }
    uint64_t same = __ballot(live);
    for (int b = 0; b < bits; ++b) {
      const uint64_t ones = __ballot((key >> b) & 1);
      same &= (key >> b) & 1 ? ones : ~ones;
    }
    const int rank = __builtin_popcountll(same & ((1ull << lane) - 1));
    volatile int* next = counts + wave * keys + key;
    const int at = live ? *next : 0;
    __builtin_amdgcn_wave_barrier();
    if (live && rank == 0) *next = at + __builtin_popcountll(same);
    __builtin_amdgcn_wave_barrier();
    if (live) {
      p.rows[at + rank] = (int)(slot0 + s);
      p.positions[slot0 + s] = at + rank;
    }
  }
}

// Exclusive prefix of `total` over the experts into `first` (LDS, E + 1 each),
// by the first wave.
__device__ __forceinline__ void prefix_experts(const int* total, int* first, int keys, int lane) {
  const int c = (keys + 63) >> 6;
  int sum = 0;
  for (int i = 0; i < c; ++i) {
    const int key = lane * c + i;
    if (key < keys) sum += total[key];
  }
  int inc = sum;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int v = __shfl_up(inc, d);
    if (lane >= d) inc += v;
  }
  int at = inc - sum;
  for (int i = 0; i < c; ++i) {
    const int key = lane * c + i;
    if (key < keys) {
      const int n = total[key];
      first[key] = at;
      at += n;
    }
  }
}

// The order of at most 64 slots: each thread counts the slots before its own,
// and before its expert's first.
__device__ __forceinline__ void order_few(const RouteParams& p, int slots, const int* experts, int tid) {
  if (tid < slots) {
    const int key = experts[tid];
    int at = 0;
    for (int i = 0; i < slots; ++i) at += experts[i] < key || (experts[i] == key && i < tid);
    p.rows[at] = tid;
    p.positions[tid] = at;
  }
  for (int key = tid; key <= p.E; key += blockDim.x) {
    int at = 0;
    for (int i = 0; i < slots; ++i) at += experts[i] < key;
    p.offsets[key] = at;
  }
}

// Choice of the block's tokens (threads / LANES at a time) and its counts per
// expert.  With ONE (all tokens in one block, at most kRouteRound) the order
// follows in the same launch.  LDS: counts; with ONE also their prefix, the
// counts per wave and the slots' experts.
template <int LANES, int NR, bool ONE>
__global__ void __launch_bounds__(kRouteThreads) route_choose_kernel(RouteParams p) {
  extern __shared__ int lds[];
  const int keys = p.E + 1;
  const int threads = blockDim.x;
  const int tid = threadIdx.x, lane = tid & 63;
  int* total = lds;
  int* slot_experts = lds + (2 + (threads >> 6)) * keys;  // ONE: unused slots as expert E
  const int64_t slots = p.T * p.k;
  const bool few = ONE && slots <= 64;  // ordered without counts
  if (!few) {
    for (int i = tid; i < keys; i += threads) total[i] = 0;
    __syncthreads();
  }
  const int64_t t0 = (int64_t)blockIdx.x * p.tokens_per_block;
  const int64_t t1 = min(p.T, t0 + p.tokens_per_block);
  for (int64_t first = t0; first < t1; first += threads / LANES) {
    const int64_t t = first + tid / LANES;
    const bool live = t < t1;
    if (__ballot(live) == 0) continue;
    int expert[2];
    float weight[2];
    choose<LANES, NR>(p, t, live, lane, expert, weight);
#pragma unroll
    for (int half = 0; half < (LANES == 16 ? 2 : 1); ++half) {
      const int j = LANES * half + (lane & (LANES - 1));
      if (live && j < p.k) {
        const int key = expert[half] < 0 ? p.E : expert[half];
        p.experts[t * p.k + j] = expert[half];
        p.weights[t * p.k + j] = weight[half];
        if (!few) atomicAdd(&total[key], 1);
        if (ONE) slot_experts[t * p.k + j] = key;
      }
    }
  }
  __syncthreads();
  if (few) {
    order_few(p, (int)slots, slot_experts, tid);
  } else if (ONE) {
    int* first = lds + keys;
    if (tid < 64) prefix_experts(total, first, keys, lane);
    __syncthreads();
    for (int i = tid; i < keys; i += threads) p.offsets[i] = first[i];
    scatter_block(p, 0, (int)slots, slot_experts, first, lds + 2 * keys, tid);
  } else {
    for (int i = tid; i < p.E; i += threads) p.hist[(int64_t)i * p.hist_ld + blockIdx.x] = (uint16_t)total[i];
  }
}

// The order, from the counts of all blocks: each block sums the counts of the
// blocks before it and of all, so that no launch lies between.  32 lanes read
// 256 blocks' counts of one expert; a wave has eight such pairs in flight.
__global__ void __launch_bounds__(kRouteThreads) route_order_kernel(RouteParams p) {
  extern __shared__ int lds[];
  const int keys = p.E + 1;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int* total = lds;
  int* before = lds + keys;
  int* first = lds + 2 * keys;
  const int64_t slot0 = (int64_t)blockIdx.x * p.tokens_per_block * p.k;
  const int64_t slots = p.T * p.k;
  constexpr int G = 8;
  for (int key0 = wave * 2 * G; key0 < p.E; key0 += kRouteThreads / 64 * 2 * G) {
    int all[G], prev[G];
#pragma unroll
    for (int g = 0; g < G; ++g) all[g] = prev[g] = 0;
    for (int b0 = 0; b0 < p.blocks; b0 += 256) {
      const int b = b0 + (lane & 31) * 8;
      u32x4 n[G];
#pragma unroll
      for (int g = 0; g < G; ++g)
        n[g] = b < p.hist_ld
                   ? *(const u32x4*)(p.hist + (int64_t)min(key0 + 2 * g + (lane >> 5), p.E - 1) * p.hist_ld + b)
                   : u32x4{0u, 0u, 0u, 0u};
#pragma unroll
      for (int g = 0; g < G; ++g)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int c = (int)((n[g][i >> 1] >> (16 * (i & 1))) & 0xffffu);
          all[g] += b + i < p.blocks ? c : 0;
          prev[g] += b + i < (int)blockIdx.x ? c : 0;
        }
    }
#pragma unroll
    for (int g = 0; g < G; ++g) {
      all[g] = half_sum(all[g]);
      prev[g] = half_sum(prev[g]);
      const int key = key0 + 2 * g + (lane >> 5);
      if ((lane & 31) == 31 && key < p.E) {
        total[key] = all[g];
        before[key] = prev[g];
      }
    }
  }
  if (tid == 0) total[p.E] = 0;  // the last prefix needs none
  __syncthreads();
  if (wave == 0) prefix_experts(total, first, keys, lane);
  // the unused slots of the blocks before: what their experts did not take
  if (wave == 1) {
    int used = 0;
    for (int i = lane; i < p.E; i += 64) used += before[i];
    used = wave_sum(used);
    if (lane == 0) before[p.E] = (int)(slot0 - used);
  }
  __syncthreads();
  for (int i = tid; i < keys; i += kRouteThreads) {
    if (blockIdx.x == 0) p.offsets[i] = first[i];
    first[i] += before[i];
  }
  __syncthreads();
  scatter_block(p, slot0, (int)min(slots - slot0, (int64_t)p.tokens_per_block * p.k), p.experts + slot0, first,
                lds + 3 * keys, tid);
}

// Gradient of the weights by the logits, one wave per token.  With q the
// softmax the weights come from (over the chosen experts, or over all) and g
// the incoming gradient, zero where nothing was chosen:
//   d logit_i = q_i (g_i - sum_j q_j g_j)
template <int NR>
__global__ void __launch_bounds__(256) route_dgrad_kernel(const float* logits, int64_t ldl, const int32_t* experts,
                                                          const float* weights, const float* dweights, float* dlogits,
                                                          int64_t ldd, int64_t T, int E, int k, int renorm) {
  const int lane = threadIdx.x & 63;
  for (int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); t < T; t += (int64_t)gridDim.x * 4) {
    int e = -1;
    float w = 0.f, d = 0.f;
    if (lane < k) {
      e = experts[t * k + lane];
      if (e >= 0) {
        w = weights[t * k + lane];
        d = w * dweights[t * k + lane];
      }
    }
    const float inner = wave_sum(d);
    float out[NR];
    if (renorm) {
      d -= w * inner;
#pragma unroll
      for (int r = 0; r < NR; ++r) out[r] = 0.f;
    } else {
      float v[NR], local = -__builtin_inff();
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        const int i = r * 64 + lane;
        v[r] = i < E ? logits[t * ldl + i] : -__builtin_inff();
        local = fmaxf(local, v[r]);
      }
      float top = wave_max(local);
      if (top == -__builtin_inff()) top = 0.f;
      float sum = 0.f;
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        v[r] = expf(v[r] - top);
        sum += v[r];
      }
      sum = wave_sum(sum);
      const float scale = sum == 0.f ? 0.f : -inner / sum;
#pragma unroll
      for (int r = 0; r < NR; ++r) out[r] = v[r] * scale;
    }
    for (int j = 0; j < k; ++j) {
      const int ej = __builtin_amdgcn_readlane(e, j);
      const float dj = lane_f32(d, j);
#pragma unroll
      for (int r = 0; r < NR; ++r)
        if (r * 64 + lane == ej) out[r] += dj;
    }
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      const int i = r * 64 + lane;
      if (i < E) dlogits[t * ldd + i] = out[r];
    }
  }
}

// --------------------------------------------------------- moving rows --
// The row kernels go token by token: a token's row is read once for all its
// slots, and slot j's row lies at positions[t, j] of the sorted matrix.  Slots
// without an expert have their places past offsets[E], where rows are never
// read and are written as zeros, all of them: by their own indexes, since the
// matrix may have more rows than there are slots, and a caller's positions
// need not name each.  Positions come from device memory: one outside the
// matrix is left out.
//
// Bound by memory: 16384 tokens, 8 slots each, 4096 columns of BF16 take 247 us
// to dispatch (4.9 TB/s), 223 to combine (5.4) and 444 for the gradients of that
// (5.1) in a training pass, which finds the token side in no cache; called again
// and again on the same rows 206, 212 and 421.
struct RowsParams {
  const void* a;   // [T, H] of the token side
  const void* b;   // [R, H] sorted rows, read
  void* out;       // what is written: [R, H] or [T, H]
  float* dweights; // [T, k]
  const int32_t* positions;
  const int32_t* routed;  // &offsets[E]
  const float* weights;   // [T, k] or null (all one)
  int64_t lda, ldb, ldo;
  int64_t T, R;
  int H, k;
  int lanes_log2;  // threads of one token
};

template <int BYTES>
struct RowVec;
template <>
struct RowVec<2> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void unpack(const u32x4& v, float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __builtin_bit_cast(float, v[i] << 16);
      f[2 * i + 1] = __builtin_bit_cast(float, v[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ u32x4 pack(const float (&f)[8]) {
    return u32x4{pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7])};
  }
};
template <>
struct RowVec<4> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void unpack(const u32x4& v, float (&f)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t bits = v[i];  // a value: a bit cast of the vector element itself reads element 0
      f[i] = __builtin_bit_cast(float, bits);
    }
  }
  static __device__ __forceinline__ u32x4 pack(const float (&f)[4]) {
    return u32x4{__builtin_bit_cast(uint32_t, f[0]), __builtin_bit_cast(uint32_t, f[1]),
                 __builtin_bit_cast(uint32_t, f[2]), __builtin_bit_cast(uint32_t, f[3])};
  }
};

// Slots whose places are read at once, so that a batch of rows is in flight.
constexpr int kSlotBatch = 8;

// STREAM: the sorted rows pass the caches by (see stream_rows).
template <bool STREAM>
__device__ __forceinline__ u32x4 load_row(const u32x4* p) {
  return STREAM ? __builtin_nontemporal_load(p) : *p;
}
template <bool STREAM>
__device__ __forceinline__ void store_row(const u32x4& v, u32x4* p) {
  if constexpr (STREAM)
    __builtin_nontemporal_store(v, p);
  else
    *p = v;
}

// rows of the sorted matrix that slots have: offsets[E] of them, as far as they exist
__device__ __forceinline__ int64_t routed_rows(const RowsParams& p) {
  return min((int64_t)max(*p.routed, 0), p.R);
}

// out[positions[t, j]] = a[t], zeros past the routed rows.
template <int BYTES, bool STREAM>
__global__ void __launch_bounds__(256) dispatch_kernel(RowsParams p) {
  const int64_t routed = routed_rows(p);
  const int lanes = 1 << p.lanes_log2, l = threadIdx.x & (lanes - 1);
  const int chunks = p.H * BYTES / 16;
  const int64_t place = ((int64_t)blockIdx.x * 256 + threadIdx.x) >> p.lanes_log2;
  const int64_t places = ((int64_t)gridDim.x * 256) >> p.lanes_log2;
  for (int64_t t = place; t < p.T; t += places) {
    for (int c = l; c < chunks; c += lanes) {
      const u32x4 v = ((const u32x4*)((const char*)p.a + t * p.lda * BYTES))[c];
      for (int j0 = 0; j0 < p.k; j0 += kSlotBatch) {
        int at[kSlotBatch];
#pragma unroll
        for (int j = 0; j < kSlotBatch; ++j) at[j] = j0 + j < p.k ? p.positions[t * p.k + j0 + j] : -1;
#pragma unroll
        for (int j = 0; j < kSlotBatch; ++j) {
          if (at[j] < 0 || at[j] >= routed) continue;
          store_row<STREAM>(v, (u32x4*)((char*)p.out + at[j] * p.ldo * BYTES) + c);
        }
      }
    }
  }
  for (int64_t r = routed + place; r < p.R; r += places)
    for (int c = l; c < chunks; c += lanes)
      store_row<STREAM>(u32x4{0u, 0u, 0u, 0u}, (u32x4*)((char*)p.out + r * p.ldo * BYTES) + c);
}

// out[t] = sum_j weights[t, j] b[positions[t, j]], in ascending j and FP32.  A
// batch's rows are all loaded before the first is used; where a slot has no
// row the first one is read and nothing of it taken.
template <int IN, int OUT, bool STREAM>
__global__ void __launch_bounds__(256) combine_kernel(RowsParams p) {
  const int64_t routed = routed_rows(p);
  const int lanes = 1 << p.lanes_log2, l = threadIdx.x & (lanes - 1);
  constexpr int N = 8;                  // columns of a thread's step
  constexpr int Q = N / RowVec<IN>::N;  // its loads of one row
  for (int64_t t = ((int64_t)blockIdx.x * 256 + threadIdx.x) >> p.lanes_log2; t < p.T;
       t += ((int64_t)gridDim.x * 256) >> p.lanes_log2) {
    for (int c = l * N; c < p.H; c += lanes * N) {
      float acc[N];
#pragma unroll
      for (int i = 0; i < N; ++i) acc[i] = 0.f;
      for (int j0 = 0; j0 < p.k && routed > 0; j0 += kSlotBatch) {
        int at[kSlotBatch];
        float w[kSlotBatch];
        u32x4 v[kSlotBatch][Q];
#pragma unroll
        for (int j = 0; j < kSlotBatch; ++j) {
          at[j] = j0 + j < p.k ? p.positions[t * p.k + j0 + j] : -1;
          w[j] = p.weights && j0 + j < p.k ? p.weights[t * p.k + j0 + j] : 1.f;
        }
#pragma unroll
        for (int j = 0; j < kSlotBatch; ++j) {
          const bool live = at[j] >= 0 && at[j] < routed;
          const char* row = (const char*)p.b + ((live ? at[j] : 0) * p.ldb + c) * IN;
          if (j0 + j < p.k)
#pragma unroll
            for (int q = 0; q < Q; ++q) v[j][q] = load_row<STREAM>((const u32x4*)row + q);
          at[j] = live;
        }
#pragma unroll
        for (int j = 0; j < kSlotBatch; ++j) {
          if (j0 + j >= p.k) break;
#pragma unroll
          for (int q = 0; q < Q; ++q) {
            float f[RowVec<IN>::N];
            RowVec<IN>::unpack(v[j][q], f);
#pragma unroll
            for (int i = 0; i < RowVec<IN>::N; ++i)
              acc[q * RowVec<IN>::N + i] = at[j] ? acc[q * RowVec<IN>::N + i] + w[j] * f[i] : acc[q * RowVec<IN>::N + i];
          }
        }
      }
      char* out = (char*)p.out + (t * p.ldo + c) * OUT;
#pragma unroll
      for (int q = 0; q < N / RowVec<OUT>::N; ++q) {
        float f[RowVec<OUT>::N];
#pragma unroll
        for (int i = 0; i < RowVec<OUT>::N; ++i) f[i] = acc[q * RowVec<OUT>::N + i];
        ((u32x4*)out)[q] = RowVec<OUT>::pack(f);
      }
    }
  }
}

// Gradients of the combination, one wave per slot: out[positions[t, j]] =
// weights[t, j] a[t] (zeros past the routed rows) and dweights[t, j] =
// <a[t], b[positions[t, j]]>, a the incoming gradient.  The waves of a token
// follow each other, so that its row of a comes from the cache but once.
template <int BYTES, bool STREAM>
__global__ void __launch_bounds__(256) combine_dgrad_kernel(RowsParams p) {
  const int lane = threadIdx.x & 63;
  const int64_t routed = routed_rows(p);
  constexpr int N = RowVec<BYTES>::N, U = 4;  // U: chunks loaded together
  const int chunks = p.H / N;
  const int64_t place = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t places = (int64_t)gridDim.x * 4;
  for (int64_t slot = place; slot < p.T * p.k; slot += places) {
    const int64_t t = slot / p.k;
    const int at = __builtin_amdgcn_readfirstlane(p.positions[slot]);
    float dot = 0.f;
    if (at >= 0 && at < routed) {
      const u32x4* dy = (const u32x4*)((const char*)p.a + t * p.lda * BYTES);
      const u32x4* row = (const u32x4*)((const char*)p.b + (int64_t)at * p.ldb * BYTES);
      u32x4* out = (u32x4*)((char*)p.out + (int64_t)at * p.ldo * BYTES);
      const float w = p.weights[slot];
      for (int c0 = lane; c0 < chunks; c0 += 64 * U) {
        u32x4 a[U], b[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int c = min(c0 + 64 * u, chunks - 1);
          a[u] = dy[c];
          b[u] = load_row<STREAM>(row + c);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (c0 + 64 * u >= chunks) break;
          float f[N], g[N];
          RowVec<BYTES>::unpack(a[u], f);
          RowVec<BYTES>::unpack(b[u], g);
#pragma unroll
          for (int i = 0; i < N; ++i) {
            dot += f[i] * g[i];
            f[i] *= w;
          }
          store_row<STREAM>(RowVec<BYTES>::pack(f), out + c0 + 64 * u);
        }
      }
    }
    dot = wave_sum(dot);
    if (lane == 0) p.dweights[slot] = dot;
  }
  for (int64_t r = routed + place; r < p.R; r += places)
    for (int c = lane; c < chunks; c += 64)
      store_row<STREAM>(u32x4{0u, 0u, 0u, 0u}, (u32x4*)((char*)p.out + r * p.ldo * BYTES) + c);
}

}  // namespace dpg

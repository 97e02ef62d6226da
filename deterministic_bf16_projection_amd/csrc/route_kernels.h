// Routing kernels: the choice of experts, the stable order of the chosen
// (token, slot) pairs by expert, rows moved into that order and back, and the
// gradients.
#pragma once
#include "device_common.h"

namespace dpg {

constexpr int kRouteThreads = 1024;
constexpr int kRouteWaves = kRouteThreads / 64;
constexpr int kRouteMaxExperts = 512;
constexpr int kRouteMaxTopK = 32;

// -------------------------------------------------------------- choice --
struct RouteParams {
  const float* logits;
  int64_t ldl;
  int64_t T;
  int E, k, renorm;
  int tokens_per_block;  // blocks of consecutive tokens
  int blocks;
  int32_t* experts;      // [T, k]
  float* weights;        // [T, k]
  int32_t* offsets;      // [E + 1]
  int32_t* rows;         // [T k]
  int32_t* positions;    // [T, k]
  int32_t* hist;         // [blocks, E + 1]
};

// One token by one wave.  The logits sit in registers, lane l holding experts
// l, 64 + l, ...; each of the k rounds takes the maximum over the wave and,
// among equal ones, the lowest expert (registers in ascending order, then the
// lowest lane of a ballot).  Only a logit of -infinity masks an expert; a NaN
// is never chosen but makes the token's weights NaN.  Lane j returns choice j.
template <int NR>
__device__ __forceinline__ void choose(const RouteParams& p, int64_t t, int lane, int& expert, float& weight) {
  const float kMasked = -__builtin_inff();
  float v[NR];
  bool nan = false;
#pragma unroll
  for (int r = 0; r < NR; ++r) {
    const int i = r * 64 + lane;
    const float x = i < p.E ? p.logits[t * p.ldl + i] : kMasked;
    nan |= x != x;
    v[r] = x != x ? kMasked : x;
  }
  const bool any_nan = __ballot(nan) != 0;
  float local = v[0];
#pragma unroll
  for (int r = 1; r < NR; ++r) local = fmaxf(local, v[r]);
  const float top = wave_max(local);
  float total = 0.f;
  if (!p.renorm && top > kMasked) {
#pragma unroll
    for (int r = 0; r < NR; ++r) total += expf(v[r] - top);
    total = wave_sum(total);
  }
  expert = -1;
  float mine = kMasked;
  float m = top;
  for (int j = 0; j < p.k && m > kMasked; ++j) {
    int at = 0;
    bool found = false;
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      const uint64_t eq = __ballot(v[r] == m);
      if (!found && eq) {
        const int l = __builtin_ctzll(eq);
        at = r * 64 + l;
        if (lane == l) v[r] = kMasked;
        found = true;
      }
    }
    if (lane == j) {
      expert = at;
      mine = m;
    }
    local = v[0];
#pragma unroll
    for (int r = 1; r < NR; ++r) local = fmaxf(local, v[r]);
    m = wave_max(local);
  }
  const float e = expert >= 0 ? expf(mine - top) : 0.f;
  if (p.renorm) total = wave_sum(e);
  weight = expert >= 0 ? e / total : 0.f;
  if (any_nan && expert >= 0) weight = __builtin_nanf("");
}

// --------------------------------------------------------- stable order --
// Slots (token * k + slot) of one block, ranked by (expert, slot): `start[e]`
// is the place of the block's first slot of expert e (experts in ascending
// order, unused slots last as expert E).  Each wave owns a run of consecutive
// slots; the counts per (wave, expert) in LDS, summed over the waves before,
// give every wave its own running places, and inside a wave the lanes with
// equal experts are found with one ballot per bit.  Integer counts: no order
// matters, the result is the same every time.
__device__ __forceinline__ void scatter_block(const RouteParams& p, int64_t slot0, int slots, const int* start,
                                              int* counts /* waves x (E + 1) */, int tid) {
  const int keys = p.E + 1;
  const int lane = tid & 63, wave = tid >> 6;
  const int per_wave = ((slots + kRouteWaves - 1) / kRouteWaves + 63) & ~63;
  const int s0 = wave * per_wave, s1 = min(slots, s0 + per_wave);
  for (int i = tid; i < kRouteWaves * keys; i += kRouteThreads) counts[i] = 0;
  __syncthreads();
  for (int s = s0 + lane; s < s1; s += 64) {
    const int e = p.experts[slot0 + s];
    atomicAdd(&counts[wave * keys + (e < 0 ? p.E : e)], 1);
  }
  __syncthreads();
  for (int key = tid; key < keys; key += kRouteThreads) {
    int at = start[key];
    for (int w = 0; w < kRouteWaves; ++w) {
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
      const int e = p.experts[slot0 + s];
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

// Choice of the block's tokens and its counts per expert.  With ONE (all
// tokens in one block) the order follows in the same launch.
template <int NR, bool ONE>
__global__ void __launch_bounds__(kRouteThreads) route_choose_kernel(RouteParams p) {
  extern __shared__ int lds[];
  const int keys = p.E + 1;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int* total = lds;
  for (int i = tid; i < keys; i += kRouteThreads) total[i] = 0;
  __syncthreads();
  const int64_t t0 = (int64_t)blockIdx.x * p.tokens_per_block;
  const int64_t t1 = min(p.T, t0 + p.tokens_per_block);
  for (int64_t t = t0 + wave; t < t1; t += kRouteWaves) {
    int expert;
    float weight;
    choose<NR>(p, t, lane, expert, weight);
    if (lane < p.k) {
      p.experts[t * p.k + lane] = expert;
      p.weights[t * p.k + lane] = weight;
      atomicAdd(&total[expert < 0 ? p.E : expert], 1);
    }
  }
  __syncthreads();
  if (ONE) {
    int* first = lds + keys;
    if (wave == 0) prefix_experts(total, first, keys, lane);
    __syncthreads();
    for (int i = tid; i < keys; i += kRouteThreads) p.offsets[i] = first[i];
    scatter_block(p, 0, (int)(p.T * p.k), first, lds + 2 * keys, tid);
  } else {
    for (int i = tid; i < keys; i += kRouteThreads) p.hist[(int64_t)blockIdx.x * keys + i] = total[i];
  }
}

// The order, from the counts of all blocks: each block sums the counts of the
// blocks before it and of all, so that no launch lies between.
__global__ void __launch_bounds__(kRouteThreads) route_order_kernel(RouteParams p) {
  extern __shared__ int lds[];
  const int keys = p.E + 1;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int* total = lds;
  int* before = lds + keys;
  int* first = lds + 2 * keys;
  for (int i = tid; i < 2 * keys; i += kRouteThreads) lds[i] = 0;
  __syncthreads();
  // a part of the threads' groups takes every blocks / groups-th block
  const int width = (keys + 63) & ~63;
  const int groups = kRouteThreads / width;
  const int g = tid / width, key = tid - g * width;
  if (g < groups && key < keys) {
    int all = 0, prev = 0;
#pragma unroll 8
    for (int b = g; b < p.blocks; b += groups) {
      const int n = p.hist[(int64_t)b * keys + key];
      all += n;
      prev += b < (int)blockIdx.x ? n : 0;
    }
    atomicAdd(&total[key], all);
    atomicAdd(&before[key], prev);
  }
  __syncthreads();
  if (wave == 0) prefix_experts(total, first, keys, lane);
  __syncthreads();
  for (int i = tid; i < keys; i += kRouteThreads) {
    if (blockIdx.x == 0) p.offsets[i] = first[i];
    first[i] += before[i];
  }
  __syncthreads();
  const int64_t slot0 = (int64_t)blockIdx.x * p.tokens_per_block * p.k;
  const int64_t left = p.T * p.k - slot0;
  scatter_block(p, slot0, (int)min(left, (int64_t)p.tokens_per_block * p.k), first, lds + 3 * keys, tid);
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
  const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (t >= T) return;
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

// --------------------------------------------------------- moving rows --
// The row kernels go token by token: a token's row is read once for all its
// slots, and slot j's row lies at positions[t, j] of the sorted matrix.  Slots
// without an expert have their places past offsets[E], where rows are written
// as zeros and never read.  Positions come from device memory: one outside the
// matrix is left out.
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

// out[positions[t, j]] = a[t], zeros past the routed rows.
template <int BYTES>
__global__ void __launch_bounds__(256) dispatch_kernel(RowsParams p) {
  const int64_t t = ((int64_t)blockIdx.x * 256 + threadIdx.x) >> p.lanes_log2;
  if (t >= p.T) return;
  const int routed = *p.routed;
  const int lanes = 1 << p.lanes_log2, l = threadIdx.x & (lanes - 1);
  const int chunks = p.H * BYTES / 16;
  for (int c = l; c < chunks; c += lanes) {
    const u32x4 v = ((const u32x4*)((const char*)p.a + t * p.lda * BYTES))[c];
    for (int j = 0; j < p.k; ++j) {
      const int at = p.positions[t * p.k + j];
      if ((uint64_t)(int64_t)at >= (uint64_t)p.R) continue;
      ((u32x4*)((char*)p.out + at * p.ldo * BYTES))[c] = at < routed ? v : u32x4{0u, 0u, 0u, 0u};
    }
  }
}

// out[t] = sum_j weights[t, j] b[positions[t, j]], in ascending j and FP32.
template <int IN, int OUT>
__global__ void __launch_bounds__(256) combine_kernel(RowsParams p) {
  const int64_t t = ((int64_t)blockIdx.x * 256 + threadIdx.x) >> p.lanes_log2;
  if (t >= p.T) return;
  const int64_t routed = min((int64_t)*p.routed, p.R);
  const int lanes = 1 << p.lanes_log2, l = threadIdx.x & (lanes - 1);
  constexpr int N = 8;  // columns of a thread's step
  for (int c = l * N; c < p.H; c += lanes * N) {
    float acc[N];
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] = 0.f;
    for (int j = 0; j < p.k; ++j) {
      const int at = p.positions[t * p.k + j];
      if (at < 0 || at >= routed) continue;
      const float w = p.weights ? p.weights[t * p.k + j] : 1.f;
      const char* row = (const char*)p.b + (at * p.ldb + c) * IN;
#pragma unroll
      for (int q = 0; q < N / RowVec<IN>::N; ++q) {
        float f[RowVec<IN>::N];
        RowVec<IN>::unpack(((const u32x4*)row)[q], f);
#pragma unroll
        for (int i = 0; i < RowVec<IN>::N; ++i) acc[q * RowVec<IN>::N + i] += w * f[i];
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

// Gradients of the combination, one wave per token: out[positions[t, j]] =
// weights[t, j] a[t] (zeros past the routed rows) and dweights[t, j] =
// <a[t], b[positions[t, j]]>, a the incoming gradient.
template <int BYTES>
__global__ void __launch_bounds__(256) combine_dgrad_kernel(RowsParams p) {
  const int lane = threadIdx.x & 63;
  const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (t >= p.T) return;
  const int64_t routed = min((int64_t)*p.routed, p.R);
  constexpr int N = RowVec<BYTES>::N;
  const int chunks = p.H / N;
  const u32x4* dy = (const u32x4*)((const char*)p.a + t * p.lda * BYTES);
  for (int j = 0; j < p.k; ++j) {
    const int at = __builtin_amdgcn_readfirstlane(p.positions[t * p.k + j]);
    float dot = 0.f;
    if (at >= 0 && at < p.R) {
      const bool live = at < routed;
      const float w = live ? p.weights[t * p.k + j] : 0.f;
      const u32x4* row = (const u32x4*)((const char*)p.b + (int64_t)at * p.ldb * BYTES);
      u32x4* out = (u32x4*)((char*)p.out + (int64_t)at * p.ldo * BYTES);
      for (int c = lane; c < chunks; c += 64) {
        float f[N], g[N];
        RowVec<BYTES>::unpack(dy[c], f);
        if (live) {
          RowVec<BYTES>::unpack(row[c], g);
#pragma unroll
          for (int i = 0; i < N; ++i) {
            dot += f[i] * g[i];
            f[i] *= w;
          }
          out[c] = RowVec<BYTES>::pack(f);
        } else {
          out[c] = u32x4{0u, 0u, 0u, 0u};
        }
      }
    }
    dot = wave_sum(dot);
    if (lane == 0) p.dweights[t * p.k + j] = dot;
  }
}

}  // namespace dpg

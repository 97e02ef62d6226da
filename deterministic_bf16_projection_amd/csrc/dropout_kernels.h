// Dropout from a counter-based generator: the mask is a function of the seed,
// a step and an element's place, so that nothing is stored and the gradient
// recomputes it.
//
// The generator is Philox4x32 with ten rounds (Salmon, Moraes, Dror and Shaw,
// "Parallel random numbers: as easy as 1, 2, 3", 2011): four 32-bit words from
// a 128-bit counter and a 64-bit key.  The counter holds the group of eight
// consecutive elements (low half) and the step (high half); each element takes
// 16 of the 128 bits, and is left out where they are below p in units of
// 2^-16.  Sixteen bits and not 32: ten rounds are 20 wide multiplications, at
// a quarter of the rate of additions, and eight elements share them.
#pragma once
#include "rows8.h"

namespace dpg {

struct DropParams {
  unsigned key0, key1;   // the seed
  const int64_t* step;   // on the device, or null: 0
  unsigned bar;          // elements whose 16 bits are below it are left out: 0 .. 65536
  float scale;           // of the others: 65536 / (65536 - bar); 0 when none is left
};

struct DropKey {
  unsigned key0, key1, step0, step1;
};
__device__ __forceinline__ DropKey drop_key(const DropParams& d) {
  const uint64_t step = d.step ? (uint64_t)*d.step : 0;
  return DropKey{d.key0, d.key1, (unsigned)step, (unsigned)(step >> 32)};
}

// The words of one counter.
__device__ __forceinline__ u32x4 philox(uint64_t group, const DropKey& k) {
  unsigned c0 = (unsigned)group, c1 = (unsigned)(group >> 32), c2 = k.step0, c3 = k.step1;
  unsigned k0 = k.key0, k1 = k.key1;
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t a = (uint64_t)c0 * 0xD2511F53u, b = (uint64_t)c2 * 0xCD9E8D57u;
    c0 = (unsigned)(b >> 32) ^ c1 ^ k0;
    c1 = (unsigned)b;
    c2 = (unsigned)(a >> 32) ^ c3 ^ k1;
    c3 = (unsigned)a;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return u32x4{c0, c1, c2, c3};
}

// Eight consecutive elements, group = (row * H + column) / 8.  What is left
// out is 0 whatever it was, infinities and NaN too.
__device__ __forceinline__ void drop8(float (&v)[8], uint64_t group, const DropKey& k, unsigned bar, float scale) {
  const u32x4 w = philox(group, k);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const unsigned bits = j & 1 ? w[j >> 1] >> 16 : w[j >> 1] & 0xffffu;
    v[j] = bits < bar ? 0.f : v[j] * scale;
  }
}

struct DropoutParams {
  Rows8 x, residual, y;  // residual.data null: none
  DropParams drop;
  int64_t T;             // rows
  int64_t groups;        // of eight elements, in all
  int per_row;           // groups of a row
  int lanes_log2;        // threads of a row
};

// 2^lanes_log2 threads to a row.  Rows without gaps come as rows of 512 groups,
// whatever the tensor's own: two groups to a thread.  Bound by memory: 16384 rows
// of 12288 BF16 columns in 127 to 131 us, 6.2 TB/s (146 through the caches and with
// one group to a thread; 136 and 160 past them with four or eight times as many).
template <bool BF16_IN, bool BF16_OUT, bool ADD, bool NT>
__global__ void __launch_bounds__(256) dropout_kernel(DropoutParams p) {
  const int lanes = 1 << p.lanes_log2, lane = threadIdx.x & (lanes - 1);
  const int64_t rows = (int64_t)gridDim.x << (8 - p.lanes_log2);
  const DropKey key = drop_key(p.drop);
  for (int64_t t = (((int64_t)blockIdx.x << 8) + threadIdx.x) >> p.lanes_log2; t < p.T; t += rows) {
    const int64_t first = t * p.per_row;
    const int n = (int)min((int64_t)p.per_row, p.groups - first);
    for (int g = lane; g < n; g += lanes) {
      float v[8];
      unpack8(load8<BF16_IN, NT>(p.x, t, g), v);
      if (p.drop.bar) drop8(v, (uint64_t)(first + g), key, p.drop.bar, p.drop.scale);
      if (ADD) {
        float r[8];
        unpack8(load8<BF16_OUT, NT>(p.residual, t, g), r);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] += r[j];
      }
      store8<BF16_OUT, NT>(p.y, t, g, v);
    }
  }
}

}  // namespace dpg

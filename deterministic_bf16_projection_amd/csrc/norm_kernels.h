// Layer norm, alone or of a residual sum whose new part passes through dropout,
// and its gradient.
//
//   v = x                  (alone)      v = residual + keep x / (1 - p)    (sum)
//   mean = sum v / H       rstd = (sum (v - mean)^2 / H + eps)^-1/2
//   n = (v - mean) rstd    y = n weight + bias
// and with u = dy weight
//   dv = rstd (u - sum u / H - n sum(u n) / H) + dsum
//   dresidual = dv         dx = keep dv / (1 - p)
//   dweight = sum over the rows of dy n        dbias = sum over the rows of dy
//
// Every kernel reads its rows once and keeps them in registers: bound by
// memory.  W waves share a row (one row to a wave, or to a workgroup), each
// lane holding C groups of eight columns, and go from row to row with the
// weights in registers, the next row's loads in flight.  Statistics and sums
// are FP32.
#pragma once
#include "dropout_kernels.h"

namespace dpg {

// Eight values of a type known at run time only (the same for all the launch).
struct Any8 {
  f32x4 a, b;
};
__device__ __forceinline__ Any8 load_any(const Rows8& m, bool bf16, int64_t row, int group) {
  Any8 r;
  if (bf16) {
    r.a = __builtin_bit_cast(f32x4, load8<true>(m, row, group).a);
    r.b = f32x4{0.f, 0.f, 0.f, 0.f};
  } else {
    const Raw8<false> w = load8<false>(m, row, group);
    r.a = w.a;
    r.b = w.b;
  }
  return r;
}
__device__ __forceinline__ void unpack_any(const Any8& r, bool bf16, float (&v)[8]) {
  if (bf16)
    unpack8(Raw8<true>{__builtin_bit_cast(u32x4, r.a)}, v);
  else
    unpack8(Raw8<false>{r.a, r.b}, v);
}
__device__ __forceinline__ void store_any(const Rows8& m, bool bf16, int64_t row, int group, const float (&v)[8]) {
  if (bf16)
    store8<true>(m, row, group, v);
  else
    store8<false>(m, row, group, v);
}

__device__ __forceinline__ void load_columns(const float* data, int group, float otherwise, float (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = otherwise;
  if (data) {
    const f32x4 a = *(const f32x4*)(data + 8 * group), b = *(const f32x4*)(data + 8 * group + 4);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[j] = a[j];
      v[j + 4] = b[j];
    }
  }
}

struct NormParams {
  Rows8 x;        // what is normalised, or the residual that a sum starts from
  Rows8 branch;   // sum: the new part
  Rows8 sum;      // sum: residual and new part, of x's type
  Rows8 y;
  const float* weight;  // or null
  const float* bias;    // or null
  float* mean;
  float* rstd;
  int64_t T;
  int H;
  float inv_h, eps;
  bool y_bf16, branch_bf16;
  DropParams drop;
};

constexpr int norm_threads(int waves) { return waves == 1 ? 256 : 64 * waves; }
constexpr int norm_rows(int waves) { return waves == 1 ? 4 : 1; }  // rows of a workgroup at once

// A row's mean and sum of squared differences from it.  The waves of a row
// each take those of their own columns and meet once, in LDS:
//   mean = sum n_w mean_w / H,   m2 = sum (m2_w + n_w (mean_w - mean)^2)
template <int W, int C>
__device__ __forceinline__ void row_statistics(const float (&v)[C][8], int groups, int lane, int wave, float inv_h,
                                               float (*shared)[2], float& mean, float& m2) {
  float s = 0.f;
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int j = 0; j < 8; ++j) s += v[c][j];
  // columns of this wave
  const auto columns = [&](int w) {
    int n = 0;
#pragma unroll
    for (int c = 0; c < C; ++c) n += min(64, max(0, groups - (c * W + w) * 64));
    return 8.f * (float)n;
  };
  const float n = columns(wave);
  s = wave_sum(s);
  float m = W == 1 ? s * inv_h : n > 0.f ? s / n : 0.f;
  float q = 0.f;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const bool have = (c * W + wave) * 64 + lane < groups;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float d = have ? v[c][j] - m : 0.f;
      q = fmaf(d, d, q);
    }
  }
  q = wave_sum(q);
  if constexpr (W > 1) {
    if (lane == 0) {
      shared[wave][0] = m;
      shared[wave][1] = q;
    }
    __syncthreads();
    m = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) m = fmaf(columns(w), shared[w][0], m);
    m *= inv_h;
    q = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float d = shared[w][0] - m;
      q += fmaf(columns(w) * d, d, shared[w][1]);
    }
  }
  mean = m;
  m2 = q;
}

template <bool X_BF16, int W, int C, bool ADD>
__global__ void __launch_bounds__(norm_threads(W)) norm_kernel(NormParams p) {
  __shared__ float shared[2][W][2];
  const int lane = threadIdx.x & 63, id = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wave = W == 1 ? 0 : id, groups = p.H >> 3;
  const int64_t stride = (int64_t)gridDim.x * norm_rows(W);
  int64_t t = (int64_t)blockIdx.x * norm_rows(W) + (W == 1 ? id : 0);
  if (t >= p.T) return;
  const auto group = [&](int c) { return (c * W + wave) * 64 + lane; };
  float w[C][8], b[C][8];
  Raw8<X_BF16> raw[C];
  Any8 part[ADD ? C : 1];
  const auto fetch = [&](int64_t row) {
#pragma unroll
    for (int c = 0; c < C; ++c)
      if (group(c) < groups) {
        raw[c] = load8<X_BF16>(p.x, row, group(c));
        if (ADD) part[c] = load_any(p.branch, p.branch_bf16, row, group(c));
      }
  };
#pragma unroll
  for (int c = 0; c < C; ++c) raw[c] = {};
  if (ADD) {
#pragma unroll
    for (int c = 0; c < C; ++c) part[c] = {};
  }
  fetch(t);
#pragma unroll
  for (int c = 0; c < C; ++c) {
    if (group(c) >= groups) continue;
    load_columns(p.weight, group(c), 1.f, w[c]);
    load_columns(p.bias, group(c), 0.f, b[c]);
  }
  DropKey key{};
  if (ADD) key = drop_key(p.drop);
  int turn = 0;
  for (; t < p.T; t += stride) {
    float v[C][8];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      unpack8(raw[c], v[c]);
      if (ADD) {
        float d[8];
        unpack_any(part[c], p.branch_bf16, d);
        if (p.drop.bar) drop8(d, (uint64_t)t * groups + group(c), key, p.drop.bar, p.drop.scale);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[c][j] += d[j];
      }
      // lanes past the row hold zeros, which a sum does not notice
#pragma unroll
      for (int j = 0; j < 8; ++j) v[c][j] = group(c) < groups ? v[c][j] : 0.f;
    }
    if (t + stride < p.T) fetch(t + stride);
    if (ADD) {
#pragma unroll
      for (int c = 0; c < C; ++c)
        if (group(c) < groups) store8<X_BF16>(p.sum, t, group(c), v[c]);
    }
    float mean, m2;
    // two places in LDS by turns: a wave may write for the next row while
    // others still read, and the barrier of the next row ends their reading
    row_statistics<W, C>(v, groups, lane, wave, p.inv_h, shared[turn], mean, m2);
    turn ^= 1;
    const float rstd = 1.f / sqrtf(m2 * p.inv_h + p.eps);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      if (group(c) >= groups) continue;
      float y[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = fmaf((v[c][j] - mean) * rstd, w[c][j], b[c][j]);
      store_any(p.y, p.y_bf16, t, group(c), y);
    }
    if (lane == 0 && wave == 0) {
      p.mean[t] = mean;
      p.rstd[t] = rstd;
    }
  }
}

// ------------------------------------------------------------- gradient --
struct NormGradParams {
  Rows8 dy, x;         // x: what was normalised
  Rows8 dsum;          // sum: the gradient that reaches the sum from elsewhere, or null
  Rows8 dx;            // of x's type; sum: the new part's, of a type of its own
  Rows8 dresidual;     // sum: of x's type
  const float* mean;
  const float* rstd;
  const float* weight;  // or null
  float* partial;       // [blocks, 2, H]: sums of dy n and of dy, or null
  int64_t T;
  int H;
  float inv_h;
  bool dy_bf16, dx_bf16;
  DropParams drop;
};

template <bool X_BF16, int W, int C, bool ADD>
__global__ void __launch_bounds__(norm_threads(W)) norm_dgrad_kernel(NormGradParams p) {
  __shared__ float shared[2][W][2];
  __shared__ float sums[W == 1 ? 4 * 2 * 512 * C : 1];
  const int lane = threadIdx.x & 63, id = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wave = W == 1 ? 0 : id, groups = p.H >> 3;
  const int64_t stride = (int64_t)gridDim.x * norm_rows(W);
  const auto group = [&](int c) { return (c * W + wave) * 64 + lane; };
  float w[C][8], dw[C][8], db[C][8];
  Raw8<X_BF16> raw[C], more[ADD ? C : 1];
  Any8 grad[C];
  float next_mean = 0.f, next_rstd = 0.f;
  const bool with_dsum = ADD && p.dsum.data;
  const auto fetch = [&](int64_t row) {
    next_mean = p.mean[row];
    next_rstd = p.rstd[row];
#pragma unroll
    for (int c = 0; c < C; ++c)
      if (group(c) < groups) {
        raw[c] = load8<X_BF16>(p.x, row, group(c));
        grad[c] = load_any(p.dy, p.dy_bf16, row, group(c));
        if (ADD && with_dsum) more[c] = load8<X_BF16>(p.dsum, row, group(c));
      }
  };
#pragma unroll
  for (int c = 0; c < C; ++c) {
    raw[c] = {};
    grad[c] = {};
    if (ADD) more[c] = {};
#pragma unroll
    for (int j = 0; j < 8; ++j) w[c][j] = dw[c][j] = db[c][j] = 0.f;
    if (group(c) < groups) load_columns(p.weight, group(c), 1.f, w[c]);
  }
  DropKey key{};
  if (ADD) key = drop_key(p.drop);
  int turn = 0;
  int64_t t = (int64_t)blockIdx.x * norm_rows(W) + (W == 1 ? id : 0);
  if (t < p.T) fetch(t);
  for (; t < p.T; t += stride) {
    float n[C][8], u[C][8], s1 = 0.f, s2 = 0.f;
    const float mean = next_mean, rstd = next_rstd;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      float dy[8];
      unpack8(raw[c], n[c]);
      unpack_any(grad[c], p.dy_bf16, dy);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        n[c][j] = (n[c][j] - mean) * rstd;
        u[c][j] = dy[j] * w[c][j];
        dw[c][j] = fmaf(dy[j], n[c][j], dw[c][j]);
        db[c][j] += dy[j];
        // a lane past the row: u is 0, n is not, and may be infinite
        s1 += u[c][j];
        s2 = group(c) < groups ? fmaf(u[c][j], n[c][j], s2) : s2;
      }
    }
    Raw8<X_BF16> extra[ADD ? C : 1];
    if (ADD) {
#pragma unroll
      for (int c = 0; c < C; ++c) extra[c] = more[c];
    }
    if (t + stride < p.T) fetch(t + stride);
    s1 = wave_sum(s1);
    s2 = wave_sum(s2);
    if constexpr (W > 1) {
      if (lane == 0) {
        shared[turn][wave][0] = s1;
        shared[turn][wave][1] = s2;
      }
      __syncthreads();
      s1 = s2 = 0.f;
#pragma unroll
      for (int i = 0; i < W; ++i) {
        s1 += shared[turn][i][0];
        s2 += shared[turn][i][1];
      }
      turn ^= 1;
    }
    s1 *= p.inv_h;
    s2 *= p.inv_h;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      if (group(c) >= groups) continue;
      float d[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) d[j] = rstd * (u[c][j] - s1 - n[c][j] * s2);
      if constexpr (ADD) {
        if (with_dsum) {
          float e[8];
          unpack8(extra[c], e);
#pragma unroll
          for (int j = 0; j < 8; ++j) d[j] += e[j];
        }
        store8<X_BF16>(p.dresidual, t, group(c), d);
        if (p.drop.bar) drop8(d, (uint64_t)t * groups + group(c), key, p.drop.bar, p.drop.scale);
        store_any(p.dx, p.dx_bf16, t, group(c), d);
      } else {
        store8<X_BF16>(p.dx, t, group(c), d);
      }
    }
  }
  if (!p.partial) return;
  float* out = p.partial + (int64_t)blockIdx.x * 2 * p.H;
  if constexpr (W == 1) {
    // four waves with rows of their own: added in the waves' order
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        sums[(id * 2 + 0) * 512 * C + 8 * group(c) + j] = dw[c][j];
        sums[(id * 2 + 1) * 512 * C + 8 * group(c) + j] = db[c][j];
      }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * p.H; i += 256) {
      const int which = i >= p.H, col = i - which * p.H;
      float s = 0.f;
#pragma unroll
      for (int k = 0; k < 4; ++k) s += sums[(k * 2 + which) * 512 * C + col];
      out[i] = s;
    }
  } else {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      if (group(c) >= groups) continue;
      float* at = out + 8 * group(c);
      *(f32x4*)at = f32x4{dw[c][0], dw[c][1], dw[c][2], dw[c][3]};
      *(f32x4*)(at + 4) = f32x4{dw[c][4], dw[c][5], dw[c][6], dw[c][7]};
      *(f32x4*)(at + p.H) = f32x4{db[c][0], db[c][1], db[c][2], db[c][3]};
      *(f32x4*)(at + p.H + 4) = f32x4{db[c][4], db[c][5], db[c][6], db[c][7]};
    }
  }
}

// dweight and dbias from the workgroups' sums, added in a fixed order: sixteen
// waves take every sixteenth block each for 64 columns and meet in LDS.
// blocks = 0 writes zeros.
__global__ void __launch_bounds__(1024) norm_wgrad_kernel(const float* partial, int blocks, int H, float* dweight,
                                                          float* dbias) {
  __shared__ float sums[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int i = blockIdx.x * 64 + lane;  // column of [2, H]
  float s = 0.f;
  if (i < 2 * H)
    for (int k = wave; k < blocks; k += 16) s += partial[(int64_t)k * 2 * H + i];
  sums[wave][lane] = s;
  __syncthreads();
  if (wave != 0 || i >= 2 * H) return;
  s = 0.f;
#pragma unroll
  for (int k = 0; k < 16; ++k) s += sums[k][lane];
  float* out = i < H ? dweight : dbias;
  if (out) out[i < H ? i : i - H] = s;
}

}  // namespace dpg

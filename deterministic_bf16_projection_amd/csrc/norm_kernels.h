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
// memory.  `waves` waves share a row, each lane holding C groups of eight
// columns, and go from row to row with the next row's loads in flight (but the
// gradient's dsum) and the weights in registers; forward with more than two
// groups to a lane, in LDS.  A workgroup has `groups` sets of such waves (or of
// lanes, where rows are short).  Statistics and sums are FP32.
//
// 16384 rows of 4096 columns, BF16: forward 47-52 us (5.2-5.7 TB/s), gradient 79 us
// (73 us and 5.6 TB/s for the rows, 5 us for the weight gradient's last sums).
// A sum of 8192 such rows, FP32 stream and BF16 branch: 78 us (5.2 TB/s); its
// gradient of 5003 x 5120 82 us (5.0).  Non-temporal accesses are level.  The
// gradient's kernels with two groups to a lane (rows of more than 8192 columns)
// spill 20 to 84 registers: 3.0 to 3.8 TB/s.
#pragma once
#include "dropout_kernels.h"

namespace dpg {

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

constexpr int kNormWaves = 16;  // of a workgroup, at most
// With more groups to a lane there are half as many, of twice the registers.
__host__ __device__ constexpr int norm_threads(int chunks) { return 64 * (chunks > 2 ? kNormWaves / 2 : kNormWaves); }

// Forward, weight and bias are in registers with up to two groups to a lane, and
// in LDS with more: the first four columns of each group, then the last four
// (lanes 16 bytes apart), the weight's before the bias's.
__host__ __device__ constexpr bool norm_shares_weights(int chunks) { return chunks > 2; }
__device__ __forceinline__ float* column_place(float* columns, int H, int which, int half, int group) {
  return columns + (2 * which + half) * (H >> 1) + 4 * group;
}
__device__ __forceinline__ void put_columns(float* columns, int H, int which, int group, const float (&v)[8]) {
  *(f32x4*)column_place(columns, H, which, 0, group) = f32x4{v[0], v[1], v[2], v[3]};
  *(f32x4*)column_place(columns, H, which, 1, group) = f32x4{v[4], v[5], v[6], v[7]};
}
__device__ __forceinline__ void get_columns(float* columns, int H, int which, int group, float (&v)[8]) {
  const f32x4 a = *(const f32x4*)column_place(columns, H, which, 0, group);
  const f32x4 b = *(const f32x4*)column_place(columns, H, which, 1, group);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[j] = a[j];
    v[j + 4] = b[j];
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
  int H, waves, groups, lanes;
  float inv_h, eps;
  DropParams drop;
};

// A lane's place: the wave among those of its row, and its row's place among the
// workgroup's.  SMALL: `lanes` (8, 16 or 32) lanes hold a row, and a wave several
// rows; else a row has whole waves.
template <bool SMALL>
struct NormPlace {
  int lane, id, wave, set, chunks, lanes;  // chunks: groups of eight columns of a row
  __device__ __forceinline__ NormPlace(int waves, int H, int lanes_of_row) {
    chunks = H >> 3;
    if constexpr (SMALL) {
      lanes = lanes_of_row;
      lane = threadIdx.x & (lanes - 1);
      set = threadIdx.x / (unsigned)lanes;
      id = wave = 0;
    } else {
      lanes = 64;
      lane = threadIdx.x & 63;
      id = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
      set = id / waves;
      wave = id - set * waves;
    }
  }
  // over the lanes of one row (of one of its waves)
  __device__ __forceinline__ float sum(float v) const {
    if constexpr (!SMALL) return wave_sum(v);
    for (int m = lanes >> 1; m > 0; m >>= 1) v += __shfl_xor(v, m);
    return v;
  }
};

// columns of wave w of a row
template <int C, bool SMALL>
__device__ __forceinline__ float row_columns(const NormPlace<SMALL>& q, int waves, int w) {
  int n = 0;
#pragma unroll
  for (int c = 0; c < C; ++c) n += min(64, max(0, q.chunks - (c * waves + w) * 64));
  return 8.f * (float)n;
}

// sum / count, inverse = 1 / count: the product and its remainder, for a quotient
// that is exact where there is one (a row of one value has that as its mean),
// without the ten dependent steps of a division in every row.
__device__ __forceinline__ float mean_of(float sum, float count, float inverse) {
  const float q = sum * inverse;
  return fabsf(q) < __builtin_inff() ? fmaf(fmaf(-q, count, sum), inverse, q) : q;
}

// A row's mean and sum of squared differences from it.  The waves of a row
// each take those of their own columns and meet once, in LDS:
//   mean = sum n_w mean_w / H,   m2 = sum (m2_w + n_w (mean_w - mean)^2)
template <int C, bool SMALL>
__device__ __forceinline__ void row_statistics(const float (&v)[C][8], const NormPlace<SMALL>& q, int waves, float inv_h,
                                               float inv_n, float (*shared)[2], float& mean, float& m2) {
  float s = 0.f;
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int j = 0; j < 8; ++j) s += v[c][j];
  const auto columns = [&](int w) { return row_columns<C, SMALL>(q, waves, w); };
  const float n = columns(q.wave);
  s = q.sum(s);
  float m = mean_of(s, n, inv_n), sq = 0.f;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const bool have = (c * waves + q.wave) * 64 + q.lane < q.chunks;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float d = have ? v[c][j] - m : 0.f;
      sq = fmaf(d, d, sq);
    }
  }
  sq = q.sum(sq);
  if (waves > 1) {
    if (q.lane == 0) {
      shared[q.id][0] = m;
      shared[q.id][1] = sq;
    }
    __syncthreads();
    const float(*own)[2] = shared + q.set * waves;
    m = 0.f;
    for (int w = 0; w < waves; ++w) m = fmaf(columns(w), own[w][0], m);
    m = mean_of(m, 8.f * (float)q.chunks, inv_h);
    sq = 0.f;
    for (int w = 0; w < waves; ++w) {
      const float d = own[w][0] - m;
      sq += fmaf(columns(w) * d, d, own[w][1]);
    }
  }
  mean = m;
  m2 = sq;
}

template <bool X_BF16, bool Y_BF16, int C, bool ADD, bool BRANCH_BF16, bool SMALL>
__global__ void __launch_bounds__(norm_threads(C)) norm_kernel(NormParams p) {
  constexpr bool SHARED = norm_shares_weights(C);
  __shared__ float shared[2][kNormWaves][2];
  extern __shared__ __attribute__((aligned(16))) float columns[];  // SHARED: weight and bias, see column_place
  const NormPlace<SMALL> q(p.waves, p.H, p.lanes);
  const int64_t stride = (int64_t)gridDim.x * p.groups;
  int64_t first = (int64_t)blockIdx.x * p.groups;  // of the workgroup's rows
  const auto chunk = [&](int c) { return (c * p.waves + q.wave) * 64 + q.lane; };
  float w[SHARED ? 1 : C][8], b[SHARED ? 1 : C][8];
  Raw8<X_BF16> raw[C];
  Raw8<BRANCH_BF16> part[ADD ? C : 1];
  const auto fetch = [&](int64_t row) {
#pragma unroll
    for (int c = 0; c < C; ++c)
      if (chunk(c) < q.chunks && row < p.T) {
        raw[c] = load8<X_BF16>(p.x, row, chunk(c));
        if (ADD) part[c] = load8<BRANCH_BF16>(p.branch, row, chunk(c));
      }
  };
#pragma unroll
  for (int c = 0; c < C; ++c) {
    raw[c] = {};
    if (ADD) part[c] = {};
  }
  fetch(first + q.set);
  if constexpr (SHARED) {
    for (int i = threadIdx.x; i < q.chunks; i += blockDim.x) {
      float v[8];
      load_columns(p.weight, i, 1.f, v);
      put_columns(columns, p.H, 0, i, v);
      load_columns(p.bias, i, 0.f, v);
      put_columns(columns, p.H, 1, i, v);
    }
    __syncthreads();
  } else {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      if (chunk(c) >= q.chunks) continue;
      load_columns(p.weight, chunk(c), 1.f, w[c]);
      load_columns(p.bias, chunk(c), 0.f, b[c]);
    }
  }
  const float own = row_columns<C, SMALL>(q, p.waves, q.wave), inv_n = own > 0.f ? 1.f / own : 0.f;
  DropKey key{};
  if (ADD) key = drop_key(p.drop);
  int turn = 0;
  for (; first < p.T; first += stride) {
    const int64_t t = first + q.set;
    const bool live = t < p.T;
    float v[C][8];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      unpack8(raw[c], v[c]);
      if (ADD) {
        float d[8];
        unpack8(part[c], d);
        if (p.drop.bar) drop8(d, (uint64_t)t * q.chunks + chunk(c), key, p.drop.bar, p.drop.scale);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[c][j] += d[j];
      }
      // lanes past the row hold zeros, which a sum does not notice
#pragma unroll
      for (int j = 0; j < 8; ++j) v[c][j] = chunk(c) < q.chunks ? v[c][j] : 0.f;
    }
    fetch(t + stride);
    if (ADD && live) {
#pragma unroll
      for (int c = 0; c < C; ++c)
        if (chunk(c) < q.chunks) store8<X_BF16>(p.sum, t, chunk(c), v[c]);
    }
    float mean, m2;
    // two places in LDS by turns: a wave may write for the next row while
    // others still read, and the barrier of the next row ends their reading
    row_statistics<C, SMALL>(v, q, p.waves, p.inv_h, inv_n, shared[turn], mean, m2);
    turn ^= 1;
    const float rstd = 1.f / sqrtf(m2 * p.inv_h + p.eps);
    if (!live) continue;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      if (chunk(c) >= q.chunks) continue;
      float y[8];
      constexpr int kOwn = SHARED ? 0 : 1;
      if constexpr (SHARED) {
        get_columns(columns, p.H, 0, chunk(c), w[0]);
        get_columns(columns, p.H, 1, chunk(c), b[0]);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = fmaf((v[c][j] - mean) * rstd, w[kOwn * c][j], b[kOwn * c][j]);
      store8<Y_BF16>(p.y, t, chunk(c), y);
    }
    if (q.lane == 0 && q.wave == 0) {
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
  int H, waves, groups, lanes;
  bool dx_bf16;         // sum
  DropParams drop;
};

// Each wave adds up dy n and dy over its rows in registers; a workgroup's sets
// of waves meet in LDS (groups * H floats), set after set, and its sums are one
// row of `partial`.
template <bool X_BF16, bool DY_BF16, int C, bool ADD, bool SMALL>
__global__ void __launch_bounds__(64 * kNormWaves) norm_dgrad_kernel(NormGradParams p) {
  __shared__ float shared[2][kNormWaves][2];
  extern __shared__ __attribute__((aligned(16))) float sums[];
  const NormPlace<SMALL> q(p.waves, p.H, p.lanes);
  const int64_t stride = (int64_t)gridDim.x * p.groups;
  const auto chunk = [&](int c) { return (c * p.waves + q.wave) * 64 + q.lane; };
  float w[C][8], dw[C][8], db[C][8];
  Raw8<X_BF16> raw[C], more[ADD ? C : 1];
  Raw8<DY_BF16> grad[C];
  float next_mean = 0.f, next_rstd = 0.f;
  const bool with_dsum = ADD && p.dsum.data;
  const auto fetch = [&](int64_t row) {
    if (row >= p.T) return;
    next_mean = p.mean[row];
    next_rstd = p.rstd[row];
#pragma unroll
    for (int c = 0; c < C; ++c)
      if (chunk(c) < q.chunks) {
        raw[c] = load8<X_BF16>(p.x, row, chunk(c));
        grad[c] = load8<DY_BF16>(p.dy, row, chunk(c));
      }
  };
#pragma unroll
  for (int c = 0; c < C; ++c) {
    raw[c] = {};
    grad[c] = {};
    if (ADD) more[c] = {};
#pragma unroll
    for (int j = 0; j < 8; ++j) w[c][j] = dw[c][j] = db[c][j] = 0.f;
    if (chunk(c) < q.chunks) load_columns(p.weight, chunk(c), 1.f, w[c]);
  }
  const float inv_h = 1.f / (float)p.H;
  DropKey key{};
  if (ADD) key = drop_key(p.drop);
  int turn = 0;
  int64_t first = (int64_t)blockIdx.x * p.groups;
  fetch(first + q.set);
  for (; first < p.T; first += stride) {
    const int64_t t = first + q.set;
    const bool live = t < p.T;
    float n[C][8], u[C][8], s1 = 0.f, s2 = 0.f;
    const float mean = next_mean, rstd = next_rstd;
    if (ADD && with_dsum) {
#pragma unroll
      for (int c = 0; c < C; ++c)
        if (chunk(c) < q.chunks && live) more[c] = load8<X_BF16>(p.dsum, t, chunk(c));
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const bool have = chunk(c) < q.chunks && live;
      float dy[8];
      unpack8(raw[c], n[c]);
      unpack8(grad[c], dy);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        n[c][j] = (n[c][j] - mean) * rstd;
        u[c][j] = dy[j] * w[c][j];
        // what is no row's column may be anything
        dw[c][j] = have ? fmaf(dy[j], n[c][j], dw[c][j]) : dw[c][j];
        db[c][j] = have ? db[c][j] + dy[j] : db[c][j];
        s1 = have ? s1 + u[c][j] : s1;
        s2 = have ? fmaf(u[c][j], n[c][j], s2) : s2;
      }
    }
    fetch(t + stride);
    s1 = q.sum(s1);
    s2 = q.sum(s2);
    if (p.waves > 1) {
      if (q.lane == 0) {
        shared[turn][q.id][0] = s1;
        shared[turn][q.id][1] = s2;
      }
      __syncthreads();
      const float(*own)[2] = shared[turn] + q.set * p.waves;
      s1 = s2 = 0.f;
      for (int i = 0; i < p.waves; ++i) {
        s1 += own[i][0];
        s2 += own[i][1];
      }
      turn ^= 1;
    }
    s1 = mean_of(s1, (float)p.H, inv_h);
    s2 = mean_of(s2, (float)p.H, inv_h);
    if (!live) continue;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      if (chunk(c) >= q.chunks) continue;
      float d[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) d[j] = rstd * (u[c][j] - s1 - n[c][j] * s2);
      if constexpr (ADD) {
        if (with_dsum) {
          float e[8];
          unpack8(more[c], e);
#pragma unroll
          for (int j = 0; j < 8; ++j) d[j] += e[j];
        }
        store8<X_BF16>(p.dresidual, t, chunk(c), d);
        if (p.drop.bar) drop8(d, (uint64_t)t * q.chunks + chunk(c), key, p.drop.bar, p.drop.scale);
        if (p.dx_bf16)
          store8<true>(p.dx, t, chunk(c), d);
        else
          store8<false>(p.dx, t, chunk(c), d);
      } else {
        store8<X_BF16>(p.dx, t, chunk(c), d);
      }
    }
  }
  if (!p.partial) return;
  // dweight's, then dbias's: the sets of waves in their order
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    float* out = p.partial + ((int64_t)blockIdx.x * 2 + which) * p.H;
    if (p.groups > 1) {
      __syncthreads();
#pragma unroll
      for (int c = 0; c < C; ++c) {
        if (chunk(c) >= q.chunks) continue;
        const float(&v)[8] = which ? db[c] : dw[c];
        float* at = sums + q.set * p.H + 8 * chunk(c);
        *(f32x4*)at = f32x4{v[0], v[1], v[2], v[3]};
        *(f32x4*)(at + 4) = f32x4{v[4], v[5], v[6], v[7]};
      }
      __syncthreads();
      for (int i = threadIdx.x; i < p.H; i += blockDim.x) {
        float s = sums[i];
        for (int g = 1; g < p.groups; ++g) s += sums[g * p.H + i];
        out[i] = s;
      }
    } else {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        if (chunk(c) >= q.chunks) continue;
        const float(&v)[8] = which ? db[c] : dw[c];
        float* at = out + 8 * chunk(c);
        *(f32x4*)at = f32x4{v[0], v[1], v[2], v[3]};
        *(f32x4*)(at + 4) = f32x4{v[4], v[5], v[6], v[7]};
      }
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
  if (i < 2 * H) {
    for (int k = wave; k < blocks; k += 256) {
      float v[16];  // sixteen loads in flight
#pragma unroll
      for (int j = 0; j < 16; ++j) v[j] = k + 16 * j < blocks ? partial[(int64_t)(k + 16 * j) * 2 * H + i] : 0.f;
#pragma unroll
      for (int j = 0; j < 16; ++j) s += v[j];
    }
  }
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

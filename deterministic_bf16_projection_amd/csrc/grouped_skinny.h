// Grouped products of few rows: forward and input gradient where a group holds
// a handful of rows, so that the weights are read once and bound the call, or
// where the large kernel's tiles are too few for the chip.
//
// A workgroup of eight waves owns a few rows by BN columns of one group and
// splits the reduction among its waves: wave w takes the steps w, w + 8, ...
// All operands go straight from memory to MFMA fragments, so a wave keeps many
// loads in flight and nothing waits at a barrier until the eight partial sums
// meet in LDS, where they are added in a fixed order: the same bits each time.
//
// The weight is a product's first operand (D rows: output columns), the token
// side its second (D columns: rows).  Three kernels:
//  forward, 16 rows by 16 columns: products of 4x4x4 with 16 blocks that lie
//    along the reduction.  Lane l loads 16 bytes of row n0 + l % 4 at k + 8 (l /
//    4), so that a load takes 256 contiguous bytes of four rows; a block holds
//    the sum over its share of k, and the blocks are added across lanes once
//    per unit.  Whole lines can be read past the caches: 256 rows of 64 groups,
//    1024 x 4096, 90 us (6.0 TB/s); with 16x16x32 fragments, whose loads take
//    64 bytes of sixteen rows, 106, and 139 past the caches.
//  forward, 32 rows by 32 columns: products of 16x16x32, lane l loading
//    W[n0 + l % 16][k + 8 (l / 16) ..]; more rows share a weight's fragment.
//  input gradient, 16 rows by 128 columns: W is contiguous along the outputs.
//    Lane l loads the 8x8 block of rows n + 8 (l / 16) .. and columns 8 (l % 16)
//    .. (256 contiguous bytes of four rows per load) and transposes it in
//    registers for products of 16x16x32: fragment f then holds the columns
//    8 i + f, i = 0 .. 15.  256 rows as above 88 us, 99 through the caches.
// A weight that only one unit reads (a group of at most 16 rows) is loaded
// non-temporally.  Rows past the group, columns past the matrix and reduction
// indexes past its end read as zero through the buffer descriptors.
//
// Included by dpg_grouped.hip after gemm_fast.h.
#pragma once

namespace dpg {

constexpr int kSkinnyThreads = 512;
constexpr int kSkinnyWaves = kSkinnyThreads / 64;

__device__ __forceinline__ f32x4 mfma16(const bf16x8& a, const bf16x8& b, const f32x4& c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

typedef short bf16x4 __attribute__((ext_vector_type(4)));

// 16 blocks of D[i][j] += sum_k A[i][k] B[k][j], 4x4x4: lane l holds row (or
// column) l % 4 of block l / 4, and D's column l % 4 in four registers; 8
// reduction elements per lane in two products
__device__ __forceinline__ f32x4 mfma4(const u32x4& a, const u32x4& b, f32x4 c) {
  const u32x2 al = {a[0], a[1]}, ah = {a[2], a[3]}, bl = {b[0], b[1]}, bh = {b[2], b[3]};
  c = __builtin_amdgcn_mfma_f32_4x4x4bf16_1k(__builtin_bit_cast(bf16x4, al), __builtin_bit_cast(bf16x4, bl), c, 0, 0, 0);
  return __builtin_amdgcn_mfma_f32_4x4x4bf16_1k(__builtin_bit_cast(bf16x4, ah), __builtin_bit_cast(bf16x4, bh), c, 0, 0, 0);
}

template <bool ONCE>
__device__ __forceinline__ u32x4 load_weight(rsrc_t r, uint32_t voff) {
  return __builtin_amdgcn_raw_buffer_load_b128(r, (int)voff, 0, ONCE ? 2 : 0);  // 2: non-temporal
}

template <class T>
__device__ __forceinline__ rsrc_t rows_rsrc(const T* base, int rows, int ld, int cols) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<T*>(base), (short)0,
                                           max(((rows - 1) * ld + cols) * (int)sizeof(T), 0), 0x00020000);
}

// One unit's products for MT row tiles of 16, this wave's share of the
// reduction, into acc.  U: steps whose loads a wave issues together.
template <bool DG, int MT, int NF, int U, bool ONCE>
__device__ __forceinline__ void skinny_products(const GroupedParams& p, const StepCursor& c, int wave, int lane,
                                                f32x4 (&acc)[MT][NF]) {
  constexpr int BN = DG ? 128 : 16 * NF;
  constexpr int STEP = DG ? 32 : 64;  // reduction elements of a step
  constexpr int XF = STEP / 32;       // token-side fragments of a step and row tile
  const int row = lane & 15, quad = lane >> 4;
  const int lda = (int)p.lda, ldb = (int)p.ldb, K = p.K;
  const int steps = (K + STEP - 1) / STEP;
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NF; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  // descriptors of the unit's rows and, forward, of its weight rows
  const rsrc_t rx = rows_rsrc((const __bf16*)p.a + ((int64_t)c.base + c.row0) * lda, min(c.count - c.row0, 16 * MT),
                              lda, K);
  const __bf16* w = (const __bf16*)p.b + (int64_t)c.b * p.batch_b + (DG ? (int64_t)c.col0 : (int64_t)c.col0 * ldb);
  const rsrc_t rw = rows_rsrc(w, min(p.N - c.col0, BN), ldb, K);
  for (int s0 = wave; s0 < steps; s0 += kSkinnyWaves * U) {
    u32x4 fx[U][XF][MT], fw[U][DG ? 8 : XF * NF];
#pragma unroll
    for (int q = 0; q < U; ++q) {
      const int k0 = (s0 + q * kSkinnyWaves) * STEP;  // past the end: zeros
      if constexpr (DG) {
        const int kr = min(K - k0, STEP);
        const rsrc_t r = rows_rsrc(w + (int64_t)min(k0, K) * ldb, kr, ldb, kr > 0 ? p.N - c.col0 : 0);
#pragma unroll
        for (int e = 0; e < 8; ++e) fw[q][e] = load_weight<ONCE>(r, (uint32_t)(((quad * 8 + e) * ldb + row * 8) * 2));
      }
#pragma unroll
      for (int h = 0; h < XF; ++h) {
        const int k = k0 + 32 * h + quad * 8;
        const uint32_t past = k >= K ? 0x80000000u : 0u;  // beyond any descriptor: zeros
        if constexpr (!DG) {
#pragma unroll
          for (int j = 0; j < NF; ++j)
            fw[q][h * NF + j] = buf_load16(rw, (uint32_t)(((j * 16 + row) * ldb + k) * 2) | past);
        }
#pragma unroll
        for (int i = 0; i < MT; ++i) fx[q][h][i] = buf_load16(rx, (uint32_t)(((i * 16 + row) * lda + k) * 2) | past);
      }
    }
#pragma unroll
    for (int q = 0; q < U; ++q) {
      if constexpr (DG) {
        u32x4 t[8];
        transpose8x8(fw[q], t);
#pragma unroll
        for (int j = 0; j < NF; ++j)
#pragma unroll
          for (int i = 0; i < MT; ++i) acc[i][j] = mfma16(as_bf16x8(t[j]), as_bf16x8(fx[q][0][i]), acc[i][j]);
      } else {
#pragma unroll
        for (int h = 0; h < XF; ++h)
#pragma unroll
          for (int j = 0; j < NF; ++j)
#pragma unroll
            for (int i = 0; i < MT; ++i)
              acc[i][j] = mfma16(as_bf16x8(fw[q][h * NF + j]), as_bf16x8(fx[q][h][i]), acc[i][j]);
      }
    }
  }
}

// The workgroup's sum of one row tile (of all waves' acc: waves 4-7 hand theirs to
// waves 0-3, whose four sums are added in ascending order) and its output rows
// from row0 of the group.
template <bool DG, int NF, int OUT>
__device__ __forceinline__ void skinny_store(const GroupedParams& p, const StepCursor& c, int row0, int tid, int wave,
                                             int lane, const f32x4 (&acc)[NF], f32x4 (*part)[NF][64]) {
  constexpr int HALF = kSkinnyWaves / 2;
  // the eight sums become four, then one
  if (wave >= HALF) {
#pragma unroll
    for (int j = 0; j < NF; ++j) part[wave - HALF][j][lane] = acc[j];
  }
  __syncthreads();
  if (wave < HALF) {
#pragma unroll
    for (int j = 0; j < NF; ++j) {
      f32x4& o = part[wave][j][lane];
      const f32x4 v = o;
      o = f32x4{acc[j][0] + v[0], acc[j][1] + v[1], acc[j][2] + v[2], acc[j][3] + v[3]};
    }
  }
  __syncthreads();
  if constexpr (DG) {
    // a thread's output: 8 consecutive columns of one row, one from each fragment
    const int l = tid >> 2, e = tid & 3;
    const int m = row0 + (l & 15), n = c.col0 + ((l >> 4) * 4 + e) * 8;
    if (tid < 256 && m < c.count && n < p.N) {
      float v[8];
#pragma unroll
      for (int f = 0; f < 8; ++f) {
        v[f] = part[0][f][l][e];
#pragma unroll
        for (int h = 1; h < HALF; ++h) v[f] += part[h][f][l][e];
      }
      const int64_t at = ((int64_t)c.base + m) * p.ldc + n;
      if constexpr (OUT == OUT_BF16) {
        *(u32x4*)((unsigned short*)p.c + at) = u32x4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                     pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
      } else {
        *(f32x4*)((float*)p.c + at) = f32x4{v[0], v[1], v[2], v[3]};
        *(f32x4*)((float*)p.c + at + 4) = f32x4{v[4], v[5], v[6], v[7]};
      }
    }
  } else {
    // a thread's output: 4 consecutive columns of one row
    const int j = tid >> 6;
    const int m = row0 + (lane & 15), n = c.col0 + j * 16 + (lane >> 4) * 4;
    if (tid < NF * 64 && m < c.count && n < p.N) {
      f32x4 v = part[0][j][lane];
#pragma unroll
      for (int h = 1; h < HALF; ++h) {
        const f32x4 o = part[h][j][lane];
        v = f32x4{v[0] + o[0], v[1] + o[1], v[2] + o[2], v[3] + o[3]};
      }
      const int64_t at = ((int64_t)c.base + m) * p.ldc + n;
      if constexpr (OUT == OUT_BF16)
        *(u32x2*)((unsigned short*)p.c + at) = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
      else
        *(f32x4*)((float*)p.c + at) = v;
    }
  }
  __syncthreads();  // before the next sums
}

template <bool DG, int MT, int NF, int U, bool ONCE, int OUT>
__device__ __forceinline__ void skinny_unit(const GroupedParams& p, const StepCursor& c, int tid, int wave, int lane,
                                            f32x4 (*part)[NF][64]) {
  f32x4 acc[MT][NF];
  skinny_products<DG, MT, NF, U, ONCE>(p, c, wave, lane, acc);
#pragma unroll
  for (int i = 0; i < MT; ++i) skinny_store<DG, NF, OUT>(p, c, c.row0 + 16 * i, tid, wave, lane, acc[i], part);
}

// DG: input gradient.  MT: row tiles of 16 in a unit; a unit with at most 16
// live rows does the work of one.  NF: weight fragments of a wave (input
// gradient: 8, one per column of a block).  U: steps loaded together by a wave
// with one row tile.
template <bool DG, int MT, int NF, int U, int OUT>
__global__ void __launch_bounds__(kSkinnyThreads, MT * NF > 16 ? 2 : 4) grouped_skinny_kernel(GroupedParams p) {
  static_assert(!DG || NF == 8, "one fragment per column of an 8x8 block");
  constexpr int BM = 16 * MT, BN = DG ? 128 : 16 * NF;
  __shared__ f32x4 part[kSkinnyWaves / 2][NF][64];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const GroupMap gm = group_map<BM, true>(p, lane);
  for (int u = blockIdx.x; u < gm.total; u += gridDim.x) {
    const StepCursor c = group_cursor<BM, BN, true>(p, gm, u);
    const int rows = min(c.count - c.row0, BM);
    if (c.b >= p.groups) {  // rows of no group
      f32x4 zero[NF];
#pragma unroll
      for (int j = 0; j < NF; ++j) zero[j] = f32x4{0.f, 0.f, 0.f, 0.f};
      for (int i = 0; i < rows; i += 16) skinny_store<DG, NF, OUT>(p, c, c.row0 + i, tid, wave, lane, zero, part);
    } else if (MT >= 2 && rows > 16) {
      skinny_unit<DG, MT, NF, (U + 1) / 2, false, OUT>(p, c, tid, wave, lane, part);
    } else if (DG && c.count <= 16) {
      skinny_unit<DG, 1, NF, U, DG, OUT>(p, c, tid, wave, lane, part);
    } else {
      skinny_unit<DG, 1, NF, U, false, OUT>(p, c, tid, wave, lane, part);
    }
  }
}

// ----------------------------------------------- forward, 16 by 16 units --
// lanes 0-31 of the result: a summed over the wave's halves, lanes 32-63: b
__device__ __forceinline__ float fold_halves(float a, float b) {
  const auto s = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b),
                                                  false, false);
  return __builtin_bit_cast(float, (uint32_t)s[0]) + __builtin_bit_cast(float, (uint32_t)s[1]);
}
// rows 0 and 2 (of 16 lanes): a summed over the rows of each half, rows 1 and 3: b
__device__ __forceinline__ float fold_rows(float a, float b) {
  const auto s = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b),
                                                  false, false);
  return __builtin_bit_cast(float, (uint32_t)s[0]) + __builtin_bit_cast(float, (uint32_t)s[1]);
}

// This wave's part of 16 columns by 4 TG rows, into part[row][column].  U: steps
// of 128 whose loads are issued together.
template <int TG, int U, bool ONCE>
__device__ __forceinline__ void rows16_products(const GroupedParams& p, const StepCursor& c, int wave, int lane,
                                                f32x4 (*part)[4]) {
  const int r4 = lane & 3, chunk = lane >> 2;
  const int lda = (int)p.lda, ldb = (int)p.ldb, K = p.K, steps = (K + 127) >> 7;
  const rsrc_t rx = rows_rsrc((const __bf16*)p.a + ((int64_t)c.base + c.row0) * lda, min(c.count - c.row0, 4 * TG),
                              lda, K);
  const rsrc_t rw = rows_rsrc((const __bf16*)p.b + (int64_t)c.b * p.batch_b + (int64_t)c.col0 * ldb,
                              min(p.N - c.col0, 16), ldb, K);
  const uint32_t xstep = 8u * (uint32_t)lda, wstep = 8u * (uint32_t)ldb;  // bytes of four rows
  const uint32_t x0 = (uint32_t)(r4 * lda + chunk * 8) * 2, w0 = (uint32_t)(r4 * ldb + chunk * 8) * 2;
  f32x4 acc[4][TG];
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int t = 0; t < TG; ++t) acc[j][t] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int s0 = wave; s0 < steps; s0 += kSkinnyWaves * U) {
    u32x4 fw[U][4], fx[U][TG];
#pragma unroll
    for (int q = 0; q < U; ++q) {
      const int k0 = (s0 + q * kSkinnyWaves) * 128;
      const uint32_t past = k0 + chunk * 8 >= K ? 0x80000000u : 0u;  // beyond any descriptor: zeros
#pragma unroll
      for (int j = 0; j < 4; ++j) fw[q][j] = load_weight<ONCE>(rw, (w0 + j * wstep + 2 * k0) | past);
#pragma unroll
      for (int t = 0; t < TG; ++t) fx[q][t] = buf_load16(rx, (x0 + t * xstep + 2 * k0) | past);
    }
#pragma unroll
    for (int q = 0; q < U; ++q)
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int t = 0; t < TG; ++t) acc[j][t] = mfma4(fw[q][j], fx[q][t], acc[j][t]);
  }
  // the 16 blocks: halves and rows of the wave while four registers become one
  // (row g of 16 lanes then holds columns 4 j + i, j = 2 (g & 1) + (g >> 1)),
  // then the four blocks of a row
  const int g = lane >> 4;
#pragma unroll
  for (int t = 0; t < TG; ++t) {
    f32x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float s = fold_rows(fold_halves(acc[0][t][i], acc[1][t][i]), fold_halves(acc[2][t][i], acc[3][t][i]));
      s += row_rotate<4>(s);
      s += row_rotate<8>(s);
      v[i] = s;
    }
    if ((lane & 12) == 0) part[4 * t + r4][2 * (g & 1) + (g >> 1)] = v;
  }
}

template <int OUT>
__global__ void __launch_bounds__(kSkinnyThreads, 4) grouped_rows16_kernel(GroupedParams p) {
  // two buffers: the other waves start the next unit while wave 0 adds up this one
  __shared__ f32x4 part[2][kSkinnyWaves][16][4];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const GroupMap gm = group_map<16, true>(p, lane);
  int odd = 0;
  for (int u = blockIdx.x; u < gm.total; u += gridDim.x, odd ^= 1) {
    const StepCursor c = group_cursor<16, 16, true>(p, gm, u);
    const int rows = min(c.count - c.row0, 16);
    const bool live = c.b < p.groups;  // else the rows of no group: zeros
    if (live) {
      if (c.count > 16)
        rows16_products<4, 1, false>(p, c, wave, lane, part[odd][wave]);
      else if (rows > 8)
        rows16_products<4, 1, true>(p, c, wave, lane, part[odd][wave]);
      else if (rows > 4)
        rows16_products<2, 2, true>(p, c, wave, lane, part[odd][wave]);
      else
        rows16_products<1, 4, true>(p, c, wave, lane, part[odd][wave]);
    }
    __syncthreads();
    if (wave == 0) {
      const int r = lane >> 2, n = c.col0 + (lane & 3) * 4;
      if (r < rows && n < p.N) {
        f32x4 v = {0.f, 0.f, 0.f, 0.f};
        if (live) {
          v = part[odd][0][r][lane & 3];
#pragma unroll
          for (int w = 1; w < kSkinnyWaves; ++w) {
            const f32x4 o = part[odd][w][r][lane & 3];
            v = f32x4{v[0] + o[0], v[1] + o[1], v[2] + o[2], v[3] + o[3]};
          }
        }
        const int64_t at = ((int64_t)c.base + c.row0 + r) * p.ldc + n;
        if constexpr (OUT == OUT_BF16)
          *(u32x2*)((unsigned short*)p.c + at) = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
        else
          *(f32x4*)((float*)p.c + at) = v;
      }
    }
  }
}

}  // namespace dpg

// AdamW over many tensors in one launch, moments in FP32 or in E4M3.
//
// Per element, with g the gradient times the optional device-side factor:
//   m = beta1 m + (1 - beta1) g
//   v = beta2 v + (1 - beta2) g^2
//   p = p (1 - lr decay) - (lr / c1) m / (sqrt(v) / sqrt(c2) + eps)
// with c = 1 - beta^step; all of it in FP32.
//
// 8-bit moments keep m and sqrt(v) -- the root halves the exponent range a
// block has to span -- as E4M3 codes with one power-of-two scale for 256
// consecutive elements of a tensor, which brings the block's largest magnitude
// to (224, 448].  The step itself uses the FP32 values before they are stored.
// Storing rounds up or down at random, up with the probability of the distance
// from the lower neighbour: a moment changes by a fraction 1 - beta of the
// difference to its target per step, far less than the 1/8 to 1/16 between
// neighbouring codes, so rounding to nearest would freeze it, while random
// rounding is right on average.  A positive root is never stored as zero:
// the next step divides by it.  NaN and infinities are stored as NaN.
#pragma once
#include "device_common.h"

namespace dpg {

constexpr int kAdamwBlock = 256;                  // elements of one scale: 4 per lane of a wave
constexpr int kAdamwSteps = 4;                    // blocks of one wave
constexpr int kAdamwChunk = 4 * kAdamwSteps * kAdamwBlock;  // elements of a workgroup's four waves
constexpr int kAdamwTensors = 48;                 // tensors of one launch: 3.5 KB of kernel arguments

struct AdamwTensor {
  float* p;
  const void* g;
  void* m;
  void* v;
  float* ms;
  float* vs;
  unsigned short* w;  // BF16 copy or null
  int64_t n;
};

struct AdamwParams {
  AdamwTensor t[kAdamwTensors];
  int chunk0[kAdamwTensors];       // first workgroup of each tensor
  unsigned key[kAdamwTensors];     // random key of each tensor
  int count;
  float beta1, rest1, beta2, rest2, decay, rate, root_scale, eps;
  const float* grad_scale;
};
static_assert(sizeof(AdamwParams) <= 4096, "kernel arguments");

// 32-bit mix of an element's place: a multiply by an odd constant (fractions
// of the golden ratio, sqrt(2) and sqrt(3)) carries low bits up, a shifted xor
// brings them down again.
__host__ __device__ __forceinline__ unsigned adamw_mix(unsigned x) {
  x ^= x >> 16;
  x *= 0x6A09E667u;
  x ^= x >> 15;
  x *= 0xBB67AE85u;
  return x ^ (x >> 16);
}
constexpr unsigned kAdamwStride = 0x9E3779B9u;

// Power of two that brings `top` (a block's largest magnitude) to (224, 448]:
// 448 = 1.75 * 2^8, so the exponent is that of `top` less 8, or less 7 when
// its mantissa is above 1.75.  The range is held to 2^-120 .. 2^127.
__device__ __forceinline__ float adamw_scale(float top) {
  const unsigned b = __builtin_bit_cast(unsigned, top);
  int e = (int)(b >> 23) - 127 - ((b & 0x7fffffu) <= 0x600000u ? 8 : 7);
  e = min(max(e, -120), 127);
  return top > 0.f ? __builtin_bit_cast(float, (unsigned)(e + 127) << 23) : 1.f;
}
// its reciprocal, exact (2^-127 is a denormal, which is a number here too)
__device__ __forceinline__ float adamw_inverse(float scale) { return 1.f / scale; }

// E4M3 code of x * inverse, rounded at random with 16 bits.  Codes of positive
// values ascend with them, so a rounding up is an addition of 20-bit fractions:
// to the FP32 pattern for normal codes, to the value in steps of 2^-9 below.
__device__ __forceinline__ unsigned adamw_code(float x, float inverse, unsigned bits16, bool floor1) {
  const float mag = fminf(fabsf(x) * inverse, 448.f);
  const unsigned r = (bits16 << 4) + 8;
  const unsigned big = ((__builtin_bit_cast(unsigned, mag) + r) >> 20) - (120u << 3);
  const unsigned small = ((unsigned)(mag * 0x1p29f) + r) >> 20;
  unsigned code = min(mag < 0x1p-6f ? small : big, 126u);
  if (floor1) code = mag > 0.f ? max(code, 1u) : code;
  if (!(fabsf(x) < __builtin_inff())) code = 127u;
  return code | (x < 0.f ? 128u : 0u);
}

template <int GRAD_BYTES, bool E4M3>
__global__ void __launch_bounds__(256) adamw_kernel(AdamwParams p) {
  // every product and sum is rounded by itself, as the formulas read: with
  // fused multiply-adds a moment would differ in its last bit from the same
  // formulas computed step by step, and now and then take another stored code
#pragma clang fp contract(off)
  int lo = 0, hi = p.count;  // the tensor of this workgroup: the last one that starts at it or before
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (p.chunk0[mid] <= (int)blockIdx.x)
      lo = mid;
    else
      hi = mid;
  }
  const AdamwTensor t = p.t[lo];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t first = (int64_t)((int)blockIdx.x - p.chunk0[lo]) * kAdamwChunk + wave * (kAdamwSteps * kAdamwBlock);
  const float gs = p.grad_scale ? *p.grad_scale : 1.f;
  // whole quads through 16-byte (FP32), 8-byte (BF16) and 4-byte (codes)
  // accesses where the tensor's pointers allow them
  const uintptr_t low = (uintptr_t)t.p | (E4M3 ? ((uintptr_t)t.m | (uintptr_t)t.v) << 2 : (uintptr_t)t.m | (uintptr_t)t.v) |
                        ((uintptr_t)t.w << 1) | (GRAD_BYTES == 2 ? (uintptr_t)t.g << 1 : (uintptr_t)t.g);
  const bool wide = (low & 15) == 0;
#pragma unroll
  for (int s = 0; s < kAdamwSteps; ++s) {
    const int64_t block = first + s * kAdamwBlock;
    if (block >= t.n) return;
    const int64_t i = block + 4 * lane;
    const int have = (int)min((int64_t)4, max((int64_t)0, t.n - i));
    const bool quad = wide && have == 4;
    float pv[4] = {0.f, 0.f, 0.f, 0.f}, g[4] = {0.f, 0.f, 0.f, 0.f};
    float m[4] = {0.f, 0.f, 0.f, 0.f}, v[4] = {0.f, 0.f, 0.f, 0.f};
    const float ms = E4M3 ? t.ms[block / kAdamwBlock] : 1.f, vs = E4M3 ? t.vs[block / kAdamwBlock] : 1.f;
    unsigned mc = 0, vc = 0;
    if (quad) {
      const f32x4 q = *(const f32x4*)(t.p + i);
#pragma unroll
      for (int e = 0; e < 4; ++e) pv[e] = q[e];
      if (GRAD_BYTES == 2) {
        const u32x2 h = *(const u32x2*)((const unsigned short*)t.g + i);
        g[0] = bf16_value(h[0] & 0xffffu);
        g[1] = __builtin_bit_cast(float, h[0] & 0xffff0000u);
        g[2] = bf16_value(h[1] & 0xffffu);
        g[3] = __builtin_bit_cast(float, h[1] & 0xffff0000u);
      } else {
        const f32x4 h = *(const f32x4*)((const float*)t.g + i);
#pragma unroll
        for (int e = 0; e < 4; ++e) g[e] = h[e];
      }
      if (E4M3) {
        mc = *(const unsigned*)((const unsigned char*)t.m + i);
        vc = *(const unsigned*)((const unsigned char*)t.v + i);
      } else {
        const f32x4 a = *(const f32x4*)((const float*)t.m + i), b = *(const f32x4*)((const float*)t.v + i);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          m[e] = a[e];
          v[e] = b[e];
        }
      }
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (e >= have) continue;
        pv[e] = t.p[i + e];
        g[e] = GRAD_BYTES == 2 ? bf16_value(((const unsigned short*)t.g)[i + e]) : ((const float*)t.g)[i + e];
        if (E4M3) {
          mc |= (unsigned)((const unsigned char*)t.m)[i + e] << (8 * e);
          vc |= (unsigned)((const unsigned char*)t.v)[i + e] << (8 * e);
        } else {
          m[e] = ((const float*)t.m)[i + e];
          v[e] = ((const float*)t.v)[i + e];
        }
      }
    }
    if (E4M3) {
      m[0] = __builtin_amdgcn_cvt_f32_fp8((int)mc, 0) * ms;
      m[1] = __builtin_amdgcn_cvt_f32_fp8((int)mc, 1) * ms;
      m[2] = __builtin_amdgcn_cvt_f32_fp8((int)mc, 2) * ms;
      m[3] = __builtin_amdgcn_cvt_f32_fp8((int)mc, 3) * ms;
      v[0] = __builtin_amdgcn_cvt_f32_fp8((int)vc, 0) * vs;
      v[1] = __builtin_amdgcn_cvt_f32_fp8((int)vc, 1) * vs;
      v[2] = __builtin_amdgcn_cvt_f32_fp8((int)vc, 2) * vs;
      v[3] = __builtin_amdgcn_cvt_f32_fp8((int)vc, 3) * vs;
    }
    float root[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float ge = g[e] * gs;
      if (E4M3) v[e] *= v[e];
      m[e] = p.beta1 * m[e] + p.rest1 * ge;
      v[e] = p.beta2 * v[e] + p.rest2 * ge * ge;
      root[e] = sqrtf(v[e]);
      pv[e] = pv[e] * p.decay - p.rate * m[e] / (root[e] * p.root_scale + p.eps);
    }
    if (E4M3) {
      float top_m = 0.f, top_r = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        top_m = e < have ? fmaxf(top_m, fabsf(m[e])) : top_m;
        top_r = e < have ? fmaxf(top_r, root[e]) : top_r;
      }
      const float new_ms = adamw_scale(wave_max(top_m)), new_vs = adamw_scale(wave_max(top_r));
      const float im = adamw_inverse(new_ms), ir = adamw_inverse(new_vs);
      // elements past 2^32 of a tensor take another key
      const unsigned key = p.key[lo] + (unsigned)(i >> 32) * 0x6A09E667u;
      mc = vc = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const unsigned word = adamw_mix((unsigned)(i + e) * kAdamwStride + key);
        mc |= adamw_code(m[e], im, word & 0xffffu, false) << (8 * e);
        vc |= adamw_code(root[e], ir, word >> 16, true) << (8 * e);
      }
      if (lane == 0) {
        t.ms[block / kAdamwBlock] = new_ms;
        t.vs[block / kAdamwBlock] = new_vs;
      }
    }
    if (quad) {
      *(f32x4*)(t.p + i) = f32x4{pv[0], pv[1], pv[2], pv[3]};
      if (t.w) *(u32x2*)(t.w + i) = u32x2{pack_bf16x2(pv[0], pv[1]), pack_bf16x2(pv[2], pv[3])};
      if (E4M3) {
        *(unsigned*)((unsigned char*)t.m + i) = mc;
        *(unsigned*)((unsigned char*)t.v + i) = vc;
      } else {
        *(f32x4*)((float*)t.m + i) = f32x4{m[0], m[1], m[2], m[3]};
        *(f32x4*)((float*)t.v + i) = f32x4{v[0], v[1], v[2], v[3]};
      }
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (e >= have) continue;
        t.p[i + e] = pv[e];
        if (t.w) t.w[i + e] = (unsigned short)bf16_bits(pv[e]);
        if (E4M3) {
          ((unsigned char*)t.m)[i + e] = (unsigned char)(mc >> (8 * e));
          ((unsigned char*)t.v)[i + e] = (unsigned char)(vc >> (8 * e));
        } else {
          ((float*)t.m)[i + e] = m[e];
          ((float*)t.v)[i + e] = v[e];
        }
      }
    }
  }
}

}  // namespace dpg

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
// consecutive elements of a tensor, which brings the block's largest finite
// magnitude to (224, 448].  The step itself uses the FP32 values before they
// are stored.  Storing rounds up or down at random, up with the probability of the distance
// from the lower neighbour: a moment changes by a fraction 1 - beta of the
// difference to its target per step, far less than the 1/8 to 1/16 between
// neighbouring codes, so rounding to nearest would freeze it, while random
// rounding is right on average.  A positive root is never stored as zero:
// the next step divides by it.  NaN and infinities are stored as NaN and have
// no part in the scale: an infinite one would leave its 255 neighbours without
// their moments, and without their parameters two steps later.
#pragma once
#include "device_common.h"

namespace dpg {

constexpr int kAdamwBlock = 256;                  // elements of one scale: 4 per lane of a wave
// Blocks of one wave, loaded before the first is worked on: four, or one where
// a call has few elements and each wave's own time counts.
constexpr int kAdamwSteps = 4;
// elements of a workgroup's four waves
constexpr int adamw_chunk(int steps) { return 4 * steps * kAdamwBlock; }
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

// Power of two that brings `top` (a block's largest finite magnitude) to (224, 448]:
// 448 = 1.75 * 2^8, so the exponent is that of `top` less 8, or less 7 when
// its mantissa is above 1.75.  The range is held to 2^-120 .. 2^127.
__device__ __forceinline__ float adamw_scale(float top) {
  const unsigned b = __builtin_bit_cast(unsigned, top);
  int e = (int)(b >> 23) - 127 - ((b & 0x7fffffu) <= 0x600000u ? 8 : 7);
  e = min(max(e, -120), 127);
  return top > 0.f ? __builtin_bit_cast(float, (unsigned)(e + 127) << 23) : 1.f;
}
// The block's largest finite magnitude, from four values of each lane: as
// integers, the pattern without its sign and moved up by what an infinity
// lacks to 2^32, so that infinities and NaN wrap to below zero's place (201
// million parameters 660 us; 655 with a maximum that infinities take part in,
// 668 with a comparison of each value to infinity).  Elements past the tensor
// are zeros, or NaN by a strange factor.
__device__ __forceinline__ float adamw_top(const float (&x)[4]) {
  constexpr unsigned kZero = 0x01000000u;
  unsigned top = kZero;
#pragma unroll
  for (int e = 0; e < 4; ++e) top = max(top, (__builtin_bit_cast(unsigned, x[e]) << 1) + kZero);
  return wave_max(__builtin_bit_cast(float, (top - kZero) >> 1));
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

// Four consecutive elements of a lane as they are in memory, and their block's
// scales.  `have` counts the valid ones; the others are zeros.
struct AdamwQuad {
  float p[4], g[4], m[4], v[4];
  unsigned mc, vc;  // E4M3 codes
  float ms, vs;
  int have;
};

// Everything is read and written once: non-temporal accesses.  201 million
// parameters, 32-bit moments, BF16 gradients and copies: 1064 us without, 980
// with, and 952 (5.9 TB/s) with four blocks of a wave in flight instead of one;
// 8-bit moments and FP32 gradients 692, 660 and 655 (5.5 TB/s).
template <class T>
__device__ __forceinline__ T adamw_load(const void* p) {
  return __builtin_nontemporal_load((const T*)p);
}

template <int GRAD_BYTES, bool E4M3>
__device__ __forceinline__ void adamw_fetch(const AdamwTensor& t, int64_t block, int lane, bool wide, AdamwQuad& q) {
  const int64_t i = block + 4 * lane;
  q.have = (int)min((int64_t)4, max((int64_t)0, t.n - i));
  q.mc = q.vc = 0;
  q.ms = E4M3 ? t.ms[block / kAdamwBlock] : 1.f;
  q.vs = E4M3 ? t.vs[block / kAdamwBlock] : 1.f;
#pragma unroll
  for (int e = 0; e < 4; ++e) q.p[e] = q.g[e] = q.m[e] = q.v[e] = 0.f;
  if (wide && q.have == 4) {
    const f32x4 p = adamw_load<f32x4>(t.p + i);
#pragma unroll
    for (int e = 0; e < 4; ++e) q.p[e] = p[e];
    if (GRAD_BYTES == 2) {
      const u32x2 h = adamw_load<u32x2>((const unsigned short*)t.g + i);
      q.g[0] = bf16_value(h[0] & 0xffffu);
      q.g[1] = __builtin_bit_cast(float, h[0] & 0xffff0000u);
      q.g[2] = bf16_value(h[1] & 0xffffu);
      q.g[3] = __builtin_bit_cast(float, h[1] & 0xffff0000u);
    } else {
      const f32x4 h = adamw_load<f32x4>((const float*)t.g + i);
#pragma unroll
      for (int e = 0; e < 4; ++e) q.g[e] = h[e];
    }
    if (E4M3) {
      q.mc = adamw_load<unsigned>((const unsigned char*)t.m + i);
      q.vc = adamw_load<unsigned>((const unsigned char*)t.v + i);
    } else {
      const f32x4 a = adamw_load<f32x4>((const float*)t.m + i), b = adamw_load<f32x4>((const float*)t.v + i);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        q.m[e] = a[e];
        q.v[e] = b[e];
      }
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (e >= q.have) continue;
      q.p[e] = t.p[i + e];
      q.g[e] = GRAD_BYTES == 2 ? bf16_value(((const unsigned short*)t.g)[i + e]) : ((const float*)t.g)[i + e];
      if (E4M3) {
        q.mc |= (unsigned)((const unsigned char*)t.m)[i + e] << (8 * e);
        q.vc |= (unsigned)((const unsigned char*)t.v)[i + e] << (8 * e);
      } else {
        q.m[e] = ((const float*)t.m)[i + e];
        q.v[e] = ((const float*)t.v)[i + e];
      }
    }
  }
}

template <bool E4M3>
__device__ __forceinline__ void adamw_update(const AdamwParams& p, const AdamwTensor& t, unsigned tensor_key, float gs,
                                             int64_t block, int lane, bool wide, AdamwQuad& q) {
  // every product and sum is rounded by itself, as the formulas read: with
  // fused multiply-adds a moment would differ in its last bit from the same
  // formulas computed step by step, and now and then take another stored code
#pragma clang fp contract(off)
  const int64_t i = block + 4 * lane;
  if (E4M3) {
    q.m[0] = __builtin_amdgcn_cvt_f32_fp8((int)q.mc, 0) * q.ms;
    q.m[1] = __builtin_amdgcn_cvt_f32_fp8((int)q.mc, 1) * q.ms;
    q.m[2] = __builtin_amdgcn_cvt_f32_fp8((int)q.mc, 2) * q.ms;
    q.m[3] = __builtin_amdgcn_cvt_f32_fp8((int)q.mc, 3) * q.ms;
    q.v[0] = __builtin_amdgcn_cvt_f32_fp8((int)q.vc, 0) * q.vs;
    q.v[1] = __builtin_amdgcn_cvt_f32_fp8((int)q.vc, 1) * q.vs;
    q.v[2] = __builtin_amdgcn_cvt_f32_fp8((int)q.vc, 2) * q.vs;
    q.v[3] = __builtin_amdgcn_cvt_f32_fp8((int)q.vc, 3) * q.vs;
  }
  float root[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float g = q.g[e] * gs;
    if (E4M3) q.v[e] *= q.v[e];
    q.m[e] = p.beta1 * q.m[e] + p.rest1 * g;
    q.v[e] = p.beta2 * q.v[e] + p.rest2 * g * g;
    root[e] = sqrtf(q.v[e]);
    q.p[e] = q.p[e] * p.decay - p.rate * q.m[e] / (root[e] * p.root_scale + p.eps);
  }
  if (E4M3) {
    const float new_ms = adamw_scale(adamw_top(q.m)), new_vs = adamw_scale(adamw_top(root));
    const float im = adamw_inverse(new_ms), ir = adamw_inverse(new_vs);
    // elements past 2^32 of a tensor take another key
    const unsigned key = tensor_key + (unsigned)(i >> 32) * 0x6A09E667u;
    q.mc = q.vc = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const unsigned word = adamw_mix((unsigned)(i + e) * kAdamwStride + key);
      q.mc |= adamw_code(q.m[e], im, word & 0xffffu, false) << (8 * e);
      q.vc |= adamw_code(root[e], ir, word >> 16, true) << (8 * e);
    }
    if (lane == 0) {
      t.ms[block / kAdamwBlock] = new_ms;
      t.vs[block / kAdamwBlock] = new_vs;
    }
  }
  if (wide && q.have == 4) {
    __builtin_nontemporal_store(f32x4{q.p[0], q.p[1], q.p[2], q.p[3]}, (f32x4*)(t.p + i));
    if (t.w)
      __builtin_nontemporal_store(u32x2{pack_bf16x2(q.p[0], q.p[1]), pack_bf16x2(q.p[2], q.p[3])}, (u32x2*)(t.w + i));
    if (E4M3) {
      __builtin_nontemporal_store(q.mc, (unsigned*)((unsigned char*)t.m + i));
      __builtin_nontemporal_store(q.vc, (unsigned*)((unsigned char*)t.v + i));
    } else {
      __builtin_nontemporal_store(f32x4{q.m[0], q.m[1], q.m[2], q.m[3]}, (f32x4*)((float*)t.m + i));
      __builtin_nontemporal_store(f32x4{q.v[0], q.v[1], q.v[2], q.v[3]}, (f32x4*)((float*)t.v + i));
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (e >= q.have) continue;
      t.p[i + e] = q.p[e];
      if (t.w) t.w[i + e] = (unsigned short)bf16_bits(q.p[e]);
      if (E4M3) {
        ((unsigned char*)t.m)[i + e] = (unsigned char)(q.mc >> (8 * e));
        ((unsigned char*)t.v)[i + e] = (unsigned char)(q.vc >> (8 * e));
      } else {
        ((float*)t.m)[i + e] = q.m[e];
        ((float*)t.v)[i + e] = q.v[e];
      }
    }
  }
}

template <int GRAD_BYTES, bool E4M3, int STEPS>
__global__ void __launch_bounds__(256) adamw_kernel(AdamwParams p) {
  int lo = 0, hi = p.count;  // the tensor of this workgroup: the last one that starts at it or before
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (p.chunk0[mid] <= (int)blockIdx.x)
      lo = mid;
    else
      hi = mid;
  }
  const AdamwTensor t = p.t[lo];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t first = (int64_t)((int)blockIdx.x - p.chunk0[lo]) * adamw_chunk(STEPS) +
                        wave * (STEPS * kAdamwBlock);
  const float gs = p.grad_scale ? *p.grad_scale : 1.f;
  // whole quads through 16-byte (FP32), 8-byte (BF16) and 4-byte (codes)
  // accesses where the tensor's pointers allow them
  const uintptr_t low = (uintptr_t)t.p | (E4M3 ? ((uintptr_t)t.m | (uintptr_t)t.v) << 2 : (uintptr_t)t.m | (uintptr_t)t.v) |
                        ((uintptr_t)t.w << 1) | (GRAD_BYTES == 2 ? (uintptr_t)t.g << 1 : (uintptr_t)t.g);
  const bool wide = (low & 15) == 0;
  AdamwQuad q[STEPS];
#pragma unroll
  for (int s = 0; s < STEPS; ++s)
    if (first + s * kAdamwBlock < t.n)
      adamw_fetch<GRAD_BYTES, E4M3>(t, first + s * kAdamwBlock, lane, wide, q[s]);
#pragma unroll
  for (int s = 0; s < STEPS; ++s) {
    if (first + s * kAdamwBlock >= t.n) return;
    adamw_update<E4M3>(p, t, p.key[lo], gs, first + s * kAdamwBlock, lane, wide, q[s]);
  }
}

}  // namespace dpg

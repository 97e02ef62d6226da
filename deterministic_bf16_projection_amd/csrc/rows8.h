// Rows of BF16 or FP32 in groups of eight consecutive elements, one group to a
// lane: 16 or 32 bytes.
#pragma once
#include "device_common.h"

namespace dpg {

struct Rows8 {
  void* data;
  int64_t ld;  // elements between rows
};

template <bool BF16>
struct Raw8;
template <>
struct Raw8<true> {
  u32x4 a;
};
template <>
struct Raw8<false> {
  f32x4 a, b;
};

// NT: past the caches
template <bool BF16, bool NT = false>
__device__ __forceinline__ Raw8<BF16> load8(const Rows8& m, int64_t row, int group) {
  const auto get = [](const auto* at) { return NT ? __builtin_nontemporal_load(at) : *at; };
  if constexpr (BF16) {
    return Raw8<true>{get((const u32x4*)((const unsigned short*)m.data + row * m.ld) + group)};
  } else {
    const f32x4* at = (const f32x4*)((const float*)m.data + row * m.ld) + 2 * group;
    return Raw8<false>{get(at), get(at + 1)};
  }
}

__device__ __forceinline__ void unpack8(const Raw8<true>& r, float (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = bf16_value(r.a[j] & 0xffffu);
    v[2 * j + 1] = __builtin_bit_cast(float, r.a[j] & 0xffff0000u);
  }
}
__device__ __forceinline__ void unpack8(const Raw8<false>& r, float (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[j] = r.a[j];
    v[j + 4] = r.b[j];
  }
}

template <bool BF16, bool NT = false>
__device__ __forceinline__ void store8(const Rows8& m, int64_t row, int group, const float (&v)[8]) {
  const auto put = [](auto* at, const auto& value) {
    if (NT)
      __builtin_nontemporal_store(value, at);
    else
      *at = value;
  };
  if constexpr (BF16) {
    put((u32x4*)((unsigned short*)m.data + row * m.ld) + group,
        u32x4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])});
  } else {
    f32x4* at = (f32x4*)((float*)m.data + row * m.ld) + 2 * group;
    put(at, f32x4{v[0], v[1], v[2], v[3]});
    put(at + 1, f32x4{v[4], v[5], v[6], v[7]});
  }
}

}  // namespace dpg

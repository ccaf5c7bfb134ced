// Rows of bf16 or fp32 in pieces of 8 elements, at any element alignment, and
// wave sums in a fixed order: what the row-streaming kernels (layer norm,
// optimizer) share.
#pragma once

#include "common.h"

namespace moe {

// gfx950 reads and writes 16 bytes at any address; the type states only the
// element's alignment, so odd widths and offset views take the same path
typedef u32x4 u32x4_a2 __attribute__((aligned(2)));
typedef u32x4 u32x4_a4 __attribute__((aligned(4)));

// 8 values as they are stored
template <typename T>
struct Raw8;
template <>
struct Raw8<uint16_t> {
  u32x4 a;
};
template <>
struct Raw8<float> {
  u32x4 a, b;
};

// n: how many of the 8 exist (the others read as 0 and are not touched)
__device__ __forceinline__ void load8(Raw8<uint16_t>& r, const uint16_t* p, int n) {
  if (n >= 8) {
    r.a = __builtin_nontemporal_load(reinterpret_cast<const u32x4_a2*>(p));
  } else {
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (i < n) w[i / 2] |= static_cast<uint32_t>(p[i]) << (16 * (i & 1));
    r.a = u32x4{w[0], w[1], w[2], w[3]};
  }
}
__device__ __forceinline__ void load8(Raw8<float>& r, const float* p, int n) {
  if (n >= 8) {
    r.a = __builtin_nontemporal_load(reinterpret_cast<const u32x4_a4*>(p));
    r.b = __builtin_nontemporal_load(reinterpret_cast<const u32x4_a4*>(p + 4));
  } else {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = i < n ? __float_as_uint(p[i]) : 0u;
    r.a = u32x4{w[0], w[1], w[2], w[3]};
    r.b = u32x4{w[4], w[5], w[6], w[7]};
  }
}

__device__ __forceinline__ void to_f32(const Raw8<uint16_t>& r, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(r.a[i] << 16);
    f[2 * i + 1] = __uint_as_float(r.a[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void to_f32(const Raw8<float>& r, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[i] = __uint_as_float(r.a[i]);
    f[4 + i] = __uint_as_float(r.b[i]);
  }
}

// rounded to the stored type (nearest even; NaN stays NaN)
__device__ __forceinline__ void from_f32(Raw8<uint16_t>& r, const float (&f)[8]) {
  r.a = u32x4{pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7])};
}
__device__ __forceinline__ void from_f32(Raw8<float>& r, const float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r.a[i] = __float_as_uint(f[i]);
    r.b[i] = __float_as_uint(f[4 + i]);
  }
}

__device__ __forceinline__ void store8(uint16_t* p, const Raw8<uint16_t>& r, int n) {
  if (n >= 8) {
    *reinterpret_cast<u32x4_a2*>(p) = r.a;
  } else {
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (i < n) p[i] = static_cast<uint16_t>(r.a[i / 2] >> (16 * (i & 1)));
  }
}
__device__ __forceinline__ void store8(float* p, const Raw8<float>& r, int n) {
  if (n >= 8) {
    *reinterpret_cast<u32x4_a4*>(p) = r.a;
    *reinterpret_cast<u32x4_a4*>(p + 4) = r.b;
  } else {
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (i < n) p[i] = __uint_as_float(i < 4 ? r.a[i & 3] : r.b[i & 3]);
  }
}

// Sum over the 64 lanes in every lane, by the same tree on every call: DPP
// moves inside 16-lane rows, then gfx950's row swaps.  Every lane of the wave
// must be active.
template <int CTRL>
__device__ __forceinline__ float dpp_f32(float v) {
  return __uint_as_float(__builtin_amdgcn_update_dpp(0u, __float_as_uint(v), CTRL, 0xF, 0xF, false));
}
__device__ __forceinline__ float wave_sum(float v) {
  v += dpp_f32<0xB1>(v);   // quad_perm [1,0,3,2]
  v += dpp_f32<0x4E>(v);   // quad_perm [2,3,0,1]
  v += dpp_f32<0x141>(v);  // row_half_mirror
  v += dpp_f32<0x140>(v);  // row_mirror
  const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

}  // namespace moe

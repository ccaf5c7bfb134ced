// Pieces of E consecutive elements of a row (bf16 or fp32) at any element
// alignment, and wave maxima: what the kernels on table rows (embedding) and on
// rows of logits (distillation and policy losses) share beside stream8.h.
//
// E is chosen so that a lane moves 16 bytes of the wider of the types it reads
// and writes: a wave's access then covers one solid kilobyte.
#pragma once

#include <float.h>

#include "stream8.h"

namespace moe {

typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef u32x2 u32x2_a2 __attribute__((aligned(2)));

// a piece as it is stored, in 32-bit words
template <typename T, int E>
struct Vec {
  static constexpr int kWords = E * static_cast<int>(sizeof(T)) / 4;
  uint32_t w[kWords];
};

template <bool STREAM, typename T, int E>
__device__ __forceinline__ void load_vec(Vec<T, E>& v, const T* p) {
  if constexpr (Vec<T, E>::kWords == 2) {  // bf16 x 4
    const u32x2_a2* q = reinterpret_cast<const u32x2_a2*>(p);
    const u32x2 a = STREAM ? u32x2(__builtin_nontemporal_load(q)) : u32x2(*q);
    v.w[0] = a[0];
    v.w[1] = a[1];
  } else {
#pragma unroll
    for (int h = 0; h < Vec<T, E>::kWords / 4; ++h) {
      u32x4 a;
      if constexpr (sizeof(T) == 2) {
        const u32x4_a2* q = reinterpret_cast<const u32x4_a2*>(p) + h;
        a = STREAM ? u32x4(__builtin_nontemporal_load(q)) : u32x4(*q);
      } else {
        const u32x4_a4* q = reinterpret_cast<const u32x4_a4*>(p) + h;
        a = STREAM ? u32x4(__builtin_nontemporal_load(q)) : u32x4(*q);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) v.w[4 * h + i] = a[i];
    }
  }
}

template <bool STREAM, typename T, int E>
__device__ __forceinline__ void store_vec(T* p, const Vec<T, E>& v) {
  if constexpr (Vec<T, E>::kWords == 2) {
    const u32x2 a = {v.w[0], v.w[1]};
    u32x2_a2* q = reinterpret_cast<u32x2_a2*>(p);
    if constexpr (STREAM) __builtin_nontemporal_store(u32x2_a2(a), q);
    else *q = a;
  } else {
#pragma unroll
    for (int h = 0; h < Vec<T, E>::kWords / 4; ++h) {
      const u32x4 a = {v.w[4 * h], v.w[4 * h + 1], v.w[4 * h + 2], v.w[4 * h + 3]};
      if constexpr (sizeof(T) == 2) {
        u32x4_a2* q = reinterpret_cast<u32x4_a2*>(p) + h;
        if constexpr (STREAM) __builtin_nontemporal_store(u32x4_a2(a), q);
        else *q = a;
      } else {
        u32x4_a4* q = reinterpret_cast<u32x4_a4*>(p) + h;
        if constexpr (STREAM) __builtin_nontemporal_store(u32x4_a4(a), q);
        else *q = a;
      }
    }
  }
}

template <typename T, int E>
__device__ __forceinline__ void vec_f32(const Vec<T, E>& v, float (&f)[E]) {
#pragma unroll
  for (int i = 0; i < E; ++i) {
    if constexpr (sizeof(T) == 2) f[i] = __uint_as_float(i % 2 == 0 ? v.w[i / 2] << 16 : v.w[i / 2] & 0xFFFF0000u);
    else f[i] = __uint_as_float(v.w[i]);
  }
}

// rounded to the stored type (nearest even; NaN stays NaN)
template <typename T, int E>
__device__ __forceinline__ void f32_vec(Vec<T, E>& v, const float (&f)[E]) {
#pragma unroll
  for (int i = 0; i < Vec<T, E>::kWords; ++i) {
    if constexpr (sizeof(T) == 2) v.w[i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
    else v.w[i] = __float_as_uint(f[i]);
  }
}

__device__ __forceinline__ void put_one(uint16_t* p, float f) { *p = static_cast<uint16_t>(pack_bf16x2(f, f)); }
__device__ __forceinline__ void put_one(float* p, float f) { *p = f; }

// Maximum over 16 lanes, and over the wave, in every lane (every lane active).
// NaN does not take part.
__device__ __forceinline__ float row16_max(float v) {
  v = fmaxf(v, dpp_f32<0xB1>(v));
  v = fmaxf(v, dpp_f32<0x4E>(v));
  v = fmaxf(v, dpp_f32<0x141>(v));
  return fmaxf(v, dpp_f32<0x140>(v));
}
__device__ __forceinline__ float wave_max(float v) {
  v = row16_max(v);
  const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}

}  // namespace moe

// Rows of bf16 or fp32 in pieces of 8 elements, at any element alignment, and
// wave sums in a fixed order: what the row-streaming kernels (layer norm,
// optimizer, balance loss) share.
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

// A lane's piece of a row of d elements: the 8 columns [c, c + 8), of which it
// owns [lo, hi).  A row's last piece is moved back to end with the row, so that
// it is loaded whole too and owns only what the piece before it does not reach;
// rows shorter than 8 have one partial piece.  lo = 8: no piece.
struct Piece {
  int c, lo, hi;
};
__device__ __forceinline__ Piece piece_of(int i, int d) {
  const int c = i * 8;
  if (d < 8) return {0, i == 0 ? 0 : 8, d};
  const int back = max(0, c + 8 - d);
  return {c - back, min(back, 8), 8};
}
__device__ __forceinline__ bool owns(const Piece& q, int j) { return j >= q.lo && j < q.hi; }

// Loads the piece (zeros where there is none, or past hi).  STREAM: past the
// caches; without it data that is still in the 256 MB cache of the package, as
// a kernel before left it, is found there.
template <bool STREAM>
__device__ __forceinline__ void load8(Raw8<uint16_t>& r, const uint16_t* p, const Piece& q) {
  r.a = u32x4{0, 0, 0, 0};
  if (q.lo >= 8) return;
  p += q.c;
  if (q.hi == 8) {
    if constexpr (STREAM) r.a = __builtin_nontemporal_load(reinterpret_cast<const u32x4_a2*>(p));
    else r.a = *reinterpret_cast<const u32x4_a2*>(p);
  } else {
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (i < q.hi) w[i / 2] |= static_cast<uint32_t>(p[i]) << (16 * (i & 1));
    r.a = u32x4{w[0], w[1], w[2], w[3]};
  }
}
template <bool STREAM>
__device__ __forceinline__ void load8(Raw8<float>& r, const float* p, const Piece& q) {
  r.a = r.b = u32x4{0, 0, 0, 0};
  if (q.lo >= 8) return;
  p += q.c;
  if (q.hi == 8) {
    if constexpr (STREAM) {
      r.a = __builtin_nontemporal_load(reinterpret_cast<const u32x4_a4*>(p));
      r.b = __builtin_nontemporal_load(reinterpret_cast<const u32x4_a4*>(p + 4));
    } else {
      r.a = *reinterpret_cast<const u32x4_a4*>(p);
      r.b = *reinterpret_cast<const u32x4_a4*>(p + 4);
    }
  } else {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = i < q.hi ? __float_as_uint(p[i]) : 0u;
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

__device__ __forceinline__ float one_f32(uint16_t v) { return bf16_to_f32(v); }
__device__ __forceinline__ float one_f32(float v) { return v; }

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

// stores the elements the piece owns, past the caches
__device__ __forceinline__ void store8(uint16_t* p, const Raw8<uint16_t>& r, const Piece& q) {
  p += q.c;
  if (q.lo == 0 && q.hi == 8) {
    __builtin_nontemporal_store(r.a, reinterpret_cast<u32x4_a2*>(p));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (owns(q, i)) p[i] = static_cast<uint16_t>(r.a[i / 2] >> (16 * (i & 1)));
  }
}
__device__ __forceinline__ void store8(float* p, const Raw8<float>& r, const Piece& q) {
  p += q.c;
  if (q.lo == 0 && q.hi == 8) {
    __builtin_nontemporal_store(r.a, reinterpret_cast<u32x4_a4*>(p));
    __builtin_nontemporal_store(r.b, reinterpret_cast<u32x4_a4*>(p + 4));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (owns(q, i)) p[i] = __uint_as_float(i < 4 ? r.a[i & 3] : r.b[i & 3]);
  }
}
// zeros the elements the piece does not own
__device__ __forceinline__ void mask8(float (&f)[8], const Piece& q) {
  if (q.lo == 0 && q.hi == 8) return;
#pragma unroll
  for (int j = 0; j < 8; ++j) f[j] = owns(q, j) ? f[j] : 0.0f;
}

// Sum over the 64 lanes in every lane, by the same tree on every call: DPP
// moves inside 16-lane rows, then gfx950's row swaps.  Every lane of the wave
// must be active.
template <int CTRL>
__device__ __forceinline__ float dpp_f32(float v) {
  return __uint_as_float(__builtin_amdgcn_update_dpp(0u, __float_as_uint(v), CTRL, 0xF, 0xF, false));
}
__device__ __forceinline__ float row16_sum(float v) {  // over 16 lanes
  v += dpp_f32<0xB1>(v);          // quad_perm [1,0,3,2]
  v += dpp_f32<0x4E>(v);          // quad_perm [2,3,0,1]
  v += dpp_f32<0x141>(v);         // row_half_mirror
  return v + dpp_f32<0x140>(v);   // row_mirror
}
__device__ __forceinline__ float wave_sum(float v) {
  v = row16_sum(v);
  const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

// the same over aligned groups of lpt lanes (a power of two); the lanes of a
// group must be active, all 64 of them for lpt = 64
__device__ __forceinline__ float group_sum(float v, int lpt) {
  if (lpt == kWave) return wave_sum(v);
  if (lpt >= 2) v += dpp_f32<0xB1>(v);
  if (lpt >= 4) v += dpp_f32<0x4E>(v);
  if (lpt >= 8) v += dpp_f32<0x141>(v);
  if (lpt >= 16) v += dpp_f32<0x140>(v);
  if (lpt >= 32) v += __shfl_xor(v, 16, kWave);
  return v;
}

}  // namespace moe

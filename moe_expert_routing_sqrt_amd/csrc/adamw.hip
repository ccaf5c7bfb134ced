// AdamW over many tensors in one launch, the states in fp32 or in 8 bits.
//
//   g' = g * scale
//   m  = b1 m + (1 - b1) g',   v = b2 v + (1 - b2) g' g'
//   w  = w (1 - lr wd) - lr/(1 - b1^t) * m / (sqrt(v)/sqrt(1 - b2^t) + eps)
//
// in fp32, each operation rounded on its own (no contraction, IEEE divide and
// root), so that the new states, and with them their 8-bit codes, are a fixed
// function of the inputs.
//
// 8-bit states hold m and r = sqrt(v) as e4m3 codes with one scale 2^j per 128
// consecutive elements, 2^j the smallest with amax <= 448 * 2^j: scaling by a
// power of two is exact, so the only loss is the code's rounding (3 bits of
// mantissa, 2^-4 relative).  The root halves the exponent range v needs: codes
// reach 2.3e5 below a tile's largest r, 5e10 below its largest v.  This step's
// weights use the moments before that rounding.  A non-finite moment gets the
// NaN code and takes no part in its tile's scale, so it stays its own element's.
//
// Bound by memory: 12 to 30 bytes an element, each touched once.  A lane takes 4
// consecutive elements, so that every fp32 access of a wave is one solid
// kilobyte (32 lanes share a tile's scale), stores pass the caches by, as do the
// loads of large launches, and a work-group ends after one quad a lane, the next
// one's loads filling its place.  Measured on 113 M bf16 weights with fp32
// masters, us (TB/s), fp32 / 8-bit states:
//   one quad, streaming loads and stores   581 (5.85) / 326 (6.31)
//   stores through the caches              632 (5.37) / 374 (5.49)
//   loads and stores through the caches    627 (5.42) / 369 (5.56)
//   two quads, four quads                  598, 583  / 350, 348
//   8 elements a lane (two half-used lines an access), two steps: 666 / 403
#pragma clang fp contract(off)

#include <type_traits>

#include "launch.h"
#include "stream8.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kPerGroup = kThreads * 4;  // elements of a work-group: one quad a lane
constexpr int kMaxTensors = 48;         // per launch: the arguments stay under 4 KB

struct Item {
  int64_t n;
  void* p;
  const void* g;
  float* w;
  void* m;
  void* v;
  float* ms;
  float* vs;
  float keep;  // 1 - lr wd
};

struct AdamArgs {
  Item item[kMaxTensors];
  int64_t first[kMaxTensors + 1];  // first work-group of each tensor
  int count;
  float b1, omb1, b2, omb2, eps, rbc2, step;
  const float* scale;
};

// the exponent scale of a tile: the smallest 2^j >= 2^-100 with amax <= 448 * 2^j
// (1 for amax = 0), and its inverse
__device__ __forceinline__ void tile_scale(float amax, float& scale, float& inv) {
  const uint32_t u = __float_as_uint(amax);
  int j = static_cast<int>(u >> 23) - 127 - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  j = amax == 0.0f ? 0 : (j < -100 ? -100 : j);
  scale = __uint_as_float(static_cast<uint32_t>(j + 127) << 23);
  inv = __uint_as_float(static_cast<uint32_t>(127 - j) << 23);
}

__device__ __forceinline__ float tile_max(float v) {  // over 32 lanes
  v = fmaxf(v, dpp_f32<0xB1>(v));
  v = fmaxf(v, dpp_f32<0x4E>(v));
  v = fmaxf(v, dpp_f32<0x141>(v));
  v = fmaxf(v, dpp_f32<0x140>(v));
  const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
}

__device__ __forceinline__ bool finite(float v) { return (__float_as_uint(v) & 0x7F800000u) != 0x7F800000u; }

// 4 consecutive elements as they are stored, at any element alignment
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef u32x2 u32x2_a2 __attribute__((aligned(2)));
typedef unsigned int u32_a1 __attribute__((aligned(1)));
template <typename T>
struct Quad;
template <>
struct Quad<float> {
  typedef u32x4 V;
  typedef u32x4_a4 A;
};
template <>
struct Quad<uint16_t> {
  typedef u32x2 V;
  typedef u32x2_a2 A;
};
template <>
struct Quad<uint8_t> {
  typedef unsigned int V;
  typedef u32_a1 A;
};

// FULL: all 4 exist; else the first n (the others read as 0)
template <bool FULL, bool STREAM, typename T>
__device__ __forceinline__ typename Quad<T>::V load4(const T* p, int n) {
  typedef typename Quad<T>::A A;
  if constexpr (FULL && STREAM) {
    return __builtin_nontemporal_load(reinterpret_cast<const A*>(p));
  } else if constexpr (FULL) {
    return *reinterpret_cast<const A*>(p);
  } else {
    T e[4] = {};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < n) e[i] = p[i];
    return __builtin_bit_cast(typename Quad<T>::V, e);
  }
}
template <bool FULL, typename T>
__device__ __forceinline__ void store4(T* p, typename Quad<T>::V v, int n) {
  typedef typename Quad<T>::A A;
  if constexpr (FULL) {
    __builtin_nontemporal_store(v, reinterpret_cast<A*>(p));
  } else {
    struct E {
      T e[4];
    };
    const E e = __builtin_bit_cast(E, v);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < n) p[i] = e.e[i];
  }
}

__device__ __forceinline__ void widen(u32x4 v, float (&f)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(v[i]);
}
__device__ __forceinline__ void widen(u32x2 v, float (&f)[4]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    f[2 * i] = __uint_as_float(v[i] << 16);
    f[2 * i + 1] = __uint_as_float(v[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void narrow(const float (&f)[4], u32x4& v) {
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = __float_as_uint(f[i]);
}
__device__ __forceinline__ void narrow(const float (&f)[4], u32x2& v) {
  v = u32x2{pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3])};
}

// the values of 4 codes (the NaN code gives NaN)
__device__ __forceinline__ void decode(uint32_t c, float scale, float (&f)[4]) {
  const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8(c, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8(c, true);
  f[0] = lo[0] * scale;
  f[1] = lo[1] * scale;
  f[2] = hi[0] * scale;
  f[3] = hi[1] * scale;
}
// the codes of 4 values and their tile's scale; the scaled values are at most
// 448, so the conversion (nearest even) never saturates.  Every lane of the
// tile has to be here.
__device__ __forceinline__ uint32_t encode(const float (&f)[4], float& scale) {
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) amax = fmaxf(amax, finite(f[i]) ? __builtin_fabsf(f[i]) : 0.0f);
  float inv, x[4];
  tile_scale(tile_max(amax), scale, inv);
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = finite(f[i]) ? f[i] * inv : __builtin_nanf("");
  int q = __builtin_amdgcn_cvt_pk_fp8_f32(x[0], x[1], 0, false);
  return static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(x[2], x[3], q, true));
}

// The quad of elements [i, i + 4) of a tensor, of which n exist (FULL: all).
template <typename TP, typename TG, bool MASTER, bool BITS8, bool STREAM, bool FULL>
__device__ __forceinline__ void adamw_quad(const AdamArgs& a, const Item& it, int64_t i, int n, float scale) {
  typedef typename std::conditional<BITS8, uint8_t, float>::type TS;
  typedef typename std::conditional<MASTER, float, TP>::type TW;
  TP* const pp = static_cast<TP*>(it.p) + i;
  TW* const pw = (MASTER ? reinterpret_cast<TW*>(it.w) : reinterpret_cast<TW*>(it.p)) + i;
  TS* const pm = static_cast<TS*>(it.m) + i;
  TS* const pv = static_cast<TS*>(it.v) + i;
  const auto rg = load4<FULL, STREAM>(static_cast<const TG*>(it.g) + i, n);
  const auto rw = load4<FULL, STREAM>(pw, n);
  const auto rm = load4<FULL, STREAM>(pm, n);
  const auto rv = load4<FULL, STREAM>(pv, n);
  float g[4], w[4], m[4], v[4], r[4];
  if constexpr (BITS8) {
    decode(rm, n > 0 ? it.ms[i / 128] : 0.0f, m);
    decode(rv, n > 0 ? it.vs[i / 128] : 0.0f, v);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = v[j] * v[j];
  } else {
    widen(rm, m);
    widen(rv, v);
  }
  widen(rg, g);
  widen(rw, w);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float gj = g[j] * scale;
    m[j] = m[j] * a.b1 + gj * a.omb1;
    v[j] = v[j] * a.b2 + (gj * gj) * a.omb2;
    r[j] = __builtin_sqrtf(v[j]);
    w[j] = w[j] * it.keep - (m[j] / (r[j] * a.rbc2 + a.eps)) * a.step;
  }
  if constexpr (BITS8) {
    float sm, sv;
    const uint32_t cm = encode(m, sm), cv = encode(r, sv);
    store4<FULL>(pm, cm, n);
    store4<FULL>(pv, cv, n);
    if (n > 0 && (threadIdx.x & 31) == 0) {
      it.ms[i / 128] = sm;
      it.vs[i / 128] = sv;
    }
  } else {
    u32x4 o;
    narrow(m, o);
    store4<FULL>(pm, o, n);
    narrow(v, o);
    store4<FULL>(pv, o, n);
  }
  if constexpr (MASTER) {
    u32x4 o;
    narrow(w, o);
    store4<FULL>(pw, o, n);
  }
  typename Quad<TP>::V o;
  narrow(w, o);
  store4<FULL>(pp, o, n);
}

// TP: the weight's type; MASTER: fp32 weights in w, p their rounded copy;
// BITS8: 8-bit states
template <typename TP, typename TG, bool MASTER, bool BITS8, bool STREAM>
__global__ __launch_bounds__(kThreads) void adamw_kernel(const AdamArgs a) {
  // the work-group's tensor (uniform)
  int lo = 0, hi = a.count;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.first[mid] <= blockIdx.x) lo = mid; else hi = mid;
  }
  const Item& it = a.item[lo];
  const int64_t at = (blockIdx.x - a.first[lo]) * (int64_t)kPerGroup;  // a tile starts here
  const int64_t i = at + threadIdx.x * 4;
  const float scale = a.scale == nullptr ? 1.0f : *a.scale;
  if (at + kPerGroup <= it.n) adamw_quad<TP, TG, MASTER, BITS8, STREAM, true>(a, it, i, 4, scale);
  else
    adamw_quad<TP, TG, MASTER, BITS8, STREAM, false>(
        a, it, i, static_cast<int>(max((int64_t)0, min((int64_t)4, it.n - i))), scale);
}

static_assert(sizeof(AdamArgs) <= 4096, "the arguments of a launch");

struct Kind {
  int p, g, state;
  bool master;
  bool operator==(const Kind& o) const { return p == o.p && g == o.g && state == o.state && master == o.master; }
};

template <typename TP, typename TG, bool MASTER>
void launch_state(const AdamArgs& a, const Kind& k, dim3 grid, hipStream_t s) {
  // loads pass the caches by when the launch touches more than the package's
  // 256 MB cache holds (28 M elements: 139 us against 156, 8-bit 83 against 89);
  // below that the gradients at least may still be there (7 M: 27 against 36)
  const double each = (k.state == MOE_E4M3 ? 4.125 : 16.0) + sizeof(TG) + 2.0 * sizeof(TP) + (MASTER ? 6.0 : 0.0);
  const bool stream = static_cast<double>(a.first[a.count]) * kPerGroup * each > 256.0 * (1 << 20);
  auto go = [&](auto bits8, auto st) {
    hipLaunchKernelGGL((adamw_kernel<TP, TG, MASTER, decltype(bits8)::value, decltype(st)::value>), grid,
                       dim3(kThreads), 0, s, a);
  };
  if (k.state == MOE_E4M3) stream ? go(std::true_type{}, std::true_type{}) : go(std::true_type{}, std::false_type{});
  else stream ? go(std::false_type{}, std::true_type{}) : go(std::false_type{}, std::false_type{});
}

template <typename TG>
void launch_param(const AdamArgs& a, const Kind& k, dim3 grid, hipStream_t s) {
  if (k.p == MOE_F32) launch_state<float, TG, false>(a, k, grid, s);
  else if (k.master) launch_state<uint16_t, TG, true>(a, k, grid, s);
  else launch_state<uint16_t, TG, false>(a, k, grid, s);
}

hipError_t launch_kind(AdamArgs& a, const Kind& k, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>(a.first[a.count]));
  if (k.g == MOE_BF16) launch_param<uint16_t>(a, k, grid, s);
  else launch_param<float>(a, k, grid, s);
  a.count = 0;
  return hipGetLastError();
}

}  // namespace

// One launch per kind (weight, gradient and state types) and kMaxTensors tensors,
// or as many of their elements as a launch reaches (17 G).
hipError_t launch_adamw(int n_tensors, const moe_adamw_tensor* t, const moe_adamw_params& h, const float* grad_scale,
                        hipStream_t s) {
  AdamArgs a;
  const double bc1 = 1.0 - __builtin_pow(h.beta1, static_cast<double>(h.step));
  const double bc2 = 1.0 - __builtin_pow(h.beta2, static_cast<double>(h.step));
  a.b1 = static_cast<float>(h.beta1);
  a.omb1 = static_cast<float>(1.0 - h.beta1);
  a.b2 = static_cast<float>(h.beta2);
  a.omb2 = static_cast<float>(1.0 - h.beta2);
  a.eps = static_cast<float>(h.eps);
  a.rbc2 = static_cast<float>(1.0 / __builtin_sqrt(bc2));
  a.step = static_cast<float>(h.lr / bc1);
  a.scale = grad_scale;
  auto kind = [](const moe_adamw_tensor& x) {
    return Kind{x.param_dtype, x.grad_dtype, x.state_dtype, x.master != nullptr};
  };
  constexpr int64_t kMaxGroups = UINT32_MAX / kThreads;  // a launch has under 2^32 threads
  auto ahead = [](const void* q, int64_t bytes) { return static_cast<char*>(const_cast<void*>(q)) + bytes; };
  for (int i = 0; i < n_tensors; ++i) {
    const Kind k = kind(t[i]);
    bool first = t[i].n > 0;
    for (int j = 0; j < i && first; ++j) first = !(t[j].n > 0 && kind(t[j]) == k);
    if (!first) continue;  // empty, or launched with an earlier tensor of its kind
    a.count = 0;
    a.first[0] = 0;
    hipError_t e;
    for (int j = i; j < n_tensors; ++j) {
      const moe_adamw_tensor& x = t[j];
      if (x.n == 0 || !(kind(x) == k)) continue;
      const int64_t bp = k.p == MOE_F32 ? 4 : 2, bg = k.g == MOE_F32 ? 4 : 2, bs = k.state == MOE_F32 ? 4 : 1;
      for (int64_t at = 0; at < x.n;) {  // at: whole work-groups, so whole tiles; one turn under 2^34 elements
        if (a.count == kMaxTensors || (a.count > 0 && a.first[a.count] == kMaxGroups)) {
          if ((e = launch_kind(a, k, s)) != hipSuccess) return e;
        }
        const int64_t left = (x.n - at + kPerGroup - 1) / kPerGroup, room = kMaxGroups - a.first[a.count];
        const int64_t groups = left < room ? left : room, n = left <= room ? x.n - at : groups * kPerGroup;
        const bool bits8 = k.state == MOE_E4M3;
        a.item[a.count] = {n, ahead(x.param, at * bp), ahead(x.grad, at * bg), k.master ? x.master + at : nullptr,
                           ahead(x.m, at * bs), ahead(x.v, at * bs), bits8 ? x.m_scale + at / 128 : nullptr,
                           bits8 ? x.v_scale + at / 128 : nullptr, static_cast<float>(1.0 - h.lr * x.weight_decay)};
        a.first[a.count + 1] = a.first[a.count] + groups;
        ++a.count;
        at += n;
      }
    }
    if (a.count > 0 && (e = launch_kind(a, k, s)) != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace moe

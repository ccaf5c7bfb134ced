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
// Bound by memory (18 to 30 bytes an element, each touched once): a lane takes
// 8 consecutive elements, so 16 lanes (one DPP row) share a tile's scale.
#pragma clang fp contract(off)

#include "launch.h"
#include "stream8.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kStep = kThreads * 8;   // elements of a work-group's step
constexpr int kSteps = 2;             // steps of a work-group
constexpr int kMaxTensors = 32;       // per launch: the arguments stay under 4 KB

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

__device__ __forceinline__ float tile_max(float v) {  // over 16 lanes
  v = fmaxf(v, dpp_f32<0xB1>(v));
  v = fmaxf(v, dpp_f32<0x4E>(v));
  v = fmaxf(v, dpp_f32<0x141>(v));
  return fmaxf(v, dpp_f32<0x140>(v));
}

__device__ __forceinline__ bool finite(float v) { return (__float_as_uint(v) & 0x7F800000u) != 0x7F800000u; }

struct Codes {
  uint32_t a, b;
};
__device__ __forceinline__ void load_codes(Codes& c, const uint8_t* p, int n) {
  if (n >= 8) {
    struct __attribute__((packed, aligned(1))) U { uint32_t a, b; };
    const U u = *reinterpret_cast<const U*>(p);
    c = {u.a, u.b};
  } else {
    c = {0, 0};
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (i < n) (i < 4 ? c.a : c.b) |= static_cast<uint32_t>(p[i]) << (8 * (i & 3));
  }
}
__device__ __forceinline__ void store_codes(uint8_t* p, const Codes& c, int n) {
  if (n >= 8) {
    struct __attribute__((packed, aligned(1))) U { uint32_t a, b; };
    *reinterpret_cast<U*>(p) = U{c.a, c.b};
  } else {
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (i < n) p[i] = static_cast<uint8_t>((i < 4 ? c.a : c.b) >> (8 * (i & 3)));
  }
}
// the values of 8 codes (the NaN code gives NaN)
__device__ __forceinline__ void decode(const Codes& c, float scale, float (&f)[8]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t u = h == 0 ? c.a : c.b;
    const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8(u, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8(u, true);
    f[4 * h] = lo[0] * scale;
    f[4 * h + 1] = lo[1] * scale;
    f[4 * h + 2] = hi[0] * scale;
    f[4 * h + 3] = hi[1] * scale;
  }
}
// the codes of 8 values and their tile's scale; the scaled values are at most
// 448, so the conversion (nearest even) never saturates
__device__ __forceinline__ Codes encode(const float (&f)[8], float& scale) {
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = fmaxf(amax, finite(f[i]) ? __builtin_fabsf(f[i]) : 0.0f);
  float inv;
  tile_scale(tile_max(amax), scale, inv);
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      x[i] = finite(f[4 * h + i]) ? f[4 * h + i] * inv : __builtin_nanf("");
    int q = __builtin_amdgcn_cvt_pk_fp8_f32(x[0], x[1], 0, false);
    q = __builtin_amdgcn_cvt_pk_fp8_f32(x[2], x[3], q, true);
    w[h] = static_cast<uint32_t>(q);
  }
  return {w[0], w[1]};
}

// TP: the weight's type; MASTER: fp32 weights in w, p their rounded copy;
// BITS8: 8-bit states
template <typename TP, typename TG, bool MASTER, bool BITS8>
__global__ __launch_bounds__(kThreads) void adamw_kernel(const AdamArgs a) {
  // the work-group's tensor (uniform)
  int lo = 0, hi = a.count;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.first[mid] <= blockIdx.x) lo = mid; else hi = mid;
  }
  const Item& it = a.item[lo];
  const int64_t at = (blockIdx.x - a.first[lo]) * (int64_t)(kStep * kSteps);
  const float scale = a.scale == nullptr ? 1.0f : *a.scale;
#pragma unroll
  for (int st = 0; st < kSteps; ++st) {
    const int64_t i = at + st * kStep + threadIdx.x * 8;
    const int64_t left = it.n - i;
    const int n = left >= 8 ? 8 : static_cast<int>(left);  // may be <= 0: the lane still joins its tile's maximum
    Raw8<TG> rg;
    Raw8<float> rw;
    Raw8<TP> rp;
    const Piece q{0, n > 0 ? 0 : 8, n};
    load8(rg, static_cast<const TG*>(it.g) + i, q);
    if constexpr (MASTER) load8(rw, it.w + i, q);
    else load8(rp, static_cast<const TP*>(it.p) + i, q);
    float g[8], w[8], m[8], v[8], r[8];
    if constexpr (BITS8) {
      Codes cm, cv;
      load_codes(cm, static_cast<const uint8_t*>(it.m) + i, n);
      load_codes(cv, static_cast<const uint8_t*>(it.v) + i, n);
      const float sm = n > 0 ? it.ms[i / 128] : 0.0f, sv = n > 0 ? it.vs[i / 128] : 0.0f;
      decode(cm, sm, m);
      decode(cv, sv, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = v[j] * v[j];
    } else {
      Raw8<float> rm, rv;
      load8(rm, static_cast<const float*>(it.m) + i, q);
      load8(rv, static_cast<const float*>(it.v) + i, q);
      to_f32(rm, m);
      to_f32(rv, v);
    }
    to_f32(rg, g);
    if constexpr (MASTER) to_f32(rw, w);
    else to_f32(rp, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float gj = g[j] * scale;
      m[j] = m[j] * a.b1 + gj * a.omb1;
      v[j] = v[j] * a.b2 + (gj * gj) * a.omb2;
      r[j] = __builtin_sqrtf(v[j]);
      w[j] = w[j] * it.keep - (m[j] / (r[j] * a.rbc2 + a.eps)) * a.step;
    }
    if constexpr (BITS8) {
      float sm, sv;
      const Codes cm = encode(m, sm), cv = encode(r, sv);
      store_codes(static_cast<uint8_t*>(it.m) + i, cm, n);
      store_codes(static_cast<uint8_t*>(it.v) + i, cv, n);
      if (n > 0 && i % 128 == 0) {
        it.ms[i / 128] = sm;
        it.vs[i / 128] = sv;
      }
    } else {
      Raw8<float> o;
      from_f32(o, m);
      store8(static_cast<float*>(it.m) + i, o, q);
      from_f32(o, v);
      store8(static_cast<float*>(it.v) + i, o, q);
    }
    if constexpr (MASTER) {
      Raw8<float> o;
      from_f32(o, w);
      store8(it.w + i, o, q);
    }
    Raw8<TP> o;
    from_f32(o, w);
    store8(static_cast<TP*>(it.p) + i, o, q);
  }
}

struct Kind {
  int p, g, state;
  bool master;
  bool operator==(const Kind& o) const { return p == o.p && g == o.g && state == o.state && master == o.master; }
};

template <typename TP, typename TG, bool MASTER>
void launch_state(const AdamArgs& a, const Kind& k, dim3 grid, hipStream_t s) {
  if (k.state == MOE_E4M3)
    hipLaunchKernelGGL((adamw_kernel<TP, TG, MASTER, true>), grid, dim3(kThreads), 0, s, a);
  else
    hipLaunchKernelGGL((adamw_kernel<TP, TG, MASTER, false>), grid, dim3(kThreads), 0, s, a);
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

// One launch per kind (weight, gradient and state types) and kMaxTensors tensors.
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
  constexpr int64_t kPerGroup = kStep * kSteps, kMaxGroups = INT32_MAX;
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
      const int64_t groups = (x.n + kPerGroup - 1) / kPerGroup;
      if (a.count == kMaxTensors || (a.count > 0 && a.first[a.count] + groups > kMaxGroups)) {
        if ((e = launch_kind(a, k, s)) != hipSuccess) return e;
      }
      a.item[a.count] = {x.n, x.param, x.grad, x.master, x.m, x.v, x.m_scale, x.v_scale,
                         static_cast<float>(1.0 - h.lr * x.weight_decay)};
      a.first[a.count + 1] = a.first[a.count] + groups;
      ++a.count;
    }
    if (a.count > 0 && (e = launch_kind(a, k, s)) != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace moe

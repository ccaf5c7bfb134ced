// Losses on rows of logits over a vocabulary and their gradients, as one kernel
// each: what the distillation loss and the policy loss share.
//
// Both take a softmax q over the V logits x of a row at temperature tau, need
// q at a few entries, and have the gradient
//     dx[v] = k (q[v] - sum_{j: i_j = v} p_j)
// with a factor k of the row and weights p_j of its entries (distillation: the
// teacher's probabilities; policy: 1 at the token).  KIND says what a row's few
// entries are and how its loss and k come from them:
//
//   Shared<NT>   what the row's threads share
//   live         whether the row may count (the same in all its threads)
//   ahead        what of a row is loaded while the row before it is at work
//   begin        before the sums: with that, loads whose results are wanted after them
//   share        wave 0 of the row, after its sums: the row's entries into Shared
//   finish       wave 0, with the row's maximum and sum: statistics, loss, k
//   factor       k, every thread (after finish where kLateFactor, else after share)
//   mine         every thread: which of its pieces hold entries
//   correct      the gradient of a piece that does: less k p_j at its entries
//   correct_one  the same for one of the last V % E logits
//   done         every thread: Shared as init left it
//   none         one thread: the outputs of a row that does not count
//
// exp is 2^((x - max) log2(e)/tau): the difference first, so that its relative
// error does not grow with the logits, the factor in two parts.  Sums are fp32, a thread's in order, then
// a fixed tree.  A row without a finite logit gives NaN; a NaN spreads over its
// row.  -inf is a logit of probability 0.
#pragma once

#include <hip/hip_runtime.h>

#include <cmath>

#include "launch.h"
#include "rowvec.h"

namespace moe {
namespace vocab {

struct Logits {
  int64_t rows;
  int V;
  const void* x;
  void* dx;             // or nullptr
  float* stats;         // [rows][2]: maximum, sum of exp((x - max)/tau); the gradient alone reads it
  const float* weight;  // [rows] or nullptr: 1 / rows
  const float* grad;    // [1] or nullptr: 1
  float* row_loss;
  float even;           // 1 / rows
  float c, c_low;       // log2(e) / tau in two parts
  float inv_tau_f;
  double inv_tau, tau;
};

inline Logits logits_of(int64_t rows, int V, double tau, const float* weight, const float* grad) {
  Logits p{};
  p.rows = rows;
  p.V = V;
  p.weight = weight;
  p.grad = grad;
  p.even = static_cast<float>(1.0 / static_cast<double>(rows));
  p.tau = tau;
  p.inv_tau = 1.0 / tau;
  p.inv_tau_f = static_cast<float>(1.0 / tau);
  // The low part is positive, so that a difference of -inf stays -inf: c is the
  // second number below.
  const double c = 1.4426950408889634 / tau;
  p.c = std::nextafter(std::nextafter(static_cast<float>(c), 0.0f), 0.0f);
  p.c_low = static_cast<float>(c - static_cast<double>(p.c));
  return p;
}

__device__ __forceinline__ float exp2_of(float v) { return __builtin_amdgcn_exp2f(v); }

// exp(v / tau).  log2(e)/tau as one fp32 number would put every term of a row off in
// the same direction, by up to 2^-24 of its exponent; so it is the rounding of one
// product.  4096 x 131072 bf16 with gradient: 2 % slower.
__device__ __forceinline__ float exp_tau(const Logits& p, float v) {
  return exp2_of(__builtin_fmaf(v, p.c, v * p.c_low));
}

// A value of an input that the kernel does not write, at an address that is the
// same in all lanes, through the scalar cache: it does not wait for the vector
// loads in flight, which return in order.
template <typename T>
__device__ __forceinline__ T scalar_of(const T* p) {
  static_assert(sizeof(T) == 4, "dwords");
  return *reinterpret_cast<const __attribute__((address_space(4))) T*>(reinterpret_cast<uintptr_t>(p));
}
// a logit likewise (of a gradient written over the logits, the kernel writes it
// only after this reading of it)
__device__ __forceinline__ float scalar_logit(const float* x, int v) { return scalar_of(x + v); }
__device__ __forceinline__ float scalar_logit(const uint16_t* x, int v) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(x + v);
  const uint32_t w = scalar_of(reinterpret_cast<const uint32_t*>(at & ~uintptr_t{3}));
  return __uint_as_float(at & 2 ? w & 0xFFFF0000u : w << 16);
}

__device__ __forceinline__ float weight_of(const Logits& p, int64_t row) {
  return p.weight != nullptr ? scalar_of(p.weight + row) : p.even;
}

// ln(v) of a normal fp32 v > 0 to 6e-8 absolute: fp32 for the mantissa, the
// exponent's share in fp64.  (libm's fp64 log would take 40 registers of
// constants out of the rows' loop.)  0, infinities and NaN as log's.
__device__ __forceinline__ double ln_of(float v) {
  if (!(v > 0.0f && v < INFINITY)) return static_cast<double>(__builtin_logf(v));
  const uint32_t u = __float_as_uint(v) - 0x3F3504F3u;  // mantissa in [0.707, 1.414)
  const int e = static_cast<int>(u) >> 23;
  const float f = __uint_as_float((u & 0x7FFFFFu) + 0x3F3504F3u);
  return static_cast<double>(e) * 0.6931471805599453 +
         static_cast<double>(__builtin_amdgcn_logf(f) * 0.6931471805599453f);
}

// Keeps the compiler from holding on to what it made of a piece: three passes
// unpack the same registers, and their fp32 values would be twice the registers.
template <typename T, int E>
__device__ __forceinline__ void pin(Vec<T, E>& v) {
#pragma unroll
  for (int i = 0; i < Vec<T, E>::kWords; ++i) asm volatile("" : "+v"(v.w[i]));
}

// What lies `at` bytes from a row's (scalar) address, and pieces by their number.
template <typename T>
__device__ __forceinline__ const T* at_byte(const T* row, uint32_t at) {
  return reinterpret_cast<const T*>(reinterpret_cast<const char*>(row) + at);
}
template <typename T>
__device__ __forceinline__ T* at_byte(T* row, uint32_t at) {
  return reinterpret_cast<T*>(reinterpret_cast<char*>(row) + at);
}
template <bool STREAM, typename T, int E>
__device__ __forceinline__ void load_at(Vec<T, E>& v, const T* row, int piece) {
  load_vec<STREAM>(v, at_byte(row, static_cast<uint32_t>(piece) * static_cast<uint32_t>(E * sizeof(T))));
}
template <typename T, int E>
__device__ __forceinline__ void store_at(T* row, const Vec<T, E>& v, int piece) {
  store_vec<true>(at_byte(row, static_cast<uint32_t>(piece) * static_cast<uint32_t>(E * sizeof(T))), v);
}
__device__ __forceinline__ float uniform(float v) {  // the same in every lane
  return __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(v)));
}
// the same number, but not one whose derived values are kept over the rows' loop
__device__ __forceinline__ int fresh(int v) {
  asm volatile("" : "+v"(v));
  return v;
}
// a row's number likewise, in scalar registers: addresses are formed from it where
// they are used instead of being carried along, a register pair each
__device__ __forceinline__ int64_t fresh(int64_t v) {
  asm volatile("" : "+s"(v));
  return v;
}

// The thread that stores a logit's gradient.  Pieces below `held` lie in stretches
// of `per` times 64, one a wave; the others, and with held = 0 all, go round the nt
// threads; the logits behind the last piece are one a thread.
// `local`: which of the thread's pieces it is.
struct Owner {
  int pieces, e, nt, per, held;
  static __host__ __device__ __forceinline__ int blocks(int pieces, int waves) {
    const int b = (pieces + kWave * waves - 1) / (kWave * waves);
    return b > 0 ? b : 1;
  }
  __device__ __forceinline__ int of(int v) const {
    const int piece = v / e;
    if (piece >= pieces) return v - pieces * e;
    if (piece < held) return piece / kWave / per * kWave + piece % kWave;
    return (piece - held) & (nt - 1);
  }
  __device__ __forceinline__ int local(int piece) const {
    return piece < held ? piece / kWave % per : held / nt + (piece - held) / nt;
  }
};
constexpr int kManyPieces = 31;  // a thread's pieces from the 31st on share the last bit of a mask

// Barrier of a row's threads (NT = 64: the wave, whose LDS accesses keep their
// order).
template <int NT>
__device__ __forceinline__ void team_sync() {
  if constexpr (NT > kWave) {
    __syncthreads();
  } else {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
}

// a piece of logits: 16 bytes
template <typename TX>
constexpr int kPiece = 16 / static_cast<int>(sizeof(TX));

constexpr int kTogether = 4;  // pieces whose maximum is taken before their exponentials (of 1, 2, 4, 8: 416, 419, 415, 431 us)
constexpr int kBlock = 256;   // threads of a work-group whose rows are narrower
// waves a SIMD holds, by the registers that NC pieces take
template <int NC>
constexpr int kWaves = NC > 8 ? 4 : NC > 6 ? 5 : 6;
template <int NT>
constexpr int kTeams = NT < kBlock ? kBlock / NT : 1;  // rows a work-group has at once
template <int NT>
constexpr int kGroup = NT < kBlock ? kBlock : NT;

// Loss, statistics and with GRAD the gradient, from one reading of the logits: a
// row lives in the registers of its NT threads (NC pieces each).  A longer
// row's other pieces (MORE) are read twice, the second time as they lie in the
// caches.
//
// A work-group walks rows gridDim.x * kTeams apart.  The next row's piece is
// loaded into each register as this row's last use of it is over, so that memory
// is busy while a row is reduced; nothing between that and the next row's first
// use waits for a vector load (the loads of a row drained before its sums: 483 us
// where this took 415 when it came, at 4096 x 131072, bf16 with gradient; 406 of
// that build without its exponentials).
//
// Bound by memory: that case now moves 2.1 GB in 405 us (5.3 TB/s), 8192 x 65536 2.0
// GB in 379.  Work-groups that each stream a row of their own stay below the 6.2 TB/s
// of an elementwise pass in address order.  No vector registers spill; scalar ones do,
// up to 82 of them into lanes.
template <typename KIND, typename TX, typename TD, int NT, int NC, bool MORE, bool GRAD>
__global__ __launch_bounds__(kGroup<NT>, kWaves<NC>) void loss_kernel(const Logits p, const typename KIND::Args k) {
  constexpr int E = kPiece<TX>, WAVES = NT / kWave;
  // two copies by turns where a wave may be a row ahead of another
  constexpr int COPIES = WAVES > 1 ? 2 : 1;
  __shared__ typename KIND::template Shared<NT> s_kind[kTeams<NT>][COPIES];
  __shared__ float s_red[COPIES][2][16];  // the waves' maxima and sums
  const int team = __builtin_amdgcn_readfirstlane(threadIdx.x / NT), tid = threadIdx.x % NT;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int V = p.V, pieces = V / E, tail = V % E;  // the last V % E logits: one a thread
  // A wave holds `per` times 64 consecutive pieces: one stretch of memory (strided
  // over the waves: 412 and 418 us where this takes 397 and 385).
  const int per = MORE ? NC : Owner::blocks(pieces, WAVES);
  const int64_t step = (int64_t)gridDim.x * kTeams<NT>;
  int64_t row = (int64_t)blockIdx.x * kTeams<NT> + team;
  if (row >= p.rows) return;  // whole teams; no barrier where a work-group has several
  for (int b = 0; b < COPIES; ++b) KIND::init(s_kind[team][b], tid);
  if (WAVES > 1 && tid < COPIES * 32) (&s_red[0][0][0])[tid] = tid % 32 < 16 ? -FLT_MAX : 0.0f;
  team_sync<NT>();
  const float g = p.grad != nullptr ? scalar_of(p.grad) : 1.0f;

  const Owner owner{pieces, E, NT, per, NC * NT};
  const TX* const x0 = static_cast<const TX*>(p.x);
  Vec<TX, E> h[NC > 0 ? NC : 1];
  TX t{};
  int ft = tid;  // tid, as `fresh` gives it
  // Without a branch (registers that a branch may or may not load are copied where
  // it ends): what a row has no piece for, and every piece of a row that is not
  // read, loads one that is there.
  auto fetch = [&](int i, const TX* x, bool read) __attribute__((always_inline)) {
    load_at<true>(h[i], x, min((wave * per + min(i, per - 1)) * kWave + (ft & 63), read ? pieces - 1 : 0));
  };
  auto fetch_tail = [&](const TX* x) __attribute__((always_inline)) {
    t = *at_byte(x, static_cast<uint32_t>(min(pieces * E + ft, V - 1)) * static_cast<uint32_t>(sizeof(TX)));
  };
  float w = weight_of(p, row);
  bool live = w != 0.0f && KIND::live(k, row, V);
  typename KIND::Ahead ahead = KIND::ahead(k, row, ft);
#pragma unroll
  for (int i = 0; i < NC; ++i) fetch(i, x0 + row * V, live);
  fetch_tail(x0 + row * V);
  int turn = 0;
  while (row < p.rows) {
    row = fresh(row);
    ft = fresh(tid);
    const int64_t next = row + step, after = next < p.rows ? next : row;
    const float w_next = weight_of(p, after);
    const bool live_next = next < p.rows && w_next != 0.0f && KIND::live(k, after, V);
    const TX* const x = x0 + row * V;
    const TX* const xn = x0 + after * V;
    TD* const dx = static_cast<TD*>(p.dx) + row * V;
    auto tail_out = [&](float v) __attribute__((always_inline)) {
      if (ft < tail) put_one(at_byte(dx, static_cast<uint32_t>(pieces * E + ft) * static_cast<uint32_t>(sizeof(TD))), v);
    };
    auto zero_row = [&]() __attribute__((always_inline)) {
      Vec<TD, E> z;
#pragma unroll
      for (int i = 0; i < Vec<TD, E>::kWords; ++i) z.w[i] = static_cast<uint32_t>(fresh(0));
      for (int i = ft; i < pieces; i += NT) store_at(dx, z, i);
      tail_out(0.0f);
    };
    auto& sh = s_kind[team][turn];
    typename KIND::template Few<TX> few{};
    if (live) few = KIND::template begin<TX>(p, k, row, x, ft, ahead);
    ahead = KIND::ahead(k, after, ft);

    // This thread's maximum and sum, a few pieces at a time as they arrive.  (There
    // is one place that loads a piece, taken by every row: with two, the registers
    // would be copied where they meet, and the copies wait for all loads.)
    const float tv = ft < tail ? one_f32(t) : -INFINITY;
    float m = fmaxf(tv, -FLT_MAX), sum = exp_tau(p, tv - m);
    constexpr int G = NC == 0 ? 1 : NC % kTogether == 0 ? kTogether : NC % 3 == 0 ? 3 : 2;
    static_assert(NC % G == 0, "whole groups");
#pragma unroll
    for (int i0 = 0; i0 < NC; i0 += G) {
      if (live && i0 < per) {
        float m1 = m, s2 = 0.0f;
#pragma unroll
        for (int i = i0; i < i0 + G; ++i) {
          float f[E];
          vec_f32(h[i], f);
#pragma unroll
          for (int j = 0; j < E; ++j) m1 = fmaxf(m1, f[j]);  // (a repeated last piece changes nothing)
        }
#pragma unroll
        for (int i = i0; i < i0 + G; ++i) {
          if (i >= per) break;  // (32768 x 10000 bf16, 5 pieces in registers for 8: 150 us, 130 with this)
          float f[E], s1 = 0.0f;
          vec_f32(h[i], f);
#pragma unroll
          for (int j = 0; j < E; ++j) s1 += exp_tau(p, f[j] - m1);
          s2 += (wave * per + i) * kWave + (ft & 63) < pieces ? s1 : 0.0f;
        }
        sum = sum * exp_tau(p, m - m1) + s2;
        m = m1;
      }
      if constexpr (!GRAD) {
#pragma unroll
        for (int i = i0; i < i0 + G; ++i) fetch(i, xn, live_next);
      }
    }
    if constexpr (!GRAD) fetch_tail(xn);
    constexpr int U = 4;
    float kr = 0.0f, ks = 0.0f;
    if (live) {
      for (int i0 = MORE ? NC * NT + ft : pieces; i0 < pieces; i0 += U * NT) {  // what the registers do not hold
        Vec<TX, E> v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) load_at<false>(v[u], x, min(i0 + u * NT, pieces - 1));
#pragma unroll
        for (int u = 0; u < U; ++u) {
          float f[E], s1 = 0.0f, m1 = m;
          vec_f32(v[u], f);
#pragma unroll
          for (int j = 0; j < E; ++j) m1 = fmaxf(m1, f[j]);
#pragma unroll
          for (int j = 0; j < E; ++j) s1 += exp_tau(p, f[j] - m1);
          sum = sum * exp_tau(p, m - m1) + (i0 + u * NT < pieces ? s1 : 0.0f);
          m = m1;
        }
      }
      // the row's
      const float mw = wave_max(m);
      sum = wave_sum(sum * exp_tau(p, m - mw));
      m = mw;
      if constexpr (WAVES > 1) {
        if ((ft & 63) == 0) {
          s_red[turn][0][wave] = m;
          s_red[turn][1][wave] = sum;
        }
      }
      if (wave == 0) KIND::template share<TX>(p, k, row, x, GRAD, owner, ft, few, sh);
      team_sync<NT>();
      if constexpr (WAVES > 1) {
        const float m1 = s_red[turn][0][ft & 15];
        sum = s_red[turn][1][ft & 15];
        m = row16_max(m1);
        sum = row16_sum(sum * exp_tau(p, m1 - m));
      }
      if (wave == 0) KIND::finish(p, k, row, g * w, m, sum, ft, sh, true);
      if constexpr (GRAD) {
        if constexpr (KIND::kLateFactor) team_sync<NT>();
        kr = uniform(KIND::factor(p, g * w, sh));
        ks = kr / sum;
      }
    } else {
      if (ft == 0) KIND::none(p, k, row);
    }
    if constexpr (GRAD) {
      // k = 0: zeros, also where the logits hold anything
      if (kr == 0.0f) zero_row();
      const auto mine = KIND::mine(owner, sh, ft, kr != 0.0f);
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        pin(h[i]);
        if (i < per && kr != 0.0f) {
          float f[E];
          vec_f32(h[i], f);
#pragma unroll
          for (int j = 0; j < E; ++j) f[j] = ks * exp_tau(p, f[j] - m);
          const int at = (wave * per + i) * kWave + (ft & 63);
          KIND::correct(sh, mine, i, at, kr, ft, f);
          Vec<TD, E> o;
          f32_vec(o, f);
          if (at < pieces) store_at(dx, o, at);
        }
        fetch(i, xn, live_next);
      }
      if (kr != 0.0f && ft < tail)
        tail_out(KIND::correct_one(sh, mine, pieces * E + ft, kr, ft, ks * exp_tau(p, tv - m)));
      fetch_tail(xn);
      for (int i0 = MORE && kr != 0.0f ? NC * NT + ft : pieces; i0 < pieces; i0 += U * NT) {
        Vec<TX, E> v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) load_at<false>(v[u], x, min(i0 + u * NT, pieces - 1));
#pragma unroll
        for (int u = 0; u < U; ++u) {
          float f[E];
          vec_f32(v[u], f);
#pragma unroll
          for (int j = 0; j < E; ++j) f[j] = ks * exp_tau(p, f[j] - m);
          KIND::correct(sh, mine, owner.local(i0 + u * NT), i0 + u * NT, kr, ft, f);
          Vec<TD, E> o;
          f32_vec(o, f);
          if (i0 + u * NT < pieces) store_at(dx, o, i0 + u * NT);
        }
      }
    }
    if (live) {
      if constexpr (GRAD) KIND::done(sh, ft);
      if constexpr (COPIES > 1) turn ^= 1;
      else team_sync<NT>();
    }
    row = next;
    w = w_next;
    live = live_next;
  }
}

// The gradient from the logits and the forward's statistics: a work-group has
// `span` pieces of a row, a multiple of NT (NT = 64: a wave has them).  The row's few
// entries are looked up while its pieces are on their way.  Runs at the rate of an
// elementwise pass: 2048 x 100003 fp32 to bf16 (1.2 GB) 192 us, 6.0 TB/s.
template <int NT>
constexpr int kGradAhead = NT > kWave ? 2 : 4;
template <typename KIND, typename TX, typename TD, int NT>
__global__ __launch_bounds__(kGroup<NT>, (NT > kWave ? 6 : 5)) void grad_kernel(const Logits p,
                                                                                const typename KIND::Args k, int splits,
                                                                                int span, int64_t units) {
  constexpr int E = kPiece<TX>, U = kGradAhead<NT>;
  __shared__ typename KIND::template Shared<NT> s_kind[kTeams<NT>];
  const int team = __builtin_amdgcn_readfirstlane(threadIdx.x / NT), tid = threadIdx.x % NT, lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int V = p.V, pieces = V / E, tail = V % E;
  const float g = p.grad != nullptr ? scalar_of(p.grad) : 1.0f;
  const Owner owner{pieces, E, NT, 1, 0};
  auto& sh = s_kind[team];
  for (int64_t unit = (int64_t)blockIdx.x * kTeams<NT> + team; unit < units; unit += (int64_t)gridDim.x * kTeams<NT>) {
    const int64_t row = unit / splits;
    const int part = static_cast<int>(unit % splits), first = part * span, last = min(pieces, first + span);
    const TX* const x = static_cast<const TX*>(p.x) + row * V;
    TD* const dx = static_cast<TD*>(p.dx) + row * V;
    const bool ends = part == splits - 1, one = ends && tid < tail;
    const float w = weight_of(p, row);
    const bool live = w != 0.0f && KIND::live(k, row, V);
    float kr = 0.0f, m = 0.0f, ks = 0.0f;
    Vec<TX, E> v[U];
    auto fetch = [&](int i0) __attribute__((always_inline)) {
#pragma unroll
      for (int u = 0; u < U; ++u) load_at<true>(v[u], x, max(0, min(i0 + u * NT, last - 1)));
    };
    if (live) {
      if (pieces > 0) fetch(first + tid);  // in flight while the row's entries are looked up
      KIND::init(sh, tid);
      team_sync<NT>();
      m = scalar_of(p.stats + 2 * row);
      const float sum = scalar_of(p.stats + 2 * row + 1);
      if (wave == 0) {
        KIND::template entries<TX>(p, k, row, x, owner, first * E, ends ? V : last * E, lane, sh);
        if constexpr (KIND::kLateFactor) KIND::finish(p, k, row, g * w, m, sum, lane, sh, false);
      }
      team_sync<NT>();
      kr = uniform(KIND::factor(p, g * w, sh));
      ks = kr / sum;
    }
    if (kr == 0.0f) {  // zeros, also where the logits hold anything
      Vec<TD, E> z;
#pragma unroll
      for (int i = 0; i < Vec<TD, E>::kWords; ++i) z.w[i] = 0;
      for (int i = first + tid; i < last; i += NT) store_at(dx, z, i);
      if (one) put_one(dx + (int64_t)pieces * E + tid, 0.0f);
    } else {
      const auto mine = KIND::mine(owner, sh, tid, true);
      for (int i0 = first + tid; i0 < last; i0 += U * NT) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          float f[E];
          vec_f32(v[u], f);
#pragma unroll
          for (int j = 0; j < E; ++j) f[j] = ks * exp_tau(p, f[j] - m);
          KIND::correct(sh, mine, owner.local(i0 + u * NT), i0 + u * NT, kr, tid, f);
          Vec<TD, E> o;
          f32_vec(o, f);
          if (i0 + u * NT < last) store_at(dx, o, i0 + u * NT);
        }
        if (i0 + U * NT < last) fetch(i0 + U * NT);
      }
      if (one) {
        const int64_t at = (int64_t)pieces * E + tid;
        const float f = ks * exp_tau(p, one_f32(x[at]) - m);
        put_one(dx + at, KIND::correct_one(sh, mine, static_cast<int>(at), kr, tid, f));
      }
    }
    team_sync<NT>();  // Shared is free again
  }
}

// ---------------------------------------------------------------- launches
template <typename KIND, typename TX, typename TD, int NT, int NC, bool MORE, bool GRAD>
hipError_t run_loss(const Logits& p, const typename KIND::Args& k, hipStream_t s) {
  const int64_t need = (p.rows + kTeams<NT> - 1) / kTeams<NT>;
  // the work-groups the chip holds at once
  const int64_t held = (int64_t)stream_cu_count(s) * 4 * kWaves<NC> * kWave / kGroup<NT>;
  const dim3 grid(static_cast<unsigned>(need < held ? need : held)), block(kGroup<NT>);
  hipLaunchKernelGGL((loss_kernel<KIND, TX, TD, NT, NC, MORE, GRAD>), grid, block, 0, s, p, k);
  return hipGetLastError();
}

template <typename KIND, typename TX, typename TD, bool GRAD>
hipError_t loss_rows(const Logits& p, const typename KIND::Args& k, hipStream_t s) {
  const int pieces = p.V / kPiece<TX>;
  // The fewest registers that hold a row, of the fewest waves.  The width alone
  // decides, so that a row's results do not depend on the rows beside it.  (Few rows
  // would be quicker cut over several work-groups, in an order of sums that V alone
  // fixes too; that is not built: 64 x 32000 bf16 with gradient takes 13 us.)
  if (pieces == 0) return run_loss<KIND, TX, TD, 64, 0, false, GRAD>(p, k, s);
  if (pieces <= 2 * 64) return run_loss<KIND, TX, TD, 64, 2, false, GRAD>(p, k, s);
  if (pieces <= 4 * 64) return run_loss<KIND, TX, TD, 64, 4, false, GRAD>(p, k, s);
  if (pieces <= 8 * 64) return run_loss<KIND, TX, TD, 64, 8, false, GRAD>(p, k, s);
  if (pieces <= 4 * 256) return run_loss<KIND, TX, TD, 256, 4, false, GRAD>(p, k, s);
  // (6 between 4 and 8: 32768 x 10000 bf16 130 -> 118 us)
  if (pieces <= 6 * 256) return run_loss<KIND, TX, TD, 256, 6, false, GRAD>(p, k, s);
  if (pieces <= 8 * 256) return run_loss<KIND, TX, TD, 256, 8, false, GRAD>(p, k, s);
  if (pieces <= 12 * 256) return run_loss<KIND, TX, TD, 256, 12, false, GRAD>(p, k, s);
  if (pieces <= 16 * 256) return run_loss<KIND, TX, TD, 256, 16, false, GRAD>(p, k, s);
  if (pieces <= 12 * 512) return run_loss<KIND, TX, TD, 512, 12, false, GRAD>(p, k, s);
  if (pieces <= 16 * 512) return run_loss<KIND, TX, TD, 512, 16, false, GRAD>(p, k, s);
  if (pieces <= 12 * 1024) return run_loss<KIND, TX, TD, 1024, 12, false, GRAD>(p, k, s);
  if (pieces <= 16 * 1024) return run_loss<KIND, TX, TD, 1024, 16, false, GRAD>(p, k, s);
  return run_loss<KIND, TX, TD, 1024, 12, true, GRAD>(p, k, s);
}

template <typename KIND, typename TX, typename TD, int NT>
hipError_t run_grad(const Logits& p, const typename KIND::Args& k, hipStream_t s) {
  // A wave has its row.  4 waves have 2 pieces a thread, so that what runs at the
  // same time lies side by side in memory (1500 x 50001 fp32: 98 us, 112 with 8
  // pieces; 2048 x 100003: 191 and 236); more where every work-group has many entries
  // to look up first.
  const int pieces = p.V / kPiece<TX>, span = (NT > kWave ? KIND::grad_pieces(k) : 8) * NT;
  const int splits = pieces <= span ? 1 : (pieces + span - 1) / span;
  const int64_t units = p.rows * splits, groups = (units + kTeams<NT> - 1) / kTeams<NT>;
  const dim3 grid(static_cast<unsigned>(groups < (1 << 20) ? groups : 1 << 20)), block(kGroup<NT>);
  hipLaunchKernelGGL((grad_kernel<KIND, TX, TD, NT>), grid, block, 0, s, p, k, splits, span, units);
  return hipGetLastError();
}

template <typename KIND, typename TX, typename TD>
hipError_t grad_rows(const Logits& p, const typename KIND::Args& k, hipStream_t s) {
  if (p.V / kPiece<TX> <= 8 * kWave) return run_grad<KIND, TX, TD, 64>(p, k, s);
  return run_grad<KIND, TX, TD, 256>(p, k, s);
}

// x_dtype, dx_dtype: MOE_F32 or MOE_BF16
template <typename KIND>
hipError_t loss_dtypes(const Logits& p, const typename KIND::Args& k, int x_dtype, int dx_dtype, hipStream_t s) {
  using B = uint16_t;
  const bool xb = x_dtype == MOE_BF16, db = dx_dtype == MOE_BF16;
  if (p.dx == nullptr)
    return xb ? loss_rows<KIND, B, float, false>(p, k, s) : loss_rows<KIND, float, float, false>(p, k, s);
  if (xb) return db ? loss_rows<KIND, B, B, true>(p, k, s) : loss_rows<KIND, B, float, true>(p, k, s);
  return db ? loss_rows<KIND, float, B, true>(p, k, s) : loss_rows<KIND, float, float, true>(p, k, s);
}
template <typename KIND>
hipError_t grad_dtypes(const Logits& p, const typename KIND::Args& k, int x_dtype, int dx_dtype, hipStream_t s) {
  using B = uint16_t;
  const bool xb = x_dtype == MOE_BF16, db = dx_dtype == MOE_BF16;
  if (xb) return db ? grad_rows<KIND, B, B>(p, k, s) : grad_rows<KIND, B, float>(p, k, s);
  return db ? grad_rows<KIND, float, B>(p, k, s) : grad_rows<KIND, float, float>(p, k, s);
}

}  // namespace vocab

// loss[0] = sum_t weight[t] row_loss[t] (weight nullptr: even), in a fixed order
hipError_t launch_loss_sum(int64_t rows, const float* row_loss, const float* weight, float even, float* loss,
                           hipStream_t s);

}  // namespace moe

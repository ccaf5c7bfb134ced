// Layer norm in front of the MoE layer, with the residual add, and its
// backward.
//
//   s = x + r (rounded once to x's type, so that the backward, which reads
//       the stored s, differentiates exactly what the forward normalised)
//   mu = sum(s)/d,  var = sum((s - mu)^2)/d,  rstd = 1/sqrt(var + eps)
//   y = (s - mu) rstd w + b
//   backward: xh = (s - mu) rstd,  q = dy w,
//       dx = rstd (q - mean(q) - xh mean(q xh)) + d_sum
//       dw = sum_t dy xh,  db = sum_t dy
//
// Both are bound by memory: each element is read once and written once.  A row
// lives in the registers of wpr waves (8 N elements a lane), so the mean and
// then the centred squares are summed from registers; two sums instead of one
// of squares keep the variance exact when the mean is large.
// Measured at 16384 x 7168: forward (bf16 with residual, 940 MB) 156 us, backward
// (fp32 gradient in, bf16 residual's added, 1.17 GB) 199 us: 6.0 and 5.9 TB/s,
// where an elementwise add of that size runs at 5.95.
#include <algorithm>
#include <type_traits>

#include "launch.h"
#include "stream8.h"

namespace moe {
namespace {

constexpr int kMaxWaves = 16;

// ---------------------------------------------------------------- forward
struct NormArgs {
  int64_t rows;
  int d, wpr, rpb, lg;  // waves per row, rows per work-group; wpr = 1: 2^lg lanes per row
  const void* x;
  const void* r;
  const float* w;
  const float* b;
  float eps;
  void* sum;
  void* y;
  float* mean;
  float* rstd;
};

// Sum over the waves of a row, the same tree on every call.  s_red: 16 slots,
// zero where there is no wave; every lane reads the slot of its place in its
// 16-lane DPP row, so one LDS read and four DPP adds end it.
__device__ __forceinline__ float row_sum(float v, float* s_red, int wpr, int lg) {
  if (wpr == 1) return group_sum(v, 1 << lg);
  v = wave_sum(v);
  if ((threadIdx.x & 63) == 0) s_red[threadIdx.x >> 6] = v;
  __syncthreads();
  return row16_sum(s_red[threadIdx.x & 15]);
}

// A work-group walks rows gridDim.x * rpb apart and issues the next row's loads
// before it reduces this one's.  Its columns' weights stay in registers up to
// N = 2; wider rows (d > 16384) read them again from cache, and with a residual
// they spill: 76 to 228 bytes a lane (fp32 to bf16 without one 20).
template <typename TX, typename TY, bool RES, int N, bool STREAM>
__global__ __launch_bounds__(kMaxWaves* kWave) void norm_fwd_kernel(const NormArgs p) {
  constexpr bool kKeep = N <= 2;
  __shared__ float s_red[2][kMaxWaves];
  if (threadIdx.x < 2 * kMaxWaves) s_red[threadIdx.x / kMaxWaves][threadIdx.x % kMaxWaves] = 0.0f;
  __syncthreads();
  const int slot = p.wpr == 1 ? threadIdx.x >> p.lg : 0;
  const int rt = threadIdx.x - (slot << p.lg);  // thread within the row
  const int64_t step = (int64_t)gridDim.x * p.rpb;
  int64_t row = (int64_t)blockIdx.x * p.rpb + slot;
  if (row >= p.rows) return;  // whole rows, and no barrier follows where rpb > 1 (then wpr = 1)
  const TX* const x = static_cast<const TX*>(p.x);
  const TX* const r = static_cast<const TX*>(p.r);
  Piece q[N];
  Raw8<TX> rx[N], rr[RES ? N : 1];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    q[i] = piece_of(i * p.wpr * kWave + rt, p.d);
    load8<STREAM>(rx[i], x + row * p.d, q[i]);
    if constexpr (RES) load8<STREAM>(rr[i], r + row * p.d, q[i]);
  }
  float w[N][8], b[N][8];
  auto weights = [&](int i) __attribute__((always_inline)) {
    Raw8<float> t;
    load8<false>(t, p.w, q[i]);
    to_f32(t, w[i]);
    if (p.b != nullptr) {
      load8<false>(t, p.b, q[i]);
      to_f32(t, b[i]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) b[i][j] = 0.0f;
    }
  };
  if constexpr (kKeep) {
#pragma unroll
    for (int i = 0; i < N; ++i) weights(i);
  }
  const float inv_d = 1.0f / static_cast<float>(p.d);
  for (; row < p.rows; row += step) {
    const int64_t base = row * p.d;
    float f[N][8];
    float acc = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      to_f32(rx[i], f[i]);
      if constexpr (RES) {
        float g[8];
        to_f32(rr[i], g);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[i][j] += g[j];
        Raw8<TX> s;
        from_f32(s, f[i]);
        store8(static_cast<TX*>(p.sum) + base, s, q[i]);
        to_f32(s, f[i]);
      }
      mask8(f[i], q[i]);
#pragma unroll
      for (int j = 0; j < 8; ++j) acc += f[i][j];
    }
    if (row + step < p.rows) {
      const int64_t next = base + step * p.d;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        load8<STREAM>(rx[i], x + next, q[i]);
        if constexpr (RES) load8<STREAM>(rr[i], r + next, q[i]);
      }
    }
    const float mean = row_sum(acc, s_red[0], p.wpr, p.lg) * inv_d;
    acc = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
#pragma unroll
      for (int j = 0; j < 8; ++j) f[i][j] -= mean;
      mask8(f[i], q[i]);
#pragma unroll
      for (int j = 0; j < 8; ++j) acc = __builtin_fmaf(f[i][j], f[i][j], acc);
    }
    const float var = row_sum(acc, s_red[1], p.wpr, p.lg) * inv_d;
    const float rstd = 1.0f / __builtin_sqrtf(var + p.eps);
    if (rt == 0 && p.mean != nullptr) {
      p.mean[row] = mean;
      p.rstd[row] = rstd;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if constexpr (!kKeep) weights(i);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[i][j] = __builtin_fmaf(f[i][j] * rstd, w[i][j], b[i][j]);
      Raw8<TY> o;
      from_f32(o, f[i]);
      store8(static_cast<TY*>(p.y) + base, o, q[i]);
    }
  }
}

// ---------------------------------------------------------------- backward
struct NormBwdArgs {
  int64_t rows;
  int d, wpr, rpb, lg;  // waves per row, rows at once in a work-group; wpr = 1: 2^lg lanes per row
  const void* dy;
  const void* x;
  const float* w;
  const float* mean;
  const float* rstd;
  const void* ds;
  void* dx;
  float* part;  // [gridDim.x][2][d]: dw, db of this work-group's rows
};

// A work-group takes every gridDim.x-th row and keeps its columns' dw and db in
// registers; their sums leave once at the end.  With one piece a lane the
// weights stay there too, and the next row's loads are issued before this one
// is reduced; rows of two (d > 8192) have no registers for either.  MULTI (rows
// of at most 4 waves): the work-group's 8 waves take several rows at once, side
// by side (several in a wave where they fit), and join their sums in registers and
// LDS, so that the parts stay one per work-group.
constexpr int kMultiWaves = 8;
template <typename TD, typename TX, typename TO, bool DS, int N, bool MULTI, bool STREAM>
__global__ __launch_bounds__(kMaxWaves* kWave) void norm_bwd_kernel(const NormBwdArgs p) {
  __shared__ float s_red[2][2][kMaxWaves];
  __shared__ float s_part[MULTI ? 2 : 1][MULTI ? kMultiWaves * kWave * 8 : 1];
  const int wave = threadIdx.x >> 6, waves = MULTI ? p.wpr : blockDim.x >> 6;
  const bool packed = MULTI && waves == 1;    // rows side by side also within a wave
  const int slot = packed ? threadIdx.x >> p.lg : MULTI ? wave / waves : 0;  // the row's place in the work-group
  const int width = packed ? 1 << p.lg : waves * kWave;
  const int tid = threadIdx.x - slot * width;  // thread within the row
  if (threadIdx.x < 4 * kMaxWaves) (&s_red[0][0][0])[threadIdx.x] = 0.0f;
  __syncthreads();
  const TD* const dy = static_cast<const TD*>(p.dy);
  const TX* const x = static_cast<const TX*>(p.x);
  const TX* const ds = static_cast<const TX*>(p.ds);
  const int64_t step = (int64_t)gridDim.x * (MULTI ? p.rpb : 1);
  int64_t row = MULTI ? (int64_t)blockIdx.x * p.rpb + slot : blockIdx.x;
  Piece q[N];
  Raw8<TD> rd[N];
  Raw8<TX> rx[N], rs[DS ? N : 1];
  float mean = 0.0f, rstd = 0.0f;
  auto load = [&](int64_t r) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      load8<STREAM>(rd[i], dy + r * p.d, q[i]);
      load8<STREAM>(rx[i], x + r * p.d, q[i]);
      if constexpr (DS) load8<STREAM>(rs[i], ds + r * p.d, q[i]);
    }
    mean = p.mean[r];
    rstd = p.rstd[r];
  };
#pragma unroll
  for (int i = 0; i < N; ++i) q[i] = piece_of(i * width + tid, p.d);
  constexpr bool kAhead = N == 1;
  float w[1][8], dw[N][8], db[N][8];
  auto weights = [&](int i, float (&f)[8]) __attribute__((always_inline)) {
    Raw8<float> t;
    load8<false>(t, p.w, q[i]);
    to_f32(t, f);
  };
  if constexpr (kAhead) {
    if (row < p.rows) load(row);
    weights(0, w[0]);
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[i][j] = db[i][j] = 0.0f;
  }
  const float inv_d = 1.0f / static_cast<float>(p.d);
  // row - slot: the same in all waves, which meet at the barriers
  for (int buf = 0; row - slot < p.rows; row += step, buf ^= 1) {
    const bool in = !MULTI || row < p.rows;
    const int64_t base = row * p.d;
    float xh[N][8], g[N][8], res[DS ? N : 1][8];
    float c1 = 0.0f, c2 = 0.0f;
    if constexpr (!kAhead) load(row);
    const float rs1 = rstd;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (!in) break;
      if constexpr (!kAhead) weights(i, w[0]);
      float (&wi)[8] = w[0];
      to_f32(rd[i], g[i]);
      to_f32(rx[i], xh[i]);
      if constexpr (DS) to_f32(rs[i], res[i]);
      mask8(g[i], q[i]);  // dy = 0 where the piece owns nothing: no term of any sum
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        xh[i][j] = (xh[i][j] - mean) * rs1;
        dw[i][j] = __builtin_fmaf(g[i][j], xh[i][j], dw[i][j]);
        db[i][j] += g[i][j];
        g[i][j] *= wi[j];
        c1 += g[i][j];
        c2 = __builtin_fmaf(g[i][j], xh[i][j], c2);
      }
    }
    if constexpr (kAhead) {
      if (row + step < p.rows) load(row + step);
    }
    if (packed) {
      c1 = group_sum(c1, width);
      c2 = group_sum(c2, width);
    } else {
      c1 = wave_sum(c1);
      c2 = wave_sum(c2);
    }
    if (waves > 1) {
      if ((tid & 63) == 0) {
        s_red[buf][0][wave] = c1;
        s_red[buf][1][wave] = c2;
      }
      __syncthreads();  // the other buffer is free again once all waves are here
      const bool mine = !MULTI || (tid & 15) < waves;
      const int at = !mine ? 0 : MULTI ? slot * waves + (tid & 15) : tid & 15;
      c1 = row16_sum(mine ? s_red[buf][0][at] : 0.0f);
      c2 = row16_sum(mine ? s_red[buf][1][at] : 0.0f);
    }
    if (!in) continue;
    c1 *= inv_d;
    c2 *= inv_d;
#pragma unroll
    for (int i = 0; i < N; ++i) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        g[i][j] = rs1 * (g[i][j] - c1 - xh[i][j] * c2);
        if constexpr (DS) g[i][j] += res[i][j];
      }
      Raw8<TO> o;
      from_f32(o, g[i]);
      store8(static_cast<TO*>(p.dx) + base, o, q[i]);
    }
  }
  float* part = p.part + (int64_t)blockIdx.x * 2 * p.d;
  if constexpr (MULTI) {
    const int at = packed ? wave : slot, n = kMultiWaves / waves;
    for (int o = width; o < kWave; o <<= 1) {  // the rows of a wave
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        dw[0][j] += __shfl_xor(dw[0][j], o, kWave);
        db[0][j] += __shfl_xor(db[0][j], o, kWave);
      }
    }
    if (!packed || (threadIdx.x & 63) < width) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (!owns(q[0], j)) continue;
        s_part[0][at * p.d + q[0].c + j] = dw[0][j];
        s_part[1][at * p.d + q[0].c + j] = db[0][j];
      }
    }
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * p.d; c += blockDim.x) {
      const int h = c >= p.d ? 1 : 0;
      float t[kMultiWaves], v = 0.0f;
#pragma unroll
      for (int k = 0; k < kMultiWaves; ++k) t[k] = s_part[h][min(k, n - 1) * p.d + c - h * p.d];
#pragma unroll
      for (int k = 0; k < kMultiWaves; ++k) v += k < n ? t[k] : 0.0f;
      part[c] = v;
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    Raw8<float> r;
    from_f32(r, dw[i]);
    store8(part, r, q[i]);
    from_f32(r, db[i]);
    store8(part + p.d, r, q[i]);
  }
}

// dw and db as the sums of the work-groups' parts: 64 columns a work-group, each
// of its 16 waves adds every 16th part in order (16 loads in flight: all of them
// at 256 parts), then the waves in order.
constexpr int kSumWaves = 16;
__global__ __launch_bounds__(kSumWaves* kWave) void norm_param_grad_kernel(const float* part, int parts, int d,
                                                                          float* dw, float* db) {
  __shared__ float s_sum[kSumWaves][kWave];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = blockIdx.x * kWave + lane;  // column of [dw | db]
  float v = 0.0f;
  if (c < 2 * d && parts > 0) {  // no rows: no parts to read, and no workspace
    const int64_t pitch = 2 * (int64_t)d;
    const float* at = part + c;
    auto batch = [&](auto n, int g) __attribute__((always_inline)) {
      constexpr int B = decltype(n)::value;
      float t[B];
#pragma unroll
      for (int i = 0; i < B; ++i) t[i] = at[min(g + i * kSumWaves, parts - 1) * pitch];
#pragma unroll
      for (int i = 0; i < B; ++i) v += g + i * kSumWaves < parts ? t[i] : 0.0f;
    };
    if (parts <= 4 * kSumWaves) {
      batch(std::integral_constant<int, 4>{}, wave);
    } else {
      for (int g = wave; g < parts; g += 16 * kSumWaves) batch(std::integral_constant<int, 16>{}, g);
    }
  }
  s_sum[wave][lane] = v;
  __syncthreads();
  if (wave == 0 && c < 2 * d) {
    v = s_sum[0][lane];
#pragma unroll
    for (int i = 1; i < kSumWaves; ++i) v += s_sum[i][lane];
    if (c < d) dw[c] = v;
    else if (db != nullptr) db[c - d] = v;
  }
}

// Loads pass the caches by when a call touches more than the package's 256 MB
// cache holds (16384 x 7168 bf16 with residual, 940 MB: 158 us against 161;
// backward 200 against 213); below that its inputs may still be there (4096 x
// 2048: 11.3 us against 14.2, backward 19.0 against 22.5).
bool streams(double bytes) { return bytes > 256.0 * (1 << 20); }

template <typename TX, typename TY, bool RES>
hipError_t fwd_n(const NormArgs& a, int n, dim3 grid, dim3 block, hipStream_t s) {
  const bool st = streams(static_cast<double>(a.rows) * a.d * (sizeof(TX) * (RES ? 3 : 1) + sizeof(TY)));
  if (n == 1 && st) hipLaunchKernelGGL((norm_fwd_kernel<TX, TY, RES, 1, true>), grid, block, 0, s, a);
  else if (n == 1) hipLaunchKernelGGL((norm_fwd_kernel<TX, TY, RES, 1, false>), grid, block, 0, s, a);
  else if (n == 2 && st) hipLaunchKernelGGL((norm_fwd_kernel<TX, TY, RES, 2, true>), grid, block, 0, s, a);
  else if (n == 2) hipLaunchKernelGGL((norm_fwd_kernel<TX, TY, RES, 2, false>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((norm_fwd_kernel<TX, TY, RES, 4, false>), grid, block, 0, s, a);
  return hipGetLastError();
}

// The same in one launch without parts, for few rows and for rows too wide to
// keep dw and db in registers: the first `row_groups` work-groups form dx, a row
// each, and the others dw and db, 64 columns each, from the rows again.
template <typename TD, typename TX, typename TO, bool DS, int N>
__global__ __launch_bounds__(kMaxWaves* kWave) void norm_bwd_split_kernel(const NormBwdArgs p, int row_groups, float* dw,
                                                                       float* db) {
  __shared__ float s_red[2][kMaxWaves][kWave];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  const TD* const dy = static_cast<const TD*>(p.dy);
  const TX* const x = static_cast<const TX*>(p.x);
  if (static_cast<int>(blockIdx.x) >= row_groups) {
    // columns: each wave adds every waves-th row, then the waves in order
    constexpr int B = 8;  // rows in flight
    const int c = (blockIdx.x - row_groups) * kWave + lane, at = min(c, p.d - 1);
    const int rows = static_cast<int>(p.rows);
    float sw = 0.0f, sb = 0.0f;
    for (int r0 = wave; r0 < rows; r0 += B * waves) {
      float g[B], v[B], mean[B], rstd[B];
#pragma unroll
      for (int i = 0; i < B; ++i) {
        const int r = min(r0 + i * waves, rows - 1);
        g[i] = one_f32(dy[(int64_t)r * p.d + at]);
        v[i] = one_f32(x[(int64_t)r * p.d + at]);
        mean[i] = p.mean[r];
        rstd[i] = p.rstd[r];
      }
#pragma unroll
      for (int i = 0; i < B; ++i) {
        if (r0 + i * waves >= rows) continue;
        sw = __builtin_fmaf(g[i], (v[i] - mean[i]) * rstd[i], sw);
        sb += g[i];
      }
    }
    s_red[0][wave][lane] = sw;
    s_red[1][wave][lane] = sb;
    __syncthreads();
    if (wave == 0 && c < p.d) {
      for (int w = 1; w < waves; ++w) {
        sw += s_red[0][w][lane];
        sb += s_red[1][w][lane];
      }
      dw[c] = sw;
      if (db != nullptr) db[c] = sb;
    }
    return;
  }
  const int64_t row = blockIdx.x, base = row * p.d;
  Piece q[N];
  Raw8<TD> rd[N];
  Raw8<TX> rx[N], rs[DS ? N : 1];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    q[i] = piece_of(i * blockDim.x + threadIdx.x, p.d);
    load8<false>(rd[i], dy + base, q[i]);
    load8<false>(rx[i], x + base, q[i]);
  }
  const float mean = p.mean[row], rstd = p.rstd[row], inv_d = 1.0f / static_cast<float>(p.d);
  float g[N][8], xh[N][8], c1 = 0.0f, c2 = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    Raw8<float> rw;
    float w[8];
    load8<false>(rw, p.w, q[i]);
    to_f32(rd[i], g[i]);
    to_f32(rx[i], xh[i]);
    to_f32(rw, w);
    mask8(g[i], q[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      xh[i][j] = (xh[i][j] - mean) * rstd;
      g[i][j] *= w[j];
      c1 += g[i][j];
      c2 = __builtin_fmaf(g[i][j], xh[i][j], c2);
    }
    if constexpr (DS) load8<false>(rs[i], static_cast<const TX*>(p.ds) + base, q[i]);
  }
  c1 = wave_sum(c1);
  c2 = wave_sum(c2);
  if (lane == 0) {
    s_red[0][0][wave] = c1;
    s_red[0][1][wave] = c2;
  }
  __syncthreads();
  c1 = row16_sum((lane & 15) < waves ? s_red[0][0][lane & 15] : 0.0f) * inv_d;
  c2 = row16_sum((lane & 15) < waves ? s_red[0][1][lane & 15] : 0.0f) * inv_d;
#pragma unroll
  for (int i = 0; i < N; ++i) {
#pragma unroll
    for (int j = 0; j < 8; ++j) g[i][j] = rstd * (g[i][j] - c1 - xh[i][j] * c2);
    if constexpr (DS) {
      float res[8];
      to_f32(rs[i], res);
#pragma unroll
      for (int j = 0; j < 8; ++j) g[i][j] += res[j];
    }
    Raw8<TO> o;
    from_f32(o, g[i]);
    store8(static_cast<TO*>(p.dx) + base, o, q[i]);
  }
}

// Lanes of a row that fits a wave: a power of two of them that covers its pieces,
// rows side by side in the wave (500000 x 128 bf16: forward 49 us against 106 with
// a wave per row, backward 79 against 153; 16384 x 128 4.2 against 7.7).
int row_lanes_log(int pieces) {
  int lg = 0;
  while (lg < 6 && (1 << lg) < pieces) ++lg;
  return lg;
}

// launch shape of the backward: pieces of 8 a lane holds, waves of a row, rows
// at once in a work-group, work-groups (= parts of the parameter gradients)
struct BwdShape {
  int n, waves, rpb, lg;
  int64_t groups;
  bool split;  // the one-launch form, which has no parts
};
// One piece a lane while a row then fits 16 waves (d <= 8192): two need over
// 128 registers (16384 x 7168: 206 us against 400).  Rows of up to 4 waves go
// side by side in work-groups of 8 (16384 x 1024 bf16: 28 us against 35).  One
// work-group per CU keeps the parts few (16384 x 7168: 206 + 5 us, 223 + 9 with
// two; 65536 x 2048 fp32: 293 against 337); rows of at most one wave take two
// where there are many (16000 x 257: 14.2 against 15.0; 250000 x 256 75.7 against
// 79.6, but 16384 x 256 13.9 against 12.7).
// The one-launch form: up to 384 rows (64 x 7168: 3.3 us against 8.1; 400 x 1024:
// 7.0 against 8.2, 400 x 200: 6.8 against 6.4), and rows of four pieces a lane,
// whose dw and db alone would be 64 registers of 128 (2000 x 20000 fp32: 157 us
// against 238 with parts).  With d_sum both forms spill beyond 8192 columns: rows
// of two pieces 16 to 44 bytes a lane, of four 36 to 128.
constexpr int kFewRows = 384;
BwdShape bwd_shape(int64_t rows, int d) {
  const int pieces = (d + 7) / 8;
  int n = 1;
  while (pieces > n * kWave * kMaxWaves) n *= 2;
  const int waves = (pieces + n * kWave - 1) / (n * kWave);
  const int lg = row_lanes_log(pieces);
  const int rpb = waves == 1 ? kMultiWaves * kWave >> lg : waves <= kMultiWaves / 2 ? kMultiWaves / waves : 1;
  const int64_t need = (rows + rpb - 1) / rpb, fill = waves == 1 && need > 4 * 256 ? 512 : 256;
  return {n, waves, rpb, lg, need < fill ? need : fill, rows > 0 && (rows <= kFewRows || n > 2)};
}

template <typename TD, typename TX, typename TO, bool DS>
hipError_t bwd_n(const NormBwdArgs& a, const BwdShape& b, float* dw, float* db, hipStream_t s) {
  if (b.split) {
    // at least 8 waves: the columns' rows are split over them
    const int rows = static_cast<int>(a.rows);
    const dim3 all(rows + (a.d + kWave - 1) / kWave), wide((b.waves > 8 ? b.waves : 8) * kWave);
    if (b.n == 1) hipLaunchKernelGGL((norm_bwd_split_kernel<TD, TX, TO, DS, 1>), all, wide, 0, s, a, rows, dw, db);
    else if (b.n == 2) hipLaunchKernelGGL((norm_bwd_split_kernel<TD, TX, TO, DS, 2>), all, wide, 0, s, a, rows, dw, db);
    else hipLaunchKernelGGL((norm_bwd_split_kernel<TD, TX, TO, DS, 4>), all, wide, 0, s, a, rows, dw, db);
    return hipGetLastError();
  }
  const dim3 grid(static_cast<unsigned>(b.groups)), block((b.rpb > 1 ? kMultiWaves / b.waves : 1) * b.waves * kWave);
  const bool st = streams(static_cast<double>(a.rows) * a.d * (sizeof(TD) + sizeof(TX) * (DS ? 2 : 1) + sizeof(TO)));
  if (b.rpb > 1) hipLaunchKernelGGL((norm_bwd_kernel<TD, TX, TO, DS, 1, true, false>), grid, block, 0, s, a);
  else if (b.n == 1 && st) hipLaunchKernelGGL((norm_bwd_kernel<TD, TX, TO, DS, 1, false, true>), grid, block, 0, s, a);
  else if (b.n == 1) hipLaunchKernelGGL((norm_bwd_kernel<TD, TX, TO, DS, 1, false, false>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((norm_bwd_kernel<TD, TX, TO, DS, 2, false, false>), grid, block, 0, s, a);
  return hipGetLastError();
}

template <typename TD, typename TX, typename TO>
hipError_t bwd_ds(const NormBwdArgs& a, const BwdShape& b, float* dw, float* db, hipStream_t s) {
  return a.ds != nullptr ? bwd_n<TD, TX, TO, true>(a, b, dw, db, s) : bwd_n<TD, TX, TO, false>(a, b, dw, db, s);
}

}  // namespace

hipError_t launch_layer_norm(int64_t rows, int d, const void* x, const void* r, int x_dtype, const float* w,
                             const float* b, float eps, void* sum, void* y, int y_dtype, float* mean, float* rstd,
                             hipStream_t s) {
  // two pieces a lane, one for narrow rows (4096 x 2048 bf16: 13.1 us against
  // 13.4; fp32 16384 x 7168: 303 against 296)
  const int pieces = (d + 7) / 8;
  int n = d <= 2048 ? 1 : 2;
  while (pieces > n * kWave * kMaxWaves) n *= 2;
  const int waves = (pieces + n * kWave - 1) / (n * kWave), lg = row_lanes_log(pieces);
  const int wg_waves = waves == 1 ? 4 : waves, rpb = waves == 1 ? wg_waves * kWave >> lg : 1;
  // Work-groups: all at once while the chip holds them; else about 24 KB of
  // loads per CU in flight (more only lengthens the queues: 16384 x 7168 bf16
  // 164 us with 256 work-groups, 180 with 512), in passes of equal length.
  const int64_t need = (rows + rpb - 1) / rpb;
  int64_t groups = need;
  if (need * wg_waves > 256 * 16) {
    const int64_t bytes = (int64_t)rpb * d * (x_dtype == MOE_BF16 ? 2 : 4) * (r != nullptr ? 2 : 1);
    const int64_t most = 256 * std::max<int64_t>(1, (24576 + bytes / 2) / bytes);
    const int64_t passes = (need + most - 1) / most;
    groups = (need + passes - 1) / passes;
  }
  const NormArgs a{rows, d, waves, rpb, lg, x, r, w, b, eps, sum, y, mean, rstd};
  const dim3 grid(static_cast<unsigned>(groups)), block(wg_waves * kWave);
  const bool xb = x_dtype == MOE_BF16, yb = y_dtype == MOE_BF16;
  if (r != nullptr) {
    if (xb) return yb ? fwd_n<uint16_t, uint16_t, true>(a, n, grid, block, s)
                      : fwd_n<uint16_t, float, true>(a, n, grid, block, s);
    return yb ? fwd_n<float, uint16_t, true>(a, n, grid, block, s)
              : fwd_n<float, float, true>(a, n, grid, block, s);
  }
  if (xb) return yb ? fwd_n<uint16_t, uint16_t, false>(a, n, grid, block, s)
                    : fwd_n<uint16_t, float, false>(a, n, grid, block, s);
  return yb ? fwd_n<float, uint16_t, false>(a, n, grid, block, s)
            : fwd_n<float, float, false>(a, n, grid, block, s);
}

size_t layer_norm_bwd_workspace_bytes(int64_t rows, int d) {
  const BwdShape b = bwd_shape(rows, d);
  return b.split ? 0 : static_cast<size_t>(b.groups) * 2 * d * sizeof(float);
}

hipError_t launch_layer_norm_bwd(int64_t rows, int d, const void* dy, int dy_dtype, const void* x, int x_dtype,
                                 const float* w, const float* mean, const float* rstd, const void* ds, void* dx,
                                 int dx_dtype, float* dw, float* db, float* ws, hipStream_t s) {
  const BwdShape b = bwd_shape(rows, d);
  if (b.groups > 0) {
    const NormBwdArgs a{rows, d, b.waves, b.rpb, b.lg, dy, x, w, mean, rstd, ds, dx, ws};
    const int key = (dy_dtype == MOE_BF16) | (x_dtype == MOE_BF16) << 1 | (dx_dtype == MOE_BF16) << 2;
    hipError_t e = hipSuccess;
    using B = uint16_t;
    switch (key) {
      case 0: e = bwd_ds<float, float, float>(a, b, dw, db, s); break;
      case 1: e = bwd_ds<B, float, float>(a, b, dw, db, s); break;
      case 2: e = bwd_ds<float, B, float>(a, b, dw, db, s); break;
      case 3: e = bwd_ds<B, B, float>(a, b, dw, db, s); break;
      case 4: e = bwd_ds<float, float, B>(a, b, dw, db, s); break;
      case 5: e = bwd_ds<B, float, B>(a, b, dw, db, s); break;
      case 6: e = bwd_ds<float, B, B>(a, b, dw, db, s); break;
      default: e = bwd_ds<B, B, B>(a, b, dw, db, s); break;
    }
    if (e != hipSuccess || b.split) return e;
  }
  hipLaunchKernelGGL(norm_param_grad_kernel, dim3((2 * d + kWave - 1) / kWave), dim3(kSumWaves * kWave), 0, s, ws,
                     static_cast<int>(b.groups), d, dw, db);
  return hipGetLastError();
}

}  // namespace moe

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
#include "launch.h"
#include "stream8.h"

namespace moe {
namespace {

constexpr int kMaxWaves = 16;

// ---------------------------------------------------------------- forward
struct NormArgs {
  int64_t rows;
  int d, wpr, rpb;  // waves per row, rows per work-group
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

// sum over the wpr waves of a row, the same tree on every call
__device__ __forceinline__ float row_sum(float v, float* s_red, int wpr) {
  v = wave_sum(v);
  if (wpr == 1) return v;
  const int wave = threadIdx.x >> 6;
  if ((threadIdx.x & 63) == 0) s_red[wave] = v;
  __syncthreads();
  float t = s_red[0];
  for (int i = 1; i < wpr; ++i) t += s_red[i];
  return t;
}

template <typename TX, typename TY, bool RES, int N>
__global__ __launch_bounds__(kMaxWaves* kWave) void norm_fwd_kernel(const NormArgs p) {
  __shared__ float s_red[2][kMaxWaves];
  const int slot = p.wpr == 1 ? threadIdx.x >> 6 : 0;
  const int rt = p.wpr == 1 ? threadIdx.x & 63 : threadIdx.x;  // thread within the row
  const int64_t row = (int64_t)blockIdx.x * p.rpb + slot;
  if (row >= p.rows) return;  // whole waves, and only where no barrier follows (rpb > 1 has wpr = 1)
  const int stride = p.wpr * kWave;
  const int64_t base = row * p.d;
  const TX* x = static_cast<const TX*>(p.x) + base;
  Raw8<TX> rx[N], rr[RES ? N : 1];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int c = (i * stride + rt) * 8;
    load8(rx[i], x + c, p.d - c);
    if constexpr (RES) load8(rr[i], static_cast<const TX*>(p.r) + base + c, p.d - c);
  }
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
      const int c = (i * stride + rt) * 8;
      Raw8<TX> s;
      from_f32(s, f[i]);
      store8(static_cast<TX*>(p.sum) + base + c, s, p.d - c);
      to_f32(s, f[i]);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) acc += f[i][j];
  }
  const float mean = row_sum(acc, s_red[0], p.wpr) / static_cast<float>(p.d);
  acc = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int left = p.d - (i * stride + rt) * 8;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      f[i][j] = j < left ? f[i][j] - mean : 0.0f;
      acc = __builtin_fmaf(f[i][j], f[i][j], acc);
    }
  }
  const float var = row_sum(acc, s_red[1], p.wpr) / static_cast<float>(p.d);
  const float rstd = 1.0f / __builtin_sqrtf(var + p.eps);
  if (rt == 0 && p.mean != nullptr) {
    p.mean[row] = mean;
    p.rstd[row] = rstd;
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int c = (i * stride + rt) * 8;
    if (c >= p.d) continue;
    float w[8], b[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const bool in = c + j < p.d;
      w[j] = in ? p.w[c + j] : 0.0f;
      b[j] = in && p.b != nullptr ? p.b[c + j] : 0.0f;
      f[i][j] = __builtin_fmaf(f[i][j] * rstd, w[j], b[j]);
    }
    Raw8<TY> o;
    from_f32(o, f[i]);
    store8(static_cast<TY*>(p.y) + base + c, o, p.d - c);
  }
}

// ---------------------------------------------------------------- backward
struct NormBwdArgs {
  int64_t rows;
  int d;
  const void* dy;
  const void* x;
  const float* w;
  const float* mean;
  const float* rstd;
  const void* ds;
  void* dx;
  float* part;  // [gridDim.x][2][d]: dw, db of this work-group's rows
};

// A work-group takes every gridDim.x-th row and keeps its columns' dw and db
// in registers; their sums leave once at the end.
template <typename TD, typename TX, typename TO, bool DS, int N>
__global__ __launch_bounds__(kMaxWaves* kWave) void norm_bwd_kernel(const NormBwdArgs p) {
  __shared__ float s_red[2][2][kMaxWaves];
  const int tid = threadIdx.x, wave = tid >> 6, waves = blockDim.x >> 6;
  float w[N][8], dw[N][8], db[N][8];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int c = (i * blockDim.x + tid) * 8;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      w[i][j] = c + j < p.d ? p.w[c + j] : 0.0f;
      dw[i][j] = db[i][j] = 0.0f;
    }
  }
  const float inv_d = 1.0f / static_cast<float>(p.d);
  int buf = 0;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x, buf ^= 1) {
    const int64_t base = row * p.d;
    Raw8<TD> rd[N];
    Raw8<TX> rx[N], rs[DS ? N : 1];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = (i * blockDim.x + tid) * 8;
      load8(rd[i], static_cast<const TD*>(p.dy) + base + c, p.d - c);
      load8(rx[i], static_cast<const TX*>(p.x) + base + c, p.d - c);
      if constexpr (DS) load8(rs[i], static_cast<const TX*>(p.ds) + base + c, p.d - c);
    }
    const float mean = p.mean[row], rstd = p.rstd[row];
    float xh[N][8], q[N][8];
    float c1 = 0.0f, c2 = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float dy[8];
      to_f32(rd[i], dy);
      to_f32(rx[i], xh[i]);
      const int left = p.d - (i * static_cast<int>(blockDim.x) + tid) * 8;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        xh[i][j] = j < left ? (xh[i][j] - mean) * rstd : 0.0f;
        q[i][j] = dy[j] * w[i][j];
        dw[i][j] = __builtin_fmaf(dy[j], xh[i][j], dw[i][j]);
        db[i][j] += dy[j];
        c1 += q[i][j];
        c2 = __builtin_fmaf(q[i][j], xh[i][j], c2);
      }
    }
    c1 = wave_sum(c1);
    c2 = wave_sum(c2);
    if (waves > 1) {
      if ((tid & 63) == 0) {
        s_red[buf][0][wave] = c1;
        s_red[buf][1][wave] = c2;
      }
      __syncthreads();  // the other buffer is free again once all waves are here
      c1 = s_red[buf][0][0];
      c2 = s_red[buf][1][0];
      for (int i = 1; i < waves; ++i) {
        c1 += s_red[buf][0][i];
        c2 += s_red[buf][1][i];
      }
    }
    c1 *= inv_d;
    c2 *= inv_d;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = (i * blockDim.x + tid) * 8;
      if (c >= p.d) continue;
      float o[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = rstd * (q[i][j] - c1 - xh[i][j] * c2);
      if constexpr (DS) {
        float g[8];
        to_f32(rs[i], g);
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] += g[j];
      }
      Raw8<TO> ro;
      from_f32(ro, o);
      store8(static_cast<TO*>(p.dx) + base + c, ro, p.d - c);
    }
  }
  float* part = p.part + (int64_t)blockIdx.x * 2 * p.d;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int c = (i * blockDim.x + tid) * 8;
    if (c >= p.d) continue;
    Raw8<float> r;
    from_f32(r, dw[i]);
    store8(part + c, r, p.d - c);
    from_f32(r, db[i]);
    store8(part + p.d + c, r, p.d - c);
  }
}

// dw and db as the sums of the work-groups' parts, each column by 4 lanes that
// take every fourth part in order, then (l0 + l1) + (l2 + l3)
__global__ __launch_bounds__(256) void norm_param_grad_kernel(const float* part, int parts, int d, float* dw,
                                                              float* db) {
  __shared__ float s_sum[4][kWave];
  const int lane = threadIdx.x & 63, q = threadIdx.x >> 6;
  const int c = blockIdx.x * kWave + lane;  // column of [dw | db]
  float v = 0.0f;
  if (c < 2 * d)
    for (int g = q; g < parts; g += 4) v += part[(int64_t)g * 2 * d + c];
  s_sum[q][lane] = v;
  __syncthreads();
  if (q == 0 && c < 2 * d) {
    v = (s_sum[0][lane] + s_sum[1][lane]) + (s_sum[2][lane] + s_sum[3][lane]);
    if (c < d) dw[c] = v;
    else if (db != nullptr) db[c - d] = v;
  }
}

template <typename TX, typename TY, bool RES>
hipError_t fwd_n(const NormArgs& a, int n, dim3 grid, dim3 block, hipStream_t s) {
  switch (n) {
    case 1: hipLaunchKernelGGL((norm_fwd_kernel<TX, TY, RES, 1>), grid, block, 0, s, a); break;
    case 2: hipLaunchKernelGGL((norm_fwd_kernel<TX, TY, RES, 2>), grid, block, 0, s, a); break;
    case 4: hipLaunchKernelGGL((norm_fwd_kernel<TX, TY, RES, 4>), grid, block, 0, s, a); break;
    default: hipLaunchKernelGGL((norm_fwd_kernel<TX, TY, RES, 8>), grid, block, 0, s, a); break;
  }
  return hipGetLastError();
}

template <typename TD, typename TX, typename TO, bool DS>
hipError_t bwd_n(const NormBwdArgs& a, int n, dim3 grid, dim3 block, hipStream_t s) {
  switch (n) {
    case 1: hipLaunchKernelGGL((norm_bwd_kernel<TD, TX, TO, DS, 1>), grid, block, 0, s, a); break;
    case 2: hipLaunchKernelGGL((norm_bwd_kernel<TD, TX, TO, DS, 2>), grid, block, 0, s, a); break;
    default: hipLaunchKernelGGL((norm_bwd_kernel<TD, TX, TO, DS, 4>), grid, block, 0, s, a); break;
  }
  return hipGetLastError();
}

template <typename TD, typename TX, typename TO>
hipError_t bwd_ds(const NormBwdArgs& a, int n, dim3 grid, dim3 block, hipStream_t s) {
  return a.ds != nullptr ? bwd_n<TD, TX, TO, true>(a, n, grid, block, s)
                         : bwd_n<TD, TX, TO, false>(a, n, grid, block, s);
}

// pieces of 8 a lane holds, and the waves that then cover a row
struct Split {
  int n, waves;
};
Split row_split(int d, int n) {
  const int pieces = (d + 7) / 8;
  while (pieces > n * kWave * kMaxWaves) n *= 2;
  return {n, (pieces + n * kWave - 1) / (n * kWave)};
}

}  // namespace

hipError_t launch_layer_norm(int64_t rows, int d, const void* x, const void* r, int x_dtype, const float* w,
                             const float* b, float eps, void* sum, void* y, int y_dtype, float* mean, float* rstd,
                             hipStream_t s) {
  const Split sp = row_split(d, d <= 512 ? 1 : 2);
  const int rpb = sp.waves == 1 ? 4 : 1;
  const NormArgs a{rows, d, sp.waves, rpb, x, r, w, b, eps, sum, y, mean, rstd};
  const dim3 grid(static_cast<unsigned>((rows + rpb - 1) / rpb)), block(sp.waves * rpb * kWave);
  const bool xb = x_dtype == MOE_BF16, yb = y_dtype == MOE_BF16;
  if (r != nullptr) {
    if (xb) return yb ? fwd_n<uint16_t, uint16_t, true>(a, sp.n, grid, block, s)
                      : fwd_n<uint16_t, float, true>(a, sp.n, grid, block, s);
    return yb ? fwd_n<float, uint16_t, true>(a, sp.n, grid, block, s)
              : fwd_n<float, float, true>(a, sp.n, grid, block, s);
  }
  if (xb) return yb ? fwd_n<uint16_t, uint16_t, false>(a, sp.n, grid, block, s)
                    : fwd_n<uint16_t, float, false>(a, sp.n, grid, block, s);
  return yb ? fwd_n<float, uint16_t, false>(a, sp.n, grid, block, s)
            : fwd_n<float, float, false>(a, sp.n, grid, block, s);
}

// work-groups of the backward (= parts of the parameter gradients)
static int64_t norm_bwd_groups(int64_t rows, int d) {
  const Split sp = row_split(d, d <= 512 ? 1 : 2);
  const int64_t fill = 256 * (sp.waves >= 8 ? 2 : 16 / sp.waves);
  return rows < fill ? rows : fill;
}

size_t layer_norm_bwd_workspace_bytes(int64_t rows, int d) {
  return static_cast<size_t>(norm_bwd_groups(rows, d)) * 2 * d * sizeof(float);
}

hipError_t launch_layer_norm_bwd(int64_t rows, int d, const void* dy, int dy_dtype, const void* x, int x_dtype,
                                 const float* w, const float* mean, const float* rstd, const void* ds, void* dx,
                                 int dx_dtype, float* dw, float* db, float* ws, hipStream_t s) {
  const int64_t groups = norm_bwd_groups(rows, d);
  if (groups > 0) {
    const Split sp = row_split(d, d <= 512 ? 1 : 2);
    const NormBwdArgs a{rows, d, dy, x, w, mean, rstd, ds, dx, ws};
    const dim3 grid(static_cast<unsigned>(groups)), block(sp.waves * kWave);
    const int key = (dy_dtype == MOE_BF16) | (x_dtype == MOE_BF16) << 1 | (dx_dtype == MOE_BF16) << 2;
    hipError_t e = hipSuccess;
    using B = uint16_t;
    switch (key) {
      case 0: e = bwd_ds<float, float, float>(a, sp.n, grid, block, s); break;
      case 1: e = bwd_ds<B, float, float>(a, sp.n, grid, block, s); break;
      case 2: e = bwd_ds<float, B, float>(a, sp.n, grid, block, s); break;
      case 3: e = bwd_ds<B, B, float>(a, sp.n, grid, block, s); break;
      case 4: e = bwd_ds<float, float, B>(a, sp.n, grid, block, s); break;
      case 5: e = bwd_ds<B, float, B>(a, sp.n, grid, block, s); break;
      case 6: e = bwd_ds<float, B, B>(a, sp.n, grid, block, s); break;
      default: e = bwd_ds<B, B, B>(a, sp.n, grid, block, s); break;
    }
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(norm_param_grad_kernel, dim3((2 * d + kWave - 1) / kWave), dim3(256), 0, s, ws,
                     static_cast<int>(groups), d, dw, db);
  return hipGetLastError();
}

}  // namespace moe

// Distillation from a teacher's top logits.  For a row's entries (index i_j,
// teacher logit t_j) with an index inside the vocabulary and a logit above -inf:
//     p = softmax(t / tau) over the entries,   q = softmax(x / tau) over V
//     l = tau^2 sum_j p_j (log p_j - log q[i_j])
//     dl/dx[v] = tau (q[v] - sum_{j: i_j = v} p_j)
// Without an entry, or with weight 0, a row adds nothing.  Indices may repeat.
//
// Beside the walk of the logits a row costs its wave 0 the entries: teacher and
// student logits there, one lane each, read while the row's sums are formed, and
// for the gradient a list for each thread that stores some of them, so that a
// piece is corrected before it is stored instead of read and written again.
// 4096 x 131072 bf16 with 64 entries and gradient 405 us (5.3 TB/s), the policy
// loss, which has one entry, 391; forward alone 175 and 172.  64 x 32000: 13 us.
#include "vocab_loss.h"

namespace moe {
namespace {

using vocab::exp_tau;
using vocab::Logits;

__device__ __forceinline__ double wave_sum_f64(double v) {
#pragma unroll
  for (int o = 1; o < kWave; o <<= 1) v += __shfl_xor(v, o, kWave);
  return v;
}

struct Distill {
  struct Args {
    const int* idx;
    const void* teacher;
    int K, wide;  // wide: the teacher's logits are fp32
  };
  // The entries, and for each thread a list of those among the logits it stores.
  template <int NT>
  struct Shared {
    int counted;
    float sum;              // of the teacher's exponentials
    float p[kMaxTeacher];   // probability (0: no entry)
    float w[kMaxTeacher];   // with that of the same index's other entries
    float u[kMaxTeacher];   // teacher's logit less the largest
    float x[kMaxTeacher];   // the student's logit
    int at[kMaxTeacher];
    int16_t next[kMaxTeacher];
    int head[NT];
  };
  static constexpr bool kLateFactor = false;
  static int grad_pieces(const Args& k) { return k.K <= 64 ? 2 : k.K <= 128 ? 4 : 8; }

  template <typename S>
  static __device__ __forceinline__ void init(S& sh, int tid) {
    sh.head[tid] = -1;
  }
  static __device__ __forceinline__ bool live(const Args&, int64_t, int) { return true; }

  // a lane's first entry
  struct Ahead {
    int id;
    float t;
  };
  static __device__ __forceinline__ Ahead entry(const Args& k, int64_t row, int j) {
    const int64_t from = row * k.K + min(j, k.K - 1);
    return {k.idx[from], k.wide ? static_cast<const float*>(k.teacher)[from]
                                : bf16_to_f32(static_cast<const uint16_t*>(k.teacher)[from])};
  }
  static __device__ __forceinline__ bool is_entry(const Logits& p, const Args& k, const Ahead& a, int j) {
    return j < k.K && static_cast<unsigned>(a.id) < static_cast<unsigned>(p.V) && a.t != -INFINITY;
  }
  static __device__ __forceinline__ Ahead ahead(const Args& k, int64_t row, int tid) {
    if (tid >= kWave) return {};
    return entry(k, row, tid);
  }
  // and the student's logit there
  template <typename TX>
  struct Few {
    Ahead a;
    TX x;
  };
  template <typename TX>
  static __device__ __forceinline__ Few<TX> begin(const Logits& p, const Args& k, int64_t, const TX* x, int tid,
                                                  const Ahead& a) {
    if (tid >= kWave) return {};
    return {a, x[is_entry(p, k, a, tid) ? a.id : 0]};
  }

  template <typename TX, typename S>
  static __device__ __forceinline__ void share(const Logits& p, const Args& k, int64_t row, const TX* x, bool grad,
                                               const vocab::Owner& owner, int lane, const Few<TX>& few, S& sh) {
    const bool ok = is_entry(p, k, few.a, lane);
    const int v = ok ? few.a.id : -1;
    uint64_t any = __ballot(ok);
    float top = ok ? few.a.t : -FLT_MAX, sum;
    if (k.K <= kWave) {  // all in this lane's registers
      top = wave_max(top);
      const float u = few.a.t - top, e = ok ? exp_tau(p, u) : 0.0f;
      sum = wave_sum(e);
      if (lane < k.K) {
        sh.u[lane] = u;
        sh.x[lane] = one_f32(few.x);
        enter(sh, owner, lane, v, e / sum, grad);
      }
    } else {
      for (int j = lane; j < k.K; j += kWave) {
        const Ahead a = j < kWave ? few.a : entry(k, row, j);
        const bool in = is_entry(p, k, a, j);
        sh.at[j] = in ? a.id : -1;
        sh.u[j] = a.t;
        sh.x[j] = one_f32(j < kWave ? few.x : x[in ? a.id : 0]);
        if (in) top = fmaxf(top, a.t);
        any |= __ballot(in);
      }
      top = wave_max(top);
      sum = weigh(p, k, top, lane, sh);
      for (int j = lane; j < k.K; j += kWave) enter(sh, owner, j, sh.at[j], sh.p[j] / sum, grad);
    }
    if (lane == 0) {
      sh.counted = any != 0;
      sh.sum = sum;
    }
  }
  // u and the exponentials' sum from the logits in u, by one wave
  template <typename S>
  static __device__ __forceinline__ float weigh(const Logits& p, const Args& k, float top, int lane, S& sh) {
    float sum = 0.0f;
    for (int j = lane; j < k.K; j += kWave) {
      const float u = sh.u[j] - top, e = sh.at[j] >= 0 ? exp_tau(p, u) : 0.0f;
      sh.u[j] = u;
      sh.p[j] = e;
      sum += e;
    }
    return wave_sum(sum);
  }
  // entry j, and where its gradient is wanted on the list of the thread that stores it
  template <typename S>
  static __device__ __forceinline__ void enter(S& sh, const vocab::Owner& owner, int j, int v, float pj, bool list) {
    sh.at[j] = v;
    sh.p[j] = pj;
    if (list && v >= 0) sh.next[j] = static_cast<int16_t>(atomicExch(&sh.head[owner.of(v)], j));
  }

  // for the gradient alone: the probabilities, and the entries among [lo, hi)
  template <typename TX, typename S>
  static __device__ __forceinline__ void entries(const Logits& p, const Args& k, int64_t row, const TX*,
                                                 const vocab::Owner& owner, int lo, int hi, int lane, S& sh) {
    Ahead a = entry(k, row, lane);
    bool ok = is_entry(p, k, a, lane);
    uint64_t any = __ballot(ok);
    float top = ok ? a.t : -FLT_MAX, sum;
    if (k.K <= kWave) {
      top = wave_max(top);
      const float e = ok ? exp_tau(p, a.t - top) : 0.0f;
      sum = wave_sum(e);
      if (lane < k.K) enter(sh, owner, lane, a.id, e / sum, ok && a.id >= lo && a.id < hi);
    } else {
      for (int j = lane; j < k.K; j += kWave) {
        if (j >= kWave) a = entry(k, row, j);
        ok = is_entry(p, k, a, j);
        sh.at[j] = ok ? a.id : -1;
        sh.u[j] = a.t;
        if (ok) top = fmaxf(top, a.t);
        any |= __ballot(ok);
      }
      top = wave_max(top);
      sum = weigh(p, k, top, lane, sh);
      for (int j = lane; j < k.K; j += kWave) {
        const int v = sh.at[j];
        enter(sh, owner, j, v, sh.p[j] / sum, v >= lo && v < hi);
      }
    }
    if (lane == 0) sh.counted = any != 0;
  }

  template <typename S>
  static __device__ __forceinline__ void finish(const Logits& p, const Args& k, int64_t row, float, float m, float sum,
                                                int lane, S& sh, bool) {
    // fp64, so that nothing is added to the two sums' own errors, which the loss carries as an
    // absolute one where student and teacher agree (512 rows of 32: 6e-8 tau^2 rms, 2e-7 at most)
    const bool counted = sh.counted != 0;
    const double shift = vocab::ln_of(sum) - vocab::ln_of(sh.sum);
    double l = 0.0;
    for (int j = lane; j < k.K; j += kWave) {
      const float pj = sh.p[j];
      if (pj != 0.0f) {
        const double d = static_cast<double>(sh.u[j]) - (static_cast<double>(sh.x[j]) - static_cast<double>(m));
        l += pj * (d * p.inv_tau + shift);
      }
    }
    l = wave_sum_f64(l);
    if (lane == 0) {
      p.row_loss[row] = counted ? static_cast<float>(l * p.tau * p.tau) : 0.0f;
      p.stats[2 * row] = counted ? m : 0.0f;
      p.stats[2 * row + 1] = counted ? sum : 0.0f;
    }
  }

  template <typename S>
  static __device__ __forceinline__ float factor(const Logits& p, float gw, const S& sh) {
    return sh.counted ? gw * static_cast<float>(p.tau) : 0.0f;
  }

  // A thread's list: its first entry in registers, the pieces that the others are in.
  struct Mine {
    int v, rest;
    float w;
    uint32_t mask;
  };
  template <typename S>
  static __device__ __forceinline__ Mine mine(const vocab::Owner& owner, S& sh, int tid, bool any) {
    Mine my{-1, -1, 0.0f, 0};
    const int j0 = any ? sh.head[tid] : -1;
    if (j0 < 0) return my;
    my.v = sh.at[j0];
    my.rest = sh.next[j0];
    my.w = sh.p[j0];
    if (my.rest < 0) return my;
    // An index that comes several times is taken once, its probabilities summed in
    // units of 2^-60: their order, which is not that of the entries, does not matter.
    for (int j = j0; j >= 0; j = sh.next[j]) {
      const int v = sh.at[j];
      if (v < 0) continue;
      float w = sh.p[j];
      uint64_t units = 0;
      for (int i = sh.next[j]; i >= 0; i = sh.next[i]) {
        if (sh.at[i] != v) continue;
        if (units == 0) units = in_units(w);
        units += in_units(sh.p[i]);
        sh.at[i] = -1;
      }
      if (units != 0 && w == w) w = static_cast<float>(units) * 0x1p-60f;  // (NaN stays)
      sh.w[j] = w;
      if (j == j0) {
        my.w = w;
        continue;
      }
      const int piece = v / owner.e;
      my.mask |= 1u << (piece < owner.pieces ? min(owner.local(piece), vocab::kManyPieces) : vocab::kManyPieces);
    }
    return my;
  }
  template <int E, typename S>
  static __device__ __forceinline__ void correct(S& sh, const Mine& my, int local, int piece, float kr, int,
                                                 float (&f)[E]) {
    auto take = [&](int v, float w) __attribute__((always_inline)) {
      const int i = v - piece * E;
      if (static_cast<unsigned>(i) >= static_cast<unsigned>(E)) return;
      const float less = kr * w;
#pragma unroll
      for (int l = 0; l < E; ++l) f[l] -= l == i ? less : 0.0f;
    };
    take(my.v, my.w);
    if ((my.mask >> min(local, vocab::kManyPieces) & 1) == 0) return;
    for (int j = my.rest; j >= 0; j = sh.next[j]) take(sh.at[j], sh.w[j]);
  }
  template <typename S>
  static __device__ __forceinline__ float correct_one(S& sh, const Mine& my, int at, float kr, int, float f) {
    if (my.v == at) f -= kr * my.w;
    if (my.mask >> vocab::kManyPieces == 0) return f;
    for (int j = my.rest; j >= 0; j = sh.next[j])
      if (sh.at[j] == at) f -= kr * sh.w[j];
    return f;
  }
  template <typename S>
  static __device__ __forceinline__ void done(S& sh, int tid) {
    sh.head[tid] = -1;
  }
  static __device__ __forceinline__ uint64_t in_units(float v) { return static_cast<uint64_t>(v * 0x1p60f); }

  static __device__ __forceinline__ void none(const Logits& p, const Args&, int64_t row) {
    p.row_loss[row] = p.stats[2 * row] = p.stats[2 * row + 1] = 0.0f;
  }
};

// 1024 threads add every 1024th row in fp64, then a fixed tree.
__global__ __launch_bounds__(1024) void loss_sum_kernel(int64_t rows, const float* row_loss, const float* weight,
                                                        float even, float* loss) {
  constexpr int B = 8;
  __shared__ double s_sum[16];
  double v = 0.0;
  for (int64_t t0 = threadIdx.x; t0 < rows; t0 += B * 1024) {
    float l[B], w[B];
#pragma unroll
    for (int i = 0; i < B; ++i) {
      const int64_t t = min(t0 + i * 1024, rows - 1);
      l[i] = row_loss[t];
      w[i] = weight != nullptr ? weight[t] : even;
    }
#pragma unroll
    for (int i = 0; i < B; ++i) {
      if (t0 + i * 1024 < rows && w[i] != 0.0f) v += static_cast<double>(w[i]) * static_cast<double>(l[i]);
    }
  }
  v = wave_sum_f64(v);
  if ((threadIdx.x & 63) == 0) s_sum[threadIdx.x >> 6] = v;
  __syncthreads();
  if (threadIdx.x >= 64) return;
  v = wave_sum_f64(threadIdx.x < 16 ? s_sum[threadIdx.x] : 0.0);
  if (threadIdx.x == 0) *loss = static_cast<float>(v);
}

}  // namespace

hipError_t launch_loss_sum(int64_t rows, const float* row_loss, const float* weight, float even, float* loss,
                           hipStream_t s) {
  hipLaunchKernelGGL(loss_sum_kernel, dim3(1), dim3(1024), 0, s, rows, row_loss, weight, even, loss);
  return hipGetLastError();
}

hipError_t launch_distill_loss(int64_t rows, int V, int K, const void* x, int x_dtype, const int32_t* idx,
                               const void* teacher, int t_dtype, double tau, const float* weight, const float* grad,
                               float* loss, float* row_loss, float* stats, void* dx, int dx_dtype, hipStream_t s) {
  if (rows > 0) {
    Logits p = vocab::logits_of(rows, V, tau, weight, grad);
    p.x = x;
    p.dx = dx;
    p.stats = stats;
    p.row_loss = row_loss;
    const Distill::Args k{idx, teacher, K, t_dtype == MOE_F32};
    const hipError_t e = vocab::loss_dtypes<Distill>(p, k, x_dtype, dx_dtype, s);
    if (e != hipSuccess) return e;
  }
  return launch_loss_sum(rows, row_loss, weight, rows > 0 ? static_cast<float>(1.0 / static_cast<double>(rows)) : 0.0f,
                         loss, s);
}

hipError_t launch_distill_loss_bwd(int64_t rows, int V, int K, const void* x, int x_dtype, const float* stats,
                                   const int32_t* idx, const void* teacher, int t_dtype, double tau,
                                   const float* weight, const float* grad, void* dx, int dx_dtype, hipStream_t s) {
  Logits p = vocab::logits_of(rows, V, tau, weight, grad);
  p.x = x;
  p.dx = dx;
  p.stats = const_cast<float*>(stats);  // read only
  const Distill::Args k{idx, teacher, K, t_dtype == MOE_F32};
  return vocab::grad_dtypes<Distill>(p, k, x_dtype, dx_dtype, s);
}

}  // namespace moe

// The router's balance loss, per-expert counts, and the loss's gradient.
//
//   a = sqrt(softplus(l)), p = a / sum_e a          per counted token
//   c[s,e] slots of sequence s on expert e, T_s its counted tokens
//   f = E c / (k T_s),  P = sum_t p / T_s
//   loss = alpha / n_seq * sum_s sum_e f P
//   dprob[s,e] = dloss / dp[t,e] = alpha f / (n_seq T_s)      (c held fixed)
//   dl[t,e] = g (dprob_e - sum_j dprob_j p_j) / S * sig(l) / (2 a)
//
// Here the affinity is a smooth function to be summed, not ranked, so fp32
// serves (the router's fp64 sequence exists for its ties):  with h = e^(-|l|/2),
// u = h h, z = u / (2 + u),
//   log1p(u) = 2 atanh(z) = u q,  q = 2/(2+u) (1 + z^2/3 + z^4/5 + ...)
// (z <= 1/3: seven terms leave 2e-8), a = sqrt(l + u q) for l >= 0 and
// h sqrt(q) for l < 0: no cancellation, and no underflow before e^(l/2) does.
// A row whose affinities all vanish has no probabilities: it adds 0.
#include "launch.h"
#include "stream8.h"

namespace moe {
namespace {

constexpr int kTile = 64;      // tokens of one work-group
constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / kWave;

struct Affinity {
  float a;   // sqrt(softplus(l))
  float da;  // its derivative sig(l) / (2 a)
};

template <bool GRAD>
__device__ __forceinline__ Affinity affinity(float l) {
  const float h = __expf(-0.5f * __builtin_fabsf(l));
  const float u = h * h;
  const float inv = __builtin_amdgcn_rcpf(2.0f + u);
  const float z = u * inv, z2 = z * z;
  float s = 1.0f / 13.0f;
  s = __builtin_fmaf(s, z2, 1.0f / 11.0f);
  s = __builtin_fmaf(s, z2, 1.0f / 9.0f);
  s = __builtin_fmaf(s, z2, 1.0f / 7.0f);
  s = __builtin_fmaf(s, z2, 1.0f / 5.0f);
  s = __builtin_fmaf(s, z2, 1.0f / 3.0f);
  s = __builtin_fmaf(s, z2, 1.0f);
  const float q = 2.0f * inv * s;
  const bool neg = l < 0.0f;
  const float t = __builtin_amdgcn_sqrtf(neg ? q : __builtin_fmaf(u, q, l));
  Affinity r;
  r.a = neg ? h * t : t;
  // sig(l) / (2 a) = h / (2 (1+u) t) for l < 0, 1 / (2 (1+u) t) for l >= 0
  r.da = GRAD ? (neg ? 0.5f * h : 0.5f) * __builtin_amdgcn_rcpf((1.0f + u) * t) : 0.0f;
  return r;
}

// The sequence of token t among offsets (nullptr: one sequence of all T
// tokens); -1 for a token outside them.
__device__ __forceinline__ int sequence_of(int64_t t, int64_t T, const int32_t* off, int n_seq) {
  if (t >= T) return -1;
  if (off == nullptr) return 0;
  if (t < off[0] || t >= off[n_seq]) return -1;
  int lo = 0, hi = n_seq;  // off[lo] <= t < off[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (off[mid] <= t) lo = mid; else hi = mid;
  }
  return lo;
}

// A row of E logits in a wave: lane groups of `lpt` lanes (a power of two)
// hold one token each, a lane 4 consecutive experts of every 256.
struct RowMap {
  int E, lpt, log_lpt;
};
template <int NR>
__device__ __forceinline__ void load_row(const float* row, const float* offset, const RowMap& m, int sub,
                                         float (&l)[NR][4]) {
#pragma unroll
  for (int r = 0; r < NR; ++r) {
    const int e = r * 256 + sub * 4;
    if (e + 4 <= m.E) {
      const u32x4 v = *reinterpret_cast<const u32x4_a4*>(row + e);
#pragma unroll
      for (int i = 0; i < 4; ++i) l[r][i] = __uint_as_float(v[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) l[r][i] = e + i < m.E ? row[e + i] : 0.0f;
    }
    if (offset != nullptr) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (e + i < m.E) l[r][i] += offset[e + i];
    }
  }
}

// sum over the aligned group of lpt lanes
__device__ __forceinline__ float group_sum(float v, int lpt) {
  for (int o = 1; o < lpt; o <<= 1) v += __shfl_xor(v, o, kWave);
  return v;
}

struct LossArgs {
  int64_t T;
  RowMap m;
  int k, n_seq;
  const float* logits;
  const float* offset;
  const int32_t* idx;
  const int32_t* seq;
  const uint8_t* mask;
  float* psum;    // [tiles + n_seq][E]
  int32_t* pcnt;  // [tiles + n_seq][E]
  int32_t* ptok;  // [tiles + n_seq]
};

// One work-group per tile of tokens.  For each sequence s with tokens in tile
// b it writes the sums of p, the slot counts and the token count to row b + s:
// along the tokens b and s only grow, so no two pairs share a row.
template <int NR>
__global__ __launch_bounds__(kThreads) void balance_part_kernel(const LossArgs p) {
  __shared__ int s_seq[kTile];
  __shared__ uint8_t s_on[kTile];
  __shared__ int s_cnt[NR * 256];
  __shared__ float s_sum[kWaves][NR * 256];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t t0 = (int64_t)blockIdx.x * kTile;
  const int ntok = static_cast<int>(min((int64_t)kTile, p.T - t0));
  if (tid < kTile) {
    s_seq[tid] = sequence_of(t0 + tid, p.T, p.seq, p.n_seq);
    s_on[tid] = tid < ntok && (p.mask == nullptr || p.mask[t0 + tid] != 0);
  }
  __syncthreads();
  const int E = p.m.E, lpt = p.m.lpt, tpw = kWave / lpt, sub = lane & (lpt - 1), which = lane >> p.m.log_lpt;
  // one sequence's run of tokens [i0, i1) at a time (uniform over the work-group)
  for (int i0 = 0, i1; i0 < ntok; i0 = i1) {
    const int s = s_seq[i0];
    i1 = i0 + 1;
    if (s < 0) continue;
    while (i1 < ntok && s_seq[i1] == s) ++i1;
    int tokens = 0;
    for (int i = i0; i < i1; ++i) tokens += s_on[i];
    for (int e = tid; e < E; e += kThreads) s_cnt[e] = 0;
    __syncthreads();
    float sum[NR][4] = {};
    for (int i = i0 + wave * tpw + which; i < i1 + tpw; i += kWaves * tpw) {
      const bool in = i < i1 && s_on[i];
      if (!__any(in)) continue;
      float l[NR][4], a[NR][4], total = 0.0f;
      load_row<NR>(p.logits + (t0 + (in ? i : i0)) * E, p.offset, p.m, sub, l);
#pragma unroll
      for (int r = 0; r < NR; ++r)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          // a token that does not count may hold anything, also NaN
          a[r][j] = in && r * 256 + sub * 4 + j < E ? affinity<false>(l[r][j]).a : 0.0f;
          total += a[r][j];
        }
      total = group_sum(total, lpt);
      const float inv = total > 0.0f ? 1.0f / total : 0.0f;
#pragma unroll
      for (int r = 0; r < NR; ++r)
#pragma unroll
        for (int j = 0; j < 4; ++j) sum[r][j] = __builtin_fmaf(a[r][j], inv, sum[r][j]);
    }
    for (int i = i0 * p.k + tid; i < i1 * p.k; i += kThreads) {
      if (!s_on[i / p.k]) continue;
      const int e = p.idx[t0 * p.k + i];
      if (e >= 0 && e < E) atomicAdd(&s_cnt[e], 1);
    }
    // the lane groups of a wave, then the waves in order
#pragma unroll
    for (int r = 0; r < NR; ++r)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float v = sum[r][j];
        for (int o = lpt; o < kWave; o <<= 1) v += __shfl_xor(v, o, kWave);
        if (which == 0) s_sum[wave][r * 256 + sub * 4 + j] = v;
      }
    __syncthreads();
    const int64_t row = (int64_t)blockIdx.x + s;
    for (int e = tid; e < E; e += kThreads) {
      float v = s_sum[0][e];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) v += s_sum[w][e];
      p.psum[row * E + e] = v;
      p.pcnt[row * E + e] = s_cnt[e];
    }
    if (tid == 0) p.ptok[row] = tokens;
    __syncthreads();
  }
}

struct SumArgs {
  int64_t T;
  int E, k, n_seq;
  float alpha;
  const int32_t* seq;
  const float* psum;
  const int32_t* pcnt;
  const int32_t* ptok;
  int32_t* counts;
  float* prob;
  float* dprob;
  float* ploss;  // [n_seq]
};

// One work-group per sequence: the parts of its tiles in order.
__global__ __launch_bounds__(kThreads) void balance_sum_kernel(const SumArgs p) {
  __shared__ float s_red[kWaves];
  const int s = blockIdx.x, tid = threadIdx.x;
  const int64_t lo = p.seq == nullptr ? 0 : max((int64_t)p.seq[s], (int64_t)0);
  const int64_t hi = p.seq == nullptr ? p.T : min((int64_t)p.seq[s + 1], p.T);
  const int64_t b0 = lo / kTile, b1 = lo < hi ? (hi - 1) / kTile + 1 : b0;
  int64_t tokens = 0;
  for (int64_t b = b0; b < b1; ++b) tokens += p.ptok[b + s];
  const float per = tokens > 0 ? 1.0f / static_cast<float>(tokens) : 0.0f;
  float part = 0.0f;
  for (int e = tid; e < p.E; e += kThreads) {
    float v = 0.0f;
    int64_t c = 0;
    for (int64_t b = b0; b < b1; ++b) {
      v += p.psum[(b + s) * p.E + e];
      c += p.pcnt[(b + s) * p.E + e];
    }
    const float f = static_cast<float>(c) * (static_cast<float>(p.E) / static_cast<float>(p.k)) * per;
    const float P = v * per;
    p.counts[(int64_t)s * p.E + e] = static_cast<int32_t>(c);
    p.prob[(int64_t)s * p.E + e] = P;
    p.dprob[(int64_t)s * p.E + e] = f * per * (p.alpha / static_cast<float>(p.n_seq));
    part = __builtin_fmaf(f, P, part);
  }
  part = wave_sum(part);
  if ((tid & 63) == 0) s_red[tid >> 6] = part;
  __syncthreads();
  if (tid == 0) {
    float t = 0.0f;
    for (int w = 0; w < kWaves; ++w) t += s_red[w];
    p.ploss[s] = t;
  }
}

__global__ __launch_bounds__(kWave) void balance_total_kernel(const float* ploss, int n_seq, float alpha,
                                                              float* loss) {
  float v = 0.0f;
  for (int s = threadIdx.x; s < n_seq; s += kWave) v += ploss[s];
  v = wave_sum(v);
  if (threadIdx.x == 0) *loss = v * (alpha / static_cast<float>(n_seq));
}

struct GradArgs {
  int64_t T;
  RowMap m;
  int n_seq;
  const float* logits;
  const float* offset;
  const int32_t* seq;
  const uint8_t* mask;
  const float* dprob;
  const float* grad;
  const float* extra;
  float* dl;
};

constexpr int kGradThreads = 256;

template <int NR>
__global__ __launch_bounds__(kGradThreads) void balance_grad_kernel(const GradArgs p) {
  __shared__ int s_seq[kTile];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t t0 = (int64_t)blockIdx.x * kTile;
  const int ntok = static_cast<int>(min((int64_t)kTile, p.T - t0));
  if (tid < kTile) {
    const int s = sequence_of(t0 + tid, p.T, p.seq, p.n_seq);
    s_seq[tid] = s >= 0 && (p.mask == nullptr || p.mask[t0 + tid] != 0) ? s : -1;
  }
  __syncthreads();
  const float g = p.grad == nullptr ? 1.0f : *p.grad;
  const int E = p.m.E, lpt = p.m.lpt, tpw = kWave / lpt, sub = lane & (lpt - 1), which = lane >> p.m.log_lpt;
  for (int i = wave * tpw + which; i < kTile; i += (kGradThreads / kWave) * tpw) {
    const bool in = i < ntok;
    if (!__any(in)) break;
    const int s = in ? s_seq[i] : -1;
    const int64_t base = (t0 + (in ? i : 0)) * E;
    float l[NR][4], dp[NR][4];
    Affinity a[NR][4];
    load_row<NR>(p.logits + base, p.offset, p.m, sub, l);
    float total = 0.0f, dot = 0.0f;
#pragma unroll
    for (int r = 0; r < NR; ++r)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int e = r * 256 + sub * 4 + j;
        a[r][j] = affinity<true>(l[r][j]);
        if (e >= E) a[r][j].a = 0.0f;
        dp[r][j] = e < E && s >= 0 ? p.dprob[(int64_t)s * E + e] : 0.0f;
        total += a[r][j].a;
        dot = __builtin_fmaf(dp[r][j], a[r][j].a, dot);
      }
    total = group_sum(total, lpt);
    dot = group_sum(dot, lpt);
    const float inv = s >= 0 && total > 0.0f ? 1.0f / total : 0.0f;
    const float mean = dot * inv, scale = g * inv;
    if (!in) continue;
#pragma unroll
    for (int r = 0; r < NR; ++r)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int e = r * 256 + sub * 4 + j;
        if (e >= E) continue;
        float v = inv == 0.0f ? 0.0f : scale * (dp[r][j] - mean) * a[r][j].da;
        if (p.extra != nullptr) v += p.extra[base + e];
        p.dl[base + e] = v;
      }
  }
}

RowMap row_map(int E) {
  int lpt = 1, lg = 0;
  while (lpt < kWave && lpt * 4 < E) {
    lpt <<= 1;
    ++lg;
  }
  return {E, lpt, lg};
}

struct LossWs {
  size_t psum, pcnt, ptok, ploss, total;
};
LossWs loss_ws(int64_t T, int E, int n_seq) {
  const size_t rows = static_cast<size_t>((T + kTile - 1) / kTile) + n_seq;
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  LossWs w;
  w.psum = 0;
  w.pcnt = up(rows * E * sizeof(float));
  w.ptok = w.pcnt + up(rows * E * sizeof(int32_t));
  w.ploss = w.ptok + up(rows * sizeof(int32_t));
  w.total = w.ploss + up(n_seq * sizeof(float));
  return w;
}

}  // namespace

size_t balance_loss_workspace_bytes(int64_t T, int E, int n_seq) { return loss_ws(T, E, n_seq).total; }

hipError_t launch_balance_loss(int64_t T, int E, int k, const float* logits, const float* offset, const int32_t* idx,
                               const int32_t* seq, int n_seq, const uint8_t* mask, float alpha, int32_t* counts,
                               float* prob, float* dprob, float* loss, void* ws, hipStream_t s) {
  const LossWs w = loss_ws(T, E, n_seq);
  char* base = static_cast<char*>(ws);
  float* psum = reinterpret_cast<float*>(base + w.psum);
  int32_t* pcnt = reinterpret_cast<int32_t*>(base + w.pcnt);
  int32_t* ptok = reinterpret_cast<int32_t*>(base + w.ptok);
  float* ploss = reinterpret_cast<float*>(base + w.ploss);
  const int64_t tiles = (T + kTile - 1) / kTile;
  hipError_t e;
  if (tiles > 0) {
    const LossArgs a{T, row_map(E), k, n_seq, logits, offset, idx, seq, mask, psum, pcnt, ptok};
    const dim3 grid(static_cast<unsigned>(tiles)), block(kThreads);
    if (E <= 256) hipLaunchKernelGGL(balance_part_kernel<1>, grid, block, 0, s, a);
    else if (E <= 512) hipLaunchKernelGGL(balance_part_kernel<2>, grid, block, 0, s, a);
    else hipLaunchKernelGGL(balance_part_kernel<4>, grid, block, 0, s, a);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  const SumArgs b{T, E, k, n_seq, alpha, seq, psum, pcnt, ptok, counts, prob, dprob, ploss};
  hipLaunchKernelGGL(balance_sum_kernel, dim3(n_seq), dim3(kThreads), 0, s, b);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  hipLaunchKernelGGL(balance_total_kernel, dim3(1), dim3(kWave), 0, s, ploss, n_seq, alpha, loss);
  return hipGetLastError();
}

hipError_t launch_balance_loss_bwd(int64_t T, int E, const float* logits, const float* offset, const int32_t* seq,
                                   int n_seq, const uint8_t* mask, const float* dprob, const float* grad,
                                   const float* extra, float* dl, hipStream_t s) {
  const GradArgs a{T, row_map(E), n_seq, logits, offset, seq, mask, dprob, grad, extra, dl};
  const dim3 grid(static_cast<unsigned>((T + kTile - 1) / kTile)), block(kGradThreads);
  if (E <= 256) hipLaunchKernelGGL(balance_grad_kernel<1>, grid, block, 0, s, a);
  else if (E <= 512) hipLaunchKernelGGL(balance_grad_kernel<2>, grid, block, 0, s, a);
  else hipLaunchKernelGGL(balance_grad_kernel<4>, grid, block, 0, s, a);
  return hipGetLastError();
}

}  // namespace moe

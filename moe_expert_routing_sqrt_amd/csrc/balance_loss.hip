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
// serves (the router's fp64 sequence exists for its ties).  With h = e^(-|l|/2)
// and u = h h in [0, 1],
//   log1p(u) = u q(u),  q the degree-8 interpolant of log1p(u)/u at the nine
//   Chebyshev nodes of [0, 1] (relative error 3.4e-8),
//   a = sqrt(l + u q) for l >= 0 and h sqrt(q) for l < 0:
// no cancellation, and no underflow before e^(l/2) itself.  Two
// transcendental instructions and 16 others an element.
// A row whose affinities all vanish has no probabilities: it adds 0.
#include "launch.h"
#include "stream8.h"

namespace moe {
namespace {

constexpr int kTile = 64;  // tokens of a forward work-group: one per lane
constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / kWave;

struct Affinity {
  float a;   // sqrt(softplus(l))
  float da;  // its derivative sig(l) / (2 a)
};

template <bool GRAD>
__device__ __forceinline__ Affinity affinity(float l) {
  const float h = __builtin_amdgcn_exp2f(__builtin_fabsf(l) * -0.72134752f);  // -log2(e)/2
  const float u = h * h;
  float q = 0x1.4ff1bap-8f;
  q = __builtin_fmaf(q, u, -0x1.dc5978p-6f);
  q = __builtin_fmaf(q, u, 0x1.3d8182p-4f);
  q = __builtin_fmaf(q, u, -0x1.1692f4p-3f);
  q = __builtin_fmaf(q, u, 0x1.86b1ccp-3f);
  q = __builtin_fmaf(q, u, -0x1.fca104p-3f);
  q = __builtin_fmaf(q, u, 0x1.552d74p-2f);
  q = __builtin_fmaf(q, u, -0x1.fffe8cp-2f);
  q = __builtin_fmaf(q, u, 0x1.fffffep-1f);
  const bool neg = l < 0.0f;
  const float t = __builtin_amdgcn_sqrtf(neg ? q : __builtin_fmaf(u, q, l));
  const float c = neg ? h : 1.0f;
  Affinity r;
  r.a = c * t;
  // sig(l) = 1/(1+u) for l >= 0, u/(1+u) for l < 0
  r.da = GRAD ? 0.5f * c * __builtin_amdgcn_rcpf(__builtin_fmaf(u, t, t)) : 0.0f;
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

// A row of E logits in a wave: aligned groups of `lpt` lanes (a power of two)
// hold one token each, a lane 4 consecutive experts of every 256.
struct RowMap {
  int E, lpt, log_lpt;
};
template <int NR>
__device__ __forceinline__ void load_row(const float* row, const RowMap& m, int sub, bool in, float fill,
                                         float (&l)[NR][4]) {
#pragma unroll
  for (int r = 0; r < NR; ++r) {
    const int e = r * 256 + sub * 4;
    if (in && e + 4 <= m.E) {
      const u32x4 v = *reinterpret_cast<const u32x4_a4*>(row + e);
#pragma unroll
      for (int i = 0; i < 4; ++i) l[r][i] = __uint_as_float(v[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) l[r][i] = in && e + i < m.E ? row[e + i] : fill;
    }
  }
}

// sum over the aligned group of lpt lanes
__device__ __forceinline__ float group_sum(float v, int lpt) {
  if (lpt == kWave) return wave_sum(v);
  if (lpt >= 2) v += dpp_f32<0xB1>(v);
  if (lpt >= 4) v += dpp_f32<0x4E>(v);
  if (lpt >= 8) v += dpp_f32<0x141>(v);
  if (lpt >= 16) v += dpp_f32<0x140>(v);
  if (lpt >= 32) v += __shfl_xor(v, 16, kWave);
  return v;
}

// ---------------------------------------------------------------- forward
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
  int* ticket;    // of the sums that follow: reset here
};

// One work-group per tile of 64 tokens, lane i of every wave knowing token i's
// sequence, so that a sequence's tokens in the tile are a ballot.  For each
// sequence s with tokens in tile b it writes the sums of p, the slot counts and
// the token count to row b + s: along the tokens b and s only grow, so no two
// pairs share a row.
template <int NR>
__global__ __launch_bounds__(kThreads) void balance_part_kernel(const LossArgs p) {
  constexpr int U = NR == 4 ? 2 : 4;  // tokens of a lane group with their loads in flight
  __shared__ int s_cnt[NR * 256];
  __shared__ float s_sum[kWaves][NR * 256];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t t0 = (int64_t)blockIdx.x * kTile;
  const int ntok = static_cast<int>(min((int64_t)kTile, p.T - t0));
  const int E = p.m.E, lpt = p.m.lpt, tpw = kWave / lpt, sub = lane & (lpt - 1), which = lane >> p.m.log_lpt;
  if (blockIdx.x == 0 && tid == 0) *p.ticket = 0;
  // a slot of the tile per thread: 64 k <= 1024
  const int my_tok = tid / p.k;
  const int my_e = my_tok < ntok ? p.idx[t0 * p.k + tid] : -1;
  const int seq = sequence_of(t0 + lane, p.T, p.seq, p.n_seq);
  const bool on = lane < ntok && (p.mask == nullptr || p.mask[t0 + lane] != 0);
  for (int e = tid; e < E; e += kThreads) s_cnt[e] = 0;
  __syncthreads();
  for (uint64_t left = __ballot(seq >= 0); left != 0;) {  // one sequence at a time, the same in every wave
    const int s = __builtin_amdgcn_readlane(seq, __builtin_ctzll(left));
    const uint64_t run = __ballot(seq == s);
    const uint64_t counted = run & __ballot(on);
    left &= ~run;
    float sum[NR][4] = {};
    for (int i0 = 0; i0 < kTile; i0 += U * kWaves * tpw) {
      float l[U][NR][4];
      bool in[U];
#pragma unroll
      for (int v = 0; v < U; ++v) {
        const int i = i0 + (v * kWaves + wave) * tpw + which;
        in[v] = i < kTile && ((counted >> (i & 63)) & 1) != 0;
        // a token that does not count may hold anything, also NaN: it is not read
        load_row<NR>(p.logits + (t0 + i) * E, p.m, sub, in[v], 0.0f, l[v]);
      }
#pragma unroll
      for (int v = 0; v < U; ++v) {
        if (!__any(in[v])) continue;
        float total = 0.0f;
#pragma unroll
        for (int r = 0; r < NR; ++r)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int e = r * 256 + sub * 4 + j;
            if (p.offset != nullptr && e < E) l[v][r][j] += p.offset[e];
            l[v][r][j] = in[v] && e < E ? affinity<false>(l[v][r][j]).a : 0.0f;
            total += l[v][r][j];
          }
        total = group_sum(total, lpt);
        const float inv = total > 0.0f ? 1.0f / total : 0.0f;
#pragma unroll
        for (int r = 0; r < NR; ++r)
#pragma unroll
          for (int j = 0; j < 4; ++j) sum[r][j] = __builtin_fmaf(l[v][r][j], inv, sum[r][j]);
      }
    }
    if (my_e >= 0 && my_e < E && ((counted >> my_tok) & 1) != 0) atomicAdd(&s_cnt[my_e], 1);
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
      s_cnt[e] = 0;
    }
    if (tid == 0) p.ptok[row] = __builtin_popcountll(counted);
    __syncthreads();
  }
}

struct SumArgs {
  int64_t T;
  int E, k, n_seq, log_w;
  float alpha;
  const int32_t* seq;
  const float* psum;
  const int32_t* pcnt;
  const int32_t* ptok;
  int32_t* counts;
  float* prob;
  float* dprob;
  float* part;  // [n_seq * column slices]: sum of f P
  int* ticket;
  float* loss;
};

// One work-group per sequence and slice of W = 2^log_w experts: thread (q, c)
// adds every (1024/W)-th part of column c, the parts of a column are then
// joined pairwise.  The last work-group to finish adds the slices' sums of f P,
// in their order, into the loss.
__global__ __launch_bounds__(kThreads) void balance_sum_kernel(const SumArgs p) {
  __shared__ float s_v[kThreads];
  __shared__ int s_c[kThreads];
  __shared__ int s_t[kThreads];
  __shared__ bool s_last;
  const int s = blockIdx.x, tid = threadIdx.x;
  const int W = 1 << p.log_w, lanes = kThreads >> p.log_w;
  const int e = blockIdx.y * W + (tid & (W - 1)), q = tid >> p.log_w;
  const int64_t lo = p.seq == nullptr ? 0 : max((int64_t)p.seq[s], (int64_t)0);
  const int64_t hi = p.seq == nullptr ? p.T : min((int64_t)p.seq[s + 1], p.T);
  const int64_t r0 = lo / kTile + s, r1 = lo < hi ? (hi - 1) / kTile + 1 + s : r0;  // its rows of parts
  float v = 0.0f;
  int c = 0, t = 0;
  for (int64_t r = r0 + tid; r < r1; r += kThreads) t += p.ptok[r];
  if (e < p.E) {
    int64_t r = r0 + q;
    for (; r + 3 * lanes < r1; r += 4 * lanes) {
      float a[4];
      int b[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        a[i] = p.psum[(r + i * lanes) * p.E + e];
        b[i] = p.pcnt[(r + i * lanes) * p.E + e];
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v += a[i];
        c += b[i];
      }
    }
    for (; r < r1; r += lanes) {
      v += p.psum[r * p.E + e];
      c += p.pcnt[r * p.E + e];
    }
  }
  s_v[tid] = v;
  s_c[tid] = c;
  s_t[tid] = t;
  __syncthreads();
  for (int o = kThreads / 2; o >= 1; o >>= 1) {
    if (tid < o) {
      s_t[tid] += s_t[tid + o];
      if (o >= W) {
        s_v[tid] += s_v[tid + o];
        s_c[tid] += s_c[tid + o];
      }
    }
    __syncthreads();
  }
  if (tid < kWave) {
    const float per = s_t[0] > 0 ? 1.0f / static_cast<float>(s_t[0]) : 0.0f;
    float part = 0.0f;
    if (tid < W && e < p.E) {
      const float f = static_cast<float>(s_c[tid]) * (static_cast<float>(p.E) / static_cast<float>(p.k)) * per;
      const float P = s_v[tid] * per;
      const int64_t at = (int64_t)s * p.E + e;
      p.counts[at] = s_c[tid];
      p.prob[at] = P;
      p.dprob[at] = f * per * (p.alpha / static_cast<float>(p.n_seq));
      part = f * P;
    }
    part = wave_sum(part);
    if (tid == 0) {
      const int total = gridDim.x * gridDim.y;
      __hip_atomic_store(&p.part[blockIdx.x * gridDim.y + blockIdx.y], part, __ATOMIC_RELAXED,
                         __HIP_MEMORY_SCOPE_AGENT);
      s_last = __hip_atomic_fetch_add(p.ticket, 1, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) == total - 1;
    }
  }
  __syncthreads();
  if (!s_last || tid >= kWave) return;
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
  float sum = 0.0f;
  for (int i = tid; i < static_cast<int>(gridDim.x * gridDim.y); i += kWave)
    sum += __hip_atomic_load(&p.part[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  sum = wave_sum(sum);
  if (tid == 0) *p.loss = sum * (p.alpha / static_cast<float>(p.n_seq));
}

// ---------------------------------------------------------------- gradient
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
constexpr int kGradWaves = kGradThreads / kWave;

// A lane group takes U tokens, all their loads in flight before the first use.
template <int NR, int U>
__global__ __launch_bounds__(kGradThreads) void balance_grad_kernel(const GradArgs p) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int E = p.m.E, lpt = p.m.lpt, tpw = kWave / lpt, sub = lane & (lpt - 1), which = lane >> p.m.log_lpt;
  const int64_t t0 = ((int64_t)blockIdx.x * kGradWaves + wave) * (U * tpw) + which;
  float l[U][NR][4], x[U][NR][4];
#pragma unroll
  for (int v = 0; v < U; ++v) {
    const int64_t t = t0 + v * tpw;
    load_row<NR>(p.logits + t * E, p.m, sub, t < p.T, 0.0f, l[v]);
    load_row<NR>(p.extra + t * E, p.m, sub, t < p.T && p.extra != nullptr, 0.0f, x[v]);
  }
  const float g = p.grad == nullptr ? 1.0f : *p.grad;
#pragma unroll
  for (int v = 0; v < U; ++v) {
    const int64_t t = t0 + v * tpw;
    int s = sequence_of(t, p.T, p.seq, p.n_seq);
    if (s >= 0 && p.mask != nullptr && p.mask[t] == 0) s = -1;
    float dp[NR][4], da[NR][4];
    load_row<NR>(p.dprob + (int64_t)s * E, p.m, sub, s >= 0, 0.0f, dp);
    float total = 0.0f, dot = 0.0f;
#pragma unroll
    for (int r = 0; r < NR; ++r)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int e = r * 256 + sub * 4 + j;
        if (p.offset != nullptr && e < E) l[v][r][j] += p.offset[e];
        Affinity a = affinity<true>(l[v][r][j]);
        if (e >= E) a.a = 0.0f;
        da[r][j] = a.da;
        total += a.a;
        dot = __builtin_fmaf(dp[r][j], a.a, dot);
      }
    total = group_sum(total, lpt);
    dot = group_sum(dot, lpt);
    const bool some = s >= 0 && total > 0.0f;
    const float inv = some ? 1.0f / total : 0.0f;
    const float mean = dot * inv, scale = g * inv;
    if (t >= p.T) continue;
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      const int e = r * 256 + sub * 4;
      u32x4 o;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        o[j] = __float_as_uint(x[v][r][j] + (some ? scale * (dp[r][j] - mean) * da[r][j] : 0.0f));
      float* at = p.dl + t * E + e;
      if (e + 4 <= E) {
        *reinterpret_cast<u32x4_a4*>(at) = o;
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (e + j < E) at[j] = __uint_as_float(o[j]);
      }
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

// expert columns of a slice: 2^log_w
int slice_log(int E) {
  int lg = 0;
  while (lg < 6 && (1 << lg) < E) ++lg;
  return lg;
}

struct LossWs {
  size_t psum, pcnt, ptok, part, ticket, total;
};
LossWs loss_ws(int64_t T, int E, int n_seq) {
  const size_t rows = static_cast<size_t>((T + kTile - 1) / kTile) + n_seq;
  const size_t slices = (E + (1 << slice_log(E)) - 1) >> slice_log(E);
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  LossWs w;
  w.psum = 0;
  w.pcnt = up(rows * E * sizeof(float));
  w.ptok = w.pcnt + up(rows * E * sizeof(int32_t));
  w.part = w.ptok + up(rows * sizeof(int32_t));
  w.ticket = w.part + up(n_seq * slices * sizeof(float));
  w.total = w.ticket + 256;
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
  int* ticket = reinterpret_cast<int*>(base + w.ticket);
  // at least one work-group: it resets the ticket
  const int64_t tiles = T > 0 ? (T + kTile - 1) / kTile : 1;
  const LossArgs a{T, row_map(E), k, n_seq, logits, offset, idx, seq, mask, psum, pcnt, ptok, ticket};
  const dim3 grid(static_cast<unsigned>(tiles)), block(kThreads);
  if (E <= 256) hipLaunchKernelGGL(balance_part_kernel<1>, grid, block, 0, s, a);
  else if (E <= 512) hipLaunchKernelGGL(balance_part_kernel<2>, grid, block, 0, s, a);
  else hipLaunchKernelGGL(balance_part_kernel<4>, grid, block, 0, s, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int lg = slice_log(E);
  const SumArgs b{T,    E,    k,      n_seq, lg,    alpha,  seq, psum, pcnt,
                  ptok, counts, prob, dprob, reinterpret_cast<float*>(base + w.part), ticket, loss};
  hipLaunchKernelGGL(balance_sum_kernel, dim3(n_seq, (E + (1 << lg) - 1) >> lg), block, 0, s, b);
  return hipGetLastError();
}

hipError_t launch_balance_loss_bwd(int64_t T, int E, const float* logits, const float* offset, const int32_t* seq,
                                   int n_seq, const uint8_t* mask, const float* dprob, const float* grad,
                                   const float* extra, float* dl, hipStream_t s) {
  const GradArgs a{T, row_map(E), n_seq, logits, offset, seq, mask, dprob, grad, extra, dl};
  auto go = [&](auto kernel, int u) {
    const int64_t per = (int64_t)kGradWaves * u * (kWave / a.m.lpt);
    hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>((T + per - 1) / per)), dim3(kGradThreads), 0, s, a);
  };
  if (E <= 256) go(balance_grad_kernel<1, 2>, 2);
  else if (E <= 512) go(balance_grad_kernel<2, 1>, 1);
  else go(balance_grad_kernel<4, 1>, 1);
  return hipGetLastError();
}

}  // namespace moe

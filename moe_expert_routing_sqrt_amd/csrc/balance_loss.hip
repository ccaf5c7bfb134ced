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
// no cancellation, and no underflow before e^(l/2) itself, at a logit of -174.
// Rounding the exponent once would cost h |l| 2^-24 of itself (a probability's
// rms error 1.5e-6 at logits near -165, 1.8e-7 near -12); its low part is carried,
// and an affinity holds 7 2^-24 at any logit (rms 7e-8 everywhere).  Two
// transcendental instructions and 22 others an element.
// A row whose affinities all vanish has no probabilities: it adds 0.  A counted
// row with a NaN has NaN for each, in the sums and in its gradient.
//
// At T = 16384, E = 256, k = 8 (17 MB, 2.9 us of HBM) the forward takes 12.2 us:
// parts whose work-groups load, compute (2.5 us), join and store one after the
// other, two thirds of it, and sums, a chain of dependent loads; the gradient
// onto others' (50 MB, 8.5 us) takes 10.5 us.  At most 64 tokens take one launch
// (T = 16, E = 64: 4.1 us against 7.3 in two).
#include <type_traits>

#include "launch.h"
#include "stream8.h"

namespace moe {
namespace {

constexpr int kTile = 64;  // tokens of a forward work-group: one per lane
constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / kWave;
constexpr int kSumGroups = 32;  // work-groups of a slice of the sums, at most

struct Affinity {
  float a;   // sqrt(softplus(l))
  float da;  // its derivative sig(l) / (2 a)
};

template <bool GRAD>
__device__ __forceinline__ Affinity affinity(float l) {
  // h = 2^e with e = -|l| log2(e)/2, the part of e past 24 bits as a factor
  // 1 + ln2 lo.  The bound on |l| keeps lo finite; h is 0 long before it.
  const float x = __builtin_fminf(__builtin_fabsf(l), 512.0f);
  const float e = x * -0x1.715476p-1f;
  const float lo = __builtin_fmaf(x, -0x1.4ae0c0p-27f, __builtin_fmaf(x, -0x1.715476p-1f, -e));
  const float h2 = __builtin_amdgcn_exp2f(e);
  const float h = __builtin_fmaf(h2, lo * 0x1.62e430p-1f, h2);
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

// Whether a row's affinities, whose sum this is, make probabilities: not where
// all vanish.  A sum that is no number does, and makes the row's NaN.
__device__ __forceinline__ bool has_share(float total) { return total != 0.0f; }

// The sequence of a lane's token t among the offsets (nullptr: one sequence of
// all T tokens); -1 for a token outside them.  Tokens must not fall from lane to
// lane, and every lane of the wave has to call.
// First the sequence of the wave's first token, by a search in scalar loads
// (few sequences: nothing of it waits behind the rows' loads) or, from 9 to 62
// sequences, a ballot over offsets loaded by the lanes when this is made; only
// where the wave's tokens leave that sequence does every lane search for its
// own.  At T = 16384 a search per lane cost 1.7 us of the gradient's 12.
struct SequenceSearch {
  int64_t T;
  const int32_t* off;
  int n, v;
  __device__ __forceinline__ SequenceSearch(int64_t T_, const int32_t* off_, int n_) : T(T_), off(off_), n(n_), v(0) {
    if (off != nullptr && n > kScalar && n <= kLanes) v = off[min(static_cast<int>(threadIdx.x & 63), n)];
  }
  __device__ __forceinline__ int operator()(int64_t t) const {
    if (off == nullptr) return t < T ? 0 : -1;
    const int ti = static_cast<int>(min(t, T));  // T fits an int
    const int t_first = __builtin_amdgcn_readfirstlane(ti);
    const int t_last = __builtin_amdgcn_readlane(ti, 63);
    int s0, end;  // the first token's sequence, and where it ends
    if (n > kScalar && n <= kLanes) {
      s0 = __builtin_popcountll(__ballot((threadIdx.x & 63) <= n && v <= t_first)) - 1;
      end = s0 >= 0 && s0 < n ? __builtin_amdgcn_readlane(v, s0 + 1) : INT32_MIN;
    } else {
      s0 = last_at_most(t_first);
      end = s0 >= 0 && s0 < n ? off[s0 + 1] : INT32_MIN;
    }
    if (t_last < end) return t < T ? s0 : -1;
    const int s = last_at_most(ti);
    return t < T && s < n ? s : -1;
  }

 private:
  static constexpr int kScalar = 8, kLanes = 62;
  // the last of the n + 1 offsets that is <= t, -1 if none is
  __device__ __forceinline__ int last_at_most(int t) const {
    int lo = 0, hi = n + 1;  // offsets before lo are <= t, from hi on > t
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (off[mid] <= t) lo = mid + 1; else hi = mid;
    }
    return lo - 1;
  }
};

// A row of E values in a wave: aligned groups of `lpt` lanes (a power of two)
// hold one token each, a lane 4 consecutive columns of every 256.  FULL: E is
// 4 lpt NR, every lane's columns exist.  Otherwise the last lane's columns are
// moved back to end with the row and lanes past it read those too, so that
// every load is a whole one and no branch stands between a load and the next
// (E < 4: single elements, the last one repeated); `lo` counts the columns at
// a lane's start that are not its own (4: none are).
template <int NR, bool FULL>
struct RowMap {
  int E, lpt, sub, which;
  int col[NR], lo[NR];
  __device__ __forceinline__ RowMap(int E_, int log_lpt) : E(E_), lpt(1 << log_lpt) {
    const int lane = threadIdx.x & 63;
    sub = lane & (lpt - 1);
    which = lane >> log_lpt;
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      const int c = r * 256 + sub * 4;
      col[r] = FULL ? c : max(0, min(c, E - 4));
      lo[r] = FULL ? 0 : min(4, c - col[r]);
    }
  }
  __device__ __forceinline__ bool owns(int r, int j) const {
    return FULL || (j >= lo[r] && col[r] + j < E);
  }
  __device__ __forceinline__ void load(const float* row, float (&l)[NR][4]) const {
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      if (FULL || E >= 4) {
        const u32x4 v = *reinterpret_cast<const u32x4_a4*>(row + col[r]);
#pragma unroll
        for (int i = 0; i < 4; ++i) l[r][i] = __uint_as_float(v[i]);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) l[r][i] = row[min(i, E - 1)];
      }
    }
  }
  // the columns a lane owns
  __device__ __forceinline__ void store(float* row, const float (&v)[NR][4]) const {
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      if (FULL || (lo[r] == 0 && E >= 4)) {
        *reinterpret_cast<u32x4_a4*>(row + col[r]) = u32x4{__float_as_uint(v[r][0]), __float_as_uint(v[r][1]),
                                                           __float_as_uint(v[r][2]), __float_as_uint(v[r][3])};
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (owns(r, i)) row[col[r] + i] = v[r][i];
      }
    }
  }
};

// ---------------------------------------------------------------- forward
struct LossArgs {
  int64_t T;
  int E, log_lpt, k, n_seq;
  const float* logits;
  const float* offset;
  const int32_t* idx;
  const int32_t* seq;
  const uint8_t* mask;
  float* psum;    // [tiles + n_seq][E]
  int32_t* pcnt;  // [tiles + n_seq][E]
  int32_t* ptok;  // [tiles + n_seq]
  unsigned long long* total;  // of the sums that follow, and their `groups` slots for
  float* left;                // shares: reset here
  int groups;
};

__device__ __forceinline__ void reset_shares(const LossArgs& p) {
  if (threadIdx.x == 0) *p.total = 0;
  for (int i = threadIdx.x; i < p.groups; i += kThreads) p.left[i] = 0.0f;
}

// One work-group per tile of 64 tokens: their probabilities are formed once, in
// registers.  Lane i of every wave knows token i's sequence, so that a
// sequence's tokens in the tile are a ballot.  For each sequence s with tokens
// in tile b the sums of p, the slot counts and the token count go to row b + s:
// along the tokens b and s only grow, so no two pairs share a row.
template <int NR, bool FULL>
__global__ __launch_bounds__(kThreads) void balance_part_kernel(const LossArgs p) {
  constexpr int U = kTile / kWaves;  // tokens of a lane group (at one token a wave)
  __shared__ int s_cnt[NR * 256];
  __shared__ __align__(16) float s_sum[kWaves][NR * 256];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t t0 = (int64_t)blockIdx.x * kTile;
  const int ntok = static_cast<int>(min((int64_t)kTile, p.T - t0));
  const int E = p.E;
  const SequenceSearch sequence_of(p.T, p.seq, p.n_seq);
  const RowMap<NR, FULL> m(E, p.log_lpt);
  const int tpw = kWave / m.lpt;
  // every load of the tile before the first wait; a token that does not count
  // may hold anything, also NaN: its row is read but never selected
  float pr[U][NR][4], off[NR][4] = {};
  if (ntok > 0) {
#pragma unroll
    for (int v = 0; v < U; ++v) {
      const int i = (v * kWaves + wave) * tpw + m.which;
      m.load(p.logits + (t0 + min(i, ntok - 1)) * E, pr[v]);
    }
    if (p.offset != nullptr) m.load(p.offset, off);
  }
  const int my_tok = tid / p.k;  // a slot of the tile per thread: 64 k <= 1024
  const int my_e = my_tok < ntok ? p.idx[t0 * p.k + tid] : -1;
  const bool on = lane < ntok && (p.mask == nullptr || p.mask[t0 + lane] != 0);
  const int seq = sequence_of(t0 + lane);
  if (blockIdx.x == 0) reset_shares(p);
  for (int e = tid; e < E; e += kThreads) s_cnt[e] = 0;
#pragma unroll
  for (int v = 0; v < U; ++v) {
    if ((v * kWaves + wave) * tpw >= ntok) break;  // uniform over the wave
    float total = 0.0f;
#pragma unroll
    for (int r = 0; r < NR; ++r)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float a = affinity<false>(pr[v][r][j] + off[r][j]).a;
        pr[v][r][j] = m.owns(r, j) ? a : 0.0f;
        total += pr[v][r][j];
      }
    total = group_sum(total, m.lpt);
    const float inv = has_share(total) ? 1.0f / total : 0.0f;
#pragma unroll
    for (int r = 0; r < NR; ++r)
#pragma unroll
      for (int j = 0; j < 4; ++j) pr[v][r][j] *= inv;
  }
  __syncthreads();
  for (uint64_t left = __ballot(seq >= 0); left != 0;) {  // one sequence at a time, the same in every wave
    const int s = __builtin_amdgcn_readlane(seq, __builtin_ctzll(left));
    const uint64_t run = __ballot(seq == s);
    const uint64_t counted = run & __ballot(on);
    left &= ~run;
    float sum[NR][4] = {};
#pragma unroll
    for (int v = 0; v < U; ++v) {
      const int i = (v * kWaves + wave) * tpw + m.which;
      const bool in = i < kTile && ((counted >> (i & 63)) & 1) != 0;
#pragma unroll
      for (int r = 0; r < NR; ++r)
#pragma unroll
        for (int j = 0; j < 4; ++j) sum[r][j] += in ? pr[v][r][j] : 0.0f;
    }
    if (my_e >= 0 && my_e < E && ((counted >> my_tok) & 1) != 0) atomicAdd(&s_cnt[my_e], 1);
    // the lane groups of a wave, then the waves in order
#pragma unroll
    for (int r = 0; r < NR; ++r)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        for (int o = m.lpt; o < kWave; o <<= 1) sum[r][j] += __shfl_xor(sum[r][j], o, kWave);
    if (m.which == 0) m.store(s_sum[wave], sum);
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
    if (left != 0) __syncthreads();
  }
}

// The runs of a tile: a run is a sequence's stretch of tokens.  Lane i holds token
// i's sequence (-1: none) and whether it counts.
struct Runs {
  uint64_t starts, ends, counted;
  int run;  // of this lane's token
  __device__ __forceinline__ Runs(int seq, bool on) {
    const int lane = threadIdx.x & 63, before = __shfl_up(seq, 1, kWave);
    starts = __ballot(seq >= 0 && (lane == 0 || before != seq));
    ends = __ballot(seq < 0 && lane != 0 && before >= 0);  // a run followed by no sequence
    counted = __ballot(on && seq >= 0);
    run = __builtin_popcountll(starts & ((2ull << lane) - 1)) - 1;
  }
  __device__ __forceinline__ int count() const { return __builtin_popcountll(starts); }
  __device__ __forceinline__ bool starts_here() const { return ((starts >> (threadIdx.x & 63)) & 1) != 0; }
  // of the run that starts at this lane's token: its end, and its tokens that count
  __device__ __forceinline__ int end(int ntok) const {
    const uint64_t after = (starts | ends) & ~((2ull << (threadIdx.x & 63)) - 1);
    return after != 0 ? __builtin_ctzll(after) : ntok;
  }
  __device__ __forceinline__ int tokens(int end) const {
    const uint64_t mine = (end >= 64 ? ~0ull : (1ull << end) - 1) & ~((1ull << (threadIdx.x & 63)) - 1);
    return __builtin_popcountll(counted & mine);
  }
};

// Loads a tile's rows for tile_probabilities, every load before the first wait;
// a token that does not count may hold anything, also NaN: its row is read but
// never selected.
template <bool FULL>
__device__ __forceinline__ void load_tile(const RowMap<1, FULL>& m, const float* logits, int ntok,
                                          float (&pr)[kTile / kWaves][1][4]) {
  const int wave = threadIdx.x >> 6, tpw = kWave / m.lpt;
#pragma unroll
  for (int v = 0; v < kTile / kWaves; ++v) {
    const int i = (v * kWaves + wave) * tpw + m.which;
    m.load(logits + static_cast<int64_t>(min(i, ntok - 1)) * m.E, pr[v]);
  }
}

// The tile's probabilities into LDS, zeros for tokens that do not count.
template <bool FULL>
__device__ __forceinline__ void tile_probabilities(const RowMap<1, FULL>& m, int ntok, uint64_t counted,
                                                   const float (&off)[1][4], float (&pr)[kTile / kWaves][1][4],
                                                   float* s_p) {
  const int wave = threadIdx.x >> 6, tpw = kWave / m.lpt;
#pragma unroll
  for (int v = 0; v < kTile / kWaves; ++v) {
    if ((v * kWaves + wave) * tpw >= ntok) break;  // uniform over the wave
    const int i = (v * kWaves + wave) * tpw + m.which;
    float total = 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float a = affinity<false>(pr[v][0][j] + off[0][j]).a;
      pr[v][0][j] = m.owns(0, j) ? a : 0.0f;
      total += pr[v][0][j];
    }
    total = group_sum(total, m.lpt);
    const bool some = i < ntok && ((counted >> (i & 63)) & 1) != 0 && has_share(total);
    const float inv = some ? 1.0f / total : 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j) pr[v][0][j] = some ? pr[v][0][j] * inv : 0.0f;
    if (i < ntok) m.store(s_p + i * m.E, pr[v]);
  }
}

// sum of column e over tokens [begin, end), in order
__device__ __forceinline__ float run_sum(const float* s_p, int E, int e, int begin, int end) {
  float v = 0.0f;
  for (int i = begin; i < end; i += 8) {  // 8 reads in flight
    float t[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) t[j] = s_p[min(i + j, end - 1) * E + e];
#pragma unroll
    for (int j = 0; j < 8; ++j) v += i + j < end ? t[j] : 0.0f;
  }
  return v;
}

// The parts for tiles of many short sequences (E <= 256).  The probabilities go to
// LDS once, and so do the slot counts of each run; then every thread takes a
// (run, expert) pair: one pass whatever the number of runs.
template <bool FULL>
__global__ __launch_bounds__(kThreads) void balance_part_short_kernel(const LossArgs p) {
  __shared__ __align__(16) float s_p[kTile * 256];
  __shared__ uint32_t s_cnt[kTile * 256 / 2];  // counts of 16 bits: 64 k <= 1024
  __shared__ int s_begin[kTile], s_end[kTile], s_seq[kTile], s_tok[kTile];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t t0 = (int64_t)blockIdx.x * kTile;
  const int ntok = static_cast<int>(min((int64_t)kTile, p.T - t0));
  const int E = p.E;
  const SequenceSearch sequence_of(p.T, p.seq, p.n_seq);
  const RowMap<1, FULL> m(E, p.log_lpt);
  float pr[kTile / kWaves][1][4], off[1][4] = {};
  if (ntok > 0) {
    load_tile<FULL>(m, p.logits + t0 * E, ntok, pr);
    if (p.offset != nullptr) m.load(p.offset, off);
  }
  const int my_tok = tid / p.k;  // a slot of the tile per thread: 64 k <= 1024
  const int my_e = my_tok < ntok ? p.idx[t0 * p.k + tid] : -1;
  const bool on = lane < ntok && (p.mask == nullptr || p.mask[t0 + lane] != 0);
  const int seq = sequence_of(t0 + lane);
  if (blockIdx.x == 0) reset_shares(p);
  const Runs runs(seq, on);
  if (wave == 0 && runs.starts_here()) {
    const int end = runs.end(ntok);
    s_begin[runs.run] = lane;
    s_end[runs.run] = end;
    s_seq[runs.run] = seq;
    s_tok[runs.run] = runs.tokens(end);
  }
  const int pairs = runs.count() * E;
  for (int i = tid; i < (pairs + 1) / 2; i += kThreads) s_cnt[i] = 0;
  __syncthreads();
  const int my_run = __shfl(runs.run, my_tok & 63, kWave);
  if (my_e >= 0 && my_e < E && ((runs.counted >> (my_tok & 63)) & 1) != 0) {
    const int at = my_run * E + my_e;
    atomicAdd(&s_cnt[at / 2], 1u << (16 * (at & 1)));
  }
  tile_probabilities<FULL>(m, ntok, runs.counted, off, pr, s_p);
  __syncthreads();
  for (int id = tid; id < pairs; id += kThreads) {
    const int r = id / E, e = id - r * E;
    const int64_t row = (int64_t)blockIdx.x + s_seq[r];
    p.psum[row * E + e] = run_sum(s_p, E, e, s_begin[r], s_end[r]);
    p.pcnt[row * E + e] = static_cast<int32_t>((s_cnt[id / 2] >> (16 * (id & 1))) & 0xFFFFu);
    if (e == 0) p.ptok[row] = s_tok[r];
  }
}

// At most a tile of tokens: everything in one work-group and one launch, without
// parts; the sums and counts of all sequences stay in LDS.
constexpr int kSmallTable = 8192, kSmallSeqs = 1024;  // sequences times experts; sequences

struct SmallArgs {
  LossArgs in;  // its parts are not used
  float alpha;
  int32_t* counts;
  float* prob;
  float* dprob;
  float* loss;
};

template <bool FULL>
__global__ __launch_bounds__(kThreads) void balance_small_kernel(const SmallArgs a) {
  __shared__ __align__(16) float s_p[kTile * 256];
  __shared__ float s_sum[kSmallTable];
  __shared__ int s_cnt[kSmallTable];
  __shared__ int s_tok[kSmallSeqs];
  __shared__ int s_begin[kTile], s_end[kTile], s_seq[kTile];
  __shared__ float s_red[kWaves];
  const LossArgs& p = a.in;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int E = p.E, ntok = static_cast<int>(p.T), table = p.n_seq * E;
  const SequenceSearch sequence_of(p.T, p.seq, p.n_seq);
  const RowMap<1, FULL> m(E, p.log_lpt);
  float pr[kTile / kWaves][1][4], off[1][4] = {};
  if (ntok > 0) {
    load_tile<FULL>(m, p.logits, ntok, pr);
    if (p.offset != nullptr) m.load(p.offset, off);
  }
  const int my_tok = tid / p.k;  // a slot per thread: 64 k <= 1024
  const int my_e = my_tok < ntok ? p.idx[tid] : -1;
  const bool on = lane < ntok && (p.mask == nullptr || p.mask[lane] != 0);
  const int seq = sequence_of(lane);
  const Runs runs(seq, on);
  for (int i = tid; i < table; i += kThreads) {
    s_sum[i] = 0.0f;
    s_cnt[i] = 0;
  }
  for (int i = tid; i < p.n_seq; i += kThreads) s_tok[i] = 0;
  __syncthreads();
  if (wave == 0 && runs.starts_here()) {
    const int end = runs.end(ntok);
    s_begin[runs.run] = lane;
    s_end[runs.run] = end;
    s_seq[runs.run] = seq;
    s_tok[seq] = runs.tokens(end);
  }
  const int my_seq = __shfl(seq, my_tok & 63, kWave);
  if (my_e >= 0 && my_e < E && ((runs.counted >> (my_tok & 63)) & 1) != 0) atomicAdd(&s_cnt[my_seq * E + my_e], 1);
  tile_probabilities<FULL>(m, ntok, runs.counted, off, pr, s_p);
  __syncthreads();
  for (int id = tid; id < runs.count() * E; id += kThreads) {
    const int r = id / E, e = id - r * E;
    s_sum[s_seq[r] * E + e] = run_sum(s_p, E, e, s_begin[r], s_end[r]);
  }
  __syncthreads();
  float loss = 0.0f;
  for (int id = tid; id < table; id += kThreads) {
    const int t = s_tok[id / E];
    const float per = t > 0 ? 1.0f / static_cast<float>(t) : 0.0f;
    const float f = static_cast<float>(s_cnt[id]) * (static_cast<float>(E) / static_cast<float>(p.k)) * per;
    const float P = s_sum[id] * per;
    a.counts[id] = s_cnt[id];
    a.prob[id] = P;
    a.dprob[id] = f * per * (a.alpha / static_cast<float>(p.n_seq));
    loss = __builtin_fmaf(f, P, loss);
  }
  loss = wave_sum(loss);
  if (lane == 0) s_red[wave] = loss;
  __syncthreads();
  if (tid < kWave) {
    loss = row16_sum(s_red[lane & 15]);
    if (tid == 0) *a.loss = loss * (a.alpha / static_cast<float>(p.n_seq));
  }
}

struct SumArgs {
  int64_t T;
  int E, k, n_seq, log_w, team;
  float alpha;
  const int32_t* seq;
  const float* psum;
  const int32_t* pcnt;
  const int32_t* ptok;
  int32_t* counts;
  float* prob;
  float* dprob;
  float one;  // 1 in units of the total
  unsigned long long* total;
  float* left;  // [gridDim.x * gridDim.y]
  float* loss;
};

// The work-groups' shares of loss / alpha meet in one 64-bit integer, so their
// sum does not depend on their order and the last one to come has it without
// another round trip: finished work-groups (11 bits, at most 32 x 32), those that
// left their share in memory instead (11 bits), and the sum of the others in
// units of 1 / one = 2^(ceil(log2 E) - 41).  The shares add up to E at most, and
// one of at least 2^23 units is a whole number of them: nothing is rounded.
// Smaller ones (a loss far below 1) and those that are no number are left in
// fp32, and the last work-group adds them in the order of the work-groups; that
// takes a release at each and an acquire (16384 x 256, four sequences: 1.1 us).
constexpr int kShareBits = 42, kLeftShift = 42, kDoneShift = 53;
constexpr float kWhole = 0x1p23f, kMostUnits = 0x1.01p41f;

// Work-group (x, y): slice y of W = 2^log_w experts.  Its waves form teams of
// `team` waves (enough for about 16 parts a thread of a sequence of average
// length), each with a sequence of its own: thread (q, c) of a team adds every
// (64 team / W)-th part of column c, and the parts of a column are joined in
// order of q.
__global__ __launch_bounds__(kThreads) void balance_sum_kernel(const SumArgs p) {
  __shared__ float s_v[kThreads];
  __shared__ int s_c[kThreads];
  __shared__ int s_t[kWaves];
  __shared__ float s_loss[kWaves];
  const int waves = blockDim.x >> 6, wave = threadIdx.x >> 6, team = wave / p.team, teams = waves / p.team;
  const int first = team * p.team * kWave;            // the team's first thread
  const int tid = static_cast<int>(threadIdx.x) - first;
  const int W = 1 << p.log_w, lanes = (p.team * kWave) >> p.log_w;
  const int e = blockIdx.y * W + (tid & (W - 1)), q = tid >> p.log_w;
  // the parts r, r + lanes, ... of column e, N of them, all in flight at once
  auto add_parts = [&](auto n, int64_t r, int64_t r1, int e, float& v, int& c) __attribute__((always_inline)) {
    constexpr int N = decltype(n)::value;
    if (r >= r1) return;
    float a[N];
    int b[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int64_t at = min(r + i * lanes, r1 - 1) * p.E + e;
      a[i] = p.psum[at];
      b[i] = p.pcnt[at];
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const bool in = r + i * lanes < r1;
      v += in ? a[i] : 0.0f;
      c += in ? b[i] : 0;
    }
  };
  float loss = 0.0f;  // of thread c < W of a team
  for (int s0 = blockIdx.x * teams; s0 < p.n_seq; s0 += gridDim.x * teams) {
    const int s = s0 + team;
    int64_t r0 = 0, r1 = 0;  // the sequence's rows of parts
    if (s < p.n_seq) {
      const int64_t lo = p.seq == nullptr ? 0 : max((int64_t)p.seq[s], (int64_t)0);
      const int64_t hi = p.seq == nullptr ? p.T : min((int64_t)p.seq[s + 1], p.T);
      r0 = lo / kTile + s;
      r1 = lo < hi ? (hi - 1) / kTile + 1 + s : r0;
    }
    float v = 0.0f;
    int c = 0, t = 0;
    for (int64_t r = r0 + tid; r < r1; r += p.team * kWave) t += p.ptok[r];
    if (e < p.E) {
      if (r1 - r0 <= 4 * lanes) add_parts(std::integral_constant<int, 4>{}, r0 + q, r1, e, v, c);
      else
        for (int64_t r = r0 + q; r < r1; r += 16 * lanes) add_parts(std::integral_constant<int, 16>{}, r, r1, e, v, c);
    }
    for (int o = 32; o >= 1; o >>= 1) t += __shfl_xor(t, o, kWave);
    s_v[threadIdx.x] = v;
    s_c[threadIdx.x] = c;
    if ((tid & 63) == 0) s_t[wave] = t;
    __syncthreads();
    if (tid < W && s < p.n_seq && e < p.E) {
      for (int i = 1; i < lanes; ++i) {
        v += s_v[first + i * W + tid];
        c += s_c[first + i * W + tid];
      }
      t = s_t[wave];
      for (int i = 1; i < p.team; ++i) t += s_t[wave + i];
      const float per = t > 0 ? 1.0f / static_cast<float>(t) : 0.0f;
      const float f = static_cast<float>(c) * (static_cast<float>(p.E) / static_cast<float>(p.k)) * per;
      const float P = v * per;
      const int64_t at = (int64_t)s * p.E + e;
      p.counts[at] = c;
      p.prob[at] = P;
      p.dprob[at] = f * per * (p.alpha / static_cast<float>(p.n_seq));
      loss = __builtin_fmaf(f, P, loss);
    }
    if (s0 + static_cast<int>(gridDim.x) * teams < p.n_seq) __syncthreads();
  }
  loss = wave_sum(loss);  // 0 in a team's other waves
  if ((tid & 63) == 0) s_loss[wave] = loss;
  __syncthreads();
  if (wave != 0) return;
  const int lane = threadIdx.x & 63, groups = gridDim.x * gridDim.y;
  loss = row16_sum((lane & 15) < waves ? s_loss[lane & 15] : 0.0f) / static_cast<float>(p.n_seq);
  if (groups > 1) {
    const float units = loss * p.one;  // exact: a power of two
    const bool whole = units == 0.0f || (units >= kWhole && units <= kMostUnits);
    const unsigned long long mine =
        (1ull << kDoneShift) + (whole ? static_cast<unsigned long long>(units) : 1ull << kLeftShift);
    unsigned long long all = 0;
    if (lane == 0) {
      if (whole) {
        all = __hip_atomic_fetch_add(p.total, mine, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) + mine;
      } else {
        __hip_atomic_store(p.left + blockIdx.y * gridDim.x + blockIdx.x, loss, __ATOMIC_RELAXED,
                           __HIP_MEMORY_SCOPE_AGENT);
        all = __hip_atomic_fetch_add(p.total, mine, __ATOMIC_RELEASE, __HIP_MEMORY_SCOPE_AGENT) + mine;
      }
    }
    all = (static_cast<unsigned long long>(__builtin_amdgcn_readfirstlane(static_cast<uint32_t>(all >> 32))) << 32) |
          static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<uint32_t>(all)));
    if (static_cast<int>(all >> kDoneShift) != groups) return;
    loss = static_cast<float>(static_cast<double>(all & ((1ull << kShareBits) - 1)) / static_cast<double>(p.one));
    if (((all >> kLeftShift) & ((1u << (kDoneShift - kLeftShift)) - 1)) != 0) {
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
      float v = 0.0f;
      for (int i = lane; i < groups; i += 4 * kWave) {  // 4 loads in flight
        float t[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          t[j] = __hip_atomic_load(p.left + min(i + j * kWave, groups - 1), __ATOMIC_RELAXED,
                                   __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
        for (int j = 0; j < 4; ++j) v += i + j * kWave < groups ? t[j] : 0.0f;
      }
      loss += wave_sum(v);
    }
  }
  if (lane == 0) *p.loss = loss * p.alpha;
}

// ---------------------------------------------------------------- gradient
struct GradArgs {
  int64_t T;
  int E, log_lpt, n_seq;
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

// One token a lane group; the loads of its logits and of the gradient to add
// are issued first, under the search for its sequence.
template <int NR, bool FULL, bool ADD>
__global__ __launch_bounds__(kGradThreads) void balance_grad_kernel(const GradArgs p) {
  const RowMap<NR, FULL> m(p.E, p.log_lpt);
  const int64_t t = ((int64_t)blockIdx.x * kGradWaves + (threadIdx.x >> 6)) * (kWave / m.lpt) + m.which;
  const int64_t at = min(t, p.T - 1) * p.E;
  const SequenceSearch sequence_of(p.T, p.seq, p.n_seq);
  float l[NR][4], x[NR][4] = {}, off[NR][4] = {}, dp[NR][4];
  m.load(p.logits + at, l);
  if constexpr (ADD) m.load(p.extra + at, x);
  if (p.offset != nullptr) m.load(p.offset, off);
  const float g = p.grad == nullptr ? 1.0f : *p.grad;
  const uint8_t on = p.mask == nullptr ? 1 : p.mask[min(t, p.T - 1)];
  int s = sequence_of(t);
  if (on == 0) s = -1;
  m.load(p.dprob + (int64_t)max(s, 0) * p.E, dp);
  float total = 0.0f, dot = 0.0f;
#pragma unroll
  for (int r = 0; r < NR; ++r)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const Affinity a = affinity<true>(l[r][j] + off[r][j]);
      const float own = m.owns(r, j) ? a.a : 0.0f;
      l[r][j] = a.da;
      total += own;
      dot = __builtin_fmaf(dp[r][j], own, dot);
    }
  total = group_sum(total, m.lpt);
  dot = group_sum(dot, m.lpt);
  const bool some = s >= 0 && has_share(total);
  const float inv = some ? 1.0f / total : 0.0f;
  const float mean = dot * inv, scale = g * inv;
#pragma unroll
  for (int r = 0; r < NR; ++r)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float v = scale * (dp[r][j] - mean) * l[r][j];
      x[r][j] += some ? v : 0.0f;
    }
  if (t < p.T) m.store(p.dl + at, x);
}

// lanes of a token: a power of two that covers E in fours
int lanes_log(int E) {
  int lg = 0;
  while (lg < 6 && (4 << lg) < E) ++lg;
  return lg;
}
bool full_rows(int E) {
  const int lane4 = 4 << lanes_log(E);
  return E == lane4 || E == 512 || E == 1024;
}

// expert columns of a slice: 2^log_w, at most kSlice
constexpr int kSlice = 32;
int slice_log(int E) {
  int lg = 0;
  while ((1 << lg) < kSlice && (1 << lg) < E) ++lg;
  return lg;
}

struct LossWs {
  size_t psum, pcnt, ptok, sum, left, total;
};
LossWs loss_ws(int64_t T, int E, int n_seq) {
  const size_t rows = static_cast<size_t>((T + kTile - 1) / kTile) + n_seq;
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  LossWs w;
  w.psum = 0;
  w.pcnt = up(rows * E * sizeof(float));
  w.ptok = w.pcnt + up(rows * E * sizeof(int32_t));
  w.sum = w.ptok + up(rows * sizeof(int32_t));
  w.left = w.sum + 256;
  w.total = w.left + up(kSumGroups * (kMaxExperts / kSlice) * sizeof(float));
  return w;
}

}  // namespace

// One work-group for at most a tile, where its tables fit in LDS: T = 1, E = 256
// 4.1 us against 7.5 in two launches, 16 x 64 4.1 against 7.3, 64 x 256 8.3 against
// 10.2; a second tile on the same CU loses (128 x 16 7.8 against 7.6, 256 x 16 12.7
// against 7.9).
static bool small_loss(int64_t T, int E, int n_seq) {
  return E <= 256 && T <= kTile && n_seq <= kSmallSeqs && static_cast<int64_t>(n_seq) * E <= kSmallTable;
}

size_t balance_loss_workspace_bytes(int64_t T, int E, int n_seq) {
  return small_loss(T, E, n_seq) ? 0 : loss_ws(T, E, n_seq).total;
}

hipError_t launch_balance_loss(int64_t T, int E, int k, const float* logits, const float* offset, const int32_t* idx,
                               const int32_t* seq, int n_seq, const uint8_t* mask, float alpha, int32_t* counts,
                               float* prob, float* dprob, float* loss, void* ws, hipStream_t s) {
  if (small_loss(T, E, n_seq)) {
    const SmallArgs a{{T, E, lanes_log(E), k, n_seq, logits, offset, idx, seq, mask, nullptr, nullptr, nullptr,
                       nullptr, nullptr, 0},
                      alpha, counts, prob, dprob, loss};
    if (full_rows(E)) hipLaunchKernelGGL(balance_small_kernel<true>, dim3(1), dim3(kThreads), 0, s, a);
    else hipLaunchKernelGGL(balance_small_kernel<false>, dim3(1), dim3(kThreads), 0, s, a);
    return hipGetLastError();
  }
  const LossWs w = loss_ws(T, E, n_seq);
  char* base = static_cast<char*>(ws);
  float* psum = reinterpret_cast<float*>(base + w.psum);
  int32_t* pcnt = reinterpret_cast<int32_t*>(base + w.pcnt);
  int32_t* ptok = reinterpret_cast<int32_t*>(base + w.ptok);
  auto* total = reinterpret_cast<unsigned long long*>(base + w.sum);
  float* left = reinterpret_cast<float*>(base + w.left);
  // at least one work-group: it resets what the shares of the loss meet in
  const int64_t tiles = T > 0 ? (T + kTile - 1) / kTile : 1;
  const int lg = slice_log(E);
  int team = 1;
  while (team < kWaves && ((team * kWave) >> lg) * 16 < tiles / n_seq) team *= 2;
  // one team a work-group while all sequences then run at once (a small
  // work-group starts sooner: 12.0 us against 12.6 at T = 16384, E = 256, four
  // sequences), else 16 waves of them
  const int teams = n_seq <= kSumGroups ? 1 : kWaves / team;
  const int groups = (n_seq + teams - 1) / teams;
  const dim3 sums(groups < kSumGroups ? groups : kSumGroups, (E + (1 << lg) - 1) >> lg);
  const LossArgs a{T, E, lanes_log(E), k, n_seq, logits, offset, idx, seq, mask, psum, pcnt, ptok, total, left,
                   static_cast<int>(sums.x * sums.y)};
  const dim3 grid(static_cast<unsigned>(tiles)), block(kThreads);
  // sequences of under a tile's length on average: each costs the first form a
  // pass of its own (29 tokens in 49 sequences, were they no single launch, 40 us
  // against 10.1; 16384 in 300, E = 100, 15.1 against 14.2), long ones the second
  // its trip through LDS (16384 in 64, E = 256, 12.7 against 14.7; 65536 in 16 25.6
  // against 40.7).  By the average alone: one long sequence among a thousand short
  // or empty ones pays for it, here and in its team below (65536 tokens in one
  // sequence 31 us, beside 1000 empty ones 59).
  const bool many = E <= 256 && T < static_cast<int64_t>(kTile) * n_seq;
  auto part = [&](auto full) {
    constexpr bool F = decltype(full)::value;
    if (many) hipLaunchKernelGGL(balance_part_short_kernel<F>, grid, block, 0, s, a);
    else if (E <= 256) hipLaunchKernelGGL((balance_part_kernel<1, F>), grid, block, 0, s, a);
    else if (E <= 512) hipLaunchKernelGGL((balance_part_kernel<2, F>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((balance_part_kernel<4, F>), grid, block, 0, s, a);
  };
  if (full_rows(E)) part(std::true_type{});
  else part(std::false_type{});
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  float one = 0x1p41f;
  for (int e2 = 1; e2 < E; e2 *= 2) one *= 0.5f;
  const SumArgs b{T,    E,   k,      n_seq, lg,    team, alpha, seq, psum, pcnt, ptok, counts,
                  prob, dprob, one, total, left, loss};
  hipLaunchKernelGGL(balance_sum_kernel, sums, dim3(teams * team * kWave), 0, s, b);
  return hipGetLastError();
}

hipError_t launch_balance_loss_bwd(int64_t T, int E, const float* logits, const float* offset, const int32_t* seq,
                                   int n_seq, const uint8_t* mask, const float* dprob, const float* grad,
                                   const float* extra, float* dl, hipStream_t s) {
  const GradArgs a{T, E, lanes_log(E), n_seq, logits, offset, seq, mask, dprob, grad, extra, dl};
  const int64_t per = (int64_t)kGradWaves * (kWave >> a.log_lpt);
  const dim3 grid(static_cast<unsigned>((T + per - 1) / per)), block(kGradThreads);
  auto go = [&](auto full, auto add) {
    constexpr bool F = decltype(full)::value, A = decltype(add)::value;
    if (E <= 256) hipLaunchKernelGGL((balance_grad_kernel<1, F, A>), grid, block, 0, s, a);
    else if (E <= 512) hipLaunchKernelGGL((balance_grad_kernel<2, F, A>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((balance_grad_kernel<4, F, A>), grid, block, 0, s, a);
  };
  auto with = [&](auto full) {
    if (extra != nullptr) go(full, std::true_type{});
    else go(full, std::false_type{});
  };
  if (full_rows(E)) with(std::true_type{});
  else with(std::false_type{});
  return hipGetLastError();
}

}  // namespace moe

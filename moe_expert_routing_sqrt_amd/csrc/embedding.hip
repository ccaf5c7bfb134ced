// The embedding lookup with scaling, and its gradient.
//
//   out[t] = scale * table[ids[t]]           (zeros for an id outside [0, V))
//   d_table[v] (+)= scale * sum_{t: ids[t] = v} d_out[t]
//
// Both are bound by memory.  The gradient first sorts the batch by id, stably,
// so that each table row's tokens are one run in token order: its sum is then
// formed in registers in a fixed order, with no atomics and one store a row.
#include <algorithm>

#include "launch.h"
#include "rowvec.h"

namespace moe {
namespace {

constexpr int kThreads = 256;

// A thread's piece of a row of d elements: E of them from c.  The row's last
// piece is moved back to end with the row and owns only what the piece before
// it does not reach (elements lo and up); rows shorter than E are one piece,
// moved element by element.  c < 0: none.
template <int E>
struct RowPiece {
  int c, lo;
  __device__ __forceinline__ RowPiece(int i, int d) {
    const int at = i * E;
    c = at >= d ? -1 : max(0, min(at, d - E));
    lo = at - c;
  }
};

template <typename T, int E>
__device__ __forceinline__ void load_piece(Vec<T, E>& v, const T* row, int c, int d) {
  if (d >= E) {
    load_vec<false>(v, row + c);
    return;
  }
#pragma unroll
  for (int i = 0; i < Vec<T, E>::kWords; ++i) v.w[i] = 0;
#pragma unroll
  for (int j = 0; j < E - 1; ++j) {
    if (j >= d) continue;
    if constexpr (sizeof(T) == 2) v.w[j / 2] |= static_cast<uint32_t>(row[j]) << (16 * (j & 1));
    else v.w[j] = __float_as_uint(row[j]);
  }
}

// stores elements [lo, min(E, d))
template <typename T, int E>
__device__ __forceinline__ void store_piece(T* row, const Vec<T, E>& v, int c, int lo, int d) {
  if (d >= E && lo == 0) {
    store_vec<true>(row + c, v);
    return;
  }
#pragma unroll
  for (int j = 0; j < E; ++j) {
    if (j < lo || j >= d) continue;
    if constexpr (sizeof(T) == 2) row[c + j] = static_cast<uint16_t>(v.w[j / 2] >> (16 * (j & 1)));
    else row[c + j] = __uint_as_float(v.w[j]);
  }
}

// ---------------------------------------------------------------- lookup
struct LookupArgs {
  const int* ids;
  const void* table;
  void* out;
  int64_t T;
  int V, d;
  float scale;
};

// NT threads a row; up to kAhead pieces of it a thread in flight.
constexpr int kAhead = 4;
template <typename TX, typename TO, int E, int NT>
__global__ __launch_bounds__(kThreads) void embedding_kernel(const LookupArgs p) {
  const int rt = threadIdx.x % NT, pieces = (p.d + E - 1) / E;
  const int64_t step = (int64_t)gridDim.x * (kThreads / NT);
  for (int64_t t = (int64_t)blockIdx.x * (kThreads / NT) + threadIdx.x / NT; t < p.T; t += step) {
    const int id = p.ids[t];
    const bool in = static_cast<unsigned>(id) < static_cast<unsigned>(p.V);
    const TX* src = static_cast<const TX*>(p.table) + (int64_t)(in ? id : 0) * p.d;
    TO* dst = static_cast<TO*>(p.out) + t * p.d;
    for (int i0 = rt; i0 < pieces; i0 += NT * kAhead) {
      Vec<TX, E> v[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
#pragma unroll
        for (int w = 0; w < Vec<TX, E>::kWords; ++w) v[u].w[w] = 0;
        const RowPiece<E> q(i0 + u * NT, p.d);
        if (in && q.c >= 0) load_piece(v[u], src, q.c, p.d);
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const RowPiece<E> q(i0 + u * NT, p.d);
        if (q.c < 0) continue;
        float f[E];
        vec_f32(v[u], f);
#pragma unroll
        for (int j = 0; j < E; ++j) f[j] = in ? f[j] * p.scale : 0.0f;
        Vec<TO, E> o;
        f32_vec(o, f);
        store_piece(dst, o, q.c, 0, p.d);  // what two pieces share is the same in both
      }
    }
  }
}

template <typename TX, typename TO, int E>
hipError_t lookup(const LookupArgs& a, hipStream_t s) {
  const int pieces = (a.d + E - 1) / E;
  const bool narrow = pieces <= kWave * kAhead;  // a wave per row
  const int64_t rows = narrow ? kThreads / kWave : 1, groups = (a.T + rows - 1) / rows;
  // (a launch holds fewer than 2^32 threads)
  const dim3 grid(static_cast<unsigned>(std::min<int64_t>(groups, 1 << 22))), block(kThreads);
  if (narrow) hipLaunchKernelGGL((embedding_kernel<TX, TO, E, kWave>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((embedding_kernel<TX, TO, E, kThreads>), grid, block, 0, s, a);
  return hipGetLastError();
}

// ---------------------------------------------------------------- sort
// One launch.  Work-group r takes the table rows [r * span, (r + 1) * span): it
// reads every id twice (they stay in the XCD's L2), each of its 16 waves one
// sixteenth of the batch, and counts those of its rows and those below them.
// The counts per wave and row give every wave its first position for every row,
// so that the second reading places its tokens in token order.
constexpr int kSortWaves = 16;
constexpr int kMaxSpan = 1024;
constexpr int kIdsAhead = 8;

struct SortArgs {
  const int* ids;
  int T, V, span, bits;  // 2^bits >= span
  int2* sorted;          // [T] (token, id) by id, then token
  int* start;            // [V + 1] each id's first position; start[V]: tokens with an id inside
};

__global__ __launch_bounds__(kSortWaves* kWave) void embedding_sort_kernel(const SortArgs p) {
  extern __shared__ int s_count[];  // [kSortWaves][span]
  __shared__ int s_below, s_total[kSortWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int first = blockIdx.x * p.span, n = min(p.span, p.V - first);
  for (int i = tid; i < kSortWaves * p.span; i += blockDim.x) s_count[i] = 0;
  if (tid == 0) s_below = 0;
  __syncthreads();
  int* const mine = s_count + wave * p.span;
  const int per = ((p.T + kSortWaves - 1) / kSortWaves + kWave - 1) / kWave * kWave;
  const int t0 = min(p.T, wave * per), t1 = min(p.T, t0 + per);
  auto batch = [&](int t, int (&id)[kIdsAhead]) __attribute__((always_inline)) {
#pragma unroll
    for (int b = 0; b < kIdsAhead; ++b) {
      const int at = t + b * kWave + lane;
      id[b] = p.ids[min(at, p.T - 1)];
      if (at >= t1) id[b] = -1;
    }
  };
  int below = 0;
  for (int t = t0; t < t1; t += kIdsAhead * kWave) {
    int id[kIdsAhead];
    batch(t, id);
#pragma unroll
    for (int b = 0; b < kIdsAhead; ++b) {
      below += id[b] >= 0 && id[b] < first;
      const int r = id[b] - first;
      if (id[b] >= 0 && static_cast<unsigned>(r) < static_cast<unsigned>(n)) atomicAdd(&mine[r], 1);
    }
  }
  if (below > 0) atomicAdd(&s_below, below);
  __syncthreads();
  // counts to first positions: over the waves of each row, then over the rows
  int total = 0;
  if (tid < n) {
    for (int w = 0; w < kSortWaves; ++w) {
      const int c = s_count[w * p.span + tid];
      s_count[w * p.span + tid] = total;
      total += c;
    }
  }
  int upto = total;
#pragma unroll
  for (int o = 1; o < kWave; o <<= 1) {
    const int v = __shfl_up(upto, o, kWave);
    if (lane >= o) upto += v;
  }
  if (lane == 63) s_total[wave] = upto;
  __syncthreads();
  int base = s_below + upto - total;
  for (int w = 0; w < wave; ++w) base += s_total[w];
  if (tid < n) {
    for (int w = 0; w < kSortWaves; ++w) s_count[w * p.span + tid] += base;
    p.start[first + tid] = base;
    if (first + tid == p.V - 1) p.start[p.V] = base + total;
  }
  __syncthreads();
  for (int t = t0; t < t1; t += kIdsAhead * kWave) {
    int id[kIdsAhead];
    batch(t, id);
#pragma unroll
    for (int b = 0; b < kIdsAhead; ++b) {
      const int r = id[b] - first;
      const bool in = id[b] >= 0 && static_cast<unsigned>(r) < static_cast<unsigned>(n);
      uint64_t same = __ballot(in);
      if (same == 0) continue;
      for (int k = 0; k < p.bits; ++k) {  // the lanes with this lane's row
        const bool bit = (r >> k) & 1;
        const uint64_t set = __ballot(bit);
        same &= bit ? set : ~set;
      }
      const int rank = __popcll(same & ((uint64_t{1} << lane) - 1));
      asm volatile("" ::: "memory");  // the wave's positions as its own last batch left them
      int pos = 0;
      if (in) pos = mine[r] + rank;
      asm volatile("" ::: "memory");
      if (in && rank == 0) mine[r] = pos + __popcll(same);
      if (in) p.sorted[pos] = make_int2(t + b * kWave + lane, id[b]);
    }
  }
}

// ---------------------------------------------------------------- gradient
// Work-groups of three kinds in one launch, by columns in y:
//   runs   kRunChunk sorted positions each: the rows whose run starts there and
//          has at most kLong tokens, summed and stored;
//   long   kLong positions each: the part of a longer run that lies there (at
//          most two, the end of one and the start of another), to `part`;
//   zeros  kZeroRows table rows each: those without a token (not when adding).
// A second launch joins the parts of every long run in order.  Every lane
// of a wave holds one sorted position (two for runs), boundaries are ballots,
// and a token's number reaches the scalar unit by a lane read.
constexpr int kLong = 64;
constexpr int kRunChunk = 8;
constexpr int kZeroRows = 8;
static_assert(kRunChunk + kLong < 2 * kWave && kLong == kWave, "positions a wave holds");

struct GradArgs {
  const int2* sorted;
  const int* start;
  const void* dy;
  void* table;
  float* part;  // [ceil(T / kLong)][2][d]
  int T, V, d, runs, longs;
  float scale;
};

__device__ __forceinline__ int lane_of(int v, int i) { return __builtin_amdgcn_readlane(v, i); }

// Sum of the rows [i, e) of `tok` (lane numbers below 128: lanes of tok0, then
// tok1), in order, TB rows in flight.
template <typename TX, int E, int U, int TB>
__device__ __forceinline__ void sum_tokens(const TX* dy, int d, const int (&c)[U], int tok0, int tok1, int i, int e,
                                           float (&acc)[U][E]) {
#pragma unroll
  for (int u = 0; u < U; ++u) {
#pragma unroll
    for (int j = 0; j < E; ++j) acc[u][j] = 0.0f;
  }
  for (; i < e; i += TB) {
    Vec<TX, E> v[TB][U];
#pragma unroll
    for (int k = 0; k < TB; ++k) {
      if (i + k >= e) break;
      const int at = i + k;
      const int tok = at < kWave ? lane_of(tok0, at) : lane_of(tok1, at - kWave);
      const TX* row = dy + (int64_t)tok * d;
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (c[u] >= 0) load_piece(v[k][u], row, c[u], d);
    }
#pragma unroll
    for (int k = 0; k < TB; ++k) {
      if (i + k >= e) break;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float f[E];
        vec_f32(v[k][u], f);
#pragma unroll
        for (int j = 0; j < E; ++j) acc[u][j] += f[j];
      }
    }
  }
}

template <typename TO, int E, bool ADD>
__device__ __forceinline__ void put_row(TO* row, int d, const RowPiece<E>& q, float (&f)[E], float scale) {
  if (q.c < 0) return;
#pragma unroll
  for (int j = 0; j < E; ++j) f[j] *= scale;
  if constexpr (ADD) {
    Vec<TO, E> old;
    float g[E];
    load_piece(old, row, q.c, d);
    vec_f32(old, g);
#pragma unroll
    for (int j = 0; j < E; ++j) f[j] += g[j];
  }
  Vec<TO, E> o;
  f32_vec(o, f);
  store_piece(row, o, q.c, ADD ? q.lo : 0, d);
}

template <typename TX, typename TO, int E, int U, bool ADD>
__global__ __launch_bounds__(kThreads) void embedding_grad_kernel(const GradArgs p) {
  constexpr int TB = U == 1 ? 8 : 4;
  const int lane = threadIdx.x & 63;
  const TX* const dy = static_cast<const TX*>(p.dy);
  TO* const table = static_cast<TO*>(p.table);
  const int i0 = blockIdx.y * U * kThreads + threadIdx.x;
  int c[U];
#pragma unroll
  for (int u = 0; u < U; ++u) c[u] = RowPiece<E>(i0 + u * kThreads, p.d).c;
  int g = blockIdx.x;
  if (g >= p.runs + p.longs) {  // zeros
    const int v0 = (g - p.runs - p.longs) * kZeroRows, v = min(v0 + (lane & 15), p.V);
    const int at = p.start[v], next = __shfl_down(at, 1, kWave);
    const uint64_t empty = __ballot(at == next && lane < kZeroRows && v < p.V);
#pragma unroll
    for (int r = 0; r < kZeroRows; ++r) {
      if (!(empty >> r & 1)) continue;
      TO* row = table + (int64_t)(v0 + r) * p.d;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        Vec<TO, E> z;
#pragma unroll
        for (int w = 0; w < Vec<TO, E>::kWords; ++w) z.w[w] = 0;
        if (c[u] >= 0) store_piece(row, z, c[u], 0, p.d);
      }
    }
    return;
  }
  const int n = p.start[p.V];  // tokens with an id inside
  float acc[U][E];
  if (g < p.runs) {
    const int p0 = g * kRunChunk;
    if (p0 >= n) return;
    const int2 a = p.sorted[min(p0 + lane, n - 1)], b = p.sorted[min(p0 + kWave + lane, n - 1)];
    const int before = p0 > 0 ? p.sorted[p0 - 1].y : -1;
    int up_a = __shfl_up(a.y, 1, kWave), up_b = __shfl_up(b.y, 1, kWave);
    if (lane == 0) {
      up_a = before;
      up_b = lane_of(a.y, 63);
    }
    // bit: a run starts here, or the batch has ended
    const uint64_t sa = __ballot(p0 + lane >= n || a.y != up_a);
    const uint64_t sb = __ballot(p0 + kWave + lane >= n || b.y != up_b);
    uint64_t here = sa & ((uint64_t{1} << kRunChunk) - 1);
    while (here != 0) {
      const int s = __builtin_ctzll(here);
      if (p0 + s >= n) break;
      here &= here - 1;
      const uint64_t later = sa & ~((uint64_t{2} << s) - 1);
      const int e = later != 0 ? __builtin_ctzll(later) : sb != 0 ? kWave + __builtin_ctzll(sb) : 2 * kWave;
      if (e - s > kLong) break;  // the positions of a long run reach past this chunk
      sum_tokens<TX, E, U, TB>(dy, p.d, c, a.x, b.x, s, e, acc);
      TO* row = table + (int64_t)lane_of(a.y, s) * p.d;
#pragma unroll
      for (int u = 0; u < U; ++u) put_row<TO, E, ADD>(row, p.d, RowPiece<E>(i0 + u * kThreads, p.d), acc[u], p.scale);
    }
    return;
  }
  g -= p.runs;
  const int p0 = g * kLong;
  if (p0 >= n) return;
  const int2 a = p.sorted[min(p0 + lane, n - 1)];
  const int used = min(kLong, n - p0);
#pragma unroll
  for (int side = 0; side < 2; ++side) {
    const int v = lane_of(a.y, side == 0 ? 0 : used - 1);
    if (side == 1 && v == lane_of(a.y, 0)) return;
    const int s = p.start[v], e = p.start[v + 1];
    if (e - s <= kLong) continue;
    sum_tokens<TX, E, U, TB>(dy, p.d, c, a.x, a.x, max(s - p0, 0), min(e - p0, used), acc);
    float* part = p.part + ((int64_t)g * 2 + side) * p.d;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (c[u] < 0) continue;
      Vec<float, E> o;
      f32_vec(o, acc[u]);
      store_piece(part, o, c[u], 0, p.d);
    }
  }
}

// The long run whose first whole-chunk position is this work-group's p0: its parts
// in order, a quarter of them by each of 4 waves, then the waves in order.
template <typename TO, bool ADD>
__global__ __launch_bounds__(kThreads) void embedding_join_kernel(const GradArgs p) {
  constexpr int E = 4, B = 8;
  __shared__ float s_sum[3][E][kWave];
  const int p0 = blockIdx.x * kLong, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  if (p0 >= p.start[p.V]) return;
  const int v = p.sorted[p0].y, s = p.start[v], e = p.start[v + 1];
  if (e - s <= kLong || s <= p0 - kLong) return;
  const RowPiece<E> q(blockIdx.y * kWave + lane, p.d);
  const int c0 = blockIdx.x, lead = s < p0 ? 1 : 0;  // a part at the end of the chunk before
  const int parts = (e - 1) / kLong - c0 + 1 + lead, per = (parts + 3) / 4;
  const int k1 = min(parts, (wave + 1) * per);
  float acc[E] = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int k0 = wave * per; k0 < k1; k0 += B) {
    Vec<float, E> t[B];
#pragma unroll
    for (int i = 0; i < B; ++i) {
      const int k = min(k0 + i, k1 - 1);
      const int64_t at = lead != 0 && k == 0 ? (int64_t)(c0 - 1) * 2 + 1 : (int64_t)(c0 + k - lead) * 2;
      if (q.c >= 0) load_piece(t[i], p.part + at * p.d, q.c, p.d);
    }
#pragma unroll
    for (int i = 0; i < B; ++i) {
      if (k0 + i >= k1 || q.c < 0) continue;
#pragma unroll
      for (int j = 0; j < E; ++j) acc[j] += __uint_as_float(t[i].w[j]);
    }
  }
  if (wave > 0) {
#pragma unroll
    for (int j = 0; j < E; ++j) s_sum[wave - 1][j][lane] = acc[j];
  }
  __syncthreads();
  if (wave > 0) return;
#pragma unroll
  for (int w = 0; w < 3; ++w) {
#pragma unroll
    for (int j = 0; j < E; ++j) acc[j] += s_sum[w][j][lane];
  }
  put_row<TO, E, ADD>(static_cast<TO*>(p.table) + (int64_t)v * p.d, p.d, q, acc, p.scale);
}

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

template <typename TX, typename TO, int E, bool ADD>
hipError_t grad(GradArgs a, hipStream_t s) {
  const int pieces = (a.d + E - 1) / E;
  const int64_t zeros = ADD ? 0 : ((int64_t)a.V + kZeroRows - 1) / kZeroRows;
  const unsigned x = static_cast<unsigned>(a.runs + a.longs + zeros);
  if (x == 0) return hipSuccess;
  const dim3 block(kThreads);
  auto y = [&](int u) { return static_cast<unsigned>((pieces + u * kThreads - 1) / (u * kThreads)); };
  if (pieces <= kThreads)
    hipLaunchKernelGGL((embedding_grad_kernel<TX, TO, E, 1, ADD>), dim3(x, y(1)), block, 0, s, a);
  else if (pieces <= 2 * kThreads)
    hipLaunchKernelGGL((embedding_grad_kernel<TX, TO, E, 2, ADD>), dim3(x, y(2)), block, 0, s, a);
  else
    hipLaunchKernelGGL((embedding_grad_kernel<TX, TO, E, 4, ADD>), dim3(x, y(4)), block, 0, s, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.longs == 0) return e;
  const int cols = kWave * 4;
  hipLaunchKernelGGL((embedding_join_kernel<TO, ADD>), dim3(a.longs, (a.d + cols - 1) / cols), block, 0, s, a);
  return hipGetLastError();
}

template <typename TX, typename TO, int E>
hipError_t grad(const GradArgs& a, bool add, hipStream_t s) {
  return add ? grad<TX, TO, E, true>(a, s) : grad<TX, TO, E, false>(a, s);
}

}  // namespace

hipError_t launch_embedding(int64_t T, int V, int d, const int32_t* ids, const void* table, int table_dtype,
                            float scale, void* out, int out_dtype, hipStream_t s) {
  const LookupArgs a{ids, table, out, T, V, d, scale};
  using B = uint16_t;
  const bool xb = table_dtype == MOE_BF16, yb = out_dtype == MOE_BF16;
  if (xb) return yb ? lookup<B, B, 8>(a, s) : lookup<B, float, 4>(a, s);
  return yb ? lookup<float, B, 4>(a, s) : lookup<float, float, 4>(a, s);
}

size_t embedding_bwd_workspace_bytes(int64_t T, int64_t V, int d) {
  if (T == 0) T = 1;
  const int64_t chunks = (T + kLong - 1) / kLong;
  return up256(T * sizeof(int2)) + up256((V + 1) * sizeof(int)) + up256(chunks * 2 * d * sizeof(float));
}

hipError_t launch_embedding_bwd(int64_t T, int V, int d, const int32_t* ids, const void* dy, int dy_dtype, float scale,
                                void* d_table, int d_table_dtype, bool add, void* ws, hipStream_t s) {
  char* w = static_cast<char*>(ws);
  SortArgs o{};
  o.ids = ids;
  o.T = static_cast<int>(T);
  o.V = V;
  // rows a work-group sorts: one work-group per CU where the counts fit LDS
  o.span = std::min(kMaxSpan, std::max(1, (V + 255) / 256));
  while ((1 << o.bits) < o.span) ++o.bits;
  o.sorted = reinterpret_cast<int2*>(w);
  w += up256(T * sizeof(int2));
  o.start = reinterpret_cast<int*>(w);
  w += up256((static_cast<size_t>(V) + 1) * sizeof(int));
  hipLaunchKernelGGL(embedding_sort_kernel, dim3((V + o.span - 1) / o.span), dim3(kSortWaves * kWave),
                     kSortWaves * o.span * sizeof(int), s, o);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const GradArgs a{o.sorted, o.start, dy, d_table, reinterpret_cast<float*>(w), o.T, V, d,
                   (o.T + kRunChunk - 1) / kRunChunk, (o.T + kLong - 1) / kLong, scale};
  using B = uint16_t;
  const bool xb = dy_dtype == MOE_BF16, yb = d_table_dtype == MOE_BF16;
  if (xb) return yb ? grad<B, B, 8>(a, add, s) : grad<B, float, 4>(a, add, s);
  return yb ? grad<float, B, 4>(a, add, s) : grad<float, float, 4>(a, add, s);
}

}  // namespace moe

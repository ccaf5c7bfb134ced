// The embedding lookup with scaling, and its gradient.
//
//   out[t] = scale * table[ids[t]]           (zeros for an id outside [0, V))
//   d_table[v] (+)= scale * sum_{t: ids[t] = v} d_out[t]
//
// Both are bound by memory.  The gradient first sorts the batch by id, stably,
// so that each table row's tokens are one run in token order: its sum is then
// formed in registers in a fixed order, with no atomics and one store a row.
// Measured: lookup of 16384 x 7168 bf16 out of 131072 rows 68 us (235 MB written,
// the rows read again where they repeat); its gradient, written whole in fp32 (3.8
// GB), 750 us, of which clearing takes 640 (5.5 TB/s, what a plain fill of that
// size reaches); 16384 x 2048 accumulated into fp32 rows 52 us in its three launches
// (sort 10, sums 37, join 5), 55 a call, 46 where the batch before was the same one.
// What is left of narrow rows is the sort and the sums' chains of loads: 16384 x 64
// accumulated 28 us.
#include <algorithm>

#include "launch.h"
#include "rowvec.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int64_t kMaxGroups = UINT32_MAX / kThreads;  // a launch holds fewer than 2^32 threads

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
template <bool STREAM, typename T, int E>
__device__ __forceinline__ void store_piece(T* row, const Vec<T, E>& v, int c, int lo, int d) {
  if (d >= E && lo == 0) {
    store_vec<STREAM>(row + c, v);
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
        store_piece<true>(dst, o, q.c, 0, p.d);  // what two pieces share is the same in both
      }
    }
  }
}

template <typename TX, typename TO, int E>
hipError_t lookup(const LookupArgs& a, hipStream_t s) {
  const int pieces = (a.d + E - 1) / E;
  const bool narrow = pieces <= kWave * kAhead;  // a wave per row
  const int64_t rows = narrow ? kThreads / kWave : 1, groups = (a.T + rows - 1) / rows;
  const dim3 grid(static_cast<unsigned>(std::min<int64_t>(groups, 1 << 22))), block(kThreads);
  if (narrow) hipLaunchKernelGGL((embedding_kernel<TX, TO, E, kWave>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((embedding_kernel<TX, TO, E, kThreads>), grid, block, 0, s, a);
  return hipGetLastError();
}

// ---------------------------------------------------------------- sort
// One launch.  Work-group r takes the table rows [r * span, (r + 1) * span): it
// goes through every id twice (they stay in the XCD's L2, or in registers), each
// of its 16 waves one sixteenth of the batch, and counts those of its rows and
// those below them.  The counts per wave and row give every wave its first
// position for every row, so that the second time it places its tokens in token
// order.
constexpr int kSortWaves = 16;
constexpr int kMaxSpan = 1024;
constexpr int kHeldIds = 16;  // ids of a thread that stay in registers: batches of up to 16384
constexpr int kFewLanes = 8;

struct SortArgs {
  const int* ids;
  int T, V, span, bits;  // 2^bits >= span
  int2* sorted;          // [T] (token, id) by id, then token
  int* start;            // [V + 1] each id's first position; start[V]: tokens with an id inside
};

template <bool HELD>
__global__ __launch_bounds__(kSortWaves* kWave) void embedding_sort_kernel(const SortArgs p) {
  constexpr int B = HELD ? kHeldIds : 8;
  extern __shared__ int s_count[];  // [kSortWaves][span]
  __shared__ int s_below, s_total[kSortWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int first = blockIdx.x * p.span, n = min(p.span, p.V - first);
  int* const mine = s_count + wave * p.span;
  const int per = ((p.T + kSortWaves - 1) / kSortWaves + kWave - 1) / kWave * kWave;
  const int t0 = min(p.T, wave * per), t1 = min(p.T, t0 + per);
  int id[B];
  auto batch = [&](int t) __attribute__((always_inline)) {
#pragma unroll
    for (int b = 0; b < B; ++b) id[b] = p.ids[max(0, min(t + b * kWave + lane, t1 - 1))];
#pragma unroll
    for (int b = 0; b < B; ++b) id[b] = t + b * kWave + lane < t1 ? id[b] : -1;
  };
  if (HELD && p.T > 0) batch(t0);
  for (int i = tid; i < kSortWaves * p.span; i += blockDim.x) s_count[i] = 0;
  if (tid == 0) s_below = 0;
  __syncthreads();
  int below = 0;
  for (int t = t0; t < t1; t += B * kWave) {
    if (!HELD) batch(t);
#pragma unroll
    for (int b = 0; b < B; ++b) {
      if (HELD && t + b * kWave >= t1) break;
      below += __popcll(__ballot(id[b] >= 0 && id[b] < first));
      const int r = id[b] - first;
      if (id[b] >= 0 && static_cast<unsigned>(r) < static_cast<unsigned>(n)) atomicAdd(&mine[r], 1);
    }
  }
  if (lane == 0 && below > 0) atomicAdd(&s_below, below);
  __syncthreads();
  // counts to first positions: over the waves of each row, then over the rows
  int total = 0, c[kSortWaves];
  if (tid < n) {
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) c[w] = s_count[w * p.span + tid];
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) {
      const int v = c[w];
      c[w] = total;
      total += v;
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
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) s_count[w * p.span + tid] = c[w] + base;
    p.start[first + tid] = base;
    if (first + tid == p.V - 1) p.start[p.V] = base + total;
  }
  __syncthreads();
  for (int t = t0; t < t1; t += B * kWave) {
    if (!HELD) batch(t);
#pragma unroll
    for (int b = 0; b < B; ++b) {
      if (HELD && t + b * kWave >= t1) break;
      const int r = id[b] - first;
      const bool in = id[b] >= 0 && static_cast<unsigned>(r) < static_cast<unsigned>(n);
      uint64_t left = __ballot(in);
      if (left == 0) continue;
      int pos = 0;
      if (__popcll(left) <= kFewLanes) {  // one row after the other
        while (left != 0) {
          const int at = __builtin_amdgcn_readlane(r, __builtin_ctzll(left));
          const uint64_t same = __ballot(in && r == at);
          const int from = mine[at];
          if (in && r == at) pos = from + __popcll(same & ((uint64_t{1} << lane) - 1));
          asm volatile("" ::: "memory");  // the wave's positions as it left them itself
          if (lane == 0) mine[at] = from + __popcll(same);
          asm volatile("" ::: "memory");
          left &= ~same;
        }
      } else {  // all at once: the lanes with this lane's row, by the bits of its number
        uint64_t same = left;
        for (int k = 0; k < p.bits; ++k) {
          const bool bit = (r >> k) & 1;
          const uint64_t set = __ballot(bit);
          same &= bit ? set : ~set;
        }
        const int rank = __popcll(same & ((uint64_t{1} << lane) - 1));
        asm volatile("" ::: "memory");
        if (in) pos = mine[r] + rank;
        asm volatile("" ::: "memory");
        if (in && rank == 0) mine[r] = pos + __popcll(same);
        asm volatile("" ::: "memory");
      }
      if (in) p.sorted[pos] = make_int2(t + b * kWave + lane, id[b]);
    }
  }
}

// ---------------------------------------------------------------- gradient
// Work-groups of three kinds in one launch:
//   runs   kRunChunk sorted positions and a block of columns each: the rows whose
//          run starts there and has at most kLong tokens, summed and stored;
//   long   kLong positions and a block of columns each: the part of a longer run
//          that lies there (at most two, the end of one and the start of another),
//          to `part`; and whether a join starts there, to `job`;
//   zeros  some table rows each: those without a token (not when adding).
// A second launch joins the parts of every long run in order.  Every lane
// of a wave holds one sorted position (two for runs), boundaries are ballots,
// and a token's number reaches the scalar unit by a lane read.
constexpr int kLong = 64;
constexpr int kRunChunk = 8;
static_assert(kRunChunk + kLong < 2 * kWave && kLong == kWave, "positions a wave holds");

struct GradArgs {
  const int2* sorted;
  const int* start;
  const void* dy;
  void* table;
  float* part;  // [longs][2][d]
  int* job;     // [longs] the row whose parts are joined from this chunk on, or -1
  int T, V, d, runs, longs, blocks, zero_rows;
  float scale;
};

__device__ __forceinline__ int lane_of(int v, int i) { return __builtin_amdgcn_readlane(v, i); }

constexpr int kRowsAhead = 16;  // rows in flight (8: 16384 x 2048 accumulated, the same batch again, 48 us, 46 so)

// scale * acc (+ old) to the row
template <typename TO, int E, bool ADD>
__device__ __forceinline__ void put_row(TO* row, int d, const RowPiece<E>& q, const float (&acc)[E],
                                        const Vec<TO, E>& old, float scale) {
  if (q.c < 0) return;
  float f[E];
#pragma unroll
  for (int j = 0; j < E; ++j) f[j] = acc[j] * scale;
  if constexpr (ADD) {
    float g[E];
    vec_f32(old, g);
#pragma unroll
    for (int j = 0; j < E; ++j) f[j] += g[j];
  }
  Vec<TO, E> o;
  f32_vec(o, f);
  store_piece<false>(row, o, q.c, ADD ? q.lo : 0, d);
}

template <typename TX, typename TO, int E, bool ADD>
__global__ __launch_bounds__(kThreads) void embedding_grad_kernel(const GradArgs p) {
  constexpr int TB = kRowsAhead;
  const int lane = threadIdx.x & 63;
  const TX* const dy = static_cast<const TX*>(p.dy);
  TO* const table = static_cast<TO*>(p.table);
  const int work = blockIdx.x;
  if (work >= (p.runs + p.longs) * p.blocks) {  // zeros
    const int v0 = (work - (p.runs + p.longs) * p.blocks) * p.zero_rows, rows = min(p.zero_rows, p.V - v0);
    const int at = p.start[min(v0 + lane, p.V)], next = __shfl_down(at, 1, kWave);
    const uint64_t empty = __ballot(lane < rows && at == next);
    const int pieces = (p.d + E - 1) / E;
    Vec<TO, E> z;
#pragma unroll
    for (int w = 0; w < Vec<TO, E>::kWords; ++w) z.w[w] = 0;
    int r = threadIdx.x / pieces, i = threadIdx.x - r * pieces;
    while (r < rows) {
      if (empty >> r & 1) store_piece<false>(table + (int64_t)(v0 + r) * p.d, z, RowPiece<E>(i, p.d).c, 0, p.d);
      for (i += kThreads; i >= pieces; i -= pieces) ++r;
    }
    return;
  }
  const bool is_long = work >= p.runs * p.blocks;
  const int g = (is_long ? work - p.runs * p.blocks : work) / p.blocks, y = work % p.blocks;
  const RowPiece<E> q(y * kThreads + threadIdx.x, p.d);
  const int n = p.start[p.V];  // tokens with an id inside
  float acc[E];
  Vec<TX, E> v[TB];
  auto clear = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < E; ++j) acc[j] = 0.0f;
  };
  // The pieces of TB tokens, tok(k) each.  No branch lies between the loads: behind
  // one, each would be waited for (1000 x 1001 fp32: 19.7 us, 16.6 so).
  const int c = max(q.c, 0);
  auto load = [&](auto tok) __attribute__((always_inline)) {
    if (p.d >= E) {
#pragma unroll
      for (int k = 0; k < TB; ++k) load_vec<false>(v[k], dy + (int64_t)tok(k) * p.d + c);
    } else {
#pragma unroll
      for (int k = 0; k < TB; ++k) load_piece(v[k], dy + (int64_t)tok(k) * p.d, 0, p.d);
    }
  };
  auto add = [&](int k) __attribute__((always_inline)) {
    float f[E];
    vec_f32(v[k], f);
#pragma unroll
    for (int j = 0; j < E; ++j) acc[j] += f[j];
  };
  if (!is_long) {
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
    const uint64_t here = sa & ((uint64_t{1} << min(kRunChunk, n - p0)) - 1);
    if (here == 0) return;
    const int last = 63 - __builtin_clzll(here);  // the last run that starts here, and its end
    const uint64_t later = sa & ~((uint64_t{2} << last) - 1);
    const int e = later != 0 ? __builtin_ctzll(later) : sb != 0 ? kWave + __builtin_ctzll(sb) : 2 * kWave;
    const int end = e - last > kLong ? last : e;  // a long run is not this kind's
    auto starts = [&](int i) __attribute__((always_inline)) { return (i < kWave ? sa >> i : sb >> (i - kWave)) & 1; };
    TO* row = table;
    Vec<TO, E> old, olds[ADD ? kRunChunk : 1];
    for (int i = __builtin_ctzll(here); i < end; i += TB) {
      load([&](int k) __attribute__((always_inline)) {
        const int at = min(i + k, end - 1);
        return at < kWave ? lane_of(a.x, at) : lane_of(b.x, at - kWave);
      });
      if constexpr (ADD) {
#pragma unroll
        for (int k = 0; k < kRunChunk; ++k) {
          const int at = i + k;
          if (at < min(kRunChunk, end) && starts(at) && q.c >= 0)
            load_piece(olds[k], table + (int64_t)lane_of(a.y, at) * p.d, q.c, p.d);
        }
      }
#pragma unroll
      for (int k = 0; k < TB; ++k) {
        const int at = i + k;
        if (at >= end) continue;
        if (k < kRunChunk && at < kRunChunk && starts(at)) {
          clear();
          row = table + (int64_t)lane_of(a.y, at) * p.d;
          if constexpr (ADD) old = olds[k < kRunChunk ? k : 0];
        }
        add(k);
        if (starts(at + 1)) put_row<TO, E, ADD>(row, p.d, q, acc, old, p.scale);
      }
    }
    return;
  }
  const int p0 = g * kLong;
  const int2 a = p.sorted[max(0, min(p0 + lane, n - 1))];
  const int used = min(kLong, n - p0);
  int job = -1;
#pragma unroll
  for (int side = 0; side < 2; ++side) {
    if (used <= 0) break;
    const int id = lane_of(a.y, side == 0 ? 0 : used - 1);
    if (side == 1 && id == lane_of(a.y, 0)) break;
    const int s = p.start[id], e = p.start[id + 1];
    if (e - s <= kLong) continue;
    if (side == 0 && s > p0 - kLong) job = id;
    clear();
    const int to = min(e - p0, used);
    for (int i = max(s - p0, 0); i < to; i += TB) {
      load([&](int k) __attribute__((always_inline)) { return lane_of(a.x, min(i + k, to - 1)); });
#pragma unroll
      for (int k = 0; k < TB; ++k) {
        if (i + k < to) add(k);
      }
    }
    float* part = p.part + ((int64_t)g * 2 + side) * p.d;
    Vec<float, E> o;
    f32_vec(o, acc);
    if (q.c >= 0) store_piece<false>(part, o, q.c, 0, p.d);
  }
  if (y == 0 && threadIdx.x == 0) p.job[g] = job;
}

// The long run whose first position at a chunk's start is this chunk's: its parts
// in order, a quarter of them by each of 4 waves, then the waves in order.
template <typename TO, bool ADD>
__global__ __launch_bounds__(kThreads) void embedding_join_kernel(const GradArgs p) {
  constexpr int E = 4, B = 8;
  __shared__ float s_sum[3][E][kWave];
  const int v = p.job[blockIdx.x], lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  if (v < 0) return;
  const int c0 = blockIdx.x, s = p.start[v], e = p.start[v + 1];
  const RowPiece<E> q(blockIdx.y * kWave + lane, p.d);
  const int lead = s < c0 * kLong ? 1 : 0;  // a part at the end of the chunk before
  const int parts = (e - 1) / kLong - c0 + 1 + lead, per = (parts + 3) / 4;
  const int k1 = min(parts, (wave + 1) * per);
  float acc[E] = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int k0 = wave * per; k0 < k1; k0 += B) {
    Vec<float, E> t[B];
#pragma unroll
    for (int i = 0; i < B; ++i) {
      const int k = min(k0 + i, k1 - 1);
      const int64_t at = lead != 0 && k == 0 ? (int64_t)(c0 - 1) * 2 + 1 : (int64_t)(c0 + k - lead) * 2;
      load_piece(t[i], p.part + at * p.d, max(q.c, 0), p.d);
    }
#pragma unroll
    for (int i = 0; i < B; ++i) {
      if (k0 + i >= k1) continue;
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
  TO* row = static_cast<TO*>(p.table) + (int64_t)v * p.d;
  Vec<TO, E> old;
  if constexpr (ADD) {
    if (q.c >= 0) load_piece(old, row, q.c, p.d);
  }
  put_row<TO, E, ADD>(row, p.d, q, acc, old, p.scale);
}

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

// column blocks of a run or a part (E elements a thread), and table rows that a
// work-group clears: about 32 KB (128 KB: 2 % slower)
int column_blocks(int d, int E) { return (d + E * kThreads - 1) / (E * kThreads); }
int rows_to_clear(int d, int bytes) {
  const int64_t rows = (int64_t{1} << 15) / ((int64_t)d * bytes);
  return static_cast<int>(std::min<int64_t>(kWave - 1, std::max<int64_t>(1, rows)));
}
int64_t run_chunks(int64_t T) { return (T + kRunChunk - 1) / kRunChunk; }
int64_t long_chunks(int64_t T) { return (T + kLong - 1) / kLong; }
int64_t grad_groups(int64_t T, int64_t V, int d, int E, int bytes, bool add) {
  const int64_t rows = rows_to_clear(d, bytes);
  return (run_chunks(T) + long_chunks(T)) * column_blocks(d, E) + (add ? 0 : (V + rows - 1) / rows);
}

template <typename TX, typename TO, int E, bool ADD>
hipError_t grad(GradArgs a, hipStream_t s) {
  a.blocks = column_blocks(a.d, E);
  a.zero_rows = rows_to_clear(a.d, sizeof(TO));
  const int64_t x = grad_groups(a.T, a.V, a.d, E, sizeof(TO), ADD);
  if (x == 0) return hipSuccess;
  if (x > kMaxGroups) return hipErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>(x)), block(kThreads);
  hipLaunchKernelGGL((embedding_grad_kernel<TX, TO, E, ADD>), grid, block, 0, s, a);
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

bool embedding_bwd_supported(int64_t T, int64_t V, int d, int d_table_dtype, bool add) {
  static_assert(MOE_MAX_EMBEDDING / (kWave * 4) <= 65535, "a grid's second axis");
  return grad_groups(T, V, d, 4, d_table_dtype == MOE_BF16 ? 2 : 4, add) <= kMaxGroups;
}

size_t embedding_bwd_workspace_bytes(int64_t T, int64_t V, int d) {
  if (T == 0) T = 1;
  const int64_t chunks = long_chunks(T);
  return up256(T * sizeof(int2)) + up256((V + 1) * sizeof(int)) + up256(chunks * sizeof(int)) +
         up256(chunks * 2 * d * sizeof(float));
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
  const dim3 grid((V + o.span - 1) / o.span), block(kSortWaves * kWave);
  const size_t lds = kSortWaves * o.span * sizeof(int);
  if (T <= kHeldIds * kSortWaves * kWave) hipLaunchKernelGGL(embedding_sort_kernel<true>, grid, block, lds, s, o);
  else hipLaunchKernelGGL(embedding_sort_kernel<false>, grid, block, lds, s, o);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  GradArgs a{};
  a.sorted = o.sorted;
  a.start = o.start;
  a.dy = dy;
  a.table = d_table;
  a.T = o.T;
  a.V = V;
  a.d = d;
  a.runs = static_cast<int>(run_chunks(T));
  a.longs = static_cast<int>(long_chunks(T));
  a.scale = scale;
  a.job = reinterpret_cast<int*>(w);
  w += up256(std::max(1, a.longs) * sizeof(int));
  a.part = reinterpret_cast<float*>(w);
  using B = uint16_t;
  const bool xb = dy_dtype == MOE_BF16, yb = d_table_dtype == MOE_BF16;
  if (xb) return yb ? grad<B, B, 8>(a, add, s) : grad<B, float, 4>(a, add, s);
  return yb ? grad<float, B, 4>(a, add, s) : grad<float, float, 4>(a, add, s);
}

}  // namespace moe

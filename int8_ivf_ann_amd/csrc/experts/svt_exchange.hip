// svt_exchange.hip - tokens sorted by expert, their rows sent to the experts and brought back with weights,
// and the gradients of both, on gfx950.
//
// Entries are the T x top (token, choice) pairs of a router; entry i = t * top + j is valid when its
// expert lies in [0, E).  The sort is stable: position[i] = offsets[e] + (valid entries of e before i).
//
//   dispatch            rows[position[t][j]] = x[t]
//   dispatch backward   dx[t] = sum_j d_rows[position[t][j]]
//   combine             y[t] = sum_j w[t][j] rows[position[t][j]]
//   combine backward    d_rows[position[t][j]] = w[t][j] dy[t],  dw[t][j] = dy[t] . rows[position[t][j]]
//
// Every exchange kernel walks tokens: a token's own row is read or written in order, its `top` rows on the experts'
// side are whole rows, and the only gather is of rows.  Each byte moves once, but that combine's gradient, which
// holds 4 rows of the experts at a time, reads dy ceil(top / 4) times (after the first from a cache: 16384 x 1024
// bfloat16, top 8, 124 us for 570 MB, as fast as top 2's 136 for 671 MB).  Sums run over j in order in float32 and no
// two threads write one address, so results never vary.  A token belongs to one wave at most, so that few tokens of
// wide rows leave compute units idle: 1 token of 4096 bfloat16, top 8, 8 us each way and 11 for combine's gradient.

#include <type_traits>

#include "svt_experts.h"

namespace svt {

namespace {

// ---- sort ----------------------------------------------------------------------------------------
//
// A counting sort.  Waves own contiguous pieces of the entries; within a piece, 64 entries at a time, an
// entry's rank among the lanes of its expert comes from one ballot per bit of the expert's number (the
// lanes that agree on every bit), added to the piece's count of that expert so far.  Ranks stay in
// registers, so the entries are read once, and no position depends on the order of atomics.
//   one launch   (up to kOneEntries): a workgroup of 16 waves ranks, scans and places.
//   two          k_sort_count: a histogram per block; k_sort_place: each block sums the histograms (few blocks
//                of many entries keep that table small), ranks its entries, orders them in LDS and writes
//                each expert's run in one piece.
// Measured: 256 entries of 32 experts 2.6 us, 4096 of 8 experts 5.1, 8192 7.8; 1 M entries of 64 experts 13.7 (12.6
// MB; all of one expert, whose count is one LDS address: 16.1), of 512 experts 27.7 (half the blocks, so that the
// table stays small).  All are chains of short steps between barriers; bytes would take 2.5 us at 1 M.

constexpr int kSortThreads = 1024, kSortWaves = kSortThreads / 64, kSortSteps = 4;
constexpr int kTileEntries = kSortThreads * kSortSteps;   // entries of a workgroup at a time
constexpr int64_t kOneEntries = 8 * kSortThreads;
constexpr int64_t kMaxBlocks = 512;                       // two per compute unit
constexpr int64_t kMaxEntries = int64_t(1) << 30;

struct SortShape {
  int64_t n;            // entries
  int64_t per_block;    // entries per block, a multiple of kTileEntries
  int32_t blocks;
};

// every block reads the whole table of histograms: at most 64 K counts
SortShape sort_shape(int64_t n, int E) {
  const int64_t tiles = (n + kTileEntries - 1) / kTileEntries;
  const int64_t most = kMaxBlocks * E > 65536 ? 65536 / E : kMaxBlocks;
  const int64_t each = (tiles + most - 1) / most;   // tiles per block
  return SortShape{n, each * kTileEntries, (int32_t)((tiles + each - 1) / each)};
}

__device__ __forceinline__ int load_expert(const int32_t *experts, int64_t i, int64_t end, int E) {
  const int e = experts[i < end ? i : end - 1];
  return i < end && (uint32_t)e < (uint32_t)E ? e : -1;
}

// count[w][e] become exclusive sums over the waves, total[e] their sum
__device__ __forceinline__ void sum_waves(int32_t (*count)[SVT_MAX_EXPERTS], int32_t *total, int E) {
  for (int e = threadIdx.x; e < E; e += kSortThreads) {
    int sum = 0;
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) {
      const int c = count[w][e];
      count[w][e] = sum;
      sum += c;
    }
    total[e] = sum;
  }
}

// start[0 .. E] = exclusive sums of total[0 .. E), by the first wave; the caller's barriers around it
__device__ __forceinline__ void scan_experts(const int32_t *total, int32_t *start, int E) {
  if (threadIdx.x >= 64) return;
  const int each = (E + 63) / 64;
  int sum = 0;
  for (int q = 0; q < each; ++q) {
    const int e = threadIdx.x * each + q;
    sum += e < E ? total[e] : 0;
  }
  const int upto = incl_sums(sum);
  int at = upto - sum;
  for (int q = 0; q < each; ++q) {
    const int e = threadIdx.x * each + q;
    if (e < E) {
      start[e] = at;
      at += total[e];
    }
  }
  if (threadIdx.x == 63) start[E] = upto;
}

template <int STEPS, int BITS>
__global__ __launch_bounds__(kSortThreads) void k_sort_one(const int32_t *experts, int64_t n, int E, int32_t *offsets,
                                                           int32_t *order, int32_t *position) {
  __shared__ int32_t count[kSortWaves][SVT_MAX_EXPERTS];
  __shared__ int32_t total[SVT_MAX_EXPERTS], start[SVT_MAX_EXPERTS + 1];
  const int tid = threadIdx.x, wv = tid / 64;
  const int64_t i0 = (int64_t)wv * (64 * STEPS) + tid % 64;
  int e[STEPS], rank[STEPS];
#pragma unroll
  for (int q = 0; q < STEPS; ++q) e[q] = n > 0 ? load_expert(experts, i0 + 64 * q, n, E) : -1;
  for (int i = tid % 64; i < E; i += 64) count[wv][i] = 0;   // its own wave's: no barrier needed
  rank_entries<STEPS, BITS>(e, rank, count[wv]);
  __syncthreads();
  sum_waves(count, total, E);
  __syncthreads();
  scan_experts(total, start, E);
  __syncthreads();
  for (int i = tid; i <= E; i += kSortThreads) offsets[i] = start[i];
  for (int64_t i = start[E] + tid; i < n; i += kSortThreads) order[i] = -1;
#pragma unroll
  for (int q = 0; q < STEPS; ++q) {
    const int64_t i = i0 + 64 * q;
    const int at = e[q] >= 0 ? start[e[q]] + count[wv][e[q]] + rank[q] : -1;
    if (i < n) position[i] = at;
    if (e[q] >= 0) order[at] = (int32_t)i;
  }
}

// counts[b * E + e]: block b's entries of expert e
__global__ __launch_bounds__(kSortThreads) void k_sort_count(const int32_t *experts, SortShape s, int E,
                                                             int32_t *counts) {
  __shared__ int32_t hist[SVT_MAX_EXPERTS];
  const int tid = threadIdx.x;
  const int64_t b0 = blockIdx.x * s.per_block, b1 = b0 + s.per_block < s.n ? b0 + s.per_block : s.n;
  for (int e = tid; e < E; e += kSortThreads) hist[e] = 0;
  __syncthreads();
  for (int64_t i0 = b0; i0 < b1; i0 += kTileEntries) {
    int e[kSortSteps];
#pragma unroll
    for (int q = 0; q < kSortSteps; ++q) e[q] = load_expert(experts, i0 + q * kSortThreads + tid, b1, E);
#pragma unroll
    for (int q = 0; q < kSortSteps; ++q)
      if (e[q] >= 0) atomicAdd(&hist[e[q]], 1);
  }
  __syncthreads();
  for (int e = tid; e < E; e += kSortThreads) counts[(int64_t)blockIdx.x * E + e] = hist[e];
}

template <int BITS>
__global__ __launch_bounds__(kSortThreads) void k_sort_place(const int32_t *experts, SortShape s, int E,
                                                             const int32_t *counts, int32_t *offsets, int32_t *order,
                                                             int32_t *position) {
  __shared__ int32_t count[kSortWaves][SVT_MAX_EXPERTS];
  __shared__ int32_t total[SVT_MAX_EXPERTS], start[SVT_MAX_EXPERTS + 1];
  __shared__ int32_t next[SVT_MAX_EXPERTS];   // the row of the block's next entry of each expert
  __shared__ int32_t entry[kTileEntries];
  __shared__ uint16_t owner[kTileEntries];
  const int tid = threadIdx.x, wv = tid / 64, b = blockIdx.x;
  const int64_t b0 = b * s.per_block, b1 = b0 + s.per_block < s.n ? b0 + s.per_block : s.n;
  const int64_t in_tile = wv * (64 * kSortSteps) + tid % 64;
  int e[kSortSteps], rank[kSortSteps];
#pragma unroll
  for (int q = 0; q < kSortSteps; ++q) e[q] = load_expert(experts, b0 + in_tile + 64 * q, b1, E);
  for (int i = tid; i < E; i += kSortThreads) total[i] = next[i] = 0;
  __syncthreads();
  {   // every expert's total and its entries in the blocks before, 2^k threads along the experts
    int along = 64;
    while (along < E) along *= 2;
    const int i = tid % along;
    int sum = 0, before = 0;
    const int step = kSortThreads / along;
    if (i < E)
      for (int r0 = tid / along; r0 < s.blocks; r0 += 8 * step) {   // 8 loads in flight
        int c[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const int r = r0 + q * step;
          c[q] = counts[(int64_t)(r < s.blocks ? r : r0) * E + i];
        }
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const int r = r0 + q * step;
          sum += r < s.blocks ? c[q] : 0;
          before += r < b ? c[q] : 0;
        }
      }
    if (i < E && sum) {
      atomicAdd(&total[i], sum);
      atomicAdd(&next[i], before);
    }
  }
  __syncthreads();
  scan_experts(total, start, E);
  __syncthreads();
  for (int i = tid; i < E; i += kSortThreads) next[i] += start[i];
  if (b == 0)
    for (int i = tid; i <= E; i += kSortThreads) offsets[i] = start[i];
  for (int64_t i = b0 + tid; i < b1; i += kSortThreads)
    if (i >= start[E]) order[i] = -1;
  for (int64_t t0 = b0; t0 < b1; t0 += kTileEntries) {
    if (t0 != b0) {
#pragma unroll
      for (int q = 0; q < kSortSteps; ++q) e[q] = load_expert(experts, t0 + in_tile + 64 * q, b1, E);
    }
    for (int i = tid % 64; i < E; i += 64) count[wv][i] = 0;
    rank_entries<kSortSteps, BITS>(e, rank, count[wv]);
    __syncthreads();   // also: start has been read
    sum_waves(count, total, E);
    __syncthreads();
    scan_experts(total, start, E);
    __syncthreads();
#pragma unroll
    for (int q = 0; q < kSortSteps; ++q) {
      const int64_t i = t0 + in_tile + 64 * q;
      int at = -1;
      if (e[q] >= 0) {
        const int in = count[wv][e[q]] + rank[q];   // among the tile's entries of the expert
        at = next[e[q]] + in;
        entry[start[e[q]] + in] = (int32_t)i;
        owner[start[e[q]] + in] = (uint16_t)e[q];
      }
      if (i < b1) position[i] = at;
    }
    __syncthreads();
    for (int p = tid; p < start[E]; p += kSortThreads) {
      const int o = owner[p];
      order[next[o] + p - start[o]] = entry[p];
    }
    __syncthreads();
    for (int i = tid; i < E; i += kSortThreads) next[i] += total[i];   // read again behind a barrier
  }
}

// f of enough bits for an expert's number as a constant
template <class F>
int with_bits(int E, F f) {
  if (E <= 8) return f(std::integral_constant<int, 3>{});
  if (E <= 64) return f(std::integral_constant<int, 6>{});
  return f(std::integral_constant<int, 9>{});
}

// ---- exchange ------------------------------------------------------------------------------------

// Bound by memory (a copy runs at 5.1 TB/s).  65536 x 1024 bfloat16 rows, top 2: sort, dispatch and combine together
// 168 us, 14 of them the sort's (5.2 TB/s); 32768 tokens, top 4: both gradients 184 us (5.1 TB/s).

constexpr int kExThreads = 256;
constexpr int64_t kExMaxBlocks = 1 << 20;
constexpr int32_t kMaxWidth = 1 << 24;

// V bytes of a row, moved by one load or store
template <int V> struct Bytes { typedef uint32_t type __attribute__((ext_vector_type(V / 4))); };
template <> struct Bytes<4> { typedef uint32_t type; };
template <> struct Bytes<2> { typedef uint16_t type; };

template <class T, int V>
struct Lanes {   // V bytes as float32 values
  static constexpr int n = V / (int)sizeof(T);
  float v[n];
  __device__ __forceinline__ explicit Lanes(typename Bytes<V>::type raw) {
    struct S { T t[n]; };
    const S s = __builtin_bit_cast(S, raw);
#pragma unroll
    for (int i = 0; i < n; ++i) v[i] = (float)s.t[i];
  }
  __device__ __forceinline__ Lanes() {
#pragma unroll
    for (int i = 0; i < n; ++i) v[i] = 0.f;
  }
  // rounded once to T
  __device__ __forceinline__ typename Bytes<V>::type raw() const {
    struct S { T t[n]; } s;
#pragma unroll
    for (int i = 0; i < n; ++i) s.t[i] = (T)v[i];
    return __builtin_bit_cast(typename Bytes<V>::type, s);
  }
};

struct ExArgs {
  int64_t n_tokens;
  int64_t n_rows;          // n_tokens * top: positions outside [0, n_rows) are skipped
  int32_t top;
  int32_t chunks;          // V-byte pieces of a row
  int32_t lanes;           // lanes that share a token: a power of two, at most 64
  const int32_t *position;
};

__device__ __forceinline__ int64_t row_at(const ExArgs &a, int64_t t, int j) {
  const int32_t p = j < a.top ? a.position[t * a.top + j] : -1;
  return (uint32_t)p < (uint64_t)a.n_rows ? p : -1;
}

// A thread takes two pieces of a row at a time, `lanes` apart, so that twice the loads are in flight.  The
// experts' rows are read once, so their loads are marked as such: 65536 x 1024 bfloat16 rows, top 2, sort,
// dispatch and combine 173 -> 168 us.
template <int V>
__global__ __launch_bounds__(kExThreads) void k_dispatch(ExArgs a, const typename Bytes<V>::type *x,
                                                         typename Bytes<V>::type *rows) {
  const int in = threadIdx.x % a.lanes;
  const int64_t per = kExThreads / a.lanes;
  for (int64_t t = blockIdx.x * per + threadIdx.x / a.lanes; t < a.n_tokens; t += gridDim.x * per)
    for (int c = in; c < a.chunks; c += 2 * a.lanes) {
      const bool two = c + a.lanes < a.chunks;
      const auto v = x[t * a.chunks + c], w = x[t * a.chunks + (two ? c + a.lanes : c)];
      for (int j = 0; j < a.top; ++j) {
        const int64_t p = row_at(a, t, j);
        if (p >= 0) {
          rows[p * a.chunks + c] = v;
          if (two) rows[p * a.chunks + c + a.lanes] = w;
        }
      }
    }
}

// y[t] = sum_j w[t][j] rows[position[t][j]] (weights NULL: every w is 1), J rows in flight together
template <class T, int V, int J>
__global__ __launch_bounds__(kExThreads) void k_combine(ExArgs a, const typename Bytes<V>::type *rows,
                                                        const float *weights, typename Bytes<V>::type *y) {
  using L = Lanes<T, V>;
  const int in = threadIdx.x % a.lanes;
  const int64_t per = kExThreads / a.lanes;
  for (int64_t t = blockIdx.x * per + threadIdx.x / a.lanes; t < a.n_tokens; t += gridDim.x * per)
    for (int c = in; c < a.chunks; c += 2 * a.lanes) {
      const bool two = c + a.lanes < a.chunks;
      L sum[2];
      for (int j0 = 0; j0 < a.top; j0 += J) {
        int64_t p[J];
        float w[J];
        typename Bytes<V>::type r[J][2];
#pragma unroll
        for (int j = 0; j < J; ++j) {
          p[j] = row_at(a, t, j0 + j);
          w[j] = weights && j0 + j < a.top ? weights[t * a.top + j0 + j] : 1.f;
        }
#pragma unroll
        for (int j = 0; j < J; ++j)
          if (p[j] >= 0) {
            r[j][0] = __builtin_nontemporal_load(&rows[p[j] * a.chunks + c]);
            r[j][1] = __builtin_nontemporal_load(&rows[p[j] * a.chunks + (two ? c + a.lanes : c)]);
          }
#pragma unroll
        for (int j = 0; j < J; ++j)
          if (p[j] >= 0) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const L v(r[j][h]);
#pragma unroll
              for (int i = 0; i < L::n; ++i) sum[h].v[i] = fmaf(w[j], v.v[i], sum[h].v[i]);
            }
          }
      }
      y[t * a.chunks + c] = sum[0].raw();
      if (two) y[t * a.chunks + c + a.lanes] = sum[1].raw();
    }
}

// d_rows[position[t][j]] = w[t][j] dy[t];  d_weights[t][j] = dy[t] . rows[position[t][j]] (0 for a dropped
// entry).  A lane sums each piece's products, kDotPieces pieces' sums, and those; then the token's lanes add theirs up.
// So no chain of additions is longer than 512 (one over a lane's whole share of 2^24 values would be 2^18), and a
// d_weight is off by at most (8 + 512 + 512 + 6) u of sum |dy r|, u = 2^-24.
constexpr int kDotPieces = 512;
template <class T, int V, int J>
__global__ __launch_bounds__(kExThreads) void k_combine_backward(ExArgs a, const typename Bytes<V>::type *dy,
                                                                 const typename Bytes<V>::type *rows,
                                                                 const float *weights,
                                                                 typename Bytes<V>::type *d_rows, float *d_weights) {
  using L = Lanes<T, V>;
  const int in = threadIdx.x % a.lanes;
  const int64_t per = kExThreads / a.lanes;
  for (int64_t t0 = blockIdx.x * per; t0 < a.n_tokens; t0 += gridDim.x * per) {
    const int64_t t = t0 + threadIdx.x / a.lanes;   // the group sums below need every lane
    const bool live = t < a.n_tokens;
    for (int j0 = 0; j0 < a.top; j0 += J) {
      int64_t p[J];
      float w[J], dot[J];
#pragma unroll
      for (int j = 0; j < J; ++j) {
        p[j] = live ? row_at(a, t, j0 + j) : -1;
        w[j] = live && j0 + j < a.top ? weights[t * a.top + j0 + j] : 0.f;
        dot[j] = 0.f;
      }
      for (int c0 = in; live && c0 < a.chunks; c0 += kDotPieces * a.lanes) {
        float part[J];
#pragma unroll
        for (int j = 0; j < J; ++j) part[j] = 0.f;
        const int end = a.chunks - c0 < kDotPieces * a.lanes ? a.chunks : c0 + kDotPieces * a.lanes;
        for (int c = c0; c < end; c += 2 * a.lanes) {
          const bool two = c + a.lanes < a.chunks;
          const int c2 = two ? c + a.lanes : c;
          const L g0(dy[t * a.chunks + c]), g1(dy[t * a.chunks + c2]);
          typename Bytes<V>::type r[J][2];
#pragma unroll
          for (int j = 0; j < J; ++j)
            if (p[j] >= 0) {
              r[j][0] = __builtin_nontemporal_load(&rows[p[j] * a.chunks + c]);
              r[j][1] = __builtin_nontemporal_load(&rows[p[j] * a.chunks + c2]);
            }
#pragma unroll
          for (int j = 0; j < J; ++j)
            if (p[j] >= 0) {
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                if (h == 1 && !two) break;
                const L &g = h ? g1 : g0;
                const L v(r[j][h]);
                L d;
                float sum = 0.f;
#pragma unroll
                for (int i = 0; i < L::n; ++i) {
                  sum = fmaf(g.v[i], v.v[i], sum);
                  d.v[i] = w[j] * g.v[i];
                }
                part[j] += sum;
                d_rows[p[j] * a.chunks + (h ? c2 : c)] = d.raw();
              }
            }
        }
#pragma unroll
        for (int j = 0; j < J; ++j) dot[j] += part[j];
      }
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const float s = group_add(dot[j], a.lanes);
        if (live && in == 0 && j0 + j < a.top) d_weights[t * a.top + j0 + j] = s;
      }
    }
  }
}

// ---- host ----------------------------------------------------------------------------------------

int check_shape(const char *who, int32_t n_tokens, int32_t top, int32_t width, int32_t dtype) {
  if (n_tokens < 0) return report(SVT_EINVAL, "%s: n_tokens %d < 0", who, n_tokens);
  if (top < 1 || top > SVT_MAX_TOP) return report(SVT_EINVAL, "%s: top %d out of [1, %d]", who, top, SVT_MAX_TOP);
  if ((int64_t)n_tokens * top > kMaxEntries)
    return report(SVT_EINVAL, "%s: %lld entries, more than 2^30", who, (long long)n_tokens * top);
  if (width < 1 || width > kMaxWidth) return report(SVT_EINVAL, "%s: width %d out of [1, %d]", who, width, kMaxWidth);
  if (!elem_size(dtype)) return report(SVT_EINVAL, "%s: unknown element type %d", who, dtype);
  return SVT_OK;
}

// the widest piece (16, 8, 4 or 2 bytes) that divides a row and every pointer's address
int piece(int32_t width, int b, std::initializer_list<const void *> ptrs) {
  uintptr_t bits = (uintptr_t)width * b;
  for (const void *p : ptrs) bits |= (uintptr_t)p;
  return (bits & 15) == 0 ? 16 : (bits & 7) == 0 ? 8 : (bits & 3) == 0 ? 4 : 2;
}

ExArgs ex_args(int32_t n_tokens, int32_t top, int32_t width, int b, int v, const int32_t *position) {
  ExArgs a{n_tokens, (int64_t)n_tokens * top, top, (int32_t)((int64_t)width * b / v), 1, position};
  while (a.lanes < 64 && a.lanes < a.chunks) a.lanes *= 2;
  return a;
}

unsigned ex_grid(const ExArgs &a) {
  const int64_t per = kExThreads / a.lanes, n = (a.n_tokens + per - 1) / per;
  return (unsigned)(n < kExMaxBlocks ? n : kExMaxBlocks);
}

// f of the piece size as a constant; T's own size is the least
template <class T, class F>
int with_piece(int v, F f) {
  if (v == 16) return f(std::integral_constant<int, 16>{});
  if (v == 8) return f(std::integral_constant<int, 8>{});
  if constexpr (sizeof(T) <= 2)
    if (v == 2) return f(std::integral_constant<int, 2>{});
  return f(std::integral_constant<int, 4>{});
}

// f of the number of rows in flight for `top` as a constant
template <class F>
int with_batch(int top, F f) {
  if (top == 1) return f(std::integral_constant<int, 1>{});
  if (top == 2) return f(std::integral_constant<int, 2>{});
  return f(std::integral_constant<int, 4>{});
}

int combine(const char *who, int32_t n_tokens, int32_t top, int32_t width, int32_t dtype, const void *rows,
            const int32_t *position, const float *weights, void *y, void *hip_stream) {
  int rc = check_shape(who, n_tokens, top, width, dtype);
  if (rc != SVT_OK || n_tokens == 0) return rc;
  if (!rows || !position || !y) return report(SVT_EINVAL, "%s: NULL input or output", who);
  const int b = elem_size(dtype);
  if (misaligned(rows, b) || misaligned(y, b) || misaligned(position, 4) || misaligned(weights, 4))
    return report(SVT_EINVAL, "%s: misaligned input or output", who);
  const size_t nt = (size_t)n_tokens * width * b, nk = (size_t)n_tokens * top * 4;
  if (overlap(y, nt, rows, nt * top) || overlap(y, nt, position, nk) || overlap(y, nt, weights, nk))
    return report(SVT_EINVAL, "%s: the output overlaps an input", who);
  const int v = piece(width, b, {rows, y});
  const ExArgs a = ex_args(n_tokens, top, width, b, v, position);
  return with_type(dtype, [&](auto ty) {
    using T = decltype(ty);
    return with_piece<T>(v, [&](auto pv) {
      return with_batch(top, [&](auto batch) {
        constexpr int V = decltype(pv)::value;
        using B = typename Bytes<V>::type;
        return launch(who, k_combine<T, V, decltype(batch)::value>, ex_grid(a), kExThreads, 0, hip_stream, a,
                      (const B *)rows, weights, (B *)y);
      });
    });
  });
}

}  // namespace

}  // namespace svt

using namespace svt;

static int check_sort(const char *who, int32_t n_tokens, int32_t top, int32_t n_experts) {
  const int rc = check_shape(who, n_tokens, top, 1, SVT_F32);
  if (rc != SVT_OK) return rc;
  if (n_experts < 1 || n_experts > SVT_MAX_EXPERTS)
    return report(SVT_EINVAL, "%s: n_experts %d out of [1, %d]", who, n_experts, SVT_MAX_EXPERTS);
  return SVT_OK;
}

static size_t sort_bytes(int64_t n, int32_t n_experts) {
  return n <= kOneEntries ? 0 : (size_t)sort_shape(n, n_experts).blocks * n_experts * 4;
}

extern "C" size_t svt_expert_sort_workspace_size(int32_t n_tokens, int32_t top, int32_t n_experts) {
  (void)report(SVT_OK, "%s", "");
  if (check_sort("svt_expert_sort_workspace_size", n_tokens, top, n_experts) != SVT_OK) return 0;
  return sort_bytes((int64_t)n_tokens * top, n_experts);
}

extern "C" int svt_expert_sort(int32_t n_tokens, int32_t top, int32_t n_experts, const int32_t *experts,
                               int32_t *offsets, int32_t *order, int32_t *position, void *workspace,
                               size_t workspace_bytes, void *hip_stream) {
  const char *who = "svt_expert_sort";
  (void)report(SVT_OK, "%s", "");
  const int rc = check_sort(who, n_tokens, top, n_experts);
  if (rc != SVT_OK) return rc;
  const int64_t n = (int64_t)n_tokens * top;
  if (!offsets || (n > 0 && (!experts || !order || !position)))
    return report(SVT_EINVAL, "%s: NULL input or output", who);
  if (misaligned(experts, 4) || misaligned(offsets, 4) || misaligned(order, 4) || misaligned(position, 4) ||
      misaligned(workspace, 4))
    return report(SVT_EINVAL, "%s: misaligned input, output or workspace", who);
  const size_t need = sort_bytes(n, n_experts), ne = (size_t)n * 4, no = ((size_t)n_experts + 1) * 4;
  if (need > 0 && (!workspace || workspace_bytes < need))
    return report(SVT_EINVAL, "%s: workspace of %zu bytes, needs %zu", who, workspace ? workspace_bytes : (size_t)0, need);
  const void *at[5] = {experts, offsets, order, position, workspace};
  const size_t bytes[5] = {ne, no, ne, ne, need};
  for (int i = 0; i < 5; ++i)
    for (int j = 0; j < i; ++j)
      if (overlap(at[i], bytes[i], at[j], bytes[j]))
        return report(SVT_EINVAL, "%s: input, outputs and workspace overlap", who);
  return with_bits(n_experts, [&](auto bits) {
    constexpr int B = decltype(bits)::value;
    auto one = [&](auto steps) {
      return launch(who, k_sort_one<decltype(steps)::value, B>, 1, kSortThreads, 0, hip_stream, experts, n, n_experts,
                    offsets, order, position);
    };
    if (n <= kSortThreads) return one(std::integral_constant<int, 1>{});
    if (n <= 4 * kSortThreads) return one(std::integral_constant<int, 4>{});
    if (n <= kOneEntries) return one(std::integral_constant<int, 8>{});
    const SortShape sh = sort_shape(n, n_experts);
    const int counted = launch(who, k_sort_count, sh.blocks, kSortThreads, 0, hip_stream, experts, sh, n_experts,
                               (int32_t *)workspace);
    if (counted != SVT_OK) return counted;   // the second kernel writes where the counts say
    return launch(who, k_sort_place<B>, sh.blocks, kSortThreads, 0, hip_stream, experts, sh, n_experts,
                  (const int32_t *)workspace, offsets, order, position);
  });
}

extern "C" int svt_expert_dispatch(int32_t n_tokens, int32_t top, int32_t width, int32_t dtype, const void *x,
                                   const int32_t *position, void *rows, void *hip_stream) {
  const char *who = "svt_expert_dispatch";
  (void)report(SVT_OK, "%s", "");
  const int rc = check_shape(who, n_tokens, top, width, dtype);
  if (rc != SVT_OK || n_tokens == 0) return rc;
  if (!x || !position || !rows) return report(SVT_EINVAL, "%s: NULL input or output", who);
  const int b = elem_size(dtype);
  if (misaligned(x, b) || misaligned(rows, b) || misaligned(position, 4))
    return report(SVT_EINVAL, "%s: misaligned input or output", who);
  const size_t nt = (size_t)n_tokens * width * b, nk = (size_t)n_tokens * top * 4;
  if (overlap(rows, nt * top, x, nt) || overlap(rows, nt * top, position, nk))
    return report(SVT_EINVAL, "%s: the output overlaps an input", who);
  const int v = piece(width, b, {x, rows});
  const ExArgs a = ex_args(n_tokens, top, width, b, v, position);
  return with_piece<uint16_t>(v, [&](auto pv) {
    constexpr int V = decltype(pv)::value;
    using B = typename Bytes<V>::type;
    return launch(who, k_dispatch<V>, ex_grid(a), kExThreads, 0, hip_stream, a, (const B *)x, (B *)rows);
  });
}

extern "C" int svt_expert_dispatch_backward(int32_t n_tokens, int32_t top, int32_t width, int32_t dtype,
                                            const void *d_rows, const int32_t *position, void *dx, void *hip_stream) {
  (void)report(SVT_OK, "%s", "");
  return combine("svt_expert_dispatch_backward", n_tokens, top, width, dtype, d_rows, position, nullptr, dx, hip_stream);
}

extern "C" int svt_expert_combine(int32_t n_tokens, int32_t top, int32_t width, int32_t dtype, const void *rows,
                                  const int32_t *position, const float *weights, void *y, void *hip_stream) {
  (void)report(SVT_OK, "%s", "");
  return combine("svt_expert_combine", n_tokens, top, width, dtype, rows, position, weights, y, hip_stream);
}

extern "C" int svt_expert_combine_backward(int32_t n_tokens, int32_t top, int32_t width, int32_t dtype, const void *dy,
                                           const void *rows, const int32_t *position, const float *weights,
                                           void *d_rows, float *d_weights, void *hip_stream) {
  const char *who = "svt_expert_combine_backward";
  (void)report(SVT_OK, "%s", "");
  const int rc = check_shape(who, n_tokens, top, width, dtype);
  if (rc != SVT_OK || n_tokens == 0) return rc;
  if (!dy || !rows || !position || !weights || !d_rows || !d_weights)
    return report(SVT_EINVAL, "%s: NULL input or output", who);
  const int b = elem_size(dtype);
  if (misaligned(dy, b) || misaligned(rows, b) || misaligned(d_rows, b) || misaligned(position, 4) ||
      misaligned(weights, 4) || misaligned(d_weights, 4))
    return report(SVT_EINVAL, "%s: misaligned input or output", who);
  const size_t nt = (size_t)n_tokens * width * b, nk = (size_t)n_tokens * top * 4;
  const void *in[4] = {dy, rows, position, weights};
  const size_t in_bytes[4] = {nt, nt * top, nk, nk};
  for (int i = 0; i < 4; ++i)
    if (overlap(d_rows, nt * top, in[i], in_bytes[i]) || overlap(d_weights, nk, in[i], in_bytes[i]))
      return report(SVT_EINVAL, "%s: an output overlaps an input", who);
  if (overlap(d_rows, nt * top, d_weights, nk)) return report(SVT_EINVAL, "%s: the outputs overlap", who);
  const int v = piece(width, b, {dy, rows, d_rows});
  const ExArgs a = ex_args(n_tokens, top, width, b, v, position);
  return with_type(dtype, [&](auto ty) {
    using T = decltype(ty);
    return with_piece<T>(v, [&](auto pv) {
      return with_batch(top, [&](auto batch) {
        constexpr int V = decltype(pv)::value;
        using B = typename Bytes<V>::type;
        return launch(who, k_combine_backward<T, V, decltype(batch)::value>, ex_grid(a), kExThreads, 0, hip_stream, a,
                      (const B *)dy, (const B *)rows, weights, (B *)d_rows, d_weights);
      });
    });
  });
}

// svt_embedding.hip - rows of a table for tokens, scaled, and the gradient in the table, on gfx950.
//
//   out[i] = scale table[ids[i]]   (zeros outside the table)
//   d_table[v] = scale sum_{i: ids[i] = v} d_out[i]
//
// The lookup moves every byte once and is bound by memory.  The gradient sorts the tokens (stable, so that a row's
// sum has one order), then walks the sorted list: a chunk of consecutive places belongs to a group of lanes, which
// adds up the runs of equal tokens in registers and writes each finished row once.  Only runs that cross a chunk's
// border leave partial sums, which one more launch joins in order, 256 columns of a run by one workgroup.  Rows that no
// token names are cleared by workgroups of their own in the launch that adds, which keeps the table's writes beside the
// gradient's reads.
//
// Measured, each kernel's average over inputs in turn: rows for 65536 tokens of 1024 bfloat16 41 us (176 MB, 4.3 TB/s; 34 at
// best), for 2048 of 128 float16 2.6.  The gradient in 131072 rows of the former 118: the sort 25 (a chain of four launches),
// sums and zeros 80 (403 MB, 5 TB/s), the join 14; of 3001 tokens of 250 float32 in 5003 rows 21: 8, 6 and 7, chains of
// dependent loads all three.  Tokens that all name one row make the join's run long: the former 149 and the latter 31; 16
// rows for all 187 and 19.  Added to a float32 table instead of zeros elsewhere, the former takes 111.

#include <type_traits>

#include "../experts/svt_experts.h"

namespace svt {

namespace {

constexpr int kThreads = 256;
constexpr int64_t kMaxTokens = int64_t(1) << 30, kMaxRows = (int64_t(1) << 31) - 2;
constexpr int32_t kMaxWidth = 1 << 24;

// M neighbouring elements, moved by one load or store (two where they take 32 bytes)
template <class T, int M>
struct alignas(M * sizeof(T) < 16 ? M * sizeof(T) : 16) Vec { T v[M]; };

// the same past the caches, for what is touched once: 16-byte pieces only, others as ever
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
template <class T, int M>
__device__ __forceinline__ Vec<T, M> load_once(const Vec<T, M> *p) {
  if constexpr (sizeof(Vec<T, M>) == 16) return __builtin_bit_cast(Vec<T, M>, __builtin_nontemporal_load((const u32x4 *)p));
  else return *p;
}
template <class T, int M>
__device__ __forceinline__ void clear_once(Vec<T, M> *p) {
  if constexpr (sizeof(Vec<T, M>) == 16) __builtin_nontemporal_store(u32x4{0u, 0u, 0u, 0u}, (u32x4 *)p);
  else *p = Vec<T, M>{};
}

// ---- lookup --------------------------------------------------------------------------------------

struct LookupArgs {
  int64_t n_tokens, n_rows;
  int32_t pieces;      // of a row
  int32_t lanes;       // that share a token: a power of two
  const int64_t *ids;
  float scale;
};

// A thread takes two pieces of a row, `lanes` apart
template <class T, int M>
__global__ __launch_bounds__(kThreads) void k_lookup(LookupArgs a, const Vec<T, M> *table, Vec<T, M> *out) {
  const int in = threadIdx.x % a.lanes;
  const int64_t per = kThreads / a.lanes;
  for (int64_t t = blockIdx.x * per + threadIdx.x / a.lanes; t < a.n_tokens; t += gridDim.x * per) {
    const int64_t id = a.ids[t];
    const bool there = (uint64_t)id < (uint64_t)a.n_rows;
    const Vec<T, M> *row = table + (there ? id : 0) * a.pieces;
    for (int c = blockIdx.y * 2 * a.lanes + in; c < a.pieces; c += gridDim.y * 2 * a.lanes) {
      const bool two = c + a.lanes < a.pieces;
      Vec<T, M> v{}, w{};
      if (there) {
        v = row[c];
        w = row[two ? c + a.lanes : c];
#pragma unroll
        for (int i = 0; i < M; ++i) {
          v.v[i] = (T)(a.scale * (float)v.v[i]);
          w.v[i] = (T)(a.scale * (float)w.v[i]);
        }
      }
      out[t * a.pieces + c] = v;
      if (two) out[t * a.pieces + c + a.lanes] = w;
    }
  }
}

// ---- sort ----------------------------------------------------------------------------------------
//
// Tokens by row, stable: a radix sort from the low digit up, up to 10 bits a digit.  Tokens outside the table get the
// key n_rows and so lie behind all others.  Ranks within a wave's piece come from ballots, as the experts' sort has
// them.  Up to kOneTokens one workgroup sorts in LDS; above that each digit takes two launches, a histogram per block
// and a placing pass that orders a tile in LDS and writes each digit's run in one piece.

constexpr int kSortThreads = 1024, kSortWaves = kSortThreads / 64;
constexpr int kMostBits = 10, kMostBins = 1 << kMostBits;
constexpr int kSteps = 4;   // tokens of a thread at a time, at most
constexpr int kOneSteps = 8;
constexpr int64_t kOneTokens = kOneSteps * kSortThreads;
constexpr int kMostCounts = 1 << 17;                       // every block reads the whole table of histograms
static_assert(kMostBins <= kSortThreads, "a thread for every bin");

struct SortShape {
  int64_t n, n_rows;
  int32_t passes, bits;                // bits a digit
  int32_t blocks;
  int32_t steps;                       // tokens of a thread at a time: 1 or kSteps
  int64_t per_block;                   // a multiple of steps times the threads
};

__device__ __forceinline__ uint32_t key_of(int64_t id, int64_t n_rows) {
  return (uint32_t)((uint64_t)id < (uint64_t)n_rows ? id : n_rows);
}

// exclusive sums over the bins, one a thread; every thread of the workgroup takes part.  `waves`: LDS, one a wave
__device__ __forceinline__ int scan_bins(int v, int32_t *waves) {
  const int incl = incl_sums(v), w = threadIdx.x / 64;
  if (lane_id() == 63) waves[w] = incl;
  __syncthreads();
  int before = 0;
#pragma unroll
  for (int i = 0; i < kSortWaves; ++i) before += i < w ? waves[i] : 0;
  return before + incl - v;
}

// count[w][bin] become exclusive sums over the waves; the bin's total is returned to its thread
__device__ __forceinline__ int sum_waves(int32_t (*count)[kMostBins], int bins) {
  int sum = 0;
  if ((int)threadIdx.x < bins) {
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) {
      const int c = count[w][threadIdx.x];
      count[w][threadIdx.x] = sum;
      sum += c;
    }
  }
  return sum;
}

template <int STEPS, int BITS>
__global__ __launch_bounds__(kSortThreads) void k_sort_tokens(const int64_t *ids, SortShape s, uint32_t *keys,
                                                              int32_t *order, int32_t *crossing) {
  __shared__ int32_t count[kSortWaves][kMostBins];
  __shared__ int32_t start[kMostBins], waves[kSortWaves];
  __shared__ uint32_t key[STEPS * kSortThreads];
  __shared__ uint16_t at[STEPS * kSortThreads];
  const int tid = threadIdx.x, wv = tid / 64, n = (int)s.n, bins = 1 << s.bits;
  const int i0 = wv * (64 * STEPS) + tid % 64;
  uint32_t k[STEPS];
  int from[STEPS];
#pragma unroll
  for (int q = 0; q < STEPS; ++q) {
    const int i = i0 + 64 * q;
    k[q] = key_of(ids[i < n ? i : n - 1], s.n_rows);
    from[q] = i;
  }
  if (tid == 0) *crossing = 0;
  for (int p = 0; p < s.passes; ++p) {
    int e[STEPS], rank[STEPS];
#pragma unroll
    for (int q = 0; q < STEPS; ++q) e[q] = i0 + 64 * q < n ? (int)((k[q] >> (p * s.bits)) & (uint32_t)(bins - 1)) : -1;
    for (int i = tid % 64; i < bins; i += 64) count[wv][i] = 0;   // its own wave's: no barrier needed
    rank_entries<STEPS, BITS>(e, rank, count[wv]);
    __syncthreads();
    const int total = sum_waves(count, bins);
    const int first = scan_bins(total, waves);
    if (tid < bins) start[tid] = first;
    __syncthreads();
    const bool last = p + 1 == s.passes;
#pragma unroll
    for (int q = 0; q < STEPS; ++q)
      if (e[q] >= 0) {
        const int to = start[e[q]] + count[wv][e[q]] + rank[q];
        if (last) {
          keys[to] = k[q];
          order[to] = from[q];
        } else {
          key[to] = k[q];
          at[to] = (uint16_t)from[q];
        }
      }
    if (last) break;
    __syncthreads();
#pragma unroll
    for (int q = 0; q < STEPS; ++q) {
      const int i = i0 + 64 * q;
      k[q] = key[i < n ? i : 0];
      from[q] = at[i < n ? i : 0];
    }
  }
}

// one digit of a token: from the ids in the first pass, later from the keys
struct Digits {
  const int64_t *ids;     // NULL after the first pass
  const uint32_t *keys;
  const int32_t *order;
  int shift;
};

__device__ __forceinline__ uint32_t load_key(const Digits &d, const SortShape &s, int64_t i) {
  return d.ids ? key_of(d.ids[i], s.n_rows) : d.keys[i];
}

template <int STEPS>
__global__ __launch_bounds__(kSortThreads) void k_sort_count(Digits d, SortShape s, int32_t *counts, int32_t *crossing) {
  __shared__ int32_t hist[kMostBins];
  const int tid = threadIdx.x, bins = 1 << s.bits;
  const int64_t b0 = blockIdx.x * s.per_block, b1 = b0 + s.per_block < s.n ? b0 + s.per_block : s.n;
  if (blockIdx.x == 0 && tid == 0) *crossing = 0;
  if (tid < bins) hist[tid] = 0;
  __syncthreads();
  for (int64_t i0 = b0; i0 < b1; i0 += STEPS * kSortThreads) {
    uint32_t k[STEPS];
#pragma unroll
    for (int q = 0; q < STEPS; ++q) {
      const int64_t i = i0 + q * kSortThreads + tid;
      k[q] = load_key(d, s, i < b1 ? i : b1 - 1);
    }
#pragma unroll
    for (int q = 0; q < STEPS; ++q)
      if (i0 + q * kSortThreads + tid < b1) atomicAdd(&hist[(k[q] >> d.shift) & (uint32_t)(bins - 1)], 1);
  }
  __syncthreads();
  if (tid < bins) counts[(int64_t)blockIdx.x * bins + tid] = hist[tid];
}

template <int STEPS, int BITS>
__global__ __launch_bounds__(kSortThreads) void k_sort_place(Digits d, SortShape s, const int32_t *counts,
                                                             uint32_t *out_keys, int32_t *out_order) {
  __shared__ int32_t count[kSortWaves][kMostBins];
  __shared__ int32_t total[kMostBins], start[kMostBins], next[kMostBins], waves[kSortWaves];
  __shared__ uint32_t key[STEPS * kSortThreads];
  __shared__ int32_t at[STEPS * kSortThreads];
  const int tid = threadIdx.x, wv = tid / 64, b = blockIdx.x, bins = 1 << s.bits;
  const int64_t b0 = b * s.per_block, b1 = b0 + s.per_block < s.n ? b0 + s.per_block : s.n;
  const int in_tile = wv * (64 * STEPS) + tid % 64;
  uint32_t k[STEPS];
  int from[STEPS];
  auto load = [&](int64_t t0) {
#pragma unroll
    for (int q = 0; q < STEPS; ++q) {
      const int64_t i = t0 + in_tile + 64 * q, j = i < b1 ? i : b1 - 1;
      k[q] = load_key(d, s, j);
      from[q] = d.ids ? (int)j : d.order[j];
    }
  };
  load(b0);
  if (tid < bins) total[tid] = next[tid] = 0;
  __syncthreads();
  {   // every bin's total and its tokens in the blocks before, 2^k threads along the bins
    int along = 64;
    while (along < bins) along *= 2;
    const int i = tid % along, step = kSortThreads / along;
    int sum = 0, before = 0;
    if (i < bins)
      for (int r0 = tid / along; r0 < s.blocks; r0 += 8 * step) {   // 8 loads in flight
        int c[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const int r = r0 + q * step;
          c[q] = counts[(int64_t)(r < s.blocks ? r : r0) * bins + i];
        }
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const int r = r0 + q * step;
          sum += r < s.blocks ? c[q] : 0;
          before += r < b ? c[q] : 0;
        }
      }
    if (i < bins && sum) {
      atomicAdd(&total[i], sum);
      atomicAdd(&next[i], before);
    }
  }
  __syncthreads();
  {
    const int first = scan_bins(tid < bins ? total[tid] : 0, waves);
    if (tid < bins) next[tid] += first;
  }
  for (int64_t t0 = b0; t0 < b1; t0 += STEPS * kSortThreads) {
    if (t0 != b0) load(t0);
    int e[STEPS], rank[STEPS];
#pragma unroll
    for (int q = 0; q < STEPS; ++q)
      e[q] = t0 + in_tile + 64 * q < b1 ? (int)((k[q] >> d.shift) & (uint32_t)(bins - 1)) : -1;
    for (int i = tid % 64; i < bins; i += 64) count[wv][i] = 0;
    rank_entries<STEPS, BITS>(e, rank, count[wv]);
    __syncthreads();   // also: the scan's and the last tile's reads of LDS are done
    const int mine = sum_waves(count, bins);
    const int first = scan_bins(mine, waves);
    if (tid < bins) start[tid] = first;
    __syncthreads();
#pragma unroll
    for (int q = 0; q < STEPS; ++q)
      if (e[q] >= 0) {
        const int to = start[e[q]] + count[wv][e[q]] + rank[q];
        key[to] = k[q];
        at[to] = from[q];
      }
    __syncthreads();
    const int here = (int)(b1 - t0 < STEPS * kSortThreads ? b1 - t0 : STEPS * kSortThreads);
    for (int p = tid; p < here; p += kSortThreads) {
      const uint32_t v = key[p];
      const int o = (int)((v >> d.shift) & (uint32_t)(bins - 1));
      const int64_t to = (int64_t)next[o] + p - start[o];
      out_keys[to] = v;
      out_order[to] = at[p];
    }
    __syncthreads();
    if (tid < bins) next[tid] += mine;   // read again behind a barrier
  }
}

// ---- sums ----------------------------------------------------------------------------------------

struct SumArgs {
  int64_t n, n_rows;
  int32_t width, pieces;       // of a row
  int32_t lanes;               // that share a chunk: a power of two, at most 64
  int32_t column_blocks;       // of 2 lanes pieces
  int32_t per;                 // places of a chunk
  int32_t chunks;
  int64_t sum_blocks;          // workgroups that add; the others clear
  int32_t clear_rows;          // rows that one of the others looks after
  float scale;
  const uint32_t *keys;        // sorted
  const int32_t *order;
  float *partial;              // [chunk][2][width]: the run that came in, the run that goes on
  int32_t *crossing;           // [0]: their number; from [2] on, pairs: a chunk whose last run starts there and goes on, its key
};

struct Pair { int32_t chunk; uint32_t run; };

// First place in [0, n) whose key is at least v, n if there is none; the whole wave asks.  64 places are looked at a time: 3
// loads one after the other for 65536 tokens, where halving takes 16.
__device__ __forceinline__ int64_t first_place(const uint32_t *keys, int64_t n, uint64_t v) {
  int64_t lo = 0, hi = n;
  while (lo < hi) {
    const int64_t step = (hi - lo + 63) / 64, probe = lo + (lane_id() + 1) * step - 1;   // the last of the lane's piece
    const bool less = probe < hi && keys[probe < hi ? probe : lo] < v;
    lo += __builtin_popcountll(__ballot(less)) * step;
    hi = lo + step - 1 < hi ? lo + step - 1 : hi;
  }
  return lo;
}

constexpr int kClearMost = 4096;   // rows of a clearing workgroup at most

// zeros for the rows first .. that no token names
template <class TD, int M>
__device__ __forceinline__ void clear_rows(const SumArgs &a, int64_t first, Vec<TD, M> *table, uint32_t *named) {
  const int64_t end = first + a.clear_rows < a.n_rows ? first + a.clear_rows : a.n_rows;
  for (int i = threadIdx.x; i < kClearMost / 32; i += kThreads) named[i] = 0u;
  __syncthreads();
  const int64_t lo = first_place(a.keys, a.n, (uint64_t)first), hi = first_place(a.keys, a.n, (uint64_t)end);
  constexpr int64_t kLeap = 64 * kThreads;
  for (int64_t p = lo; p < hi; p += kThreads) {
    while (p + kLeap < hi && a.keys[p] == a.keys[p + kLeap]) p += kLeap;   // inside a long run
    if (p + threadIdx.x < hi) {
      const uint32_t r = a.keys[p + threadIdx.x] - (uint32_t)first;
      atomicOr(&named[r / 32], 1u << (r % 32));
    }
  }
  __syncthreads();
  const int in = threadIdx.x % a.lanes;
  for (int r = threadIdx.x / a.lanes; first + r < end; r += kThreads / a.lanes)
    if (!(named[r / 32] >> (r % 32) & 1u))
      for (int c = in; c < a.pieces; c += a.lanes) clear_once(&table[(first + r) * a.pieces + c]);
}

template <class TD, int M, bool ADD>
__device__ __forceinline__ void put_row(Vec<TD, M> *at, const float (&sum)[M], float scale) {
  Vec<TD, M> r;
  if (ADD) r = *at;
#pragma unroll
  for (int i = 0; i < M; ++i) r.v[i] = (TD)(ADD ? fmaf(scale, sum[i], (float)r.v[i]) : scale * sum[i]);
  *at = r;
}

// TWO: rows of more pieces than lanes; J: places in flight
template <class T, class TD, int M, bool ADD, bool TWO>
__global__ __launch_bounds__(kThreads) void k_sum_rows(SumArgs a, const Vec<T, M> *d_out, Vec<TD, M> *table) {
  __shared__ uint32_t named[ADD ? 1 : kClearMost / 32];
  if (const int64_t cleared = block_number() - a.sum_blocks; cleared >= 0) {
    const int64_t first = cleared * a.clear_rows;
    if (!ADD && first < a.n_rows) clear_rows<TD, M>(a, first, table, named);
    return;
  }
  constexpr int J = TWO ? 4 : 8;
  const int in = threadIdx.x % a.lanes;
  const int64_t unit = block_number() * (kThreads / a.lanes) + threadIdx.x / a.lanes;
  const int64_t chunk = unit / a.column_blocks;
  if (chunk >= a.chunks) return;
  const int block = (int)(unit - chunk * a.column_blocks);
  const int c = block * 2 * a.lanes + in;
  const bool one = c < a.pieces, two = TWO && c + a.lanes < a.pieces;
  const int c1 = one ? c : 0, c2 = two ? c + a.lanes : c1;
  const int64_t p0 = chunk * a.per, p1 = p0 + a.per < a.n ? p0 + a.per : a.n;
  const uint32_t none = (uint32_t)a.n_rows;
  uint32_t run = a.keys[p0];
  bool whole = p0 == 0 || a.keys[p0 - 1] != run;   // the run starts here
  float s1[M], s2[M];
#pragma unroll
  for (int i = 0; i < M; ++i) s1[i] = s2[i] = 0.f;
  auto leave = [&](bool ends) {
    if (run == none) return;
    if (whole && ends) {
      if (one) put_row<TD, M, ADD>(&table[(int64_t)run * a.pieces + c], s1, a.scale);
      if (two) put_row<TD, M, ADD>(&table[(int64_t)run * a.pieces + c + a.lanes], s2, a.scale);
    } else {
      float *to = a.partial + (chunk * 2 + (whole ? 1 : 0)) * a.width;
#pragma unroll
      for (int i = 0; i < M; ++i) {
        if (one) to[c1 * M + i] = s1[i];
        if (two) to[c2 * M + i] = s2[i];
      }
      if (whole && block == 0 && in == 0)
        reinterpret_cast<Pair *>(a.crossing)[1 + atomicAdd(a.crossing, 1)] = Pair{(int32_t)chunk, run};
    }
  };
  // the places after the next J are looked up while the next J's rows are on their way
  uint32_t k[J], k_next[J];
  int32_t o_next[J];
  Vec<T, M> v[J], w[J];
  auto look_up = [&](int64_t p) {
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int64_t q = p + j < p1 ? p + j : p1 - 1;
      k_next[j] = a.keys[q];
      o_next[j] = a.order[q];
    }
  };
  look_up(p0);
  for (int64_t p = p0; p < p1; p += J) {
#pragma unroll
    for (int j = 0; j < J; ++j) {
      k[j] = k_next[j];
      const int64_t row = (int64_t)o_next[j] * a.pieces;
      v[j] = load_once(&d_out[row + c1]);
      if (TWO) w[j] = load_once(&d_out[row + c2]);
    }
    look_up(p + J);
#pragma unroll
    for (int j = 0; j < J; ++j)
      if (p + j < p1) {
        if (k[j] != run) {
          leave(true);
          run = k[j];
          whole = true;
#pragma unroll
          for (int i = 0; i < M; ++i) s1[i] = s2[i] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < M; ++i) {
          s1[i] += (float)v[j].v[i];
          if (TWO) s2[i] += (float)w[j].v[i];
        }
      }
  }
  leave(p1 == a.n || a.keys[p1] != run);
}

// Sums of the runs that cross chunks, 256 columns of one at a time.  Most cross once or twice: a wave each.  Those of more
// than kJoinAlone chunks are put off until the workgroup's waves share them, each a contiguous part, added in order.
// (200000 tokens of 300 rows, chunks of 8: 117 us with four waves to every run, 47 like this.)  What a run needs is asked for
// together: the number of runs with its chunk and key, its length with its first two parts (3001 x 250 float32, the whole
// gradient 23.3 us one after the other, 20.6 like this).
constexpr int kJoinColumns = 256, kJoinThreads = 1024, kJoinWaves = kJoinThreads / 64, kJoinAlone = 16;

struct __attribute__((packed, aligned(4))) FourSums { float v[4]; };

// part i of a run that begins in a chunk (row 1 of the first, row 0 of the others), `left` columns from `from` on
__device__ __forceinline__ FourSums part(const float *from, int64_t i, int64_t width, int left) {
  const float *at = from + (i ? 2 * i : 1) * width;
  if (left >= 4) return *reinterpret_cast<const FourSums *>(at);
  FourSums v{};
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (k < left) v.v[k] = at[k];
  return v;
}

// parts i0 .. i1 - 1 are added to `sum`, in order
__device__ __forceinline__ void add_parts(FourSums &sum, const float *from, int64_t i0, int64_t i1, int64_t width, int left) {
  int64_t i = i0;
  if (left >= 4)
    for (; i + 8 <= i1; i += 8) {
      FourSums v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = part(from, i + j, width, left);
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k) sum.v[k] += v[j].v[k];
    }
  for (; i < i1; ++i) {
    const FourSums v = part(from, i, width, left);
#pragma unroll
    for (int k = 0; k < 4; ++k) sum.v[k] += v.v[k];
  }
}

template <class TD, bool ADD>
__global__ __launch_bounds__(kJoinThreads) void k_join_runs(SumArgs a, TD *table) {
  __shared__ FourSums parts[kJoinWaves][64];
  __shared__ int64_t put_off[kJoinWaves], length[kJoinWaves];
  const int columns = (a.width + kJoinColumns - 1) / kJoinColumns, wave = threadIdx.x / 64;
  const int64_t units = (int64_t)a.crossing[0] * columns;
  auto pair_of = [&](int64_t u) {
    return reinterpret_cast<const Pair *>(a.crossing)[1 + (u / columns < a.chunks ? u / columns : 0)];
  };
  auto column_of = [&](int64_t u) { return (int)(u % columns) * kJoinColumns + lane_id() * 4; };
  Pair mine = pair_of(blockIdx.x + (int64_t)wave * gridDim.x);   // beside the number of runs, so perhaps behind the last of them
  auto put = [&](const FourSums &sum, int col, uint32_t run) {
    TD *at = table + (int64_t)run * a.width + col;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (col + k < a.width) at[k] = (TD)(ADD ? fmaf(a.scale, sum.v[k], (float)at[k]) : a.scale * sum.v[k]);
  };
  // neighbouring runs go to different workgroups: the long ones among a few are spread
  for (int64_t u0 = blockIdx.x; u0 < units; u0 += (int64_t)gridDim.x * kJoinWaves) {
    const int64_t u = u0 + (int64_t)wave * gridDim.x;
    int64_t n = 0;   // chunks that the run lies in: where it begins, and those that begin with it
    if (u < units) {
      const int64_t chunk = mine.chunk;
      const uint32_t run = mine.run;
      const int col = column_of(u);
      const float *from = a.partial + chunk * 2 * a.width + col;
      const int left = a.width - col;
      const int64_t c = chunk + 1 + lane_id();
      const uint32_t key = a.keys[(c < a.chunks ? c : chunk) * a.per];
      // two there are in any case: on their way while the run's length is found
      FourSums sum = part(from, 0, a.width, left);
      const FourSums next = part(from, 1, a.width, left);
      const uint64_t goes_on = __ballot(c < a.chunks && key == run);
      n = ~goes_on ? 1 + __builtin_ctzll(~goes_on) : (first_place(a.keys, a.n, (uint64_t)run + 1) - 1) / a.per - chunk + 1;
      if (n <= kJoinAlone) {
#pragma unroll
        for (int k = 0; k < 4; ++k) sum.v[k] += next.v[k];
        add_parts(sum, from, 2, n, a.width, left);
        put(sum, col, run);
      }
    }
    if (lane_id() == 0) {
      put_off[wave] = n > kJoinAlone ? u : -1;
      length[wave] = n;
    }
    __syncthreads();
    for (int w = 0; w < kJoinWaves; ++w) {
      if (put_off[w] < 0) continue;   // the same for all
      const Pair p = pair_of(put_off[w]);
      const int col = column_of(put_off[w]);
      const int64_t each = (length[w] + kJoinWaves - 1) / kJoinWaves, i0 = wave * each;
      const int64_t i1 = i0 + each < length[w] ? i0 + each : length[w];
      FourSums sum{};
      add_parts(sum, a.partial + (int64_t)p.chunk * 2 * a.width + col, i0, i1, a.width, a.width - col);
      parts[wave][lane_id()] = sum;
      __syncthreads();
      if (wave == 0) {
#pragma unroll
        for (int j = 1; j < kJoinWaves; ++j)
#pragma unroll
          for (int k = 0; k < 4; ++k) sum.v[k] += parts[j][lane_id()].v[k];
        put(sum, col, p.run);
      }
      __syncthreads();
    }
    mine = pair_of(u + (int64_t)gridDim.x * kJoinWaves);
    __syncthreads();   // put_off has been read
  }
}

// ---- host ----------------------------------------------------------------------------------------

// M, the widest piece of a row: at most 16 bytes of T, and every array's rows aligned to it (d_table's to 16 bytes
// where a piece takes 32)
int piece_elems(int32_t width, int b, const void *x, int tb, const void *table) {
  for (int m = 16 / b; m > 1; m /= 2) {
    const int x_bytes = m * b, t_bytes = m * tb < 16 ? m * tb : 16;
    if (width % m == 0 && !misaligned(x, x_bytes) && !misaligned(table, t_bytes)) return m;
  }
  return 1;
}

template <class T, class F>
int with_elems(int m, F f) {
  if constexpr (sizeof(T) == 2)
    if (m == 8) return f(std::integral_constant<int, 8>{});
  if (m == 4) return f(std::integral_constant<int, 4>{});
  if (m == 2) return f(std::integral_constant<int, 2>{});
  return f(std::integral_constant<int, 1>{});
}

SortShape sort_shape(int64_t n, int64_t n_rows) {
  SortShape s{n, n_rows, 0, 0, 1, 1, 0};
  const int bits = 64 - __builtin_clzll((uint64_t)n_rows);   // of the key n_rows
  s.passes = (bits + kMostBits - 1) / kMostBits;
  s.bits = (bits + s.passes - 1) / s.passes;
  // up to 128 blocks of one token a thread (65536 tokens: a placing pass 7.9 us, with four tokens a thread 9.3)
  s.steps = n <= 128 * kSortThreads ? 1 : kSteps;
  const int64_t tile = s.steps * kSortThreads, tiles = (n + tile - 1) / tile, most = kMostCounts >> s.bits;
  const int64_t each = tiles > most ? (tiles + most - 1) / most : 1;
  s.per_block = each * tile;
  s.blocks = (int32_t)(n ? (n + s.per_block - 1) / s.per_block : 1);
  return s;
}

// Places of a chunk, 8 to 256 (a sum is a chain of at most that many, then one over the chunks): few enough for 4096 waves,
// of which 512 columns fill one.  65536 tokens x 1024 bfloat16, with half as many waves 126 us, so 121; 200000 x 256 float32
// of 50000 rows, in chunks of 128 the sums alone 146, of 32 61.
int32_t chunk_places(int64_t n, int32_t width) {
  const int64_t want = n * (width < 512 ? width : 512) / (512 * 4096);
  int32_t per = 8;
  while (per < 256 && per < want) per *= 2;
  return per;
}

struct Space {   // of the workspace: byte offsets
  size_t keys[2], order[2], counts, partial, crossing, bytes;
};

Space space(int64_t n, int64_t n_rows, int32_t width) {
  Space s{};
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t was = at;
    at += (bytes + 15) & ~(size_t)15;
    return was;
  };
  if (n > 0) {
    const SortShape sh = sort_shape(n, n_rows);
    const int sets = n <= kOneTokens || sh.passes == 1 ? 1 : 2;
    for (int i = 0; i < 2; ++i) {
      s.keys[i] = i < sets ? take((size_t)n * 4) : s.keys[0];
      s.order[i] = i < sets ? take((size_t)n * 4) : s.order[0];
    }
    s.counts = n <= kOneTokens ? at : take(((size_t)sh.blocks << sh.bits) * 4);
    const int32_t per = chunk_places(n, width);
    const size_t chunks = (size_t)((n + per - 1) / per);
    s.partial = take(chunks * 2 * (size_t)width * 4);
    s.crossing = take((chunks + 1) * sizeof(Pair));
  }
  s.bytes = at;
  return s;
}

int check_embedding(const char *who, int64_t n_tokens, int64_t n_rows, int32_t width) {
  if (n_tokens < 0 || n_tokens > kMaxTokens)
    return report(SVT_EINVAL, "%s: n_tokens %lld out of [0, 2^30]", who, (long long)n_tokens);
  if (n_rows < 1 || n_rows > kMaxRows)
    return report(SVT_EINVAL, "%s: n_rows %lld out of [1, 2^31 - 2]", who, (long long)n_rows);
  if (width < 1 || width > kMaxWidth) return report(SVT_EINVAL, "%s: width %d out of [1, %d]", who, width, kMaxWidth);
  return SVT_OK;
}

bool finite(float f) { return f - f == 0.f; }

template <class T, class TD, int M, bool ADD>
int embedding_backward(const char *who, SumArgs a, const SortShape &sh, const Space &sp, const int64_t *ids,
                       const void *d_out, void *d_table, char *ws, void *stream) {
  int sorted = 0;
  if (a.n > 0) {
    auto with_bits = [&](auto f) {
      if (sh.bits <= 6) return f(std::integral_constant<int, 6>{});
      if (sh.bits <= 8) return f(std::integral_constant<int, 8>{});
      if (sh.bits <= 9) return f(std::integral_constant<int, 9>{});
      return f(std::integral_constant<int, 10>{});
    };
    int32_t *crossing = (int32_t *)(ws + sp.crossing);
    auto keys = [&](int i) { return (uint32_t *)(ws + sp.keys[i]); };
    auto order = [&](int i) { return (int32_t *)(ws + sp.order[i]); };
    const int rc = with_bits([&](auto bits) {
      constexpr int B = decltype(bits)::value;
      auto one = [&](auto steps) {
        return launch(who, k_sort_tokens<decltype(steps)::value, B>, 1, kSortThreads, 0, stream, ids, sh, keys(0), order(0),
                      crossing);
      };
      if (a.n <= kSortThreads) return one(std::integral_constant<int, 1>{});
      if (a.n <= kSteps * kSortThreads) return one(std::integral_constant<int, kSteps>{});
      if (a.n <= kOneTokens) return one(std::integral_constant<int, kOneSteps>{});
      int32_t *counts = (int32_t *)(ws + sp.counts);
      for (int p = 0; p < sh.passes; ++p) {
        const Digits d{p ? nullptr : ids, keys(sorted), order(sorted), p * sh.bits};
        if (p) sorted ^= 1;
        auto pass = [&](auto steps) {
          constexpr int S = decltype(steps)::value;
          const int rc = launch(who, k_sort_count<S>, sh.blocks, kSortThreads, 0, stream, d, sh, counts, crossing);
          if (rc != SVT_OK) return rc;
          return launch(who, k_sort_place<S, B>, sh.blocks, kSortThreads, 0, stream, d, sh, (const int32_t *)counts,
                        keys(sorted), order(sorted));
        };
        const int rc = sh.steps == 1 ? pass(std::integral_constant<int, 1>{}) : pass(std::integral_constant<int, kSteps>{});
        if (rc != SVT_OK) return rc;
      }
      return (int)SVT_OK;
    });
    if (rc != SVT_OK) return rc;
    a.keys = keys(sorted);
    a.order = order(sorted);
    a.partial = (float *)(ws + sp.partial);
    a.crossing = crossing;
    a.per = chunk_places(a.n, a.width);
    a.chunks = (int32_t)((a.n + a.per - 1) / a.per);
    a.column_blocks = (a.pieces + 2 * a.lanes - 1) / (2 * a.lanes);
    const int64_t units = (int64_t)a.chunks * a.column_blocks, each = kThreads / a.lanes;
    const int64_t blocks = (units + each - 1) / each;
    a.sum_blocks = blocks;
  }
  int64_t clear_blocks = 0;
  if (!ADD) {   // at most 256 KiB of rows for each, and work for every compute unit
    const int64_t row = (int64_t)a.width * sizeof(TD), share = (a.n_rows + 1023) / 1024;
    a.clear_rows = (int32_t)(row >= 262144 ? 1 : 262144 / row < kClearMost ? 262144 / row : kClearMost);
    if (share < a.clear_rows) a.clear_rows = (int32_t)share;
    clear_blocks = (a.n_rows + a.clear_rows - 1) / a.clear_rows;
  }
  if (!fits(a.sum_blocks + clear_blocks))
    return report(SVT_EINVAL, "%s: too large a table or batch for one call", who);
  auto sum = [&](auto two) {
    return launch(who, k_sum_rows<T, TD, M, ADD, decltype(two)::value>, grid_of(a.sum_blocks + clear_blocks), kThreads, 0,
                  stream, a, (const Vec<T, M> *)d_out, (Vec<TD, M> *)d_table);
  };
  const int rc = a.pieces > a.lanes ? sum(std::true_type{}) : sum(std::false_type{});
  if (rc != SVT_OK || a.chunks < 2) return rc;
  const int64_t most = (int64_t)(a.chunks - 1) * ((a.width + kJoinColumns - 1) / kJoinColumns);
  return launch(who, k_join_runs<TD, ADD>, (unsigned)(most < 512 ? most : 512), kJoinThreads, 0, stream, a, (TD *)d_table);
}

}  // namespace

}  // namespace svt

using namespace svt;

extern "C" int svt_embedding(int64_t n_tokens, int64_t n_rows, int32_t width, int32_t dtype, const void *table,
                             const int64_t *ids, float scale, void *out, void *hip_stream) {
  const char *who = "svt_embedding";
  (void)report(SVT_OK, "%s", "");
  const int rc = check_embedding(who, n_tokens, n_rows, width);
  if (rc != SVT_OK) return rc;
  if (!elem_size(dtype)) return report(SVT_EINVAL, "%s: unknown element type %d", who, dtype);
  if (!finite(scale)) return report(SVT_EINVAL, "%s: scale %g is not finite", who, scale);
  if (n_tokens == 0) return SVT_OK;
  if (!table || !ids || !out) return report(SVT_EINVAL, "%s: NULL input or output", who);
  const int b = elem_size(dtype);
  if (misaligned(table, b) || misaligned(ids, 8) || misaligned(out, b))
    return report(SVT_EINVAL, "%s: misaligned input or output", who);
  const size_t row = (size_t)width * b;
  if (overlap(out, n_tokens * row, table, n_rows * row) || overlap(out, n_tokens * row, ids, (size_t)n_tokens * 8))
    return report(SVT_EINVAL, "%s: the output overlaps an input", who);
  return with_type(dtype, [&](auto ty) {
    using T = decltype(ty);
    return with_elems<T>(piece_elems(width, b, table, b, out), [&](auto elems) {
      constexpr int M = decltype(elems)::value;
      LookupArgs a{n_tokens, n_rows, width / M, 1, ids, scale};
      while (a.lanes < 64 && a.lanes < a.pieces) a.lanes *= 2;
      const int64_t per = kThreads / a.lanes, n = (n_tokens + per - 1) / per;
      const int columns = (a.pieces + 2 * a.lanes - 1) / (2 * a.lanes);
      // few tokens of wide rows: the columns over workgroups too
      const dim3 grid((unsigned)(n < (1 << 20) ? n : (1 << 20)), n >= 2048 ? 1 : columns < 64 ? columns : 64);
      return launch(who, k_lookup<T, M>, grid, kThreads, 0, hip_stream, a, (const Vec<T, M> *)table, (Vec<T, M> *)out);
    });
  });
}

extern "C" size_t svt_embedding_backward_workspace_size(int64_t n_tokens, int64_t n_rows, int32_t width) {
  (void)report(SVT_OK, "%s", "");
  if (check_embedding("svt_embedding_backward_workspace_size", n_tokens, n_rows, width) != SVT_OK) return 0;
  return space(n_tokens, n_rows, width).bytes;
}

extern "C" int svt_embedding_backward(int64_t n_tokens, int64_t n_rows, int32_t width, int32_t dtype, const void *d_out,
                                      const int64_t *ids, float scale, int32_t accumulate, int32_t table_type,
                                      void *d_table, void *workspace, size_t workspace_bytes, void *hip_stream) {
  const char *who = "svt_embedding_backward";
  (void)report(SVT_OK, "%s", "");
  const int rc = check_embedding(who, n_tokens, n_rows, width);
  if (rc != SVT_OK) return rc;
  if (!elem_size(dtype)) return report(SVT_EINVAL, "%s: unknown element type %d", who, dtype);
  if (table_type != dtype && table_type != SVT_F32)
    return report(SVT_EINVAL, "%s: table type %d is neither the rows' nor SVT_F32", who, table_type);
  if (accumulate != 0 && accumulate != 1) return report(SVT_EINVAL, "%s: accumulate %d is not 0 or 1", who, accumulate);
  if (!finite(scale)) return report(SVT_EINVAL, "%s: scale %g is not finite", who, scale);
  if (n_tokens == 0 && accumulate) return SVT_OK;
  if (!d_table || (n_tokens > 0 && (!d_out || !ids))) return report(SVT_EINVAL, "%s: NULL input or output", who);
  const int b = elem_size(dtype), tb = elem_size(table_type);
  if (misaligned(d_out, b) || misaligned(ids, 8) || misaligned(d_table, tb) || misaligned(workspace, 16))
    return report(SVT_EINVAL, "%s: misaligned input, output or workspace", who);
  const Space sp = space(n_tokens, n_rows, width);
  if (sp.bytes > 0 && (!workspace || workspace_bytes < sp.bytes))
    return report(SVT_EINVAL, "%s: workspace of %zu bytes, needs %zu", who, workspace ? workspace_bytes : (size_t)0,
                  sp.bytes);
  const void *at[4] = {d_out, ids, d_table, workspace};
  const size_t bytes[4] = {(size_t)n_tokens * width * b, (size_t)n_tokens * 8, (size_t)n_rows * width * tb, sp.bytes};
  for (int i = 2; i < 4; ++i)
    for (int j = 0; j < i; ++j)
      if (overlap(at[i], bytes[i], at[j], bytes[j]))
        return report(SVT_EINVAL, "%s: inputs, output and workspace overlap", who);
  const SortShape sh = sort_shape(n_tokens, n_rows);
  return with_type(dtype, [&](auto ty) {
    using T = decltype(ty);
    auto typed = [&](auto table_ty) {
      using TD = decltype(table_ty);
      return with_elems<T>(piece_elems(width, b, d_out, tb, d_table), [&](auto elems) {
        constexpr int M = decltype(elems)::value;
        SumArgs a{};
        a.n = n_tokens;
        a.n_rows = n_rows;
        a.width = width;
        a.pieces = width / M;
        a.lanes = 1;
        while (a.lanes < 64 && a.lanes < a.pieces) a.lanes *= 2;
        a.scale = scale;
        return accumulate ? embedding_backward<T, TD, M, true>(who, a, sh, sp, ids, d_out, d_table, (char *)workspace, hip_stream)
                          : embedding_backward<T, TD, M, false>(who, a, sh, sp, ids, d_out, d_table, (char *)workspace, hip_stream);
      });
    };
    return table_type == dtype ? typed(T{}) : typed(float{});
  });
}

// svt_logprobs.hip - log probabilities of given tokens on gfx950, with the entropy and the best alternatives of each
// row, and the gradient of both back to the logits.
//
//   z_i = scale l_i;  p = softmax(z) over the open tokens (a logit of -inf or NaN shuts its token)
//   logp_t = z_t - log sum exp z;   H = -sum p_i log p_i
//   dl_i = scale (d (1[i = t] - p_i) - dH p_i (log p_i + H)),  0 at shut tokens
//
// Forward: one pass over the logits.  A thread keeps the largest logit m it saw, Z = sum 2^x and S = sum x 2^x with
// x = (l - m) scale log2 e, and moves Z and S to a new m only where a piece of 8 logits brings a larger one.  Partial
// sums join as  m' = max,  Z' = Z 2^(m - m'),  S' = (S + Z (m - m')) 2^(m - m'):  within a wave by lane moves, between
// waves through LDS, between the workgroups of a split row by a second launch.  log2 Z and S / Z give logp and H.  x is
// held in [-1000, 0]: 2^-1000 is 0 and 0 * 1000 too, so that shut tokens (-inf, NaN) and masks of the type's lowest
// value need no branch, and +inf counts as the largest float32.
//
// Best alternatives: a wave sees its tokens in ascending order, so that a later token only enters above its `top`-th
// best so far (ties go to the lower token).  Tokens above that bound go to a list in LDS; a full list is cut to its
// `top` best, which raises the bound.  The first piece's bound is the top-th largest of the lanes' own maxima.
//
// Measured, the forward pass alone over inputs in turn: 4096 rows of 49152 bfloat16 81 us (5.0 TB/s: bound by memory), of
// 50021, whose rows begin at odd addresses, 108 (3.8 TB/s); 49152 float32 with the 16 best 191 (4.2 TB/s).  The gradient of
// the first two 146 and 161, of forward and gradient one after the other 246 and 280: behind the gradient's writes the
// forward pass of 50021 takes 125.  Loads and conversions of a piece stand apart, and the pieces of the next step are asked
// for before this step's are used.  256 rows of 2048 float32, top 16: 8.0 us, the gradient 4.6.  One row of 131072 bfloat16,
// top 8: 7.7 us in 32 splits, 4.5 to join them.

#include <type_traits>

#include "../experts/svt_experts.h"

namespace svt {

namespace {

constexpr int kThreads = 256, kWaves = kThreads / 64;
constexpr int kPiece = 8;                       // logits of a load
constexpr int kList = 512;                      // a wave's candidates
constexpr int32_t kMaxVocab = 1 << 30;
constexpr float kLog2e = 1.44269504088896341f, kLn2 = 0.693147180559945309f;
constexpr float kFar = -1000.f;
constexpr float kMostScale = 0x1p127f;          // scale log2 e stays finite: 0 times it is 0

struct LogprobArgs {
  int64_t n_tokens;
  int32_t vocab, top, splits;
  int32_t pieces;           // of a split: kPiece logits each
  float scale;
  const int64_t *tokens;
  float *logprobs, *entropy, *norms;
  int64_t *top_tokens;
  float *top_logprobs;
  float *sums;              // [row][split][3], where rows are split
  uint64_t *best;           // [row][split][top]
};

// float -> uint32 whose unsigned order is the float order (-0 as 0, +inf as the largest finite value); 0: shut
__device__ __forceinline__ uint32_t order_of(float f) {
  const uint32_t b = __float_as_uint(fminf(f, FLT_MAX) + 0.f);
  return f > -INFINITY ? ((b & 0x80000000u) ? ~b : (b | 0x80000000u)) : 0u;
}
__device__ __forceinline__ float of_order(uint32_t o) {
  return __uint_as_float((o & 0x80000000u) ? (o & 0x7FFFFFFFu) : ~o);
}
// a logit and its token; greater: (logit desc, token asc); 0: none
__device__ __forceinline__ uint64_t key_of(float f, int token) {
  const uint32_t o = order_of(f);
  return o ? (uint64_t)o << 32 | (0xFFFFFFFFu - (uint32_t)token) : 0ull;
}
__device__ __forceinline__ float key_logit(uint64_t k) { return of_order((uint32_t)(k >> 32)); }
__device__ __forceinline__ int64_t key_token(uint64_t k) { return k ? (int64_t)(0xFFFFFFFFu - (uint32_t)k) : -1; }

__device__ __forceinline__ float wave_max(float v) {
  return __uint_as_float(group_reduce(__float_as_uint(v), 64, [](uint32_t a, uint32_t b) {
    return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
  }));
}
__device__ __forceinline__ uint64_t wave_best(uint64_t k) {
  const uint32_t hi = group_max((uint32_t)(k >> 32), 64);
  const uint64_t same = __ballot((uint32_t)(k >> 32) == hi);
  // equal logits, of which the lower token counts, are rare
  const uint32_t lo = (same & (same - 1)) == 0ull
                          ? (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)k, __builtin_ctzll(same))
                          : group_max((uint32_t)(k >> 32) == hi ? (uint32_t)k : 0u, 64);
  return (uint64_t)hi << 32 | lo;
}

// f, a signalling NaN quieted: the maximum of one and a number is a NaN, and the next maximum drops that and what was before.
// (The conversion from float16 quiets by itself; that from bfloat16 is a move of bits.)
template <class T>
__device__ __forceinline__ float quiet(float f) {
  if constexpr (std::is_same<T, f16>::value) return f;
  else return __builtin_canonicalizef(f);
}

// (l - m) scale log2 e, in [kFar, 0]; kFar for a NaN (the instruction's median of a NaN is the least of the others)
__device__ __forceinline__ float exponent(float l, float m, float c) {
  return __builtin_amdgcn_fmed3f((l - m) * c, kFar, 0.f);
}

// m: the largest logit (raw); z = sum 2^x, s = sum x 2^x
struct Sums {
  float m, z, s;
  __device__ __forceinline__ static Sums none() { return {-FLT_MAX, 0.f, 0.f}; }
  __device__ __forceinline__ void move(float to, float c) {   // to >= m
    const float x = exponent(m, to, c), f = __builtin_amdgcn_exp2f(x);
    s = (s + z * x) * f;
    z *= f;
    m = to;
  }
  __device__ __forceinline__ void join(Sums o, float c) {
    const float to = fmaxf(m, o.m);
    move(to, c);
    o.move(to, c);
    z += o.z;
    s += o.s;
  }
};

__device__ __forceinline__ Sums wave_sums(Sums a, float c) {
  a.move(wave_max(a.m), c);
  a.z = group_add(a.z, 64);
  a.s = group_add(a.s, 64);
  return a;
}

// between LDS operations of one wave, which the hardware keeps in order
__device__ __forceinline__ void wave_order() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// the `top` best of the wave's keys, N a lane: the j-th best in lane j (0 where there are fewer)
template <int N>
__device__ __forceinline__ uint64_t wave_top(uint64_t (&k)[N], int top) {
  uint64_t kept = 0ull;
  for (int j = 0; j < top; ++j) {
    uint64_t mine = k[0];
#pragma unroll
    for (int i = 1; i < N; ++i) mine = k[i] > mine ? k[i] : mine;
    const uint64_t best = wave_best(mine);
    if (lane_id() == j) kept = best;
#pragma unroll
    for (int i = 0; i < N; ++i) k[i] = k[i] == best ? 0ull : k[i];
  }
  return kept;
}

// how many of the keys of lanes 0 .. n - 1 are greater than this lane's
__device__ __forceinline__ int rank_of(uint64_t k, int n) {
  int rank = 0;
#pragma unroll 4
  for (int j = 0; j < n; ++j) {
    const uint64_t o = (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(k >> 32), j) << 32 |
                       (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)k, j);
    rank += o > k ? 1 : 0;
  }
  return rank;
}
// the `top` best of the keys of lanes 0 .. n - 1, no two alike but 0, in order in lanes 0 .. top - 1; through 16 places of LDS
__device__ __forceinline__ uint64_t in_order(uint64_t k, int n, int top, uint64_t *lds) {
  const int rank = rank_of(k, n);
  wave_order();
  if (lane_id() < SVT_MAX_TOP) lds[lane_id()] = 0ull;
  wave_order();
  if (k != 0ull && rank < top) lds[rank] = k;
  wave_order();
  return lane_id() < top ? lds[lane_id()] : 0ull;
}

// The same, by ranks or by rounds that take the best.  The whole forward pass by ranks and by rounds in us, top 4, 8 and 16:
// 256 rows of 2048 float32 6.3 and 5.9, 6.9 and 7.3, 8.0 and 10.0; 4096 of them 26 and 24, 30 and 31, 35 and 44; one row of 131072
// bfloat16 10.1 and 8.9, 12.3 and 11.6, 20.6 and 20.9; 16384 rows of 900 24 and 24, 28 and 30, 36 and 40
__device__ __forceinline__ uint64_t best_of_wave(uint64_t k, int n, int top, uint64_t *lds) {
  if (top > 8) return in_order(k, n, top, lds);
  uint64_t one[1] = {k};
  return wave_top(one, top);
}

// a wave's candidates
struct Candidates {
  uint64_t *list;     // LDS [kList]
  int count, top;
  float bound;        // a later token enters above it

  __device__ __forceinline__ uint64_t cut() {
    uint64_t kept;
    wave_order();
    if (count <= 64) {   // the first piece's, most often
      kept = best_of_wave(lane_id() < count ? list[lane_id()] : 0ull, count, top, list);
    } else {
      uint64_t k[kList / 64];
#pragma unroll
      for (int i = 0; i < kList / 64; ++i) k[i] = i * 64 + lane_id() < count ? list[i * 64 + lane_id()] : 0ull;
      kept = wave_top(k, top);
    }
    if (lane_id() < top) list[lane_id()] = kept;
    wave_order();
    const uint64_t full = __ballot(lane_id() < top && kept != 0ull);
    count = __builtin_popcountll(full);
    const uint32_t last = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(kept >> 32), top - 1);
    bound = last ? of_order(last) : -INFINITY;
    return kept;
  }

  // the bound of a first piece: just below the top-th largest of the lanes' maxima
  __device__ __forceinline__ void start(float most) {
    uint32_t o = order_of(most), best = 0u;
    for (int j = 0; j < top; ++j) {
      best = group_max(o, 64);
      const uint64_t same = __ballot(o == best);
      if (lane_id() == __builtin_ctzll(same)) o = 0u;
    }
    // two steps lower: one may lead from 0 to -0, which compares as equal.  No number lies two steps below the lowest.
    bound = best > 0x00800002u ? of_order(best - 2u) : -INFINITY;
  }

  // a piece for each lane.  One bound for all of it: its tokens do not come in order, lane after lane for each i
  __device__ __forceinline__ void offer(const float (&v)[kPiece], float most, int first) {
    const float above = bound;
    if (!__ballot(most > above)) return;
#pragma unroll
    for (int i = 0; i < kPiece; ++i) {
      const bool in = v[i] > above;
      const uint64_t who = __ballot(in);
      if (who) {
        if (in) list[count + mbcnt(who)] = key_of(v[i], first + i);
        count += __builtin_popcountll(who);
        if (count > kList - 64) (void)cut();
      }
    }
    if (count >= top + 64) (void)cut();
  }
};

// aligned to its elements alone: the order of a row's sums does not depend on where the row lies
template <class T> struct __attribute__((packed, aligned(sizeof(T)))) Piece { uint32_t v[kPiece * sizeof(T) / 4]; };
template <class T> struct Eight { T v[kPiece]; };

template <class T>
__device__ __forceinline__ Piece<T> raw_piece(const T *row, int first) {
  return *reinterpret_cast<const Piece<T> *>(row + first);
}
template <class T>
__device__ __forceinline__ void widen(const Piece<T> &raw, float (&v)[kPiece]) {
  const Eight<T> p = __builtin_bit_cast(Eight<T>, raw);
#pragma unroll
  for (int i = 0; i < kPiece; ++i) v[i] = (float)p.v[i];
}

// Logits first .. first + 7 of a row, shut past its end: the token of v[0] is returned.  A piece that would run past the end
// is the row's last 8 logits, of which those before `first` are shut (one load; 8 for rows of fewer).
template <class T>
__device__ __forceinline__ int load_piece(const T *row, int first, int vocab, float (&v)[kPiece]) {
  if (vocab < kPiece) {
#pragma unroll
    for (int i = 0; i < kPiece; ++i) {
      const float f = (float)row[i < vocab ? i : vocab - 1];
      v[i] = first == 0 && i < vocab ? f : -INFINITY;
    }
    return 0;
  }
  const int at = first + kPiece <= vocab ? first : vocab - kPiece;
  widen(raw_piece(row, at), v);
#pragma unroll
  for (int i = 0; i < kPiece; ++i) v[i] = at + i >= first ? v[i] : -INFINITY;
  return at;
}

// the pieces of a thread at a time, in flight together
template <int U>
__device__ __forceinline__ void add_pieces(Sums &a, const float (&v)[U][kPiece], float most, float c) {
  most = fminf(most, FLT_MAX);
  if (most > a.m) a.move(most, c);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    float z = 0.f, s = 0.f;
#pragma unroll
    for (int i = 0; i < kPiece; ++i) {
      const float x = exponent(v[u][i], a.m, c), e = __builtin_amdgcn_exp2f(x);
      z += e;
      s = fmaf(x, e, s);
    }
    a.z += z;
    a.s += s;
  }
}

// a row's token and its logit
struct Given { int64_t token; float logit; };
template <class T>
__device__ __forceinline__ Given given(const LogprobArgs &a, const T *row, int64_t token) {
  return {token, (float)row[(uint64_t)token < (uint64_t)a.vocab ? token : 0]};
}

// logp, H, norms and the alternatives of row t, by one wave: lane j holds the j-th best
__device__ __forceinline__ void finish(const LogprobArgs &a, Given g, int64_t t, Sums sum, uint64_t best) {
  const bool any = sum.z > 0.f;
  const float log_z = any ? __builtin_amdgcn_logf(sum.z) : 0.f;   // base 2; z >= 1
  const float peak = any ? sum.m : 0.f;
  auto logp = [&](float l) { return (fminf(l, FLT_MAX) - peak) * a.scale - log_z * kLn2; };
  if (lane_id() == 0) {
    float lp = 0.f;
    if ((uint64_t)g.token < (uint64_t)a.vocab) lp = g.logit > -INFINITY ? logp(g.logit) : -INFINITY;
    a.logprobs[t] = lp;
    a.entropy[t] = any ? (log_z - sum.s / sum.z) * kLn2 : 0.f;
    a.norms[2 * t] = peak;
    a.norms[2 * t + 1] = log_z;
  }
  if (lane_id() < a.top) {
    a.top_tokens[t * a.top + lane_id()] = key_token(best);
    a.top_logprobs[t * a.top + lane_id()] = best ? logp(key_logit(best)) : -INFINITY;
  }
}

// W waves share a row (or a split of one): 1 or kWaves; a thread takes U pieces at a time
template <class T, int W, bool TOP, bool SPLIT>
__global__ __launch_bounds__(kThreads) void k_logprobs(LogprobArgs a, const T *logits) {
  constexpr int U = 2;
  __shared__ uint64_t lists[TOP ? kWaves : 1][TOP ? kList : 1];
  __shared__ Sums parts[kWaves];
  const int wave = threadIdx.x / 64;
  const int in = threadIdx.x % (64 * W);
  const float c = a.scale * kLog2e;
  const int64_t units = a.n_tokens * a.splits;
  constexpr int kUnits = kWaves / W;   // of a workgroup
  for (int64_t u0 = blockIdx.x * (int64_t)kUnits; u0 < units; u0 += (int64_t)gridDim.x * kUnits) {
    const int64_t u = u0 + wave / W;
    if (W < kWaves && u >= units) return;   // whole waves, which wait for no other
    const int64_t t = SPLIT ? u / a.splits : u;
    const int part = SPLIT ? (int)(u - t * a.splits) : 0;
    const T *row = logits + t * a.vocab;
    const int64_t token = SPLIT ? -1 : a.tokens[t];
    const int pieces = (a.vocab + kPiece - 1) / kPiece;
    const int p0 = part * a.pieces, p1 = SPLIT ? (p0 + a.pieces < pieces ? p0 + a.pieces : pieces) : pieces;
    Sums sum = Sums::none();
    Candidates best{TOP ? lists[wave] : nullptr, 0, a.top, -INFINITY};
    // N pieces of a thread from place q on, 64 W apart; all lanes of a wave act together
    auto take = [&](int q, auto &v, int token) {   // token: of v[0][0]
      constexpr int N = sizeof(v) / sizeof(v[0]);
      float most = -INFINITY;   // of a NaN and a number, the number
#pragma unroll
      for (int n = 0; n < N; ++n) {
        float m = -INFINITY;
#pragma unroll
        for (int i = 0; i < kPiece; ++i) m = fmaxf(m, quiet<T>(v[n][i]));
        if (TOP) {
          if (n == 0 && q == p0) best.start(m);
          best.offer(v[n], m, token + n * 64 * W * kPiece);
        }
        most = fmaxf(most, m);
      }
      add_pieces<N>(sum, v, most, c);
    };
    // whole pieces for every thread, the next ones in flight; then what is left, one a thread, shut past the end
    constexpr int hop = U * 64 * W;
    const int whole = a.vocab / kPiece, p2 = p1 < whole ? p1 : whole;
    int q = p0;
    if (q + hop <= p2) {
      Piece<T> raw[U];
      auto ask = [&](int at) {
#pragma unroll
        for (int n = 0; n < U; ++n) raw[n] = raw_piece(row, (at + n * 64 * W + in) * kPiece);
      };
      ask(q);
      for (; q + hop <= p2; q += hop) {
        float v[U][kPiece];
#pragma unroll
        for (int n = 0; n < U; ++n) widen(raw[n], v[n]);
        ask(q + 2 * hop <= p2 ? q + hop : q);   // behind the last, the same again
        take(q, v, (q + in) * kPiece);
      }
    }
    Given g{};
    if (!SPLIT) g = given(a, row, token);   // in flight beside the rest
    for (; q < p1; q += 64 * W) {
      float v[1][kPiece];
      const int at = load_piece(row, q + in < p1 ? (q + in) * kPiece : a.vocab, a.vocab, v[0]);
      take(q, v, at);
    }
    sum = wave_sums(sum, c);
    uint64_t mine = TOP ? best.cut() : 0ull;
    if (W > 1) {
      if (lane_id() == 0) parts[wave] = sum;
      __syncthreads();
      if (wave == 0) {
        sum = parts[0];
        for (int w = 1; w < kWaves; ++w) sum.join(parts[w], c);
        if (TOP) {   // kWaves x top <= 64 keys
          const int from = lane_id() / 16, j = lane_id() % 16;
          static_assert(SVT_MAX_TOP == 16 && kWaves == 4, "a lane for every wave's keys");
          mine = best_of_wave(j < a.top ? lists[from][j] : 0ull, 64, a.top, &lists[0][64]);
        }
      }
    }
    if (W == 1 || wave == 0) {
      if (SPLIT) {
        if (lane_id() == 0) {
          a.sums[3 * u] = sum.m;
          a.sums[3 * u + 1] = sum.z;
          a.sums[3 * u + 2] = sum.s;
        }
        if (lane_id() < a.top) a.best[u * a.top + lane_id()] = mine;
      } else {
        finish(a, g, t, sum, mine);
      }
    }
    if (W > 1) __syncthreads();   // parts and lists are free again
  }
}

// joins the splits of a row, one wave a row
template <class T, bool TOP>
__global__ __launch_bounds__(64) void k_logprobs_join(LogprobArgs a, const T *logits) {
  __shared__ uint64_t ordered[SVT_MAX_TOP];
  const float c = a.scale * kLog2e;
  for (int64_t t = blockIdx.x; t < a.n_tokens; t += gridDim.x) {
    const Given g = given(a, logits + t * a.vocab, a.tokens[t]);
    Sums sum = Sums::none();
    for (int p = lane_id(); p < a.splits; p += 64) {
      const float *s = a.sums + 3 * (t * a.splits + p);
      sum.join({s[0], s[1], s[2]}, c);
    }
    sum = wave_sums(sum, c);
    uint64_t best = 0ull;
    if (TOP) {
      const int n = a.splits * a.top;
      if (n <= 64) best = best_of_wave(lane_id() < n ? a.best[t * n + lane_id()] : 0ull, n, a.top, ordered);
      for (int i0 = 0; n > 64 && i0 < n; i0 += 64 * 7) {
        uint64_t k[8];
#pragma unroll
        for (int i = 0; i < 7; ++i) k[i] = i0 + 64 * i + lane_id() < n ? a.best[t * n + i0 + 64 * i + lane_id()] : 0ull;
        k[7] = best;   // the best so far, in the first `top` lanes
        best = wave_top(k, a.top);
      }
    }
    finish(a, g, t, sum, best);
  }
}

// dl_i = p_i (A + B x_i), and scale d more at the token;  x the base-2 exponent, p = 2^(x - log2 Z),
// A = -scale (d + dH (H - ln Z)), B = -scale dH ln 2
template <class T, int W>
__global__ __launch_bounds__(kThreads) void k_logprobs_backward(LogprobArgs a, const T *logits, const float *d_logprobs,
                                                                const float *d_entropy, T *d_logits) {
  const int in = threadIdx.x % (64 * W);
  const float c = a.scale * kLog2e;
  const int64_t units = a.n_tokens * a.splits;
  constexpr int kUnits = kWaves / W;
  for (int64_t u = blockIdx.x * (int64_t)kUnits + threadIdx.x / (64 * W); u < units; u += (int64_t)gridDim.x * kUnits) {
    const int64_t t = u / a.splits;
    const int part = (int)(u - t * a.splits);
    const T *row = logits + t * a.vocab;
    T *out = d_logits + t * a.vocab;
    const int pieces = (a.vocab + kPiece - 1) / kPiece;
    const int p0 = part * a.pieces, p1 = p0 + a.pieces < pieces ? p0 + a.pieces : pieces;
    const float peak = a.norms[2 * t], log_z = a.norms[2 * t + 1];
    const int64_t token = a.tokens[t];
    const bool given = (uint64_t)token < (uint64_t)a.vocab;
    const float d = given ? d_logprobs[t] * a.scale : 0.f;
    const float dh = d_entropy ? d_entropy[t] * a.scale : 0.f;
    const float A = -(d + dh * (a.entropy[t] - log_z * kLn2)), B = -dh * kLn2;
    const int at = given ? (int)token : -kPiece;
    auto slopes = [&](float (&v)[kPiece], int first) {
#pragma unroll
      for (int i = 0; i < kPiece; ++i) {
        const float x = exponent(v[i], peak, c);
        const float g = __builtin_amdgcn_exp2f(x - log_z) * fmaf(B, x, A);
        v[i] = first + i == at && v[i] > -INFINITY ? g + d : g;
      }
    };
    auto narrow = [&](const float (&v)[kPiece], int first) {
      Eight<T> r;
#pragma unroll
      for (int i = 0; i < kPiece; ++i) r.v[i] = (T)v[i];
      *reinterpret_cast<Piece<T> *>(out + first) = __builtin_bit_cast(Piece<T>, r);
    };
    constexpr int U = 2, hop = U * 64 * W;   // pieces of a thread in flight
    const int whole = a.vocab / kPiece, p2 = p1 < whole ? p1 : whole;
    int q = p0;
    for (; q + hop <= p2; q += hop) {
      Piece<T> raw[U];
#pragma unroll
      for (int n = 0; n < U; ++n) raw[n] = raw_piece(row, (q + n * 64 * W + in) * kPiece);
#pragma unroll
      for (int n = 0; n < U; ++n) {
        const int first = (q + n * 64 * W + in) * kPiece;
        float v[kPiece];
        widen(raw[n], v);
        slopes(v, first);
        narrow(v, first);
      }
    }
    for (int p = q + in; p < p1; p += 64 * W) {
      const int first = p * kPiece;
      float v[kPiece];
      const int from = load_piece(row, first, a.vocab, v);
      slopes(v, from);
      if (first + kPiece <= a.vocab) {
        narrow(v, first);
      } else {
#pragma unroll
        for (int i = 0; i < kPiece; ++i)
          if (from + i >= first && from + i < a.vocab) out[from + i] = (T)v[i];
      }
    }
  }
}

// ---- host ----------------------------------------------------------------------------------------

constexpr int kSplitPieces = 2 * kThreads;   // least pieces of a split: two for each thread

int pieces_of(int32_t vocab) { return (vocab + kPiece - 1) / kPiece; }

// rows that give fewer workgroups than two for each compute unit are split
int32_t splits_of(int64_t n_tokens, int32_t vocab) {
  const int64_t want = n_tokens > 0 ? 512 / n_tokens : 1, most = (pieces_of(vocab) + kSplitPieces - 1) / kSplitPieces;
  return (int32_t)(want < 1 ? 1 : want < most ? want : most);
}

size_t split_bytes(int64_t n_tokens, int32_t vocab, int32_t top) {
  const int64_t n = splits_of(n_tokens, vocab);
  return n == 1 ? 0 : (size_t)(n_tokens * n) * (16 + 8 * (size_t)top);   // 12 for the sums, in 8-byte steps
}

int check_logprobs(const char *who, int32_t n_tokens, int32_t vocab, int32_t top, int32_t dtype) {
  if (n_tokens < 0) return report(SVT_EINVAL, "%s: n_tokens %d < 0", who, n_tokens);
  if (vocab < 1 || vocab > kMaxVocab) return report(SVT_EINVAL, "%s: vocab %d out of [1, %d]", who, vocab, kMaxVocab);
  if (top < 0 || top > SVT_MAX_TOP || top > vocab)
    return report(SVT_EINVAL, "%s: top %d out of [0, min(%d, vocab)]", who, top, SVT_MAX_TOP);
  if (!elem_size(dtype)) return report(SVT_EINVAL, "%s: unknown element type %d", who, dtype);
  return SVT_OK;
}

unsigned row_grid(int64_t units, int per_block) {
  const int64_t n = (units + per_block - 1) / per_block;
  return (unsigned)(n < (1 << 20) ? n : (1 << 20));
}

}  // namespace

}  // namespace svt

using namespace svt;

extern "C" size_t svt_token_logprobs_workspace_size(int32_t n_tokens, int32_t vocab, int32_t top) {
  (void)report(SVT_OK, "%s", "");
  if (check_logprobs("svt_token_logprobs_workspace_size", n_tokens, vocab, top, SVT_F32) != SVT_OK) return 0;
  return split_bytes(n_tokens, vocab, top);
}

extern "C" int svt_token_logprobs(int32_t n_tokens, int32_t vocab, int32_t top, int32_t dtype, const void *logits,
                                  const int64_t *tokens, float scale, float *logprobs, float *entropy, float *norms,
                                  int64_t *top_tokens, float *top_logprobs, void *workspace, size_t workspace_bytes,
                                  void *hip_stream) {
  const char *who = "svt_token_logprobs";
  (void)report(SVT_OK, "%s", "");
  int rc = check_logprobs(who, n_tokens, vocab, top, dtype);
  if (rc != SVT_OK) return rc;
  if (!(scale > 0.f && scale <= kMostScale)) return report(SVT_EINVAL, "%s: scale %g out of (0, 2^127]", who, scale);
  if (n_tokens == 0) return SVT_OK;
  if (!logits || !tokens || !logprobs || !entropy || !norms || (top > 0 && (!top_tokens || !top_logprobs)))
    return report(SVT_EINVAL, "%s: NULL input or output", who);
  const int b = elem_size(dtype);
  if (misaligned(logits, b) || misaligned(tokens, 8) || misaligned(logprobs, 4) || misaligned(entropy, 4) ||
      misaligned(norms, 4) || misaligned(top_tokens, 8) || misaligned(top_logprobs, 4) || misaligned(workspace, 8))
    return report(SVT_EINVAL, "%s: misaligned input, output or workspace", who);
  const size_t need = split_bytes(n_tokens, vocab, top), n = (size_t)n_tokens;
  if (need > 0 && (!workspace || workspace_bytes < need))
    return report(SVT_EINVAL, "%s: workspace of %zu bytes, needs %zu", who, workspace ? workspace_bytes : (size_t)0, need);
  const void *at[8] = {logits, tokens, logprobs, entropy, norms, top_tokens, top_logprobs, workspace};
  const size_t bytes[8] = {n * vocab * b, n * 8, n * 4, n * 4, n * 8, n * top * 8, n * top * 4, need};
  for (int i = 2; i < 8; ++i)
    for (int j = 0; j < i; ++j)
      if (overlap(at[i], bytes[i], at[j], bytes[j]))
        return report(SVT_EINVAL, "%s: an output or the workspace overlaps an input or another output", who);
  LogprobArgs a{};
  a.n_tokens = n_tokens;
  a.vocab = vocab;
  a.top = top;
  a.splits = splits_of(n_tokens, vocab);
  a.pieces = (pieces_of(vocab) + a.splits - 1) / a.splits;
  a.scale = scale;
  a.tokens = tokens;
  a.logprobs = logprobs;
  a.entropy = entropy;
  a.norms = norms;
  a.top_tokens = top_tokens;
  a.top_logprobs = top_logprobs;
  a.best = (uint64_t *)workspace;
  a.sums = (float *)(a.best + n * a.splits * top);
  return with_type(dtype, [&](auto ty) {
    using T = decltype(ty);
    auto with_top = [&](auto f) { return top ? f(std::true_type{}) : f(std::false_type{}); };
    return with_top([&](auto tp) {
      constexpr bool TOP = decltype(tp)::value;
      if (a.splits > 1) {
        const int parted = launch(who, k_logprobs<T, kWaves, TOP, true>, row_grid(a.n_tokens * a.splits, 1), kThreads, 0,
                                  hip_stream, a, (const T *)logits);
        if (parted != SVT_OK) return parted;
        return launch(who, k_logprobs_join<T, TOP>, row_grid(a.n_tokens, 1), 64, 0, hip_stream, a, (const T *)logits);
      }
      if (vocab <= 1024)
        return launch(who, k_logprobs<T, 1, TOP, false>, row_grid(a.n_tokens, kWaves), kThreads, 0, hip_stream, a,
                      (const T *)logits);
      return launch(who, k_logprobs<T, kWaves, TOP, false>, row_grid(a.n_tokens, 1), kThreads, 0, hip_stream, a,
                    (const T *)logits);
    });
  });
}

extern "C" int svt_token_logprobs_backward(int32_t n_tokens, int32_t vocab, int32_t dtype, const void *logits,
                                           const int64_t *tokens, float scale, const float *norms, const float *entropy,
                                           const float *d_logprobs, const float *d_entropy, void *d_logits,
                                           void *hip_stream) {
  const char *who = "svt_token_logprobs_backward";
  (void)report(SVT_OK, "%s", "");
  int rc = check_logprobs(who, n_tokens, vocab, 0, dtype);
  if (rc != SVT_OK) return rc;
  if (!(scale > 0.f && scale <= kMostScale)) return report(SVT_EINVAL, "%s: scale %g out of (0, 2^127]", who, scale);
  if (n_tokens == 0) return SVT_OK;
  if (!logits || !tokens || !norms || !entropy || !d_logprobs || !d_logits)
    return report(SVT_EINVAL, "%s: NULL input or output", who);
  const int b = elem_size(dtype);
  if (misaligned(logits, b) || misaligned(tokens, 8) || misaligned(norms, 4) || misaligned(entropy, 4) ||
      misaligned(d_logprobs, 4) || misaligned(d_entropy, 4) || misaligned(d_logits, b))
    return report(SVT_EINVAL, "%s: misaligned input or output", who);
  const size_t n = (size_t)n_tokens, nl = n * vocab * b;
  const void *at[6] = {logits, tokens, norms, entropy, d_logprobs, d_entropy};
  const size_t bytes[6] = {nl, n * 8, n * 8, n * 4, n * 4, n * 4};
  for (int i = 0; i < 6; ++i)
    if (overlap(d_logits, nl, at[i], bytes[i])) return report(SVT_EINVAL, "%s: d_logits overlaps an input", who);
  LogprobArgs a{};
  a.n_tokens = n_tokens;
  a.vocab = vocab;
  a.scale = scale;
  a.tokens = tokens;
  a.norms = const_cast<float *>(norms);
  a.entropy = const_cast<float *>(entropy);
  // nothing joins here: pieces of 4 for each thread
  a.pieces = 4 * kThreads;
  a.splits = (pieces_of(vocab) + a.pieces - 1) / a.pieces;
  return with_type(dtype, [&](auto ty) {
    using T = decltype(ty);
    if (vocab <= 1024)
      return launch(who, k_logprobs_backward<T, 1>, row_grid(a.n_tokens * a.splits, kWaves), kThreads, 0, hip_stream, a,
                    (const T *)logits, d_logprobs, d_entropy, (T *)d_logits);
    return launch(who, k_logprobs_backward<T, kWaves>, row_grid(a.n_tokens * a.splits, 1), kThreads, 0, hip_stream, a,
                  (const T *)logits, d_logprobs, d_entropy, (T *)d_logits);
  });
}

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
  const uint32_t lo = group_max((uint32_t)(k >> 32) == hi ? (uint32_t)k : 0u, 64);
  return (uint64_t)hi << 32 | lo;
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

// a wave's candidates
struct Candidates {
  uint64_t *list;     // LDS [kList]
  int count, top;
  float bound;        // a later token enters above it

  __device__ __forceinline__ uint64_t cut() {
    uint64_t k[kList / 64];
    wave_order();
#pragma unroll
    for (int i = 0; i < kList / 64; ++i) k[i] = i * 64 + lane_id() < count ? list[i * 64 + lane_id()] : 0ull;
    const uint64_t kept = wave_top(k, top);
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
template <class T> struct __attribute__((packed, aligned(sizeof(T)))) Piece { uint8_t v[kPiece * sizeof(T)]; };
template <class T> struct Eight { T v[kPiece]; };

// logits first .. first + 7 of a row (shut past its end)
template <class T>
__device__ __forceinline__ void load_piece(const T *row, int first, int vocab, float (&v)[kPiece]) {
  if (first + kPiece <= vocab) {
    const Eight<T> p = __builtin_bit_cast(Eight<T>, *reinterpret_cast<const Piece<T> *>(row + first));
#pragma unroll
    for (int i = 0; i < kPiece; ++i) v[i] = (float)p.v[i];
  } else {
#pragma unroll
    for (int i = 0; i < kPiece; ++i) v[i] = first + i < vocab ? (float)row[first + i] : -INFINITY;
  }
}

__device__ __forceinline__ void add_piece(Sums &a, const float (&v)[kPiece], float most, float c) {
  most = fminf(most, FLT_MAX);
  if (most > a.m) a.move(most, c);
#pragma unroll
  for (int i = 0; i < kPiece; ++i) {
    const float x = exponent(v[i], a.m, c), e = __builtin_amdgcn_exp2f(x);
    a.z += e;
    a.s = fmaf(x, e, a.s);
  }
}

// logp, H, norms and the alternatives of row t, by one wave: lane j holds the j-th best
template <class T>
__device__ __forceinline__ void finish(const LogprobArgs &a, const T *row, int64_t t, Sums sum, uint64_t best) {
  const bool any = sum.z > 0.f;
  const float log_z = any ? __builtin_amdgcn_logf(sum.z) : 0.f;   // base 2; z >= 1
  const float peak = any ? sum.m : 0.f;
  auto logp = [&](float l) { return (fminf(l, FLT_MAX) - peak) * a.scale - log_z * kLn2; };
  if (lane_id() == 0) {
    const int64_t token = a.tokens[t];
    float lp = 0.f;
    if ((uint64_t)token < (uint64_t)a.vocab) {
      const float l = (float)row[token];
      lp = l > -INFINITY ? logp(l) : -INFINITY;
    }
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

// W waves share a row (or a split of one): 1 or kWaves
template <class T, int W, bool TOP, bool SPLIT>
__global__ __launch_bounds__(kThreads) void k_logprobs(LogprobArgs a, const T *logits) {
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
    const int pieces = (a.vocab + kPiece - 1) / kPiece;
    const int p0 = part * a.pieces, p1 = SPLIT ? (p0 + a.pieces < pieces ? p0 + a.pieces : pieces) : pieces;
    Sums sum = Sums::none();
    Candidates best{TOP ? lists[wave] : nullptr, 0, a.top, -INFINITY};
    auto take = [&](const float (&v)[kPiece], int p, bool first) {
      float most = -INFINITY;   // of a NaN and a number, the number
#pragma unroll
      for (int i = 0; i < kPiece; ++i) most = fmaxf(most, v[i]);
      if (TOP) {
        if (first) best.start(most);
        best.offer(v, most, p * kPiece);
      }
      add_piece(sum, v, most, c);
    };
    // a piece past the end is shut; the loop's bounds are the wave's, as its lanes act together
    for (int q = p0; q < p1; q += 2 * 64 * W) {
      float v[kPiece], w[kPiece];
      const int p = q + in, p2 = p + 64 * W;
      const bool two = q + 64 * W < p1;
      load_piece(row, p < p1 ? p * kPiece : a.vocab, a.vocab, v);
      if (two) load_piece(row, p2 < p1 ? p2 * kPiece : a.vocab, a.vocab, w);
      take(v, p, q == p0);
      if (two) take(w, p2, false);
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
          uint64_t k[1] = {j < a.top ? lists[from][j] : 0ull};
          mine = wave_top(k, a.top);
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
        finish(a, row, t, sum, mine);
      }
    }
    if (W > 1) __syncthreads();   // parts and lists are free again
  }
}

// joins the splits of a row, one wave a row
template <class T, bool TOP>
__global__ __launch_bounds__(64) void k_logprobs_join(LogprobArgs a, const T *logits) {
  const float c = a.scale * kLog2e;
  for (int64_t t = blockIdx.x; t < a.n_tokens; t += gridDim.x) {
    Sums sum = Sums::none();
    for (int p = lane_id(); p < a.splits; p += 64) {
      const float *s = a.sums + 3 * (t * a.splits + p);
      sum.join({s[0], s[1], s[2]}, c);
    }
    sum = wave_sums(sum, c);
    uint64_t best = 0ull;
    if (TOP) {
      const int n = a.splits * a.top;
      for (int i0 = 0; i0 < n; i0 += 64 * 7) {
        uint64_t k[8];
#pragma unroll
        for (int i = 0; i < 7; ++i) k[i] = i0 + 64 * i + lane_id() < n ? a.best[t * n + i0 + 64 * i + lane_id()] : 0ull;
        k[7] = best;   // the best so far, in the first `top` lanes
        best = wave_top(k, a.top);
      }
    }
    finish(a, logits + t * a.vocab, t, sum, best);
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
    for (int p = p0 + in; p < p1; p += 64 * W) {
      const int first = p * kPiece;
      float v[kPiece];
      load_piece(row, first, a.vocab, v);
      const int at = given ? (int)token - first : -1;
#pragma unroll
      for (int i = 0; i < kPiece; ++i) {
        const float x = exponent(v[i], peak, c);
        const float g = __builtin_amdgcn_exp2f(x - log_z) * fmaf(B, x, A);
        v[i] = i == at && v[i] > -INFINITY ? g + d : g;
      }
      if (first + kPiece <= a.vocab) {
        Eight<T> r;
#pragma unroll
        for (int i = 0; i < kPiece; ++i) r.v[i] = (T)v[i];
        *reinterpret_cast<Piece<T> *>(out + first) = __builtin_bit_cast(Piece<T>, r);
      } else {
#pragma unroll
        for (int i = 0; i < kPiece; ++i)
          if (first + i < a.vocab) out[first + i] = (T)v[i];
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
  if (!(scale > 0.f && scale <= FLT_MAX)) return report(SVT_EINVAL, "%s: scale %g is not positive and finite", who, scale);
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
  if (!(scale > 0.f && scale <= FLT_MAX)) return report(SVT_EINVAL, "%s: scale %g is not positive and finite", who, scale);
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

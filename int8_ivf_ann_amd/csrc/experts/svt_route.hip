// svt_route.hip - the router of a mixture of experts on gfx950: softmax over a token's expert logits, the
// `top` best experts and their weights; and the gradient of those weights back to the logits.
//
//   p = softmax(l)                  over the open experts (a logit of -inf or NaN shuts its expert)
//   s_j = the top best experts by (l desc, id asc)
//   w_j = p_{s_j},  or renormalised over the chosen ones: exp(l_{s_j}) / sum_m exp(l_{s_m})
//   dl_i = P_i (sum_{j: s_j = i} dw_j - sum_j dw_j w_j), with P = p, or (renormalised) w on the chosen
//          experts and 0 elsewhere
//
// A token belongs to a group of L lanes (L = 1 .. 64, the least power of two with kPer logits a lane), so
// a wave holds 64 / L tokens and a row of logits is read once into registers.  Each lane sorts its logits
// (a network of 19 exchanges).  Up to 8 choices, the lanes then merge their lists pairwise: of two descending
// lists the 8 best are max(a_i, b_{7-i}), put in order by 12 exchanges; log2 L merges, no branch.  Above 8,
// `top` rounds take the group's best head by DPP moves, and the lane that held it moves up.  Logits become integers
// of the same order, so ties go to the lowest expert in every type; with 16-bit logits one integer holds the logit
// and the expert.  Maximum, sums and weights are float32.
//
// Measured, 65536 tokens, 64 experts, top 8, softmax over all experts: the choice 7.8 us for bfloat16, 7.7 for
// float16, 12.7 for float32 (12.6 and 21 MB, so 1.6 TB/s), the gradient 9.6, 9.5 and 11.6 (23 and 40 MB); one after
// the other, the logits still in a cache, 16.5 for bfloat16.  A wave loads, computes and stores once, and all waves
// that fit the card run in step, so that the memory waits while they compute: without the lists' sort and merges the
// choice still takes 5.9 us.  Rounds instead of merges: 8.0 against 7.6.

#include <type_traits>

#include "svt_experts.h"

namespace svt {

namespace {

constexpr int kPer = 8;            // logits per lane
constexpr int kRouteThreads = 256;
static_assert(SVT_MAX_EXPERTS == 64 * kPer, "one wave holds the widest row");

// float -> uint32 whose unsigned order is the float order (-0 as 0, +inf as the largest finite value, so that they tie
// and its weight is a number); 0 for a shut expert (-inf or NaN)
__device__ __forceinline__ uint32_t logit_order(float f) {
  const uint32_t b = __float_as_uint(fminf(f, FLT_MAX) + 0.f);
  return f > -INFINITY ? ((b & 0x80000000u) ? ~b : (b | 0x80000000u)) : 0u;
}
// its inverse
__device__ __forceinline__ float order_logit(uint32_t o) {
  return __uint_as_float((o & 0x80000000u) ? (o & 0x7FFFFFFFu) : ~o);
}

// v of a lane in the neighbouring aligned group of STEP lanes (any of them: they agree)
template <int STEP>
__device__ __forceinline__ uint32_t half_other(uint32_t v) {
  if constexpr (STEP == 1) return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, true);
  else if constexpr (STEP == 2) return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, true);
  else if constexpr (STEP == 4) return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x141, 0xF, 0xF, true);
  else if constexpr (STEP == 8) return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x140, 0xF, 0xF, true);
  else return (uint32_t)__shfl_xor((int)v, STEP);
}

// exp(x) for x <= 0, and for NaN 0 (which stands for a shut expert), for +inf 1 (+inf counts as the peak).
// x log2 e = n + f with n a whole number and |f| <= 1/2 (to the last bit: the product is subtracted unrounded, and its
// constant's rest added), exp = 2^f 2^n.  f is off by u, the hardware's 2^f by 1 ulp, so the result by 3 u; below
// 2^-126, which the hardware's 2^x would flush, 2^n rounds it to a subnormal.  0 below -200.
__device__ __forceinline__ float exp_below(float x) {
  constexpr float kLog2e = 1.44269502e+0f, kLog2eRest = 1.92596299e-8f;
  x = fminf(fmaxf(x, -200.f), 0.f);
  const float n = __builtin_rintf(x * kLog2e);
  const float f = fmaf(x, kLog2eRest, fmaf(x, kLog2e, -n));
  return ldexpf(__builtin_amdgcn_exp2f(f), (int)n);
}

// A logit and its expert; greater: (logit desc, expert asc).
// 16-bit logits: one integer, the logit's bits made ascending (0: shut) above 65535 - expert.
template <class T>
struct Choice {
  uint32_t key;
  __device__ __forceinline__ static Choice make(float f, int expert) {
    uint32_t b = (uint32_t)__builtin_bit_cast(uint16_t, (T)f) << 16;   // exact: f was a T
    b = b == 0x80000000u ? 0u : b;                                     // -0 as 0
    const uint32_t o = b ^ (uint32_t)((int32_t)b >> 31 | (int32_t)0x80000000);
    return {f > -INFINITY ? (o & 0xFFFF0000u) | (uint32_t)(65535 - expert) : 0u};
  }
  __device__ __forceinline__ bool open() const { return key != 0u; }
  __device__ __forceinline__ float logit() const {
    const uint32_t o = key >> 16;
    return fminf((float)__builtin_bit_cast(T, (uint16_t)((o & 0x8000u) ? o & 0x7FFFu : ~o)), FLT_MAX);
  }
  __device__ __forceinline__ int expert() const { return 65535 - (int)(key & 0xFFFFu); }
  __device__ __forceinline__ bool same(Choice c) const { return key == c.key; }
  __device__ __forceinline__ static void order(Choice &a, Choice &b) {   // a the greater
    const uint32_t x = a.key, y = b.key;
    a.key = x > y ? x : y;
    b.key = x > y ? y : x;
  }
  __device__ __forceinline__ static Choice best(Choice c, int L) { return {group_max(c.key, L)}; }
  template <int STEP>
  __device__ __forceinline__ Choice other() const { return {half_other<STEP>(key)}; }
};
template <>
struct Choice<float> {
  uint32_t o, id;
  __device__ __forceinline__ static Choice make(float f, int expert) { return {logit_order(f), (uint32_t)expert}; }
  __device__ __forceinline__ bool open() const { return o != 0u; }
  __device__ __forceinline__ float logit() const { return order_logit(o); }
  __device__ __forceinline__ int expert() const { return (int)id; }
  __device__ __forceinline__ bool same(Choice c) const { return id == c.id && o == c.o; }
  __device__ __forceinline__ static void order(Choice &a, Choice &b) {
    const bool swap = b.o > a.o || (b.o == a.o && b.id < a.id);
    const Choice x = a, y = b;
    a = swap ? y : x;
    b = swap ? x : y;
  }
  __device__ __forceinline__ static Choice best(Choice c, int L) {
    const uint32_t m = group_max(c.o, L);
    return {m, ~group_max(c.o == m ? ~c.id : 0u, L)};
  }
  template <int STEP>
  __device__ __forceinline__ Choice other() const { return {half_other<STEP>(o), half_other<STEP>(id)}; }
};

struct __attribute__((packed, aligned(2))) Eight16 { uint16_t v[8]; };
struct __attribute__((packed, aligned(4))) Eight32 { float v[8]; };

// the lane's kPer logits, kPer * lane .. of a row of E (shut past its end)
template <class T>
__device__ __forceinline__ void load_logits(const T *row, int first, int E, float (&v)[kPer]) {
  if (first + kPer <= E) {
    if constexpr (sizeof(T) == 4) {
      const Eight32 r = *reinterpret_cast<const Eight32 *>(row + first);
#pragma unroll
      for (int i = 0; i < kPer; ++i) v[i] = r.v[i];
    } else {
      const Eight16 r = *reinterpret_cast<const Eight16 *>(row + first);
#pragma unroll
      for (int i = 0; i < kPer; ++i) v[i] = (float)__builtin_bit_cast(T, r.v[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < kPer; ++i) v[i] = first + i < E ? (float)row[first + i] : -INFINITY;
  }
}

// descending, by a network of 19 exchanges
template <class C>
__device__ __forceinline__ void sort_eight(C (&c)[kPer]) {
  constexpr int pairs[19][2] = {{0, 1}, {2, 3}, {4, 5}, {6, 7}, {0, 2}, {1, 3}, {4, 6}, {5, 7}, {1, 2}, {5, 6},
                                {0, 4}, {1, 5}, {2, 6}, {3, 7}, {2, 4}, {3, 5}, {1, 2}, {3, 4}, {5, 6}};
#pragma unroll
  for (int i = 0; i < 19; ++i) C::order(c[pairs[i][0]], c[pairs[i][1]]);
}

// the 8 best of the lists (descending) of lane groups STEP apart, in both
template <int STEP, class C>
__device__ __forceinline__ void merge_eight(C (&c)[kPer]) {
  C o[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) o[i] = c[kPer - 1 - i].template other<STEP>();
#pragma unroll
  for (int i = 0; i < kPer; ++i) C::order(c[i], o[i]);
#pragma unroll
  for (int d = kPer / 2; d > 0; d /= 2)
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (!(i & d)) C::order(c[i], c[i + d]);
}

template <class T, int L, bool ROUNDS>
__global__ __launch_bounds__(kRouteThreads) void k_route(const T *logits, int64_t n_tokens, int E, int top,
                                                         int renormalise, int32_t *out_experts, float *out_weights) {
  using C = Choice<T>;
  const int in = threadIdx.x % L, first = in * kPer;
  // entries a lane keeps (entry j with lane j % L): top <= 16, and top <= E <= kPer L
  constexpr int kMost = ROUNDS ? SVT_MAX_TOP : kPer;
  constexpr int kTop = kMost < kPer * L ? kMost : kPer * L, kKept = (kTop + L - 1) / L;
  const int64_t per_block = kRouteThreads / L;
  for (int64_t t0 = blockIdx.x * per_block; t0 < n_tokens; t0 += gridDim.x * per_block) {
    // every lane of the wave takes part in the group moves: a token past the end is a copy of the last
    const int64_t t = t0 + threadIdx.x / L;
    const int64_t tr = t < n_tokens ? t : n_tokens - 1;
    float v[kPer];
    load_logits(logits + tr * E, first, E, v);
    C c[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) c[i] = C::make(v[i], first + i);
    sort_eight(c);
    C kept[kKept];
    C peak{};
    if constexpr (ROUNDS) {
#pragma unroll
      for (int j = 0; j < kTop; ++j)
        if (j < top) {
          const C best = C::best(c[0], L);
          if (j == 0) peak = best;
          if (in == j % L) kept[j / L] = best;
          const bool mine = c[0].same(best);
#pragma unroll
          for (int i = 0; i + 1 < kPer; ++i) c[i] = mine ? c[i + 1] : c[i];
          if (mine) c[kPer - 1] = C{};
        }
    } else {
      if constexpr (L >= 2) merge_eight<1>(c);
      if constexpr (L >= 4) merge_eight<2>(c);
      if constexpr (L >= 8) merge_eight<4>(c);
      if constexpr (L >= 16) merge_eight<8>(c);
      if constexpr (L >= 32) merge_eight<16>(c);
      if constexpr (L >= 64) merge_eight<32>(c);
      peak = c[0];
#pragma unroll
      for (int q = 0; q < kKept; ++q) {
        kept[q] = c[q * L < kPer ? q * L : 0];
#pragma unroll
        for (int i = 1; i < L && q * L + i < kPer; ++i)
          if (in == i) kept[q] = c[q * L + i];
      }
    }
    const float high = peak.open() ? peak.logit() : 0.f;
    float e[kKept], sum = 0.f;
#pragma unroll
    for (int q = 0; q < kKept; ++q) {
      const bool open = q * L + in < top && kept[q].open();
      e[q] = open ? exp_below(kept[q].logit() - high) : 0.f;
      sum += e[q];
    }
    if (!renormalise) {
      sum = 0.f;
#pragma unroll
      for (int i = 0; i < kPer; ++i) sum += exp_below(v[i] - high);
    }
    sum = group_add(sum, L);
    const float scale = sum > 0.f ? sum : 1.f;
    if (t < n_tokens) {
#pragma unroll
      for (int q = 0; q < kKept; ++q) {
        const int j = q * L + in;
        if (j < top) {
          out_experts[t * top + j] = kept[q].open() ? kept[q].expert() : -1;
          out_weights[t * top + j] = e[q] / scale;
        }
      }
    }
  }
}

// between LDS operations of one wave that reach the same addresses: the hardware keeps them in order, so that only the
// compiler has to
__device__ __forceinline__ void wave_order() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// The weights' gradients reach their experts' lanes through LDS.  An expert named more than once gets every part, in
// the order of the choices: each choice's additions are an instruction of their own, and a wave's LDS operations stay
// in order (one instruction for all lanes' choices would add them in no defined order).  A token's lanes lie in one wave,
// so no workgroup barrier is needed.
template <class T, int L>
__global__ __launch_bounds__(kRouteThreads) void k_route_backward(const T *logits, int64_t n_tokens, int E, int top,
                                                                  int renormalise, const int32_t *experts,
                                                                  const float *weights, const float *d_weights,
                                                                  T *d_logits) {
  __shared__ __attribute__((aligned(16))) float spread[kRouteThreads][kPer];
  const int in = threadIdx.x % L, first = in * kPer;
  constexpr int kTop = SVT_MAX_TOP < kPer * L ? SVT_MAX_TOP : kPer * L, kKept = (kTop + L - 1) / L;
  float *own = spread[threadIdx.x], *token = spread[threadIdx.x - in];
  const int64_t per_block = kRouteThreads / L;
  for (int64_t t0 = blockIdx.x * per_block; t0 < n_tokens; t0 += gridDim.x * per_block) {
    const int64_t t = t0 + threadIdx.x / L;
    const int64_t tr = t < n_tokens ? t : n_tokens - 1;
    float v[kPer];
    load_logits(logits + tr * E, first, E, v);
#pragma unroll
    for (int i = 0; i < kPer; ++i) own[i] = 0.f;
    int id[kKept];   // entry q L + in; -1: none
    float w[kKept], d[kKept], dot = 0.f;
#pragma unroll
    for (int q = 0; q < kKept; ++q) {
      const int j = q * L + in < top ? q * L + in : 0;
      id[q] = experts[tr * top + j];
      w[q] = weights[tr * top + j];
      d[q] = d_weights[tr * top + j];
      if (q * L + in >= top || (uint32_t)id[q] >= (uint32_t)E) id[q] = -1;
      dot += id[q] >= 0 ? d[q] * w[q] : 0.f;
    }
    dot = group_add(dot, L);
    wave_order();
#pragma unroll
    for (int q = 0; q < kKept; ++q) {
      const float part = renormalise ? w[q] * (d[q] - dot) : d[q];
#pragma unroll 1
      for (int i = 0; i < L && q * L + i < top; ++i) {
        if (in == i && id[q] >= 0) atomicAdd(&token[id[q]], part);
        wave_order();   // the compiler may not join two choices' additions
      }
    }
    float g[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) g[i] = own[i];
    if (!renormalise) {
      uint32_t best = 0u;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const uint32_t o = logit_order(v[i]);
        best = o > best ? o : best;
      }
      best = group_max(best, L);
      const float high = best ? order_logit(best) : 0.f;
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        v[i] = exp_below(v[i] - high);
        sum += v[i];
      }
      sum = group_add(sum, L);
      const float inv = sum > 0.f ? 1.f / sum : 0.f;
#pragma unroll
      for (int i = 0; i < kPer; ++i) g[i] = v[i] * inv * (g[i] - dot);
    }
    if (t >= n_tokens) continue;
    T *out = d_logits + t * E + first;
    if (first + kPer <= E) {
      if constexpr (sizeof(T) == 4) {
        Eight32 r;
#pragma unroll
        for (int i = 0; i < kPer; ++i) r.v[i] = g[i];
        *reinterpret_cast<Eight32 *>(out) = r;
      } else {
        Eight16 r;
#pragma unroll
        for (int i = 0; i < kPer; ++i) r.v[i] = __builtin_bit_cast(uint16_t, (T)g[i]);
        *reinterpret_cast<Eight16 *>(out) = r;
      }
    } else {
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (first + i < E) out[i] = (T)g[i];
    }
  }
}

// f of the group width for E experts as a constant
template <class F>
int with_lanes(int E, F f) {
  const int need = (E + kPer - 1) / kPer;
  if (need <= 1) return f(std::integral_constant<int, 1>{});
  if (need <= 2) return f(std::integral_constant<int, 2>{});
  if (need <= 4) return f(std::integral_constant<int, 4>{});
  if (need <= 8) return f(std::integral_constant<int, 8>{});
  if (need <= 16) return f(std::integral_constant<int, 16>{});
  if (need <= 32) return f(std::integral_constant<int, 32>{});
  return f(std::integral_constant<int, 64>{});
}

unsigned route_grid(int64_t n_tokens, int lanes) {
  const int64_t per = kRouteThreads / lanes, n = (n_tokens + per - 1) / per;
  return (unsigned)(n < 65536 ? n : 65536);
}

int check_route(const char *who, int32_t n_tokens, int32_t n_experts, int32_t top, int32_t dtype,
                int32_t renormalise) {
  if (n_tokens < 0) return report(SVT_EINVAL, "%s: n_tokens %d < 0", who, n_tokens);
  if (n_experts < 1 || n_experts > SVT_MAX_EXPERTS)
    return report(SVT_EINVAL, "%s: n_experts %d out of [1, %d]", who, n_experts, SVT_MAX_EXPERTS);
  if (top < 1 || top > SVT_MAX_TOP || top > n_experts)
    return report(SVT_EINVAL, "%s: top %d out of [1, min(%d, n_experts)]", who, top, SVT_MAX_TOP);
  if (!elem_size(dtype)) return report(SVT_EINVAL, "%s: unknown element type %d", who, dtype);
  if (renormalise != 0 && renormalise != 1) return report(SVT_EINVAL, "%s: renormalise %d is not 0 or 1", who, renormalise);
  return SVT_OK;
}

}  // namespace

}  // namespace svt

using namespace svt;

extern "C" int svt_route(int32_t n_tokens, int32_t n_experts, int32_t top, int32_t dtype, const void *logits,
                         int32_t renormalise, int32_t *out_experts, float *out_weights, void *hip_stream) {
  const char *who = "svt_route";
  (void)report(SVT_OK, "%s", "");
  int rc = check_route(who, n_tokens, n_experts, top, dtype, renormalise);
  if (rc != SVT_OK || n_tokens == 0) return rc;
  if (!logits || !out_experts || !out_weights) return report(SVT_EINVAL, "%s: NULL logits or output", who);
  if (misaligned(logits, elem_size(dtype)) || misaligned(out_experts, 4) || misaligned(out_weights, 4))
    return report(SVT_EINVAL, "%s: misaligned logits or output", who);
  const size_t nl = (size_t)n_tokens * n_experts * elem_size(dtype), no = (size_t)n_tokens * top * 4;
  if (overlap(logits, nl, out_experts, no) || overlap(logits, nl, out_weights, no) ||
      overlap(out_experts, no, out_weights, no))
    return report(SVT_EINVAL, "%s: an output overlaps the logits or the other output", who);
  return with_type(dtype, [&](auto ty) {
    using T = decltype(ty);
    return with_lanes(n_experts, [&](auto lanes) {
      constexpr int L = decltype(lanes)::value;
      auto go = [&](auto rounds) {
        return launch(who, k_route<T, L, decltype(rounds)::value>, route_grid(n_tokens, L), kRouteThreads, 0, hip_stream,
                      (const T *)logits, n_tokens, n_experts, top, renormalise, out_experts, out_weights);
      };
      if constexpr (L > 1)   // one lane holds at most kPer experts
        if (top > kPer) return go(std::true_type{});
      return go(std::false_type{});
    });
  });
}

extern "C" int svt_route_backward(int32_t n_tokens, int32_t n_experts, int32_t top, int32_t dtype, const void *logits,
                                  int32_t renormalise, const int32_t *experts, const float *weights,
                                  const float *d_weights, void *d_logits, void *hip_stream) {
  const char *who = "svt_route_backward";
  (void)report(SVT_OK, "%s", "");
  int rc = check_route(who, n_tokens, n_experts, top, dtype, renormalise);
  if (rc != SVT_OK || n_tokens == 0) return rc;
  if (!logits || !experts || !weights || !d_weights || !d_logits)
    return report(SVT_EINVAL, "%s: NULL input or output", who);
  const int b = elem_size(dtype);
  if (misaligned(logits, b) || misaligned(d_logits, b) || misaligned(experts, 4) || misaligned(weights, 4) ||
      misaligned(d_weights, 4))
    return report(SVT_EINVAL, "%s: misaligned input or output", who);
  const size_t nl = (size_t)n_tokens * n_experts * b, nk = (size_t)n_tokens * top * 4;
  if (overlap(d_logits, nl, logits, nl) || overlap(d_logits, nl, experts, nk) || overlap(d_logits, nl, weights, nk) ||
      overlap(d_logits, nl, d_weights, nk))
    return report(SVT_EINVAL, "%s: d_logits overlaps an input", who);
  return with_type(dtype, [&](auto ty) {
    using T = decltype(ty);
    return with_lanes(n_experts, [&](auto lanes) {
      constexpr int L = decltype(lanes)::value;
      return launch(who, k_route_backward<T, L>, route_grid(n_tokens, L), kRouteThreads, 0, hip_stream,
                    (const T *)logits, n_tokens, n_experts, top, renormalise, experts, weights, d_weights, (T *)d_logits);
    });
  });
}

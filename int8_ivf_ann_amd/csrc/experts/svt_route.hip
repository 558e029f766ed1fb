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
// (a network of 19 exchanges); then `top` rounds take the group's best head by DPP moves, and the lane that
// held it moves up.  Logits become integers of the same order, so ties go to the lowest expert in every type;
// with 16-bit logits one integer holds the logit and the expert.  Maximum, sums and weights are float32.

#include <type_traits>

#include "svt_experts.h"

namespace svt {

namespace {

constexpr int kPer = 8;            // logits per lane
constexpr int kRouteThreads = 256;
static_assert(SVT_MAX_EXPERTS == 64 * kPer, "one wave holds the widest row");

// float -> uint32 whose unsigned order is the float order (-0 as 0); 0 for a shut expert (-inf or NaN)
__device__ __forceinline__ uint32_t logit_order(float f) {
  const uint32_t b = __float_as_uint(f + 0.f);
  return f > -INFINITY ? ((b & 0x80000000u) ? ~b : (b | 0x80000000u)) : 0u;
}
// its inverse; +inf counts as the largest finite value, so that its weight is a number
__device__ __forceinline__ float order_logit(uint32_t o) {
  return fminf(__uint_as_float((o & 0x80000000u) ? (o & 0x7FFFFFFFu) : ~o), FLT_MAX);
}

// exp(x) for x <= 0 (0 below -200, long past the smallest float): 2^y with y = x log2 e and the product's
// rounding put back, so that the result is off by 3 u and not by |x| u.  Half the instructions of expf.
__device__ __forceinline__ float exp_below(float x) {
  constexpr float kLog2e = 1.44269502e+0f, kLog2eRest = 1.92596299e-8f, kLn2 = 6.93147182e-1f;
  x = fmaxf(x, -200.f);
  const float y = x * kLog2e;
  const float rest = fmaf(x, kLog2eRest, fmaf(x, kLog2e, -y));
  const float e = __builtin_amdgcn_exp2f(y);
  return fmaf(e, rest * kLn2, e);
}

// A logit and its expert; greater: (logit desc, expert asc).
// 16-bit logits: one integer, the logit's bits made ascending (0: shut) above 65535 - expert.
template <class T>
struct Choice {
  uint32_t key;
  __device__ __forceinline__ static Choice make(float f, int expert) {
    const uint32_t b = __builtin_bit_cast(uint16_t, (T)(f + 0.f));   // exact; -0 as 0
    const uint32_t o = (b & 0x8000u) ? ~b & 0xFFFFu : b | 0x8000u;
    return {f > -INFINITY ? (o << 16) | (uint32_t)(65535 - expert) : 0u};
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

template <class T, int L>
__global__ __launch_bounds__(kRouteThreads) void k_route(const T *logits, int64_t n_tokens, int E, int top,
                                                         int renormalise, int32_t *out_experts, float *out_weights) {
  using C = Choice<T>;
  const int in = threadIdx.x % L, first = in * kPer;
  // entries a lane keeps (entry j with lane j % L): top <= 16, and top <= E <= kPer L
  constexpr int kTop = SVT_MAX_TOP < kPer * L ? SVT_MAX_TOP : kPer * L, kKept = (kTop + L - 1) / L;
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
      for (int i = 0; i < kPer; ++i) sum += logit_order(v[i]) ? exp_below(fminf(v[i], FLT_MAX) - high) : 0.f;
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

// The weights' gradients reach their experts' lanes through LDS (added there: an expert named twice gets
// both).
template <class T, int L>
__global__ __launch_bounds__(kRouteThreads) void k_route_backward(const T *logits, int64_t n_tokens, int E, int top,
                                                                  int renormalise, const int32_t *experts,
                                                                  const float *weights, const float *d_weights,
                                                                  T *d_logits) {
  __shared__ __attribute__((aligned(16))) float spread[kRouteThreads][kPer];
  const int in = threadIdx.x % L, first = in * kPer;
  float *own = spread[threadIdx.x], *token = spread[threadIdx.x - in];
  const int64_t per_block = kRouteThreads / L;
  for (int64_t t0 = blockIdx.x * per_block; t0 < n_tokens; t0 += gridDim.x * per_block) {
    const int64_t t = t0 + threadIdx.x / L;
    const int64_t tr = t < n_tokens ? t : n_tokens - 1;
    float v[kPer];
    load_logits(logits + tr * E, first, E, v);
#pragma unroll
    for (int i = 0; i < kPer; ++i) own[i] = 0.f;
    float dot = 0.f;
    for (int j = in; j < top; j += L) {
      const bool ok = (uint32_t)experts[tr * top + j] < (uint32_t)E;
      dot += ok ? d_weights[tr * top + j] * weights[tr * top + j] : 0.f;
    }
    dot = group_add(dot, L);
    __syncthreads();
    for (int j = in; j < top; j += L) {
      const int id = experts[tr * top + j];
      const float d = d_weights[tr * top + j];
      if ((uint32_t)id < (uint32_t)E) atomicAdd(&token[id], renormalise ? weights[tr * top + j] * (d - dot) : d);
    }
    __syncthreads();
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
        v[i] = logit_order(v[i]) ? exp_below(fminf(v[i], FLT_MAX) - high) : 0.f;
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

// calls f with the group width for E experts as a constant
template <class F>
void with_lanes(int E, F f) {
  const int need = (E + kPer - 1) / kPer;
  if (need <= 1) f(std::integral_constant<int, 1>{});
  else if (need <= 2) f(std::integral_constant<int, 2>{});
  else if (need <= 4) f(std::integral_constant<int, 4>{});
  else if (need <= 8) f(std::integral_constant<int, 8>{});
  else if (need <= 16) f(std::integral_constant<int, 16>{});
  else if (need <= 32) f(std::integral_constant<int, 32>{});
  else f(std::integral_constant<int, 64>{});
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
  with_type(dtype, [&](auto ty) {
    using T = decltype(ty);
    with_lanes(n_experts, [&](auto lanes) {
      constexpr int L = decltype(lanes)::value;
      k_route<T, L><<<route_grid(n_tokens, L), kRouteThreads, 0, (hipStream_t)hip_stream>>>(
          (const T *)logits, n_tokens, n_experts, top, renormalise, out_experts, out_weights);
    });
  });
  return launched(who);
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
  with_type(dtype, [&](auto ty) {
    using T = decltype(ty);
    with_lanes(n_experts, [&](auto lanes) {
      constexpr int L = decltype(lanes)::value;
      k_route_backward<T, L><<<route_grid(n_tokens, L), kRouteThreads, 0, (hipStream_t)hip_stream>>>(
          (const T *)logits, n_tokens, n_experts, top, renormalise, experts, weights, d_weights, (T *)d_logits);
    });
  });
  return launched(who);
}

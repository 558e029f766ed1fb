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
// a wave holds 64 / L tokens and a row of logits is read once into registers.  The choice takes `top`
// rounds: each lane's best remaining logit as an ordered integer, the group's maximum by DPP moves, the
// lowest lane that holds it (a ballot), which strikes it out.  Ordered integers compare exactly, so ties
// go to the lowest expert in every type.  Logits, maximum and sums are float32.

#include <type_traits>

#include "svt_experts.h"

namespace svt {

namespace {

constexpr int kPer = 8;            // logits per lane
constexpr int kRouteThreads = 256;
static_assert(SVT_MAX_EXPERTS == 64 * kPer, "one wave holds the widest row");

// float -> uint32 whose unsigned order is the float order; 0 for a shut expert (-inf or NaN).  +inf
// counts as the largest finite value, so that its weight is a number.
__device__ __forceinline__ uint32_t logit_order(float f) {
  if (!(f > -INFINITY)) return 0u;
  const uint32_t b = __float_as_uint(fminf(f, FLT_MAX));
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float order_logit(uint32_t o) {
  return __uint_as_float((o & 0x80000000u) ? (o & 0x7FFFFFFFu) : ~o);
}

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

template <class T, int L>
__global__ __launch_bounds__(kRouteThreads) void k_route(const T *logits, int64_t n_tokens, int E, int top,
                                                         int renormalise, int32_t *out_experts, float *out_weights) {
  const int l = threadIdx.x % 64, in = l % L, first = in * kPer;
  const uint64_t mine = (L == 64 ? ~0ull : ((1ull << (L & 63)) - 1)) << (l - in);   // this group's lanes
  // entries a lane keeps: top <= 16, and top <= E <= kPer L
  constexpr int kKept = ((SVT_MAX_TOP < kPer * L ? SVT_MAX_TOP : kPer * L) + L - 1) / L;
  const int64_t per_block = kRouteThreads / L;
  for (int64_t t0 = blockIdx.x * per_block; t0 < n_tokens; t0 += gridDim.x * per_block) {
    // every lane of the wave takes part in the group moves: a token past the end is a copy of the last
    const int64_t t = t0 + threadIdx.x / L;
    const int64_t tr = t < n_tokens ? t : n_tokens - 1;
    float v[kPer];
    load_logits(logits + tr * E, first, E, v);
    uint32_t o[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) o[i] = logit_order(v[i]);
    float peak = 0.f, total = 0.f;
    float kept_e[kKept];   // entry j stays with lane j % L until the sum is known
    int32_t kept_id[kKept];
    for (int j = 0; j < top; ++j) {
      uint32_t best = o[0];
      int at = 0;
#pragma unroll
      for (int i = 1; i < kPer; ++i)
        if (o[i] > best) { best = o[i]; at = i; }
      const uint32_t gbest = group_max(best, L);
      const int winner = __ffsll((long long)(__ballot(best == gbest) & mine)) - 1;
      const bool open = gbest != 0u;
      const int picked = L == 1 ? first + at : __shfl(first + at, winner);
      const int id = open ? picked : -1;
      if (l == winner) {
#pragma unroll
        for (int i = 0; i < kPer; ++i)
          if (i == at) o[i] = 0u;
      }
      const float x = order_logit(gbest);
      if (j == 0) {
        peak = open ? x : 0.f;
        if (!renormalise) {
          float s = 0.f;
#pragma unroll
          for (int i = 0; i < kPer; ++i) s += logit_order(v[i]) ? expf(fminf(v[i], FLT_MAX) - peak) : 0.f;
          total = group_add(s, L);
        }
      }
      const float e = open ? expf(x - peak) : 0.f;
      if (renormalise) total += e;
      if (in == j % L) {
#pragma unroll
        for (int q = 0; q < kKept; ++q)
          if (q == j / L) {
            kept_e[q] = e;
            kept_id[q] = id;
          }
      }
    }
    const float scale = total > 0.f ? total : 1.f;
    if (t < n_tokens) {
#pragma unroll
      for (int q = 0; q < kKept; ++q) {
        const int j = q * L + in;
        if (j < top) {
          out_experts[t * top + j] = kept_id[q];
          out_weights[t * top + j] = kept_e[q] / scale;
        }
      }
    }
  }
}

template <class T, int L>
__global__ __launch_bounds__(kRouteThreads) void k_route_backward(const T *logits, int64_t n_tokens, int E, int top,
                                                                  int renormalise, const int32_t *experts,
                                                                  const float *weights, const float *d_weights,
                                                                  T *d_logits) {
  const int l = threadIdx.x % 64, in = l % L, first = in * kPer;
  const int64_t per_block = kRouteThreads / L;
  for (int64_t t0 = blockIdx.x * per_block; t0 < n_tokens; t0 += gridDim.x * per_block) {
    const int64_t t = t0 + threadIdx.x / L;
    const int64_t tr = t < n_tokens ? t : n_tokens - 1;
    const int32_t *ids = experts + tr * top;
    const float *w = weights + tr * top, *dw = d_weights + tr * top;
    float dot = 0.f;
    for (int j = 0; j < top; ++j) dot += (uint32_t)ids[j] < (uint32_t)E ? dw[j] * w[j] : 0.f;
    float g[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) g[i] = 0.f;
    if (renormalise) {
      for (int j = 0; j < top; ++j) {
        const int at = ids[j] - first;
        const float d = w[j] * (dw[j] - dot);
#pragma unroll
        for (int i = 0; i < kPer; ++i) g[i] += at == i ? d : 0.f;
      }
    } else {
      float v[kPer];
      load_logits(logits + tr * E, first, E, v);
      uint32_t best = 0u;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const uint32_t o = logit_order(v[i]);
        best = o > best ? o : best;
      }
      best = group_max(best, L);
      const float peak = best ? order_logit(best) : 0.f;
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        v[i] = logit_order(v[i]) ? expf(fminf(v[i], FLT_MAX) - peak) : 0.f;
        s += v[i];
      }
      s = group_add(s, L);
      const float scale = s > 0.f ? s : 1.f;
      for (int j = 0; j < top; ++j) {
        const int at = ids[j] - first;
        const float d = dw[j];
#pragma unroll
        for (int i = 0; i < kPer; ++i) g[i] += at == i ? d : 0.f;
      }
#pragma unroll
      for (int i = 0; i < kPer; ++i) g[i] = v[i] / scale * (g[i] - dot);
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

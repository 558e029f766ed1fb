// svt_experts.h - shared by the routed-expert operators (svt_route.hip, svt_exchange.hip, svt_quant.hip):
// element types, conversions, lane-group reductions and host-side argument checks.  Not installed.
#pragma once

#include <hip/hip_runtime.h>
#include <float.h>
#include <stdint.h>

#include "svt.h"
#include "../svt_device.h"
#include "../svt_internal.h"

namespace svt {

typedef _Float16 f16;
typedef __bf16 bf16;

// ---- host ----------------------------------------------------------------------------------------

inline int elem_size(int32_t dtype) { return dtype == SVT_F32 ? 4 : (dtype == SVT_F16 || dtype == SVT_BF16) ? 2 : 0; }

inline bool misaligned(const void *p, size_t n) { return ((uintptr_t)p & (n - 1)) != 0; }

// whether [a, a + na) and [b, b + nb) share a byte
inline bool overlap(const void *a, size_t na, const void *b, size_t nb) {
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return a && b && na && nb && x < y + nb && y < x + na;
}

// f of a value of the element type that dtype names (dtype was checked)
template <class F>
int with_type(int32_t dtype, F f) {
  switch (dtype) {
    case SVT_F32: return f(float{});
    case SVT_F16: return f(f16{});
    default: return f(bf16{});
  }
}

// Launches a kernel: SVT_OK, or its failure reported.  The status is this launch's own (an error that an earlier call
// left unread is its caller's, and stays), so that a call of several launches can end at the one that failed.
template <class... P, class... A>
int launch(const char *who, void (*kernel)(P...), dim3 grid, unsigned threads, size_t lds, void *stream, A... args) {
  static_assert(sizeof...(P) == sizeof...(A), "one argument per parameter");
  return [&](P... values) {   // converted to the kernel's types
    void *ptrs[] = {(void *)&values...};
    const hipError_t e = hipLaunchKernel((const void *)kernel, grid, dim3(threads), ptrs, lds, (hipStream_t)stream);
    if (e == hipSuccess) return (int)SVT_OK;
    (void)hipGetLastError();   // reported here
    return report(SVT_EDEVICE, "%s: launch: %s", who, hipGetErrorString(e));
  }(args...);
}

// ---- device --------------------------------------------------------------------------------------

// Reductions over aligned groups of L lanes (a power of two, at most 64); every lane gets the result.
// Within 16 lanes: DPP moves (lane ^ 1 and ^ 2 as quad permutations, then mirrors of 8 and of 16 lanes,
// which pair the already uniform halves); beyond: shuffles.
template <class Op>
__device__ __forceinline__ uint32_t group_reduce(uint32_t v, int L, Op op) {
  if (L >= 2) v = op(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, true));
  if (L >= 4) v = op(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, true));
  if (L >= 8) v = op(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xF, 0xF, true));
  if (L >= 16) v = op(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x140, 0xF, 0xF, true));
  if (L >= 32) v = op(v, (uint32_t)__shfl_xor((int)v, 16));
  if (L >= 64) v = op(v, (uint32_t)__shfl_xor((int)v, 32));
  return v;
}
__device__ __forceinline__ uint32_t group_max(uint32_t v, int L) {
  return group_reduce(v, L, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}
__device__ __forceinline__ float group_add(float v, int L) {
  return __uint_as_float(group_reduce(__float_as_uint(v), L, [](uint32_t a, uint32_t b) {
    return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
  }));
}

// inclusive sums over the wave's lanes: shifts inside rows of 16 lanes, then each row's last lane to the next
// row (1 and 3), then lane 31 to the upper half
__device__ __forceinline__ int incl_sums(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, true);    // row_shr:1
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);   // row_bcast:15
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);   // row_bcast:31
  return v;
}

}  // namespace svt

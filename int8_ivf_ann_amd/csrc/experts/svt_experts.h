// svt_experts.h - shared by the operators of experts/ and scorer/: element types, conversions, lane-group reductions,
// ranks by bin and host-side argument checks.  Not installed.
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

// The grid of a kernel that numbers its workgroups by block_number(): rows of 2^22, so that the threads along x stay below
// 2^32; at most 2^32 workgroups, which arrays that fit the memory stay far below.  The last row may not be full.
constexpr int64_t kGridRow = 1 << 22;
inline bool fits(int64_t blocks) { return blocks < int64_t(1) << 32; }
inline dim3 grid_of(int64_t blocks) {
  return blocks <= kGridRow ? dim3((unsigned)blocks) : dim3((unsigned)kGridRow, (unsigned)((blocks + kGridRow - 1) / kGridRow));
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

__device__ __forceinline__ int64_t block_number() { return blockIdx.y * (int64_t)gridDim.x + blockIdx.x; }

// Reductions over aligned groups of L lanes (a power of two, at most 64); every lane gets the result.
// Within 16 lanes: DPP moves (lane ^ 1 and ^ 2 as quad permutations, then mirrors of 8 and of 16 lanes,
// which pair the already uniform halves); beyond: moves that exchange rows of 16 lanes, then halves of the wave.
template <class Op>
__device__ __forceinline__ uint32_t group_reduce(uint32_t v, int L, Op op) {
  if (L >= 2) v = op(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, true));
  if (L >= 4) v = op(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, true));
  if (L >= 8) v = op(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xF, 0xF, true));
  if (L >= 16) v = op(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x140, 0xF, 0xF, true));
  if (L >= 32) {
    const auto p = __builtin_amdgcn_permlane16_swap(v, v, false, false);   // (even rows twice, odd rows twice)
    v = op(p[0], p[1]);
  }
  if (L >= 64) {
    const auto p = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    v = op(p[0], p[1]);
  }
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

// the lanes of this wave whose bin e, below 2^BITS, equals this lane's (0 for a lane without one, e < 0)
template <int BITS>
__device__ __forceinline__ uint64_t same_bin(int e) {
  uint64_t same = __ballot(e >= 0);
#pragma unroll
  for (int b = 0; b < BITS; ++b) {
    const uint64_t one = __ballot((e >> b) & 1);
    same &= ((e >> b) & 1) ? one : ~one;
  }
  return e >= 0 ? same : 0ull;
}

// ranks of a wave's entries by bin, step by step: rank[q] = entries of the same bin before it in the wave's piece;
// count[e] (the wave's own, cleared) becomes the piece's entries of e
template <int STEPS, int BITS>
__device__ __forceinline__ void rank_entries(const int (&e)[STEPS], int (&rank)[STEPS], volatile int32_t *count) {
  const int l = lane_id();
#pragma unroll
  for (int q = 0; q < STEPS; ++q) {
    const uint64_t same = same_bin<BITS>(e[q]);
    rank[q] = 0;
    if (e[q] >= 0) {
      rank[q] = count[e[q]] + mbcnt(same);
      // the last lane of each bin moves the count on; a wave's LDS operations stay in order
      if ((same >> l) == 1ull) count[e[q]] = rank[q] + 1;
    }
  }
}

}  // namespace svt

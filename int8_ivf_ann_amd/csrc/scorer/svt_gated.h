// svt_gated.h - the kernels of products with a gate and of their gradients (svt_gated_*.hip instantiate them, one file
// per type; svt_gated.hip checks arguments and calls).
//
//   g = x Wg^T,  u = x Wu^T,  h = act(g) u                          rows r, inputs k, outputs n
//   dg = dh u act'(g),  du = dh act(g)
//   dx = dg Wg + du Wu,  dWg = dg^T x,  dWu = du^T x
//
// All three products run on the matrix cores with float32 accumulation (16 x 16 x 32 instructions for two-byte types,
// 16 x 16 x 4 for float32).  A workgroup computes a tile of `Q rows x P columns` of the result; per step it brings 128
// bytes of the reduced index of each side to LDS, straight from memory (two buffers, so that a step's loads are in flight
// while the step before is multiplied).
//   side P   the columns of the result, which lie together in memory: the first operand, so that a lane ends up with four
//            neighbouring columns of one row
//   side Q   its rows
// A side is read in one of two forms:
//   along    the reduced index lies together (x and W forward; dg, du for dx): rows of 128 bytes in LDS, a fragment is
//            one 16-byte read
//   across   the other index lies together (W for dx; x, dg, du for dW): rows of the tile's width for each reduced index,
//            and the transposing read of LDS (float32: single values) collects a fragment
// In both, the 16-byte pieces of a row are permuted by the row's number, so that the lanes of a read spread over the
// banks.  Pieces outside the matrix are zeros: their address lies outside the buffer's range.  Rows need only begin at
// multiples of 4 bytes: the loads ask for no more, the range ends with the array (every 4 bytes are checked by themselves),
// and a piece that runs on into the next row is cleared in LDS, in the last step alone.
#pragma once

#include <type_traits>

#include "../experts/svt_experts.h"

namespace svt {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef f16 f16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
typedef __attribute__((address_space(3))) void lds_void;

constexpr int32_t kGatedMax = 1 << 20;   // inputs, outputs

// ---- activations ---------------------------------------------------------------------------------

constexpr float kGateLog2e = 1.44269504088896341f;

// 2^x, x <= 0.  The instruction gives 0 below 2^-126, which a factor of 100 would bring back up: its argument is moved.
__device__ __forceinline__ float exp2_below(float x) {
  const bool low = x < -126.f;
  return __builtin_amdgcn_exp2f(low ? x + 64.f : x) * (low ? 0x1p-64f : 1.f);
}

// 2^32 / (1 + e^-v), with e^-v as a square: neither it nor the reciprocal's result leaves the normal range where v times the
// whole is above 2^-126 (8192 x 2048 x 8192 bfloat16: e^-v itself, unscaled, 564 us, e^-|v| with its two cases 577, this 569).
// The exponential instruction's rounded argument is off by |v| 2^-24, which two-byte results do not show; float32's take the
// library's function.
template <class T>
__device__ __forceinline__ float logistic(float v) {
  float h;
  if constexpr (sizeof(T) == 4) h = expf(-0.5f * v);
  else h = __builtin_amdgcn_exp2f(-0.5f * kGateLog2e * v);
  return __builtin_amdgcn_rcpf(fmaf(h * 0x1p-32f, h, 0x1p-32f));
}

// v times the whole, l its 2^32-fold, which alone may leave the normal range (two-byte results do not show that either)
template <class T>
__device__ __forceinline__ float silu(float v, float l) {
  if constexpr (sizeof(T) == 4) return v < 0.f ? v * l * 0x1p-32f : v * (l * 0x1p-32f);
  else return v * (l * 0x1p-32f);
}

// the normal distribution's integral up to v and its density at v, times v
struct Normal { float below, slope; };
template <class T>
__device__ __forceinline__ Normal normal(float v) {
  constexpr float c = 0.39894228040143268f, r = 0.70710678118654752f;
  if constexpr (sizeof(T) == 4) {   // with what v^2 and the error function's argument were rounded by
    const float w = __builtin_amdgcn_fmed3f(v, -16.f, 16.f), q = w * w, off = fmaf(w, w, -q);
    const float t = expf(-0.25f * q);   // a square again, for the range
    const float a = -r * w, rest = fmaf(-r, w, -a) - (float)(0.70710678118654752440 - (double)r) * w;
    const float slope = c * w * t * t * fmaf(-0.5f, off, 1.f);
    return {fmaf(-0.56418958354775629f * rest * t, t, 0.5f * erfcf(a)), v == v ? slope : v};
  } else {
    return {0.5f * erfcf(-r * v), c * v * exp2_below(-0.5f * kGateLog2e * v * v)};
  }
}

template <int ACT, class T>
__device__ __forceinline__ float act_value(float v) {
  if constexpr (ACT == SVT_ACT_RELU) return v < 0.f ? 0.f : v;   // NaN stays NaN
  else if constexpr (ACT == SVT_ACT_SILU) return silu<T>(v, logistic<T>(v));
  else if constexpr (ACT == SVT_ACT_GELU) return v * normal<T>(v).below;
  else return v;
}

// value and slope
template <int ACT, class T>
__device__ __forceinline__ void act_both(float v, float &value, float &slope) {
  if constexpr (ACT == SVT_ACT_RELU) {
    value = v < 0.f ? 0.f : v;
    slope = v > 0.f ? 1.f : 0.f;
  } else if constexpr (ACT == SVT_ACT_SILU) {
    const float l = logistic<T>(v), s = l * 0x1p-32f;
    value = silu<T>(v, l);
    slope = fmaf(value, 1.f - s, s);
  } else if constexpr (ACT == SVT_ACT_GELU) {
    const Normal n = normal<T>(v);
    value = v * n.below;
    slope = n.slope + n.below;
  } else {
    value = v;
    slope = 1.f;
  }
}

// ---- fragments -----------------------------------------------------------------------------------

// 16 bytes of a lane: row lane % 16, reduced indexes (16 / size) (lane / 16) ..
template <class T> struct Mul;
template <> struct Mul<bf16> {
  typedef bf16x8 frag;
  static __device__ __forceinline__ f32x4 add(frag p, frag q, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(p, q, c, 0, 0, 0);
  }
};
template <> struct Mul<f16> {
  typedef f16x8 frag;
  static __device__ __forceinline__ f32x4 add(frag p, frag q, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(p, q, c, 0, 0, 0);
  }
};
template <> struct Mul<float> {
  typedef f32x4 frag;
  static __device__ __forceinline__ f32x4 add(frag p, frag q, f32x4 c) {
#pragma unroll
    for (int j = 0; j < 4; ++j) c = __builtin_amdgcn_mfma_f32_16x16x4f32(p[j], q[j], c, 0, 0, 0);
    return c;
  }
};

// ---- tiles ---------------------------------------------------------------------------------------

constexpr int kStepBytes = 128;                    // of the reduced index
constexpr uint32_t kOutside = 0x80000000u;         // an offset past every buffer's range
constexpr int kRange = 0x7FFFFFF0;

// Q x P columns of the result, waves WQ x WP, buffers
template <int Q, int P, int WQ_, int WP_, int BUFFERS>
struct Cut {
  static constexpr int q = Q, p = P, WQ = WQ_, WP = WP_, buffers = BUFFERS;
  static constexpr int threads = 64 * WQ * WP;
  static constexpr int nq = Q / WQ / 16, np = P / WP / 16;   // 16 x 16 blocks of a wave
};

// where a step's pieces begin: the side's first row (of its upper half), at the step's first reduced index
struct Base { const char *at, *upper, *end, *upper_end; };   // end: of the arrays

// One side of a tile.  ROWS: the tile's size along the side's own index; HALVES: two matrices' rows, half a tile each.
template <class T, int ROWS, int THREADS, bool ACROSS, bool HALVES = false>
struct Side {
  static constexpr int b = sizeof(T), each = 16 / b, step = kStepBytes / b;   // elements of a piece, of a step
  static constexpr int bytes = ROWS * kStepBytes;
  static constexpr int pieces = bytes / 16 / THREADS;                         // of a thread
  static constexpr int row_pieces = ACROSS ? ROWS * b / 16 : kStepBytes / 16;
  static_assert(pieces >= 1 && bytes % (16 * THREADS) == 0, "whole pieces for every thread");
  static_assert(!HALVES || (!ACROSS && pieces % 2 == 0), "a thread's pieces change matrix half way");

  // which piece of row `row` lies at its place `at` (an involution)
  static __device__ __forceinline__ int permuted(int row, int at) {
    static_assert((row_pieces & (row_pieces - 1)) == 0, "a place stays inside its row");
    if constexpr (!ACROSS) return at ^ ((row >> 1) & 7);
    else if constexpr (b == 2) return at ^ ((2 * ((row & 3) | ((row >> 3) & 1) << 2)) & (row_pieces - 1));
    else return at ^ ((4 * ((row >> 2) & 3)) & (row_pieces - 1));
  }

  uint32_t offset[pieces];   // of the thread's pieces; kOutside: zeros
  uint32_t gone;             // bit j: piece j is outside in a last step

  static __device__ __forceinline__ int row_of(int j) { return (j * THREADS + (int)threadIdx.x) / row_pieces; }
  static __device__ __forceinline__ int piece_of(int j) {
    return permuted(row_of(j), (j * THREADS + (int)threadIdx.x) % row_pieces);
  }

  // pitch: bytes of a memory row; own: valid indexes of the side (of each half); reduced: those of a last step
  __device__ __forceinline__ void init(uint32_t pitch, int own, int reduced) {
    gone = 0u;
#pragma unroll
    for (int j = 0; j < pieces; ++j) {
      const int row = row_of(j), piece = piece_of(j), mine = HALVES ? row % (ROWS / 2) : row;
      const bool out = ACROSS ? piece * each >= own : mine >= own;
      offset[j] = out ? kOutside : (uint32_t)mine * pitch + (uint32_t)piece * 16u;
      gone |= (ACROSS ? row >= reduced : piece * each >= reduced) ? 1u << j : 0u;
    }
  }

  // A step's pieces to LDS, straight from memory.  The loads are written out, as the compiler
  // would have every later read of LDS wait for them; whoever reads waits by loads_done() and a barrier.  (They have no
  // result in registers.)  The buffer's words may come from v_readfirstlane right before: a load reads such a register only
  // five wait states later, which nothing but the asm itself counts (the move of m0 one, the s_nop four).
  __device__ __forceinline__ void load(Base from, uint32_t lds, bool final) const {
    const uint32_t wave = (uint32_t)__builtin_amdgcn_readfirstlane((int)threadIdx.x / 64);
    auto buffer = [](const char *p, const char *end) {
      const uint64_t v = (uint64_t)(uintptr_t)p;
      const int64_t range = end - p;   // may be negative for an unused upper half
      const uint32_t bytes = range <= 0 ? 0u : range < kRange ? (uint32_t)range : (uint32_t)kRange;
      return u32x4{(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)v),
                   (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(v >> 32)) & 0xFFFFu,
                   (uint32_t)__builtin_amdgcn_readfirstlane((int)bytes), 0x00020000u};
    };
    const u32x4 lower = buffer(from.at, from.end);
    const u32x4 upper = HALVES ? buffer(from.upper, from.upper_end) : lower;
    const uint32_t out = final ? gone : 0u;
#pragma unroll
    for (int j = 0; j < pieces; ++j) {
      const uint32_t to = lds + (j * THREADS + wave * 64) * 16, at = out >> j & 1u ? kOutside : offset[j];
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"   // m0 is reserved, but the compiler's own uses of it have to see the write
      asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(to), "v"(at),
                   "s"(HALVES && 2 * j >= pieces ? upper : lower)
                   : "memory", "m0");
#pragma clang diagnostic pop
    }
  }

  // clears what lies behind the `reduced` valid elements of a last step in the piece that they end in
  static __device__ __forceinline__ void clear_tail(char *lds, int reduced) {
    static_assert(!ACROSS, "across, whole rows lie outside");
    for (int row = (int)threadIdx.x; row < ROWS; row += THREADS) {
      T *at = reinterpret_cast<T *>(lds + row * kStepBytes + permuted(row, reduced / each) * 16);
      for (int i = reduced % each; i < each; ++i) at[i] = (T)0.f;
    }
  }

  // the fragment of block `block` (16 own indexes), half `h` of the step
  static __device__ __forceinline__ typename Mul<T>::frag fragment(const char *lds, int block, int h) {
    const int i = lane_id() % 16, g = lane_id() / 16;
    if constexpr (!ACROSS) {
      return *reinterpret_cast<const typename Mul<T>::frag *>(lds + (block * 16 + i) * kStepBytes +
                                                              ((4 * h + g) ^ (i >> 1)) * 16);
    } else if constexpr (b == 2) {   // two transposing reads: reduced indexes 8 g .. 8 g + 3 and 8 g + 4 .. 8 g + 7
      s16x4 v[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int row = 32 * h + 8 * g + 4 * k + i / 4;
        v[k] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (lds_s16x4 *)(lds + row * (ROWS * b) + permuted(row, 2 * block + i % 4 / 2) * 16 + i % 2 * 8));
      }
      struct { s16x4 a, b; } both{v[0], v[1]};
      return __builtin_bit_cast(typename Mul<T>::frag, both);
    } else {
      typename Mul<T>::frag f;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int row = 16 * h + 4 * g + k;
        f[k] = *reinterpret_cast<const float *>(lds + row * (ROWS * b) + permuted(row, 4 * block + i / 4) * 16 + i % 4 * 4);
      }
      return f;
    }
  }
};

// all loads of this wave but the LATER latest, to registers or to LDS, have arrived
template <int LATER>
__device__ __forceinline__ void loads_done() {
  static_assert(LATER < 64, "six bits");
  __builtin_amdgcn_s_waitcnt(0x0F70 | (LATER & 15) | (LATER >> 4) << 14);
}

// acc[b][a] += the product of `steps` steps: lane l holds rows 16 b + l % 16 of its wave's part, columns
// 16 a + 4 (l / 16) .. + 3.  base(s, p, q): where step s begins; last(s): whether its pieces may end early.
// With HALVES of side P, the first np / 2 blocks are its lower, the others its upper half's.
template <class T, class C, bool PA, bool QA, bool HALVES>
struct Product {
  using SP = Side<T, C::p, C::threads, PA, HALVES>;
  using SQ = Side<T, C::q, C::threads, QA>;
  static constexpr int bytes = SP::bytes + SQ::bytes, lds_bytes = C::buffers * bytes;
  SP P;
  SQ Q;

  // a wave's fragments of half h of a step
  struct Fragments {
    typename Mul<T>::frag p[C::np], q[C::nq];
    __device__ __forceinline__ void read(const char *lds, int wq, int wp, int h) {
#pragma unroll
      for (int i = 0; i < C::np; ++i) {
        constexpr int half = C::np / 2;
        const int block = !HALVES ? wp * C::np + i : i < half ? wp * half + i : C::p / 32 + wp * half + i - half;
        p[i] = SP::fragment(lds, block, h);
      }
#pragma unroll
      for (int i = 0; i < C::nq; ++i) q[i] = SQ::fragment(lds + SP::bytes, wq * C::nq + i, h);
    }
    __device__ __forceinline__ void multiply(f32x4 (&acc)[C::nq][C::np]) const {
#pragma unroll
      for (int i = 0; i < C::nq; ++i)
#pragma unroll
        for (int j = 0; j < C::np; ++j) acc[i][j] = Mul<T>::add(p[j], q[i], acc[i][j]);
    }
  };

  // A step, with the loads of a later one.  Large parts with one workgroup a compute unit ask for both halves' fragments at
  // once, so that their waves wait for LDS once (dx of 16384 rows, 1024 inputs, 2048 outputs, 256 x 256: 119 us half by
  // half, 111 like this); where workgroups share a compute unit that costs registers for nothing (128 x 128: 122 and 127).
  template <class Next>
  static __device__ __forceinline__ void step(const char *lds, int wq, int wp, f32x4 (&acc)[C::nq][C::np], Next next) {
    Fragments f[2];
    if constexpr (C::nq * C::np > 16) {
      f[0].read(lds, wq, wp, 0);
      f[1].read(lds, wq, wp, 1);
      __builtin_amdgcn_sched_barrier(0);
      next();
      f[0].multiply(acc);
      f[1].multiply(acc);
    } else {
      next();
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        f[h].read(lds, wq, wp, h);
        f[h].multiply(acc);
      }
    }
  }

  // ragged: the valid elements of a last step where its last pieces have to be cleared (both sides along), or 0
  template <class At, class Last>
  __device__ __forceinline__ void run(int steps, int ragged, char *lds, At base, Last last,
                                      f32x4 (&acc)[C::nq][C::np]) const {
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x / 64), wq = wave / C::WP, wp = wave % C::WP;
    if (steps <= 0) return;
    const uint32_t at = (uint32_t)(uintptr_t)(lds_void *)lds;
    constexpr int ahead = C::buffers - 1;   // steps whose loads are in flight
    int in = 0, out = 0;                    // buffers, as byte offsets
    auto load = [&](int s) {
      Base p, q;
      base(s, p, q);
      const bool f = last(s);
      P.load(p, at + in, f);
      Q.load(q, at + in + SP::bytes, f);
      in = in + bytes == C::buffers * bytes ? 0 : in + bytes;
    };
    for (int s = 0; s < ahead && s < steps; ++s) load(s);
    for (int s = 0; s < steps; ++s) {
      if (s + ahead <= steps) loads_done<(ahead - 1) * (SP::pieces + SQ::pieces)>();   // later steps' are in flight
      else loads_done<0>();
      __syncthreads();   // the step's pieces are there, and the buffer before it has been read
      if constexpr (!PA && !QA)
        if (ragged && last(s)) {
          SP::clear_tail(lds + out, ragged);
          SQ::clear_tail(lds + out + SP::bytes, ragged);
          __syncthreads();
        }
      step(lds + out, wq, wp, acc, [&] {
        if (s + ahead < steps) load(s + ahead);
      });
      out = out + bytes == C::buffers * bytes ? 0 : out + bytes;
    }
  }
};

// ---- rows by expert ------------------------------------------------------------------------------

struct Rows { int matrix; int64_t first, end; };

__device__ __forceinline__ int64_t clamped(int64_t v, int64_t n) { return v < 0 ? 0 : v < n ? v : n; }

// rows of matrix e: [first, end)
__device__ __forceinline__ Rows rows_of_matrix(const int32_t *offsets, int64_t n_rows, int e) {
  if (!offsets) return {e, 0, n_rows};
  const int64_t a = clamped(offsets[e], n_rows), z = clamped(offsets[e + 1], n_rows);
  return {e, a, z > a ? z : a};
}

// blocks of `per` rows of matrices e0 .. e0 + 63, one a lane; of a matrix without rows `least`
__device__ __forceinline__ int blocks_of(const int32_t *offsets, int n_matrices, int64_t n_rows, int e0, int64_t per,
                                         int least, Rows &r) {
  const int e = e0 + lane_id();
  r = {e, 0, 0};
  if (e >= n_matrices) return 0;
  r = rows_of_matrix(offsets, n_rows, e);
  const int64_t n = (r.end - r.first + per - 1) / per;
  return n > least ? (int)n : least;
}

// all blocks of `per` rows; the whole wave asks, as below
__device__ __forceinline__ int64_t count_units(const int32_t *offsets, int n_matrices, int64_t n_rows, int per) {
  if (!offsets) return (n_rows + per - 1) / per;
  int64_t all = 0;
  for (int e0 = 0; e0 < n_matrices; e0 += 64) {
    Rows r;
    all += __builtin_amdgcn_readlane(incl_sums(blocks_of(offsets, n_matrices, n_rows, e0, per, 0, r)), 63);
  }
  return all;
}

// the unit-th of them; matrix -1: there is none.  part: its number among the blocks of matrices that have several, or -1
__device__ __forceinline__ Rows rows_of_unit(const int32_t *offsets, int n_matrices, int64_t n_rows, int64_t unit, int64_t per,
                                             int least = 0, int64_t *part = nullptr) {
  if (!offsets) {
    const int64_t first = unit * per;
    if (part) *part = n_rows <= per ? -1 : unit;
    return {first < n_rows || unit < least ? 0 : -1, first, first + per < n_rows ? first + per : n_rows};
  }
  int64_t before = 0, parts = 0;
  for (int e0 = 0; e0 < n_matrices; e0 += 64) {
    Rows r;
    const int blocks = blocks_of(offsets, n_matrices, n_rows, e0, per, least, r);
    const int upto = incl_sums(blocks);
    const uint64_t past = __ballot(before + upto > unit);
    if (past) {
      const int l = __builtin_ctzll(past);
      const int skip = (int)(unit - before) - (__builtin_amdgcn_readlane(upto, l) - __builtin_amdgcn_readlane(blocks, l));
      const int64_t first = __builtin_amdgcn_readlane((int)r.first, l) + (int64_t)skip * per;
      const int64_t end = __builtin_amdgcn_readlane((int)r.end, l);
      if (part) {
        const int several = blocks > 1 ? blocks : 0, upto_several = incl_sums(several);
        *part = __builtin_amdgcn_readlane(blocks, l) == 1
                    ? -1
                    : parts + __builtin_amdgcn_readlane(upto_several, l) - __builtin_amdgcn_readlane(several, l) + skip;
      }
      return {e0 + l, first, first + per < end ? first + per : end};
    }
    before += __builtin_amdgcn_readlane(upto, 63);
    if (part) parts += __builtin_amdgcn_readlane(incl_sums(blocks > 1 ? blocks : 0), 63);
  }
  return {-1, 0, 0};
}

__host__ __device__ inline int64_t eighths(int64_t tiles) { return (tiles + 7) / 8 * 8; }

// The tile of workgroup b: workgroups b, b + 8, .. share an L2, so each eighth takes neighbouring tiles; within them,
// bands of 8 units go through the columns together.  False: none left.
__device__ __forceinline__ bool tile_of(int64_t b, int64_t units, int columns, int64_t &unit, int &column) {
  const int64_t n = units * columns, each = (n + 7) / 8, t = b % 8 * each + b / 8;
  if (b / 8 >= each || t >= n) return false;
  const int64_t band = t / (8 * (int64_t)columns), in = t - band * 8 * columns;
  const int64_t high = units - band * 8 < 8 ? units - band * 8 : 8;
  unit = band * 8 + in % high;
  column = (int)(in / high);
  return true;
}

struct GatedArgs {
  int64_t n_rows, units;
  int32_t ins, outs, n_matrices, columns;   // columns: tiles across
  int32_t act;
  int32_t few;                // forward: blocks of 16 rows for the kernel of few rows, or 0
  const int32_t *offsets;
  const void *x, *w_gate, *w_up;
  void *h, *gate, *up;        // gate, up: NULL where they are not kept
  // gradients
  const void *dh;
  void *dx, *dw_gate, *dw_up;
  char *d_both;               // dg, then du: [n_rows][pitch] each
  int64_t pitch;              // bytes
  int64_t in_pitch;           // bytes of a row of x, w_gate and w_up: a multiple of 4, but for few rows
  char *padded;               // their copies with such rows, where they are not so: x, then w_gate, then w_up
  int32_t splits;             // dx: parts of the reduced index
  int64_t per;                // dW: rows of a matrix that are reduced at once
  int64_t dx_blocks;          // workgroups: dx's, with its parts
  int64_t dw_early, dw_late;  // dW's, before and behind them; where both are there, blocks of more than dw_long rows come early
  int64_t dw_long;
  int64_t dw_partial;         // where dW's parts begin in `partial`, behind dx's
  int64_t dw_slots;           // for so many parts there is room: more are not written, offsets that fall would give some
  float *partial;
};

template <class T>
__device__ __forceinline__ void store_four(T *at, const float (&v)[4], int left) {
  if (left >= 4) {
    struct Four { T t[4]; } r{{(T)v[0], (T)v[1], (T)v[2], (T)v[3]}};
    struct __attribute__((packed, aligned(sizeof(T)))) Raw { uint32_t v[sizeof(T)]; };
    *reinterpret_cast<Raw *>(at) = __builtin_bit_cast(Raw, r);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < left) at[i] = (T)v[i];
  }
}

// f of the activation as a constant
template <class F>
__device__ __forceinline__ void with_act(int act, F f) {
  switch (act) {
    case SVT_ACT_RELU: return f(std::integral_constant<int, SVT_ACT_RELU>{});
    case SVT_ACT_SILU: return f(std::integral_constant<int, SVT_ACT_SILU>{});
    case SVT_ACT_GELU: return f(std::integral_constant<int, SVT_ACT_GELU>{});
    default: return f(std::integral_constant<int, SVT_ACT_NONE>{});
  }
}

// ---- results -------------------------------------------------------------------------------------
//
// A wave's registers hold 16 rows of four columns each, 32 bytes of a row per store.  So a tile goes through LDS, where
// its rows meet, and leaves as pieces of 16 bytes, a whole row of the tile after the other: forward at 8192 rows, 2048
// inputs and 8192 outputs, kept gate and up, 704 us with direct stores, 457 without any.
template <class C, class O, int COLUMNS>   // COLUMNS of O
struct Staged {
  static constexpr int pitch = COLUMNS * (int)sizeof(O) + 16;   // 16: neighbouring rows on other banks
  static constexpr int most = (C::q + C::p) * kStepBytes * 2 + 8192;
  static constexpr int fit() {
    int n = C::nq;
    while (C::WQ * 16 * n * pitch > most) n /= 2;
    return n;
  }
  static constexpr int blocks = fit();                           // of a wave at a time
  static constexpr int rows = C::WQ * 16 * blocks, bytes = rows * pitch;
  static_assert(blocks >= 1 && C::nq % blocks == 0, "whole passes");

  // value(b, c): a wave's four values of its block b of rows and c of NC blocks of columns.  Rows first .. end - 1 of `out`,
  // whose rows have `width` values, columns from c0 on.  The whole workgroup calls; lds is free before and after.
  template <int NC, class Value>
  static __device__ __forceinline__ void store(char *lds, int64_t first, int64_t end, int c0, int width, O *out, Value value) {
    const int wave = (int)threadIdx.x / 64, wq = wave / C::WP, wp = wave % C::WP, i = lane_id() % 16, g = lane_id() / 16;
    struct alignas(4 * sizeof(O) < 16 ? 4 * sizeof(O) : 16) Four { O t[4]; };
    struct __attribute__((packed, aligned(sizeof(O)))) Raw { uint32_t v[4]; };
    constexpr int each = 16 / sizeof(O), row_pieces = COLUMNS / each;
#pragma unroll
    for (int b0 = 0; b0 < C::nq; b0 += blocks) {
      __syncthreads();
#pragma unroll
      for (int b = 0; b < blocks; ++b)
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          float v[4];
          value(b0 + b, c, v);
          *reinterpret_cast<Four *>(lds + ((wq * blocks + b) * 16 + i) * pitch +
                                    ((wp * NC + c) * 16 + 4 * g) * (int)sizeof(O)) = Four{{(O)v[0], (O)v[1], (O)v[2], (O)v[3]}};
        }
      __syncthreads();
      for (int q = (int)threadIdx.x; q < rows * row_pieces; q += C::threads) {
        const int r = q / row_pieces, piece = q % row_pieces;
        // row r of this pass is row (r / (16 blocks)) nq 16 + b0 16 + r % (16 blocks) of the tile
        const int64_t row = first + (r / (16 * blocks) * C::nq + b0) * 16 + r % (16 * blocks);
        const int col = c0 + piece * each, left = width - col;
        if (row >= end || left <= 0) continue;
        const Raw raw = *reinterpret_cast<const Raw *>(lds + r * pitch + piece * 16);
        O *to = out + row * width + col;
        if (left >= each) *reinterpret_cast<Raw *>(to) = raw;
        else {
          struct Values { O t[each]; } v = __builtin_bit_cast(Values, raw);
#pragma unroll
          for (int k = 0; k < each; ++k)
            if (k < left) to[k] = v.t[k];
        }
      }
    }
  }
};

// a tile's result, to `out` or, one part of a split, to `part`
template <class T, class C>
__device__ __forceinline__ void store_tile(const f32x4 (&acc)[C::nq][C::np], char *lds, int64_t first, int64_t end, int c0,
                                           int width, T *out, float *part) {
  auto value = [&](int b, int c, float (&v)[4]) {
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = acc[b][c][k];
  };
  if (part) Staged<C, float, C::p>::template store<C::np>(lds, first, end, c0, width, part, value);
  else Staged<C, T, C::p>::template store<C::np>(lds, first, end, c0, width, out, value);
}

constexpr int larger(int a, int b) { return a > b ? a : b; }

// ---- forward -------------------------------------------------------------------------------------

// side P: half a tile of Wg's rows and the same outputs' of Wu; side Q: rows of x
template <class T, class C>
__global__ __launch_bounds__(C::threads) void k_gated(GatedArgs a) {
  using Pr = Product<T, C, false, false, true>;
  constexpr int outs = C::p / 2;   // of a tile
  __shared__ __attribute__((aligned(1024))) char lds[larger(Pr::lds_bytes, Staged<C, T, outs>::bytes)];
  int64_t unit;
  int column;
  // the matrices' own blocks, not as many as there may be, are shared out over the L2s (dx_tile has the figures)
  const int64_t units = count_units(a.offsets, a.n_matrices, a.n_rows, C::q);
  if (!tile_of(block_number(), units, a.columns, unit, column)) return;
  const Rows rows = rows_of_unit(a.offsets, a.n_matrices, a.n_rows, unit, C::q);
  if (rows.matrix < 0) return;
  const int n0 = column * outs;
  const int64_t pitch = a.in_pitch;
  const int steps = (a.ins + Pr::SP::step - 1) / Pr::SP::step, tail = a.ins - (steps - 1) * Pr::SP::step;
  Pr product;
  product.P.init((uint32_t)pitch, a.outs - n0 < outs ? a.outs - n0 : outs, tail);
  product.Q.init((uint32_t)pitch, (int)(rows.end - rows.first), tail);
  const int64_t w0 = ((int64_t)rows.matrix * a.outs + n0) * pitch;
  const char *wg = (const char *)a.w_gate + w0, *wu = (const char *)a.w_up + w0;
  const char *x = (const char *)a.x + rows.first * pitch, *x_end = (const char *)a.x + a.n_rows * pitch;
  const int64_t w_bytes = (int64_t)a.n_matrices * a.outs * pitch;
  const char *wg_end = (const char *)a.w_gate + w_bytes, *wu_end = (const char *)a.w_up + w_bytes;
  f32x4 acc[C::nq][C::np] = {};
  product.run(
      steps, tail % Pr::SP::each ? tail : 0, lds,
      [&](int s, Base &p, Base &q) {
        const int64_t k = (int64_t)s * kStepBytes;
        p = {wg + k, wu + k, wg_end, wu_end};
        q = {x + k, nullptr, x_end, nullptr};
      },
      [&](int s) { return s + 1 == steps; }, acc);
  constexpr int half = C::np / 2;
  using St = Staged<C, T, outs>;
  if (a.gate) {
    St::template store<half>(lds, rows.first, rows.end, n0, a.outs, (T *)a.gate, [&](int b, int c, float (&v)[4]) {
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = acc[b][c][k];
    });
    St::template store<half>(lds, rows.first, rows.end, n0, a.outs, (T *)a.up, [&](int b, int c, float (&v)[4]) {
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = acc[b][half + c][k];
    });
  }
  with_act(a.act, [&](auto act) {
    St::template store<half>(lds, rows.first, rows.end, n0, a.outs, (T *)a.h, [&](int b, int c, float (&v)[4]) {
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = act_value<decltype(act)::value, T>(acc[b][c][k]) * acc[b][half + c][k];
    });
  });
}

// ---- forward, few rows ---------------------------------------------------------------------------
//
// Up to 16 MT rows of one matrix against 16 outputs: the weights' bytes are the cost, so they go straight to registers,
// each once, 64 bytes of a row at a time and U such pieces in flight.  The waves share the inputs out and their sums meet
// in LDS.  Four waves and few pieces each, so that several workgroups share a compute unit: 1 row of 32768 x 4096 bfloat16
// 97 us (5.5 TB/s), with 8 waves of 8 pieces 104; 64 rows over 128 experts of 1024 x 1024 46 and 64.


// 16 bytes of a row from index k on, zeros past its end
template <class T>
__device__ __forceinline__ typename Mul<T>::frag load_sixteen(const T *row, int k, int end) {
  constexpr int each = 16 / sizeof(T);
  struct Values { T t[each]; };
  struct __attribute__((packed, aligned(sizeof(T)))) Raw { uint32_t v[4]; };
  if (k + each <= end)
    return __builtin_bit_cast(typename Mul<T>::frag, *reinterpret_cast<const Raw *>(row + k));
  Values v{};
#pragma unroll
  for (int i = 0; i < each; ++i)
    if (k + i < end) v.t[i] = row[k + i];
  return __builtin_bit_cast(typename Mul<T>::frag, v);
}

template <class T, int MT, int U, int WAVES>
__global__ __launch_bounds__(64 * WAVES, 4) void k_gated_few(GatedArgs a) {
  __shared__ f32x4 sums[WAVES][2 * MT][64];
  const int64_t unit = blockIdx.x / a.columns;
  const int column = (int)(blockIdx.x - unit * a.columns);
  const Rows rows = rows_of_unit(a.offsets, a.n_matrices, a.n_rows, unit, 16 * MT);
  if (rows.matrix < 0) return;
  const int wave = (int)threadIdx.x / 64, i = lane_id() % 16, g = lane_id() / 16;
  constexpr int each = 16 / sizeof(T), step = 4 * each;
  const int n = column * 16 + i < a.outs ? column * 16 + i : a.outs - 1;   // a copy's sums go nowhere
  const int64_t at = ((int64_t)rows.matrix * a.outs + n) * a.ins;
  const T *wg = (const T *)a.w_gate + at, *wu = (const T *)a.w_up + at;
  const T *x[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int64_t r = rows.first + 16 * m + i;
    x[m] = (const T *)a.x + (r < rows.end ? r : rows.end - 1) * a.ins;
  }
  f32x4 acc[2 * MT] = {};
  for (int k0 = wave * U * step; k0 < a.ins; k0 += WAVES * U * step) {
    typename Mul<T>::frag fg[U], fu[U], fx[MT][U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = k0 + u * step + g * each;
      fg[u] = load_sixteen(wg, k, a.ins);
      fu[u] = load_sixteen(wu, k, a.ins);
#pragma unroll
      for (int m = 0; m < MT; ++m) fx[m][u] = load_sixteen(x[m], k, a.ins);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        acc[2 * m] = Mul<T>::add(fg[u], fx[m][u], acc[2 * m]);
        acc[2 * m + 1] = Mul<T>::add(fu[u], fx[m][u], acc[2 * m + 1]);
      }
  }
#pragma unroll
  for (int m = 0; m < 2 * MT; ++m) sums[wave][m][lane_id()] = acc[m];
  __syncthreads();
  if (wave >= MT) return;
  f32x4 s[2] = {};
#pragma unroll
  for (int w = 0; w < WAVES; ++w) {
    s[0] += sums[w][2 * wave][lane_id()];
    s[1] += sums[w][2 * wave + 1][lane_id()];
  }
  const int64_t row = rows.first + 16 * wave + i;
  const int n0 = column * 16 + 4 * g, left = a.outs - n0;
  if (row >= rows.end || left <= 0) return;
  float h[4], gate[4], up[4];
  with_act(a.act, [&](auto act) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      gate[k] = s[0][k];
      up[k] = s[1][k];
      h[k] = act_value<decltype(act)::value, T>(gate[k]) * up[k];
    }
  });
  const int64_t to = row * a.outs + n0;
  store_four((T *)a.h + to, h, left);
  if (a.gate) {
    store_four((T *)a.gate + to, gate, left);
    store_four((T *)a.up + to, up, left);
  }
}

// ---- rows of any alignment -----------------------------------------------------------------------
//
// The loads that go straight to LDS want rows that begin at multiples of 4 bytes.  Others (two-byte values, an odd number
// in a row or an odd address) are copied first, to rows of whole pieces with zeros behind: 2 (x + w) bytes more to move.  A
// path of its own through registers took longer than copy and product together (gradients of 1001 x 250 x 999 float32, when
// every row that does not begin at 16 bytes went there: 86 us, with the copy 52).
template <class T>
__global__ __launch_bounds__(256) void k_gated_pad(GatedArgs a, int lanes) {
  constexpr int each = 16 / sizeof(T);
  const int64_t w_rows = (int64_t)a.n_matrices * a.outs;
  const T *from = (const T *)(blockIdx.z == 0 ? a.x : blockIdx.z == 1 ? a.w_gate : a.w_up);
  if (!from) return;
  char *to = a.padded + (blockIdx.z == 0 ? 0 : (a.n_rows + (blockIdx.z == 1 ? 0 : w_rows)) * a.in_pitch);
  int64_t first = 0, end = w_rows;
  if (blockIdx.z == 0) {   // rows that no matrix names are not read
    first = a.offsets ? clamped(a.offsets[0], a.n_rows) : 0;
    end = a.offsets ? clamped(a.offsets[a.n_matrices], a.n_rows) : a.n_rows;
  }
  const int pieces = (int)(a.in_pitch / 16), in = threadIdx.x % lanes;
  const int64_t per = 256 / lanes;
  for (int64_t r = first + blockIdx.x * per + threadIdx.x / lanes; r < end; r += gridDim.x * per)
    for (int c = blockIdx.y * lanes + in; c < pieces; c += gridDim.y * lanes)
      *reinterpret_cast<typename Mul<T>::frag *>(to + r * a.in_pitch + c * 16) =
          load_sixteen(from + r * a.ins, c * each, a.ins);
}

// ---- gradients -----------------------------------------------------------------------------------

// dg and du of the rows that some matrix names, with zeros up to the pitch.  They are rounded to the rows' type, as the
// matrix instructions take them: that is the rounding a gradient kept between two layers has.  (In two parts each, which would
// keep 16 bits of bfloat16's, the products would take twice the instructions.)
constexpr int kBothThreads = 256;

template <class T>
__global__ __launch_bounds__(kBothThreads) void k_gated_both(GatedArgs a, int lanes) {
  constexpr int each = 16 / sizeof(T);
  struct Values { T t[each]; };
  struct __attribute__((packed, aligned(sizeof(T)))) Raw { uint32_t v[4]; };
  const int64_t first = a.offsets ? clamped(a.offsets[0], a.n_rows) : 0;
  const int64_t end = a.offsets ? clamped(a.offsets[a.n_matrices], a.n_rows) : a.n_rows;
  const int pieces = (int)(a.pitch / 16), in = threadIdx.x % lanes;
  const int64_t per = kBothThreads / lanes;
  with_act(a.act, [&](auto act) {
    for (int64_t r = first + blockIdx.x * per + threadIdx.x / lanes; r < end; r += gridDim.x * per)
      for (int c = blockIdx.y * lanes + in; c < pieces; c += gridDim.y * lanes) {
        const int n = c * each;
        const int64_t at = r * a.outs + n;
        Values g{}, u{}, d{};
        if (n + each <= a.outs) {
          g = __builtin_bit_cast(Values, *reinterpret_cast<const Raw *>((const T *)a.gate + at));
          u = __builtin_bit_cast(Values, *reinterpret_cast<const Raw *>((const T *)a.up + at));
          d = __builtin_bit_cast(Values, *reinterpret_cast<const Raw *>((const T *)a.dh + at));
        } else {
#pragma unroll
          for (int i = 0; i < each; ++i)
            if (n + i < a.outs) {
              g.t[i] = ((const T *)a.gate)[at + i];
              u.t[i] = ((const T *)a.up)[at + i];
              d.t[i] = ((const T *)a.dh)[at + i];
            }
        }
#pragma unroll
        for (int i = 0; i < each; ++i) {
          float value, slope;
          act_both<decltype(act)::value, T>((float)g.t[i], value, slope);
          const float dh = (float)d.t[i];
          g.t[i] = (T)(dh * (float)u.t[i] * slope);
          u.t[i] = (T)(dh * value);
        }
        char *to = a.d_both + r * a.pitch + c * 16;
        *reinterpret_cast<u32x4 *>(to) = __builtin_bit_cast(u32x4, g);
        *reinterpret_cast<u32x4 *>(to + a.n_rows * a.pitch) = __builtin_bit_cast(u32x4, u);
      }
  });
}

// dx: side P: columns of Wg, then of Wu (across); side Q: rows of dg, then of du (along)
template <class T, class C>
__device__ __forceinline__ void dx_tile(const GatedArgs &a, char *lds, int64_t b, int part) {
  using Pr = Product<T, C, true, false, false>;
  int64_t unit;
  int column;
  // the matrices' own blocks, not as many as there may be, are shared out over the L2s (8 even experts of 2048 rows, 1024
  // tiles in a grid for 1088: 179 us by what there may be, 121 like this)
  const int64_t units = count_units(a.offsets, a.n_matrices, a.n_rows, C::q);
  if (!tile_of(b, units, a.columns, unit, column)) return;
  const Rows rows = rows_of_unit(a.offsets, a.n_matrices, a.n_rows, unit, C::q);
  if (rows.matrix < 0) return;
  const int k0 = column * C::p;
  const int64_t pitch = a.in_pitch;
  const int half = (a.outs + Pr::SP::step - 1) / Pr::SP::step, tail = a.outs - (half - 1) * Pr::SP::step;
  const int each = (2 * half + a.splits - 1) / a.splits, s0 = part * each;
  const int steps = 2 * half - s0 < each ? 2 * half - s0 : each;   // none, or fewer, for the last part
  Pr product;
  product.P.init((uint32_t)pitch, a.ins - k0 < C::p ? a.ins - k0 : C::p, tail);
  product.Q.init((uint32_t)a.pitch, (int)(rows.end - rows.first), tail);
  const int64_t w0 = (int64_t)rows.matrix * a.outs * pitch + (int64_t)k0 * sizeof(T);
  const char *wg = (const char *)a.w_gate + w0, *wu = (const char *)a.w_up + w0;
  const int64_t w_bytes = (int64_t)a.n_matrices * a.outs * pitch;
  const char *dg = a.d_both + rows.first * a.pitch, *du = dg + a.n_rows * a.pitch, *d_end = a.d_both + 2 * a.n_rows * a.pitch;
  f32x4 acc[C::nq][C::np] = {};
  product.run(
      steps, 0, lds,
      [&](int t, Base &p, Base &q) {
        const int s = s0 + t, in = s < half ? s : s - half;
        const char *w = (s < half ? wg : wu) + (int64_t)in * Pr::SP::step * pitch;
        const char *d = (s < half ? dg : du) + (int64_t)in * kStepBytes;
        p = {w, nullptr, (const char *)(s < half ? a.w_gate : a.w_up) + w_bytes, nullptr};
        q = {d, nullptr, d_end, nullptr};
      },
      [&](int t) { return s0 + t + 1 == half || s0 + t + 1 == 2 * half; }, acc);
  store_tile<T, C>(acc, lds, rows.first, rows.end, k0, a.ins, (T *)a.dx,
                   a.splits > 1 ? a.partial + (int64_t)part * a.n_rows * a.ins : nullptr);
}

// dWg and dWu: side P: columns of x (across), side Q: columns of dg or du (across); the rows are reduced, a.per of a matrix
// at a time: the products of a matrix with more rows than that are parts, which k_gated_join adds
template <class T, class C>
__device__ __forceinline__ void dw_tile(const GatedArgs &a, char *lds, int64_t b, bool early) {
  using Pr = Product<T, C, true, true, false>;
  const int tiles = (a.outs + C::q - 1) / C::q;
  const int64_t own = eighths((int64_t)2 * tiles * a.columns), block = b / own;   // a block's tiles use all L2s
  int64_t in;
  int column;
  if (!tile_of(b % own, 2 * tiles, a.columns, in, column)) return;
  int64_t part = -1;
  const Rows rows = rows_of_unit(a.offsets, a.n_matrices, a.n_rows, block, a.per, 1, &part);
  if (rows.matrix < 0 || part >= a.dw_slots) return;
  if (a.dw_early && a.dw_late && (rows.end - rows.first > a.dw_long) != early) return;
  const bool up = in >= tiles;
  const int n0 = (int)(up ? in - tiles : in) * C::q, k0 = column * C::p;
  const int64_t len = rows.end - rows.first, pitch = a.in_pitch;
  const int steps = (int)((len + Pr::SP::step - 1) / Pr::SP::step), tail = (int)(len - (int64_t)(steps - 1) * Pr::SP::step);
  Pr product;
  product.P.init((uint32_t)pitch, a.ins - k0 < C::p ? a.ins - k0 : C::p, tail);
  product.Q.init((uint32_t)a.pitch, a.outs - n0 < C::q ? a.outs - n0 : C::q, tail);
  const char *x = (const char *)a.x + rows.first * pitch + (int64_t)k0 * sizeof(T);
  const char *d = a.d_both + (up ? a.n_rows * a.pitch : 0) + rows.first * a.pitch + (int64_t)n0 * sizeof(T);
  const char *x_end = (const char *)a.x + a.n_rows * pitch, *d_end = a.d_both + 2 * a.n_rows * a.pitch;
  f32x4 acc[C::nq][C::np] = {};
  product.run(
      steps, 0, lds,
      [&](int t, Base &p, Base &q) {
        const int64_t s = (int64_t)t * Pr::SP::step;
        p = {x + s * pitch, nullptr, x_end, nullptr};
        q = {d + s * a.pitch, nullptr, d_end, nullptr};
      },
      [&](int t) { return t + 1 == steps; }, acc);
  const int64_t size = (int64_t)a.outs * a.ins;
  store_tile<T, C>(acc, lds, n0, a.outs, k0, a.ins, (T *)(up ? a.dw_up : a.dw_gate) + rows.matrix * size,
                   part < 0 ? nullptr : a.partial + a.dw_partial + (part * 2 + up) * size);
}

// dx and dW are tiles of one grid, so that the last of the one leave no compute unit idle beside the other: 1001 x 250 x 999
// float32 51 us in two launches, 42 in one.  Tiles that reduce more come first: rows of few experts make dW's tiles the longest
// of all, those of many the shortest (16384 rows over 8 uneven experts, 1024 inputs, 2048 outputs: 427 in two launches; in one
// with dW first 388, dx first 403, with dW's long blocks before dx and the short ones behind 364; even experts 318, 322, 325).
template <class T, class C>
__global__ __launch_bounds__(C::threads) void k_gated_gradients(GatedArgs a) {
  __shared__ __attribute__((aligned(1024))) char lds[larger(Product<T, C, true, false, false>::lds_bytes,
                                                            larger(Staged<C, T, C::p>::bytes, Staged<C, float, C::p>::bytes))];
  const int64_t b = block_number() - a.dw_early;
  if (b >= a.dx_blocks + a.dw_late) return;   // the last row of a grid is not full
  if (b >= 0 && b < a.dx_blocks) {
    const int64_t own = a.dx_blocks / a.splits;
    dx_tile<T, C>(a, lds, b % own, (int)(b / own));
  } else {
    dw_tile<T, C>(a, lds, b < 0 ? b + a.dw_early : b - a.dx_blocks, b < 0);
  }
}

struct __attribute__((packed, aligned(4))) FourParts { float v[4]; };

// to[i ..] = the sum of `parts` float32 arrays at from, `stride` apart, in order; up to four values, `left` of them
template <class T>
__device__ __forceinline__ void join_four(const float *from, int parts, int64_t stride, int64_t left, T *to) {
  FourParts sum{};
  if (left >= 4) {
    sum = *reinterpret_cast<const FourParts *>(from);
#pragma unroll 4
    for (int z = 1; z < parts; ++z) {
      const FourParts v = *reinterpret_cast<const FourParts *>(from + z * stride);
#pragma unroll
      for (int k = 0; k < 4; ++k) sum.v[k] += v.v[k];
    }
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (k < left) {
        sum.v[k] = from[k];
        for (int z = 1; z < parts; ++z) sum.v[k] += from[z * stride + k];
      }
  }
  store_four(to, sum.v, (int)(left < 4 ? left : 4));
}

// The parts' sums.  blockIdx.y: dx (0; rows that no matrix names keep their values), then dWg and dWu of the matrices whose
// rows were cut into blocks, one after the other.
template <class T>
__global__ __launch_bounds__(256) void k_gated_join(GatedArgs a) {
  const int64_t at = (blockIdx.x * 256ll + threadIdx.x) * 4, hop = gridDim.x * 1024ll;
  if (blockIdx.y == 0) {
    if (!a.dx || a.splits < 2) return;
    const int64_t size = a.n_rows * a.ins;
    const int64_t first = a.offsets ? clamped(a.offsets[0], a.n_rows) * a.ins : 0;
    const int64_t end = a.offsets ? clamped(a.offsets[a.n_matrices], a.n_rows) * a.ins : size;
    for (int64_t i = first + at; i < end; i += hop) join_four(a.partial + i, a.splits, size, end - i, (T *)a.dx + i);
    return;
  }
  if (!a.dw_gate) return;
  int64_t before = 0;   // parts of the matrices before it
  int skip = blockIdx.y - 1, matrix = -1, parts = 0;
  for (int e0 = 0; e0 < a.n_matrices && matrix < 0; e0 += 64) {
    Rows r;
    int blocks = 0;
    if (a.offsets) blocks = blocks_of(a.offsets, a.n_matrices, a.n_rows, e0, a.per, 1, r);
    else if (lane_id() == 0) blocks = (int)((a.n_rows + a.per - 1) / a.per);
    const int several = blocks > 1 ? blocks : 0, upto = incl_sums(several);
    uint64_t cut = __ballot(several > 0);
    const int here = __builtin_popcountll(cut);
    if (skip < here) {
      for (; skip > 0; --skip) cut &= cut - 1;
      const int l = __builtin_ctzll(cut);
      matrix = e0 + l;
      parts = __builtin_amdgcn_readlane(several, l);
      before += __builtin_amdgcn_readlane(upto, l) - parts;
    } else {
      skip -= here;
      before += __builtin_amdgcn_readlane(upto, 63);
    }
  }
  if (matrix < 0 || before + parts > a.dw_slots) return;
  const int64_t size = (int64_t)a.outs * a.ins;
  for (int64_t i = at; i < 2 * size; i += hop) {
    const int64_t gate = size - i;   // four values may lie in both halves
    const float *from = a.partial + a.dw_partial + before * 2 * size + i;
    if (gate > 0) join_four(from, parts, 2 * size, gate, (T *)a.dw_gate + matrix * size + i);
    const int64_t skip = gate <= 0 ? 0 : gate < 4 ? gate : 4;
    if (skip < 4 && i + skip < 2 * size)
      join_four(from + skip, parts, 2 * size, 2 * size - i - skip < 4 - skip ? 2 * size - i - skip : 4 - skip,
                (T *)a.dw_up + matrix * size + (i + skip - size));
  }
}

// ---- calls ---------------------------------------------------------------------------------------

// How a product runs; the same for the workspace's size.
struct GatedPlan {
  int cut;            // of the four below
  int64_t units;      // tiles along the rows of h or dx, at most
  int columns;
  int splits;         // dx: parts of the reduced index
  int64_t per;        // dW: rows reduced at once
  int64_t dw_units;   // blocks of them, at most
};

// The cuts, and microseconds of a step of 128 bytes: with one workgroup on a compute unit, and for each further one that
// shares it (the 256 x 256 cut has none beside it: they follow each other).  Measured with products of two-byte and of
// float32 values, 200 x 512 x 2048 to 16384 x 1024 x 2048.  Its choices are within 10 % of the best cut's time there; gradients
// in us, four sets of inputs in turn: bfloat16 4096 x 4096 x 4096 530, 4096 x 1024 x 2048 100, 1024 x 1024 x 1024 34,
// 300 x 300 x 300 13; float32 1001 x 250 x 999 45, 4096 x 1024 x 2048 630.  The steps were timed with operands in the caches: few
// tiles whose weights come from memory wait for each step's loads (64 x 2048 x 2048 bfloat16 14 us in the caches, 26 from memory).
struct CutCost { int q, p; float alone[2], shared[2]; };
constexpr int kCuts = 4;
constexpr CutCost kCutCost[kCuts] = {{32, 64, {0.28f, 0.46f}, {0.15f, 0.29f}},
                                     {64, 128, {0.5f, 1.17f}, {0.34f, 1.05f}},
                                     {128, 128, {0.62f, 2.15f}, {0.53f, 2.0f}},
                                     {256, 256, {1.65f, 7.5f}, {1.65f, 7.5f}}};

// blocks of rows at most: every matrix may end inside one
inline int64_t row_units(int64_t n_rows, int n_matrices, bool by_expert, int per) {
  return by_expert ? n_rows / per + (n_rows < n_matrices ? n_rows : n_matrices) : (n_rows + per - 1) / per;
}

// the cut with the least time by the table above
inline GatedPlan plan_forward(const GatedArgs &a, int elem) {
  GatedPlan best{};
  double least = 0;
  const int type = elem == 4, step = kStepBytes / elem;
  for (int cut = 0; cut < kCuts; ++cut) {
    const CutCost &c = kCutCost[cut];
    const GatedPlan p{cut, row_units(a.n_rows, a.n_matrices, a.offsets != nullptr, c.q), (2 * a.outs + c.p - 1) / c.p, 1, 1, 1};
    const int64_t load = (p.units * p.columns + 255) / 256;
    const double time = (double)((a.ins + step - 1) / step) * (c.alone[type] + (double)(load - 1) * c.shared[type]);
    if (cut == 0 || time < least) {
      least = time;
      best = p;
    }
  }
  return best;
}

// The cut, dx's parts and dW's blocks of rows with the least time for both, whichever of them are wanted: what the compute
// units have to do, but at least what the longest tile takes, and for parts 4 us and 2.4 for each million partial values that
// are written and read again.  Only products of fewer tiles than compute units are cut into parts.  By expert one matrix may
// have all rows, which only the GPU knows: dW's blocks are as long as what each compute unit has to do, so that no tile
// outlasts the others (16384 rows, 8 uneven experts, 1024 inputs, 2048 outputs: whole 358 us, at most 8192 rows 346, 4096 366,
// the device's least times, where a call takes 365 to 385;
// 32 experts, 1024 x 1024: 252, 255, 244; 8192 rows, 8 experts, 2048 x 2048: 338 whole, at most 4096 rows 367).  A tile costs
// two steps beside its own (100 rows, 16 experts, 1024 x 1024, which small tiles without that count would take: 57 us and 51).
inline GatedPlan plan_backward(const GatedArgs &a, int elem) {
  GatedPlan best{};
  double least = 0;
  const int type = elem == 4, step = kStepBytes / elem, experts = a.offsets ? a.n_matrices : 1;
  const int64_t dx_steps = 2 * (int64_t)((a.outs + step - 1) / step), dw_steps = (a.n_rows + step - 1) / step;
  for (int cut = 0; cut < kCuts; ++cut) {
    const CutCost &c = kCutCost[cut];
    const int columns = (a.ins + c.p - 1) / c.p;
    const int64_t units = row_units(a.n_rows, a.n_matrices, a.offsets != nullptr, c.q);
    const int64_t dx_tiles = units * columns, dw_tiles = (int64_t)2 * ((a.outs + c.q - 1) / c.q) * columns;
    const double load = ((double)dx_tiles * dx_steps + (double)dw_tiles * (dw_steps + 0.5 * experts)) / 256;
    for (int splits = 1; splits <= 32 && (splits == 1 || (dx_tiles < 256 && dx_steps >= 2 * splits)); splits *= 2)
      for (int parts = 1; parts <= 32 && (parts == 1 || (dw_tiles < 256 && dw_steps >= 2 * parts)); parts *= 2) {
        const int64_t blocks = (dw_steps + parts - 1) / parts;
        if (a.offsets && (double)blocks > load && parts < 32 && dw_tiles < 256 && dw_steps >= 4 * parts) continue;
        const double longest = (double)larger((int)((dx_steps + splits - 1) / splits), (int)blocks);
        const double alone = longest * c.alone[type], shared = load * c.shared[type] + 0.3 * alone;
        double time = alone > shared ? alone : shared;
        if (splits > 1 || parts > 1) time += 4;
        if (splits > 1) time += 2.4e-6 * splits * (double)a.n_rows * a.ins;
        if (parts > 1) time += (a.offsets ? 3.6e-6 : 2.4e-6) * parts * 2.0 * a.outs * a.ins;
        if (best.columns == 0 || time < least) {
          least = time;
          const int64_t per = blocks > 0 ? blocks * step : 1;
          best = {cut, units, columns, splits, per, a.offsets ? a.n_rows / per + experts : (a.n_rows + per - 1) / per};
        }
      }
  }
  if (best.dw_units < 1) best.dw_units = 1;   // zeros for no rows
  return best;
}

// the workgroups of a plan's gradients: dW's before dx's, dx's, dW's behind
struct GradientBlocks {
  int64_t early, dx, late;
  int64_t all() const { return early + dx + late; }
};
inline int64_t long_rows(const GatedPlan &p, int32_t outs) { return 2 * (int64_t)outs / p.splits; }
inline GradientBlocks gradient_blocks(const GatedPlan &p, int32_t outs, bool dx, bool dw, bool by_expert) {
  const int q = kCutCost[p.cut].q;
  const int64_t n = dw ? eighths((int64_t)2 * ((outs + q - 1) / q) * p.columns) * p.dw_units : 0;
  const int64_t early = p.per > long_rows(p, outs) ? n : 0;
  return {early, dx ? eighths(p.units * p.columns) * p.splits : 0, early == 0 || (dx && by_expert) ? n : 0};
}

// Whether the forward pass takes the kernel for few rows: 1 or 2 blocks of 16, or 0.  Few: up to 32 (32 rows of bfloat16, weights
// from memory: 2048 x 2048 12.8 us there, 26 with tiles; 4096 x 8192 43 and 55).  Above that it reads the weights once for every 32
// rows, and which is faster depends on the outputs: 64 x 2048 x 2048 13 and 26, 64 x 4096 x 8192 70 and 57, 128 x 4096 x 8192 127
// and 65.  By expert up to 4 on average (32 experts of 1024 x 1024, 128 rows 32 and 30, 512 rows 38 and 30), or 32 where tiles
// would need copies.
inline int few_rows(const GatedArgs &a, bool copies) {
  const int64_t rows = a.offsets ? (a.n_rows + a.n_matrices - 1) / a.n_matrices : a.n_rows;
  if (rows > (a.offsets && !copies ? 4 : 32)) return 0;
  const int mt = rows <= 16 ? 1 : 2;
  return row_units(a.n_rows, a.n_matrices, a.offsets != nullptr, 16 * mt) * ((a.outs + 15) / 16) < (1 << 22) ? mt : 0;
}

// bytes of a row at a multiple of 16, and of the copies of x and both weights with such rows
inline int64_t gated_pitch(int32_t outs, int elem) { return ((int64_t)outs * elem + 15) & ~(int64_t)15; }

inline size_t gated_copies(const GatedArgs &a, int elem) {
  return (size_t)(a.n_rows + 2 * (int64_t)a.n_matrices * a.outs) * gated_pitch(a.ins, elem);
}

// values of dx's parts; dW's parts: matrices with several blocks have at most 2 n_rows / per together; their values
inline int64_t dx_parts(const GatedArgs &a, const GatedPlan &p) { return p.splits > 1 ? p.splits * a.n_rows * a.ins : 0; }
inline int64_t dw_slots(const GatedArgs &a, const GatedPlan &p) { return p.per < a.n_rows ? 2 * a.n_rows / p.per : 0; }
inline int64_t dw_parts(const GatedArgs &a, const GatedPlan &p) { return dw_slots(a, p) * 2 * a.outs * a.ins; }

// one type's calls
template <class T> int gated_forward(const char *who, GatedArgs a, const GatedPlan &p, void *stream);
template <class T> int gated_backward(const char *who, GatedArgs a, const GatedPlan &p, void *stream);

#ifdef SVT_GATED_INSTANTIATE

template <class F>
int with_cut(int cut, F f) {
  if (cut == 3) return f(Cut<256, 256, 2, 4, 2>{});
  if (cut == 2) return f(Cut<128, 128, 2, 2, 2>{});
  if (cut == 1) return f(Cut<64, 128, 1, 4, 2>{});
  return f(Cut<32, 64, 2, 2, 2>{});
}

// threads of a workgroup side by side on a row of so many pieces, and the grid for so many rows
struct RowGrid {
  int lanes = 1;
  dim3 grid;
  RowGrid(int64_t pieces, int64_t rows, int z) {
    while (lanes < 256 && lanes < pieces) lanes *= 2;
    const int64_t blocks = (rows + 256 / lanes - 1) / (256 / lanes), columns = (pieces + lanes - 1) / lanes;
    grid = dim3((unsigned)(blocks < 8192 ? blocks : 8192), (unsigned)(columns < 64 ? columns : 64), z);
  }
};

// x, w_gate and w_up (those that a has) with rows at multiples of 4 bytes: the caller's own, or copies
template <class T>
int align_rows(const char *who, GatedArgs &a, void *stream) {
  if (!a.padded) return SVT_OK;
  const int64_t w_rows = (int64_t)a.n_matrices * a.outs;
  const RowGrid g(a.in_pitch / 16, a.n_rows > w_rows ? a.n_rows : w_rows, 3);
  const int rc = launch(who, k_gated_pad<T>, g.grid, 256, 0, stream, a, g.lanes);
  if (a.x) a.x = a.padded;
  if (a.w_gate) a.w_gate = a.padded + a.n_rows * a.in_pitch;
  if (a.w_up) a.w_up = a.padded + (a.n_rows + w_rows) * a.in_pitch;
  return rc;
}

template <class T>
int gated_forward(const char *who, GatedArgs a, const GatedPlan &p, void *stream) {
  if (const int mt = a.few) {
    a.units = row_units(a.n_rows, a.n_matrices, a.offsets != nullptr, 16 * mt);
    a.columns = (a.outs + 15) / 16;
    const unsigned grid = (unsigned)(a.units * a.columns);
    if (mt == 1) return launch(who, k_gated_few<T, 1, 4, 4>, grid, 256, 0, stream, a);
    return launch(who, k_gated_few<T, 2, 2, 4>, grid, 256, 0, stream, a);
  }
  const int rc = align_rows<T>(who, a, stream);
  if (rc != SVT_OK) return rc;
  a.units = p.units;
  a.columns = p.columns;
  return with_cut(p.cut, [&](auto cut) {
    using C = decltype(cut);
    return launch(who, k_gated<T, C>, grid_of(eighths(a.units * a.columns)), C::threads, 0, stream, a);
  });
}

template <class T>
int gated_backward(const char *who, GatedArgs a, const GatedPlan &p, void *stream) {
  int rc = SVT_OK;
  if (a.n_rows > 0) {
    rc = align_rows<T>(who, a, stream);
    if (rc != SVT_OK) return rc;
    const RowGrid g(a.pitch / 16, a.n_rows, 1);
    rc = launch(who, k_gated_both<T>, g.grid, kBothThreads, 0, stream, a, g.lanes);
    if (rc != SVT_OK) return rc;
  }
  a.columns = p.columns;
  a.splits = p.splits;
  a.per = p.per;
  a.dw_slots = dw_slots(a, p);
  const GradientBlocks blocks = gradient_blocks(p, a.outs, a.dx != nullptr, a.dw_gate != nullptr, a.offsets != nullptr);
  a.dx_blocks = blocks.dx;
  a.dw_long = long_rows(p, a.outs);
  a.dw_early = blocks.early;
  a.dw_late = blocks.late;
  if (blocks.all() == 0) return SVT_OK;
  rc = with_cut(p.cut, [&](auto cut) {
    using C = decltype(cut);
    return launch(who, k_gated_gradients<T, C>, grid_of(blocks.all()), C::threads, 0, stream, a);
  });
  const bool dx_parted = a.dx && dx_parts(a, p) > 0, dw_parted = a.dw_gate && dw_parts(a, p) > 0;
  if (rc != SVT_OK || (!dx_parted && !dw_parted)) return rc;
  const int64_t dx_values = dx_parted ? a.n_rows * a.ins : 0, dw_values = dw_parted ? (int64_t)2 * a.outs * a.ins : 0;
  const int64_t pieces = ((dx_values > dw_values ? dx_values : dw_values) + 1023) / 1024;
  int64_t cut = dw_parted ? a.n_rows / (p.per + 1) : 0;   // matrices with more rows than a block
  if (dw_parted && (cut < 1 || !a.offsets)) cut = 1;
  if (cut > a.n_matrices) cut = a.n_matrices;
  return launch(who, k_gated_join<T>, dim3((unsigned)(pieces < 2048 ? pieces : 2048), (unsigned)(1 + cut)), 256, 0, stream, a);
}

#endif   // SVT_GATED_INSTANTIATE

}  // namespace svt

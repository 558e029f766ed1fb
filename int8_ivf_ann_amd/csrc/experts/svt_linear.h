// svt_linear.h - the kernel of products with 4-bit weights (svt_linear_*.hip instantiate it, one file per type
// of the rows; svt_quant.hip packs the weights, checks arguments and calls).
//
//   W[n][k] = s[n][g] (q[n][k] - z[n][g]),  g = k / group,  q in 0 .. 15
//   y[r][n] = act(bias[n] + sum_k x[r][k] W[n][k])
//           = act(bias[n] + sum_g s[n][g] (sum_{k in g} x[r][k] q[n][k] - z[n][g] sum_{k in g} x[r][k]))
//
// The inner sums run on the matrix cores (v_mfma_f32_16x16x32, 16 outputs x 16 rows x 32 k) with whole numbers as
// bf16 or f16, which hold -255 .. 255 exactly, and float32 accumulation: no weight is rounded, and s is applied to
// float32 group sums.  Two forms:
//   q - z   (outputs of float32) is formed before the instruction, so that the sums' roundings are in proportion to
//           sum |x| |q - z|, as those of the product itself: a weight of 0 adds exactly 0.
//   q       (outputs of two bytes, whose own rounding is 2^7 (float16) or 2^10 (bfloat16) times the 2.5e-6 below) and
//           z sum x from the group's sum, which the same instruction gives with a matrix of ones; where every zero
//           point is 8, a matrix of -8 gives what the products then start from.  Its roundings are in proportion to
//           sum |x| (q + z).  Forming q - z takes 12 more instructions for 8 weights (bf16), 4 (f16).
// 13 rows, 1024 inputs, groups of 128 with zero points, rows behind a relu: the relative error of float32 rows is 1.2e-7
// with q - z formed before, 2.5e-6 after (a float32 product 1.9e-7).  In us, before and after: 1 row of 16384 x 4096,
// float32 rows 18.1 and 14.8, bfloat16 rows with float32 outputs 13.4 and 10.7, float16 rows likewise 11.9 and 10.9;
// 1024 rows of 4096 x 1024, 38.0 and 35.9, 22.6 and 19.8, 20.9 and 20.0.
// q reaches bf16/f16 two at a time: the byte 0000qqqq read as an 8-bit float with 3 mantissa bits is
// q * 2^-9 (its subnormals and its first binade share one spacing), and v_cvt_scalef32_pk_* turns two such
// bytes into two exact numbers with the scale 2^9.
// float32 rows are split into three bf16 parts of 8 bits each (24 bits: exact), one instruction per part.
#pragma once

#include <algorithm>
#include <type_traits>

#include "svt_experts.h"

namespace svt {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef f16 f16x2 __attribute__((ext_vector_type(2)));
typedef f16 f16x8 __attribute__((ext_vector_type(8)));

constexpr int kTileN = 16;        // outputs of a tile
constexpr int kBlockK = 128;      // k of a block: 4 instructions, 16 bytes of q per lane
constexpr int kGroupsAt = 1024;   // of a record: its groups, after q
constexpr int kMaxIn = 1 << 20, kMaxOut = 1 << 19;

// Layout of the packed weights: per matrix (its stride a multiple of 256 bytes) a record for each block of
// 128 k and tile of 16 outputs, [block][tile], holding
//   q       [lane][16]: lane l holds output l % 16, k = 128 block + 32 s + 8 (l / 16) + i for s = 0..3 in dword
//           s, whose byte i (0..3) holds i in its low and i + 4 in its high half
//   scales  [h][g]: what lane (., h) of the instruction's result needs, together: the scales of outputs
//           4 h .. 4 h + 3 for group g of the block
//   zeros   [output][g], where there are zero points: a byte each
// Outputs and groups past the end have scale 0.  A wave reads whole records, and workgroups that run
// together read neighbouring ones.
struct QuantShape {
  int32_t n_out, n_in, group, has_zeros;
  int32_t tiles, blocks;
  int32_t zeros_at, record;   // of a record: where its zero points begin, its bytes
  size_t stride;
};

inline QuantShape quant_shape(const svt_quant_weights &w) {
  QuantShape s;
  s.n_out = w.n_out;
  s.n_in = w.n_in;
  s.group = w.group;
  s.has_zeros = w.has_zeros;
  s.tiles = (w.n_out + kTileN - 1) / kTileN;
  s.blocks = (w.n_in + kBlockK - 1) / kBlockK;
  s.zeros_at = kGroupsAt + kTileN * (kBlockK / w.group) * elem_size(w.scale_type);
  s.record = s.zeros_at + (w.has_zeros ? kTileN * (kBlockK / w.group) : 0);
  s.stride = ((size_t)s.tiles * s.blocks * s.record + 255) & ~(size_t)255;
  return s;
}

struct LinearArgs {
  QuantShape s;
  int64_t n_rows, n_units;
  int32_t n_matrices;
  int32_t direct;              // with offsets: a unit is a matrix (all its rows), not a block of rows
  int32_t lds_rows;            // rows that the launch has LDS for: min(16 MT, n_rows)
  const uint8_t *packed;
  const int32_t *offsets;      // NULL: one matrix, every row
  const float *bias;
  int32_t relu, out_f32;
  int32_t wide_store;          // four neighbouring outputs lie in one aligned piece
  const void *x;
  void *y;
};

// one product with rows of type T (scale type and group are those of a.s); launches on stream
template <class T>
int linear_rows(const char *who, LinearArgs a, int32_t scale_type, void *stream);

// what a 16 x 16 x 32 instruction takes for rows of type T, and how many parts a row value has
template <class T> struct Mma;
template <> struct Mma<bf16> {
  typedef bf16x8 frag;
  typedef bf16x2 two;
  typedef float zero;   // there is no packed bf16 subtraction
  static constexpr int parts = 1;
  static __device__ __forceinline__ f32x4 mul(frag w, frag x, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, x, c, 0, 0, 0);
  }
  // q of 8 weights
  static __device__ __forceinline__ frag weights(uint32_t d) {
    struct { bf16x2 p[4]; } u;
    const uint32_t a = d & 0x0F0F0F0Fu, b = (d >> 4) & 0x0F0F0F0Fu;
    u.p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 512.f, false);
    u.p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 512.f, true);
    u.p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 512.f, false);
    u.p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 512.f, true);
    return __builtin_bit_cast(frag, u);
  }
  // q - z
  static __device__ __forceinline__ frag weights(uint32_t d, zero z) {
    struct { bf16x2 p[4]; } u;
    const uint32_t a = d & 0x0F0F0F0Fu, b = (d >> 4) & 0x0F0F0F0Fu;
    auto less = [&](auto v) { return bf16x2{(bf16)(v[0] - z), (bf16)(v[1] - z)}; };
    u.p[0] = less(__builtin_amdgcn_cvt_scalef32_pk_f32_fp8(a, 512.f, false));
    u.p[1] = less(__builtin_amdgcn_cvt_scalef32_pk_f32_fp8(a, 512.f, true));
    u.p[2] = less(__builtin_amdgcn_cvt_scalef32_pk_f32_fp8(b, 512.f, false));
    u.p[3] = less(__builtin_amdgcn_cvt_scalef32_pk_f32_fp8(b, 512.f, true));
    return __builtin_bit_cast(frag, u);
  }
  // c + 0 v: NaN if v holds an infinity or NaN
  static __device__ __forceinline__ float nothing(two v, float c) {
    return __builtin_amdgcn_fdot2_f32_bf16(v, two{(bf16)0.f, (bf16)0.f}, c, false);
  }
};
template <> struct Mma<f16> {
  typedef f16x8 frag;
  typedef f16x2 two;
  typedef f16 zero;
  static constexpr int parts = 1;
  static __device__ __forceinline__ f32x4 mul(frag w, frag x, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(w, x, c, 0, 0, 0);
  }
  static __device__ __forceinline__ frag weights(uint32_t d) {
    struct { f16x2 p[4]; } u;
    const uint32_t a = d & 0x0F0F0F0Fu, b = (d >> 4) & 0x0F0F0F0Fu;
    u.p[0] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, 512.f, false);
    u.p[1] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, 512.f, true);
    u.p[2] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, 512.f, false);
    u.p[3] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, 512.f, true);
    return __builtin_bit_cast(frag, u);
  }
  static __device__ __forceinline__ frag weights(uint32_t d, zero z) {
    frag w = weights(d);
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      const two v = two{w[i], w[i + 1]} - two{z, z};
      w[i] = v[0];
      w[i + 1] = v[1];
    }
    return w;
  }
  static __device__ __forceinline__ float nothing(two v, float c) {
    return __builtin_amdgcn_fdot2(v, two{(f16)0.f, (f16)0.f}, c, false);
  }
};
template <> struct Mma<float> : Mma<bf16> {
  static constexpr int parts = 3;
};

// how the zero points enter: all are 8 (products start from -8 sum x), after the group's products, or before them
enum Zeros { kEight, kAfter, kBefore };

template <class T> struct __attribute__((packed, aligned(sizeof(T)))) Eight { T v[8]; };

// The parts of 8 row values, most significant first.
// An infinity becomes NaN in every form: of float32 rows as inf - inf, of two-byte ones as inf q - inf z or, where z is
// taken off before (NONFINITE), here (0x7FFF is a NaN of both types).
template <class T, bool NONFINITE>
__device__ __forceinline__ void row_parts(const Eight<T> &r, typename Mma<T>::frag (&f)[Mma<T>::parts]) {
  if constexpr (sizeof(T) == 2) {
    struct Four { uint32_t d[4]; } v = __builtin_bit_cast(Four, r);
    if constexpr (NONFINITE) {
      float bad = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) bad = Mma<T>::nothing(__builtin_bit_cast(typename Mma<T>::two, v.d[i]), bad);
      const uint32_t nan = bad == 0.f ? 0u : 0x7FFF7FFFu;
#pragma unroll
      for (int i = 0; i < 4; ++i) v.d[i] |= nan;
    }
    f[0] = __builtin_bit_cast(typename Mma<T>::frag, v);
  } else {
    struct { uint32_t d[4]; } hi, mid, lo;
    float a[8], b[8], c[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {   // by truncation, so that no part overflows: 8 + 8 + 8 bits
      a[i] = __uint_as_float(__float_as_uint(r.v[i]) & 0xFFFF0000u);
      const float rest = r.v[i] - a[i];
      b[i] = __uint_as_float(__float_as_uint(rest) & 0xFFFF0000u);
      c[i] = rest - b[i];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {   // the upper halves of two floats
      hi.d[i] = __builtin_amdgcn_perm(__float_as_uint(a[2 * i + 1]), __float_as_uint(a[2 * i]), 0x07060302u);
      mid.d[i] = __builtin_amdgcn_perm(__float_as_uint(b[2 * i + 1]), __float_as_uint(b[2 * i]), 0x07060302u);
      lo.d[i] = __builtin_amdgcn_perm(__float_as_uint(c[2 * i + 1]), __float_as_uint(c[2 * i]), 0x07060302u);
    }
    f[0] = __builtin_bit_cast(bf16x8, hi);
    f[1] = __builtin_bit_cast(bf16x8, mid);
    f[2] = __builtin_bit_cast(bf16x8, lo);
  }
}

__device__ __forceinline__ int64_t row_end(const LinearArgs &a, int e) {
  const int64_t o = a.offsets[e];
  return o < 0 ? 0 : o > a.n_rows ? a.n_rows : o;
}

// With offsets: the matrix and the rows [*r0, *r1) of a unit; false if there are none.  A unit is a block of
// `most` rows of one matrix (every wave counts the matrices' blocks up), or all rows of a matrix (direct).
// Every lane of the wave gets the same answer.
__device__ __forceinline__ bool find_rows(const LinearArgs &a, int64_t unit, int most, int *matrix, int64_t *r0,
                                          int64_t *r1) {
  if (a.direct) {
    *matrix = (int)unit;
    *r0 = row_end(a, (int)unit);
    *r1 = row_end(a, (int)unit + 1);
    return *r0 < *r1;
  }
  const int l = lane_id();
  int before = 0, owner = -1, rest = 0;
#pragma unroll 1
  for (int e0 = 0; e0 < a.n_matrices; e0 += 64) {   // 64 matrices at a time
    const int e = e0 + l;
    const int64_t n = e < a.n_matrices ? row_end(a, e + 1) - row_end(a, e) : 0;
    const int mine = n > 0 ? (int)((n + most - 1) / most) : 0;
    const int upto = before + incl_sums(mine);
    const uint64_t above = __ballot(upto > unit);
    if (above != 0ull) {
      const int at = __ffsll((long long)above) - 1;
      owner = e0 + at;
      rest = (int)unit - __builtin_amdgcn_readlane(upto - mine, at);
      break;
    }
    before = __builtin_amdgcn_readlane(upto, 63);
  }
  if (owner < 0 || rest < 0) return false;   // rest < 0: offsets that do not ascend, their counts past 2^31
  const int64_t end = row_end(a, owner + 1);
  *matrix = owner;
  *r0 = row_end(a, owner) + (int64_t)rest * most;
  *r1 = *r0 + most < end ? *r0 + most : end;
  return *r0 < *r1;
}

// the scales of a record that one lane needs
template <class S, int NG>
struct Scales {
  struct __attribute__((aligned(4 * sizeof(S)))) Four { S s[4]; } g[NG];
};

// and its zero points: of the four outputs that the lane gets results of (after), of the one whose q it holds (before)
template <int NG, Zeros Z> struct ZeroPoints {};
template <int NG> struct ZeroPoints<NG, kAfter> {
  struct __attribute__((aligned(4 * NG))) Bytes { uint32_t d[NG]; } v;   // [output][g]
  __device__ __forceinline__ void load(const uint8_t *zeros, int h, int) {
    v = *reinterpret_cast<const Bytes *>(zeros + (uint32_t)(4 * NG * h));
  }
  __device__ __forceinline__ float of(int i, int g) const {
    const int at = i * NG + g;
    return (float)((v.d[at / 4] >> (8 * (at % 4))) & 255u);
  }
};
template <int NG> struct ZeroPoints<NG, kBefore> {
  uint32_t v;
  __device__ __forceinline__ void load(const uint8_t *zeros, int, int output) {
    const uint8_t *at = zeros + (uint32_t)(NG * output);
    if constexpr (NG == 4) v = *reinterpret_cast<const uint32_t *>(at);
    else if constexpr (NG == 2) v = *reinterpret_cast<const uint16_t *>(at);
    else v = *at;
  }
  __device__ __forceinline__ float of(int g) const { return (float)((v >> (8 * g)) & 255u); }
};

// the first `left` of four values
template <class O>
__device__ __forceinline__ void store_four(O *p, f32x4 v, int left, int wide) {
  if (wide) {
    struct __attribute__((aligned(4 * sizeof(O)))) Four { O v[4]; } f;
#pragma unroll
    for (int i = 0; i < 4; ++i) f.v[i] = (O)v[i];
    *reinterpret_cast<Four *>(p) = f;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < left) p[i] = (O)v[i];
  }
}

// A workgroup of WK x WN waves computes 16 NT WN outputs of a block of 16 MT rows (at most).  k goes by in
// chunks of WK U blocks: wave (ik, in) multiplies blocks ik U .. ik U + U - 1 of a chunk for its NT output
// tiles, with the weights in registers, straight from memory, and the rows in LDS, where every wave needs
// them: 0 past K, and float32 rows as their three parts, split once.  Rows are requested before weights:
// waiting for them leaves the weights in flight; other workgroups multiply meanwhile.  At the end the WK waves'
// sums meet in LDS, added in the waves' order.  OCC: waves per SIMD to leave registers for.
template <class T, int WK, int U>
struct Stage {
  static constexpr int kChunk = WK * U * kBlockK;      // k of a chunk
  static constexpr int kRow = kChunk * 2 + 16;         // bytes of a row of one part: lanes of one h in 64 banks
  static constexpr int kParts = Mma<T>::parts;
  static constexpr size_t bytes(int rows) { return (size_t)kParts * rows * kRow; }
};

template <class T, class S, int G, Zeros Z, int MT, int NT, int U, int WK, int WN, int OCC>
__global__ __launch_bounds__(64 * WK * WN, OCC) void k_linear(LinearArgs a) {
  using M = Mma<T>;
  using St = Stage<T, WK, U>;
  constexpr int P = M::parts, NG = kBlockK / G, kSteps = G / 32, MN = MT * NT, kThreads = 64 * WK * WN;
  constexpr int kPieces = St::kChunk / 8;                            // 8 values each, of a row of a chunk
  constexpr int kEach = (16 * MT * kPieces + kThreads - 1) / kThreads;   // pieces of a thread at most
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  const int64_t unit = (int64_t)blockIdx.z * gridDim.y + blockIdx.y;
  int matrix = 0;
  int64_t first, last;
  if (unit >= a.n_units) return;   // the whole workgroup
  if (a.offsets) {
    if (!find_rows(a, unit, 16 * MT, &matrix, &first, &last)) return;   // the whole workgroup
  } else {
    first = unit * (16 * MT);
    last = first + 16 * MT < a.n_rows ? first + 16 * MT : a.n_rows;
  }
  const int tid = threadIdx.x, l = tid % 64, wv = __builtin_amdgcn_readfirstlane(tid / 64);
  const int ik = wv % WK, in = wv / WK;
  const int j = l % 16, h = l / 16;
  const QuantShape &s = a.s;
  const int K = s.n_in, tile0 = (blockIdx.x * WN + in) * NT;
  const int n_chunks = (s.blocks + WK * U - 1) / (WK * U);
  const uint8_t *base = a.packed + (size_t)matrix * s.stride;
  const uint8_t *record[NT];   // of the wave, at block 0; a lane adds its own offset
  const size_t block_step = (size_t)s.tiles * s.record;
#pragma unroll
  for (int n = 0; n < NT; ++n)   // tiles past the last one compute a copy of it, never stored
    record[n] = base + (size_t)(tile0 + n < s.tiles ? tile0 + n : s.tiles - 1) * s.record;
  struct Weights {
    uint4 d[U][NT];
    Scales<S, NG> s[U][NT];
    ZeroPoints<NG, Z> z[U][NT];
  };
  // kBefore without zero points: bytes of the scales, which are not used, so that no load is conditional
  const uint32_t zeros_at = s.has_zeros ? kGroupsAt + kTileN * NG * (uint32_t)sizeof(S) : kGroupsAt;
  auto load_weights = [&](Weights &w, int chunk) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int b = chunk * (WK * U) + ik * U + u;   // past the last block: a copy of it, multiplied by 0
      const size_t at = (size_t)(b < s.blocks ? b : s.blocks - 1) * block_step;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        w.d[u][n] = *reinterpret_cast<const uint4 *>(record[n] + at + (uint32_t)(l * 16));
        w.s[u][n] = *reinterpret_cast<const Scales<S, NG> *>(record[n] + at + kGroupsAt +
                                                             (uint32_t)(h * (int)sizeof(Scales<S, NG>)));
        if constexpr (Z != kEight) w.z[u][n].load(record[n] + at + zeros_at, h, j);
      }
    }
  };
  typename M::frag fixed;
#pragma unroll
  for (int i = 0; i < 8; ++i) fixed[i] = Z == kEight ? -8.f : 1.f;
  for (int64_t r0 = first; r0 < last; r0 += 16 * MT) {
    const int n_rows = last - r0 < 16 * MT ? (int)(last - r0) : 16 * MT;
    const T *rows = (const T *)a.x + r0 * K;
    // pieces tid, tid + kThreads, ..: piece p is values 8 (p % kPieces) .. of row p / kPieces.  A piece that
    // reaches past K is read further left (its value is not used), so that no load is conditional.
    auto load_rows = [&](Eight<T> (&x)[kEach], int chunk) {
#pragma unroll
      for (int e = 0; e < kEach; ++e) {
        if (K < 8 || e * kThreads >= n_rows * kPieces) break;
        const int p = e * kThreads + tid, r = p / kPieces, k = chunk * St::kChunk + 8 * (p % kPieces);
        x[e] = *reinterpret_cast<const Eight<T> *>(rows + (int64_t)(r < n_rows ? r : 0) * K + (k + 8 <= K ? k : K - 8));
      }
    };
    auto put_piece = [&](int p, int r, const Eight<T> &e) {
      typename M::frag f[P];
      row_parts<T, Z == kBefore>(e, f);
#pragma unroll
      for (int q = 0; q < P; ++q)
        *reinterpret_cast<typename M::frag *>(lds + (q * a.lds_rows + r) * St::kRow + 16 * (p % kPieces)) = f[q];
    };
    auto store_rows = [&](const Eight<T> (&x)[kEach], int chunk) {
#pragma unroll
      for (int e = 0; e < kEach; ++e) {
        if (e * kThreads >= n_rows * kPieces) break;
        const int p = e * kThreads + tid, r = p / kPieces, k = chunk * St::kChunk + 8 * (p % kPieces);
        if (r < n_rows && (k + 8 <= K || k >= K)) put_piece(p, r, k < K ? x[e] : Eight<T>{});
      }
      if ((chunk + 1) * St::kChunk > K && K % 8) {   // the piece that K ends inside: a thread per row
        for (int r = tid; r < n_rows; r += kThreads) {
          const int k = K / 8 * 8;
          Eight<T> e{};
#pragma unroll
          for (int i = 0; i < 7; ++i) {
            const T v = rows[(int64_t)r * K + (k + i < K ? k + i : k)];
            e.v[i] = k + i < K ? v : T(0.f);
          }
          put_piece((k - chunk * St::kChunk) / 8, r, e);
        }
      }
    };
    f32x4 acc[MT][NT];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n) acc[m][n] = f32x4{0.f, 0.f, 0.f, 0.f};
    int row_at[MT];   // lanes past the last row compute a copy of it, never stored
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const int r = 16 * m + j;
      row_at[m] = (r < n_rows ? r : n_rows - 1) * St::kRow + ik * (U * kBlockK * 2) + 16 * h;
    }
    auto multiply = [&](const Weights &k) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        auto row_frag = [&](int p, int m, int st) {
          return *reinterpret_cast<const typename M::frag *>(lds + p * a.lds_rows * St::kRow + row_at[m] +
                                                             (u * kBlockK + 32 * st) * 2);
        };
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          // xs = sum x over the group (or, without zero points, -8 sum x, which the products start from)
          f32x4 part[MT][NT], xs[MT];
#pragma unroll
          for (int m = 0; m < MT; ++m) xs[m] = f32x4{0.f, 0.f, 0.f, 0.f};
          if constexpr (Z != kBefore) {
#pragma unroll
            for (int st = g * kSteps; st < (g + 1) * kSteps; ++st)
#pragma unroll
              for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int p = 0; p < P; ++p) xs[m] = M::mul(fixed, row_frag(p, m, st), xs[m]);
          }
          typename M::zero z[NT];
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            if constexpr (Z == kBefore) z[n] = s.has_zeros ? (typename M::zero)k.z[u][n].of(g) : (typename M::zero)8.f;
#pragma unroll
            for (int m = 0; m < MT; ++m) part[m][n] = Z == kEight ? xs[m] : f32x4{0.f, 0.f, 0.f, 0.f};
          }
#pragma unroll
          for (int st = g * kSteps; st < (g + 1) * kSteps; ++st) {
            typename M::frag w[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              const uint32_t d = st == 0 ? k.d[u][n].x : st == 1 ? k.d[u][n].y : st == 2 ? k.d[u][n].z : k.d[u][n].w;
              if constexpr (Z == kBefore) w[n] = M::weights(d, z[n]);
              else w[n] = M::weights(d);
            }
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
              for (int p = 0; p < P; ++p) {
                const typename M::frag x = row_frag(p, m, st);
#pragma unroll
                for (int n = 0; n < NT; ++n) part[m][n] = M::mul(w[n], x, part[m][n]);
              }
          }
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float sv = (float)k.s[u][n].g[g].s[i];
              if constexpr (Z == kAfter) {
                const float zv = k.z[u][n].of(i, g);
#pragma unroll
                for (int m = 0; m < MT; ++m)
                  acc[m][n][i] = fmaf(sv, fmaf(-zv, xs[m][i], part[m][n][i]), acc[m][n][i]);
              } else {
#pragma unroll
                for (int m = 0; m < MT; ++m) acc[m][n][i] = fmaf(sv, part[m][n][i], acc[m][n][i]);
              }
            }
        }
      }
    };
    if (r0 != first) __syncthreads();   // the rows before, or their sums, have been read
    f32x4 bias[NT];   // requested here; outputs past the end repeat the last one's, never stored
#pragma unroll
    for (int n = 0; n < NT; ++n) bias[n] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (a.bias && ik == 0) {
      const float *row = a.bias + (size_t)matrix * s.n_out;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int o = (tile0 + n) * kTileN + 4 * h + i;
          bias[n][i] = row[o < s.n_out ? o : s.n_out - 1];
        }
    }
    Eight<T> x[kEach];
#pragma unroll 1
    for (int c = 0; c < n_chunks; ++c) {
      Weights now;
      load_rows(x, c);
      load_weights(now, c);
      if (c > 0) __syncthreads();   // the chunk before has been read
      store_rows(x, c);
      __syncthreads();
      multiply(now);
    }
    f32x4 *sums = reinterpret_cast<f32x4 *>(lds);   // [in][ik - 1][MT * NT][64]
    if constexpr (WK > 1) {
      __syncthreads();   // the rows have been read
      if (ik > 0) {
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int n = 0; n < NT; ++n) sums[((in * (WK - 1) + ik - 1) * MN + m * NT + n) * 64 + l] = acc[m][n];
      }
      __syncthreads();
    }
    if (ik == 0) {
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          f32x4 v = acc[m][n];
#pragma unroll
          for (int w = 0; w < WK - 1; ++w) {
            const f32x4 u = sums[((in * (WK - 1) + w) * MN + m * NT + n) * 64 + l];
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] += u[i];
          }
          // lane (j, h) holds outputs 4 h .. 4 h + 3 of row j
          const int64_t r = r0 + 16 * m + j;
          const int o = (tile0 + n) * kTileN + 4 * h;
          if (r < last && o < s.n_out) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              v[i] += bias[n][i];
              if (a.relu) v[i] = v[i] < 0.f ? 0.f : v[i];   // NaN stays
            }
            if (a.out_f32) store_four((float *)a.y + r * s.n_out + o, v, s.n_out - o, a.wide_store);
            else store_four((T *)a.y + r * s.n_out + o, v, s.n_out - o, a.wide_store);
          }
        }
    }
  }
}

template <class T, class S, int G, Zeros Z, int MT, int NT, int U, int WK, int WN, int OCC>
int launch_linear(const char *who, LinearArgs a, void *stream) {
  using St = Stage<T, WK, U>;
  static_assert(St::bytes(16 * MT) <= 160 * 1024, "the rows of a chunk fit a compute unit's LDS");
  const int64_t blocks = (a.n_rows + 16 * MT - 1) / (16 * MT);
  a.direct = a.offsets && blocks <= 4;
  a.n_units = !a.offsets ? blocks : a.direct ? a.n_matrices : blocks + a.n_matrices;
  a.lds_rows = (int32_t)std::min<int64_t>(a.n_rows, 16 * MT);
  const int64_t y = a.n_units < 32768 ? a.n_units : 32768, z = (a.n_units + y - 1) / y;
  const dim3 grid((unsigned)((a.s.tiles + NT * WN - 1) / (NT * WN)), (unsigned)y, (unsigned)z);
  const size_t lds = std::max(St::bytes(a.lds_rows), (size_t)WN * (WK - 1) * MT * NT * 1024);
  return launch(who, k_linear<T, S, G, Z, MT, NT, U, WK, WN, OCC>, grid, 64 * WK * WN, lds, stream, a);
}

template <class F>
int with_group(int32_t group, F f) {
  if (group == 32) return f(std::integral_constant<int, 32>{});
  if (group == 64) return f(std::integral_constant<int, 64>{});
  return f(std::integral_constant<int, 128>{});
}

// How a product is cut: rows x outputs of a workgroup and how its waves share them, by the number of workgroups that
// each cut gives.  The largest cut that still gives 512 (two per compute unit, so that one loads while the other
// multiplies; the 8 waves of the 64 x 256 cut do with 256) is taken.  All figures are us in a replayed graph over
// rotating inputs; bfloat16 rows, scales and outputs, groups of 128, no zero points, unless stated; the chosen cut
// first.
//   4096 rows, 4096 x 4096:  32 x 256 cut 199,  32 x 128 235,   64 x 256 255
//   1024 rows, 4096 x 1024:  32 x 256 cut 18.0, 64 x 256 19.9,  32 x 128 21.8
//    512 rows, 4096 x 1024:  32 x 128 cut 11.7, 32 x 256 13.6
//   1024 rows, 1024 x 1024:  32 x  64 cut  9.4, 32 x 128 11.3
//    256 rows, 1024 x 1024:  16 x  32 cut  5.8, 32 x  64  8.0,  16 x  16  8.2
//     16 rows, 4096 x 1024:  16 x  16 cut  4.3, 16 x  32  4.9
// The 32 x 256 cut keeps four tiles' scales and weights: with groups of 32 64 x 256 is ahead (1024 rows, 4096 x 1024:
// 21.7 against 22.8), with groups of 64 the two are within 4 % (20.6 and 19.9).  Where q - z is formed, 64 x 256
// makes it for twice the rows (the same product with float32 outputs: 22.2 against 26.6; of float32 rows 36.7 against
// 37.9, with groups of 32 39.9 against 48.0).
// Up to 16 rows of a large matrix (a decoding step) are bound by the weights' bytes and want about 8 waves on every
// compute unit, each with two tiles in flight, of two blocks where they stay in registers: four or eight along k.
//   1 row, 16384 x 4096: 16 x 32 cut of two blocks 10.7, of one 12.5, 16 x 64 13.2, 16 x 16 16.1; float32 rows, one
//   block, 18.1, 16 rows 26.4 (two blocks 16.6 and, as 16 rows' parts then fill most of LDS, 37.5).
// 17 to 64 rows: 16 x 64 while that gives 512 (64 rows, 8192 x 2048: 9.9, 16 x 32 11.0).  Fewer: 8 waves along k for
// as many workgroups as compute units, 16 x 32 (64 rows, 2048 x 4096: 9.0, 16 x 16 12.4; float32 rows 14.7, 22.0) or,
// up to 128 of those, 16 x 16; each wave with two blocks of a long k (1 row, 4096 x 4096: 5.3, one block 5.6; 8 rows,
// 2048 x 8192: 8.7, 10.0).
// Rows by expert: a cut of 32 rows is mostly empty below 8 rows per expert on average (64 rows, 64 experts of 2048 x
// 1024: 16 x 64 cut 10.2, 32 x 128 12.4; 1024 rows: 32 x 128 26.1, 16 x 64 28.2, 16 x 32 33.6), and one of 64 rows
// loses to 32 by the experts' uneven numbers of rows (4096 rows, 8 experts: 42.4, 64 x 256 57.2).  32 x 256 wins over
// 32 x 128 where enough workgroups are left: 8192 rows, 8 experts of 4096 x 4096 434 against 467; 32 experts of 2048
// x 1024, 1024 rows (384 workgroups) 19.1 against 20.7; 8 experts, 1408 rows (384) 18.7 against 19.9, but 1024 rows
// (288) 17.3 against 15.9: from 384 (4096 rows, 8 experts of 2048 x 1024, is an exception: 44.4 against 42.4).
// Below 8 rows per expert 16 x 64 wins over 16 x 32 likewise: 8 experts of 2048 x 512, 64 rows (256 workgroups) 7.2
// against 6.4, 80 rows (288) 5.5 against 5.6, 64 experts of 2048 x 1024, 64 rows 10.2 against 10.6: from 288.
// Where two tiles of two blocks do not stay in registers, one block each: groups of 32, 400 rows, 64 experts 20.8
// against 22.5; float32 rows, 256 rows, 64 experts 21.7 against 25.4.
// OCC: the waves per SIMD that registers are limited for; 25 of the 612 kinds (mostly float scales with zero points)
// spill 12 to 60 bytes per lane all the same.  32 x 128: three (4096 rows by 8 experts of 2048 x 1024, float32 rows,
// groups of 64, 89 against 108 with two; bfloat16 with zero points, groups of 64, 51 against 62), for float32 rows
// with groups of 128 two (85.1 against 86.8).  16 x 64: three (64 rows by 64 experts of 2048 x 1024, zero points,
// groups of 64, 11.3 against 12.0), for float32 rows two (15.4 against 16.0).  16 x 32: four (64 rows by 64 experts of
// 1024 x 1024, zero points, 8.3 against 8.6), with groups of 32 two (9.6 against 10.2).
template <class T, class S, int G, Zeros Z>
int linear_cut(const char *who, LinearArgs a, void *stream) {
  constexpr bool kShort = sizeof(T) == 2;
  constexpr int kWaves32 = kShort || G <= 64 ? 3 : 2, kWaves16 = kShort && G >= 64 ? 4 : 2;
  constexpr bool kFew = kShort && G >= 64;                   // two tiles of two blocks stay in registers
  constexpr bool kWide = Z != kBefore && G == 128;           // 32 x 256 rather than 64 x 256
  const int64_t rows = a.n_rows, tiles = a.s.tiles, blocks = a.s.blocks;
  auto groups = [&](int64_t r, int64_t t) { return ((rows + r - 1) / r) * ((tiles + t - 1) / t); };
  auto cut_16_64 = [&] { return launch_linear<T, S, G, Z, 1, 2, kFew ? 2 : 1, 2, 2, kFew ? 3 : 2>(who, a, stream); };
  auto cut_16_32 = [&] { return launch_linear<T, S, G, Z, 1, 1, 2, 2, 2, kWaves16>(who, a, stream); };
  if (a.offsets) {
    const int64_t some = std::min<int64_t>(a.n_matrices, rows) / 2;   // half-filled blocks, about
    const bool full = rows >= 8 * (int64_t)a.n_matrices;
    if constexpr (kWide)
      if (full && (rows / 32 + some) * ((tiles + 15) / 16) >= 384)
        return launch_linear<T, S, G, Z, 2, 4, 1, 1, 4, 2>(who, a, stream);
    if (full && (rows / 32 + some) * ((tiles + 7) / 8) >= 256)
      return launch_linear<T, S, G, Z, 2, 2, 1, 1, 4, kWaves32>(who, a, stream);
    if ((rows / 16 + some) * ((tiles + 3) / 4) >= 288) return cut_16_64();
    return cut_16_32();
  }
  if constexpr (kWide) {
    if (groups(32, 16) >= 512) return launch_linear<T, S, G, Z, 2, 4, 1, 1, 4, 2>(who, a, stream);
  } else {
    if (groups(64, 16) >= 256) return launch_linear<T, S, G, Z, 4, 2, 1, 1, 8, 2>(who, a, stream);
  }
  if (groups(32, 8) >= 512) return launch_linear<T, S, G, Z, 2, 2, 1, 1, 4, kWaves32>(who, a, stream);
  if (groups(32, 4) >= 512) return launch_linear<T, S, G, Z, 2, 2, 1, 2, 2, 2>(who, a, stream);
  if (rows <= 16 && groups(16, 2) >= 512 && blocks >= 8)
    return launch_linear<T, S, G, Z, 1, 2, kFew ? 2 : 1, 4, 1, 2>(who, a, stream);
  if (groups(16, 4) >= 512) return cut_16_64();
  if (blocks < 8 || groups(16, 2) > (rows <= 16 ? 511 : 256)) return cut_16_32();
  if (groups(16, 2) > 128) {
    if constexpr (kShort)   // float32 rows of two blocks: not in LDS
      if (blocks >= 16) return launch_linear<T, S, G, Z, 1, 2, 2, 8, 1, 2>(who, a, stream);
    return launch_linear<T, S, G, Z, 1, 2, 1, 8, 1, 2>(who, a, stream);
  }
  if constexpr (kShort)
    if (blocks >= 16) return launch_linear<T, S, G, Z, 1, 1, 2, 8, 1, 2>(who, a, stream);
  return launch_linear<T, S, G, Z, 1, 1, 1, 8, 1, 2>(who, a, stream);
}

template <class T>
int linear_rows(const char *who, LinearArgs a, int32_t scale_type, void *stream) {
  return with_type(scale_type, [&](auto ts) {
    return with_group(a.s.group, [&](auto g) {
      using S = decltype(ts);
      constexpr int G = decltype(g)::value;
      if constexpr (sizeof(T) == 2)
        if (!a.out_f32)
          return a.s.has_zeros ? linear_cut<T, S, G, kAfter>(who, a, stream) : linear_cut<T, S, G, kEight>(who, a, stream);
      return linear_cut<T, S, G, kBefore>(who, a, stream);
    });
  });
}

}  // namespace svt

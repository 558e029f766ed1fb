// svt_quant.hip - products with 4-bit weights and group scales on gfx950: one matrix for all rows, or one
// matrix per expert for rows sorted by expert.
//
//   W[n][k] = s[n][g] (q[n][k] - z[n][g]),  g = k / group,  q in 0 .. 15
//   y[r][n] = act(bias[n] + sum_k x[r][k] W[n][k])
//           = act(bias[n] + sum_g s[n][g] (sum_{k in g} x[r][k] q[n][k] - z[n][g] sum_{k in g} x[r][k]))
//
// The inner sums run on the matrix cores (v_mfma_f32_16x16x32, 16 outputs x 16 rows x 32 k) with q as bf16
// or f16, which hold 0 .. 15 exactly, and float32 accumulation: no weight is rounded, and s and z are
// applied to float32 group sums.  sum x comes from the same instruction with a matrix of ones, in the
// lanes that need it.
// q reaches bf16/f16 two at a time: the byte 0000qqqq read as an 8-bit float with 3 mantissa bits is
// q * 2^-9 (its subnormals and its first binade share one spacing), and v_cvt_scalef32_pk_* turns two such
// bytes into two exact numbers with the scale 2^9.
// float32 rows are split into three bf16 parts of 8 bits each (24 bits: exact), one instruction per part.

#include <type_traits>

#include "svt_experts.h"

namespace svt {

namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef f16 f16x2 __attribute__((ext_vector_type(2)));
typedef f16 f16x8 __attribute__((ext_vector_type(8)));

constexpr int kTileN = 16;        // outputs of a tile
constexpr int kBlockK = 128;      // k of a block: 4 instructions, 16 bytes of q per lane
constexpr int kMaxWaves = 8;
constexpr int kMaxIn = 1 << 20, kMaxOut = 1 << 19;

// Layout of the packed weights, per matrix (all sizes in bytes, the matrix's stride a multiple of 256):
//   q       [tile][block][lane][16]: lane l holds outputs l % 16, k = 128 block + 32 s + 8 (l / 16) + i for
//           s = 0..3 in dword s, whose byte i (0..3) holds i in its low and i + 4 in its high half
//   scales  [tile][group][16], zeros [tile][group][16] (one byte each, where there are any)
// Outputs and groups past the end have scale 0.
struct QuantShape {
  int32_t n_out, n_in, group, has_zeros;
  int32_t tiles, blocks, groups;   // groups: with the last block's padding
  size_t scale_at, zero_at, stride;
};

QuantShape quant_shape(const svt_quant_weights &w) {
  QuantShape s;
  s.n_out = w.n_out;
  s.n_in = w.n_in;
  s.group = w.group;
  s.has_zeros = w.has_zeros;
  s.tiles = (w.n_out + kTileN - 1) / kTileN;
  s.blocks = (w.n_in + kBlockK - 1) / kBlockK;
  s.groups = s.blocks * (kBlockK / w.group);
  s.scale_at = (size_t)s.tiles * s.blocks * 1024;
  s.zero_at = s.scale_at + (size_t)s.tiles * s.groups * kTileN * elem_size(w.scale_type);
  s.stride = s.zero_at + (w.has_zeros ? (size_t)s.tiles * s.groups * kTileN : 0);
  s.stride = (s.stride + 255) & ~(size_t)255;
  return s;
}

// ---- pack ----------------------------------------------------------------------------------------

constexpr int kPackThreads = 256;

__global__ __launch_bounds__(kPackThreads) void k_pack_q(QuantShape s, int64_t n_pieces, const uint8_t *nibbles,
                                                         uint8_t *packed) {
  const int64_t row_bytes = (s.n_in + 1) / 2;
  const int64_t per_matrix = (int64_t)s.tiles * s.blocks * 64;
  for (int64_t p = (int64_t)blockIdx.x * kPackThreads + threadIdx.x; p < n_pieces; p += (int64_t)gridDim.x * kPackThreads) {
    const int64_t m = p / per_matrix, r = p % per_matrix;
    const int lane = (int)(r % 64);
    const int64_t tb = r / 64;
    const int block = (int)(tb % s.blocks);
    const int n = (int)(tb / s.blocks) * kTileN + lane % 16;
    const uint8_t *row = nibbles + (m * s.n_out + n) * row_bytes;
    uint4 out;
    uint32_t *o = &out.x;
    for (int st = 0; st < 4; ++st) {
      const int k0 = block * kBlockK + 32 * st + 8 * (lane / 16);
      uint32_t d = 0u;
      for (int i = 0; i < 8; ++i) {
        const int k = k0 + i;
        const uint32_t q = (n < s.n_out && k < s.n_in) ? (row[k / 2] >> (4 * (k % 2))) & 15u : 0u;
        d |= q << (8 * (i % 4) + 4 * (i / 4));
      }
      o[st] = d;
    }
    *reinterpret_cast<uint4 *>(packed + m * s.stride + r * 16) = out;
  }
}

template <class T>
__global__ __launch_bounds__(kPackThreads) void k_pack_groups(QuantShape s, int64_t n_values, int src_groups, size_t at,
                                                              const T *src, uint8_t *packed) {
  const int64_t per_matrix = (int64_t)s.tiles * s.groups * kTileN;
  for (int64_t p = (int64_t)blockIdx.x * kPackThreads + threadIdx.x; p < n_values; p += (int64_t)gridDim.x * kPackThreads) {
    const int64_t m = p / per_matrix, r = p % per_matrix;
    const int64_t tg = r / kTileN;
    const int g = (int)(tg % s.groups);
    const int n = (int)(tg / s.groups) * kTileN + (int)(r % kTileN);
    const T v = (n < s.n_out && g < src_groups) ? src[(m * s.n_out + n) * src_groups + g] : T(0);
    reinterpret_cast<T *>(packed + m * s.stride + at)[r] = v;
  }
}

// ---- product -------------------------------------------------------------------------------------

struct LinearArgs {
  QuantShape s;
  int64_t n_rows;
  int32_t n_matrices, n_waves;
  int64_t n_units;             // blocks of rows
  const uint8_t *packed;
  const int32_t *offsets;      // NULL: one matrix, every row
  const float *bias;
  int32_t relu, out_f32;
  const void *x;
  void *y;
};

// what a 16 x 16 x 32 instruction takes for rows of type T, and how many parts a row value has
template <class T> struct Mma;
template <> struct Mma<bf16> {
  typedef bf16x8 frag;
  static constexpr int parts = 1;
  static __device__ __forceinline__ f32x4 mul(frag w, frag x, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, x, c, 0, 0, 0);
  }
  static __device__ __forceinline__ frag weights(uint32_t d) {
    struct { bf16x2 p[4]; } u;
    const uint32_t a = d & 0x0F0F0F0Fu, b = (d >> 4) & 0x0F0F0F0Fu;
    u.p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 512.f, false);
    u.p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 512.f, true);
    u.p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 512.f, false);
    u.p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 512.f, true);
    return __builtin_bit_cast(frag, u);
  }
};
template <> struct Mma<f16> {
  typedef f16x8 frag;
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
};
template <> struct Mma<float> : Mma<bf16> {
  static constexpr int parts = 3;
};

template <class T> struct __attribute__((packed, aligned(sizeof(T)))) Eight { T v[8]; };

// 8 values of a row from k on; values at or past K are 0
template <class T>
__device__ __forceinline__ Eight<T> load_row(const T *row, int k, int K, bool whole) {
  Eight<T> r;
  if (whole) {
    r = *reinterpret_cast<const Eight<T> *>(row + k);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) r.v[i] = k + i < K ? row[k + i] : T(0.f);
  }
  return r;
}

// the parts of 8 row values, most significant first
template <class T>
__device__ __forceinline__ void row_parts(const Eight<T> &r, typename Mma<T>::frag (&f)[Mma<T>::parts]) {
  if constexpr (sizeof(T) == 2) {
    f[0] = __builtin_bit_cast(typename Mma<T>::frag, r);
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

// block `unit` of at most `most` rows: its matrix and rows [*r0, *r1); false if there is none.  Every lane
// of the wave gets the same answer.  Offsets are clamped to [0, n_rows].
__device__ __forceinline__ bool find_rows(const LinearArgs &a, int64_t unit, int most, int *matrix, int64_t *r0,
                                          int64_t *r1) {
  if (!a.offsets) {
    *matrix = 0;
    *r0 = unit * most;
    *r1 = *r0 + most < a.n_rows ? *r0 + most : a.n_rows;
    return *r0 < a.n_rows;
  }
  const int l = lane_id(), each = (a.n_matrices + 63) / 64;
  auto clamped = [&](int e) {
    const int64_t o = a.offsets[e];
    return o < 0 ? 0 : o > a.n_rows ? a.n_rows : o;
  };
  int mine = 0;
  for (int i = 0; i < each; ++i) {
    const int e = l * each + i;
    if (e < a.n_matrices) {
      const int64_t n = clamped(e + 1) - clamped(e);
      mine += n > 0 ? (int)((n + most - 1) / most) : 0;
    }
  }
  const int upto = wave_incl_scan(mine);
  const uint64_t above = __ballot(upto > unit);
  if (above == 0ull) return false;
  const int owner = __ffsll((long long)above) - 1;
  int rest = (int)unit - __shfl(upto - mine, owner), e = owner * each;
  for (int i = 0; i < each; ++i, ++e) {
    if (e >= a.n_matrices) return false;
    const int64_t n = clamped(e + 1) - clamped(e);
    const int b = n > 0 ? (int)((n + most - 1) / most) : 0;
    if (rest < b) break;
    rest -= b;
  }
  if (e >= a.n_matrices) return false;
  const int64_t end = clamped(e + 1);
  *matrix = __builtin_amdgcn_readfirstlane(e);
  *r0 = clamped(e) + (int64_t)rest * most;
  *r1 = *r0 + most < end ? *r0 + most : end;
  return *r0 < *r1;
}

template <class S>
__device__ __forceinline__ f32x4 load_scales(const S *p) {
  struct __attribute__((aligned(4 * sizeof(S)))) Four { S v[4]; };
  const Four r = *reinterpret_cast<const Four *>(p);
  return f32x4{(float)r.v[0], (float)r.v[1], (float)r.v[2], (float)r.v[3]};
}

// A workgroup computes 16 NT outputs of one block of 16 MT rows.  Its waves split k (block i goes to wave
// i % n_waves); their sums meet in LDS, added in the waves' order.
template <class T, class S, int G, int MT, int NT>
__global__ __launch_bounds__(64 * kMaxWaves) void k_linear(LinearArgs a) {
  using M = Mma<T>;
  constexpr int P = M::parts, NG = kBlockK / G;
  extern __shared__ f32x4 sums[];   // [wave][MT * NT][64]
  const int64_t unit = (int64_t)blockIdx.z * gridDim.y + blockIdx.y;
  int matrix;
  int64_t r0, r1;
  if (unit >= a.n_units || !find_rows(a, unit, 16 * MT, &matrix, &r0, &r1)) return;   // the whole workgroup
  const int l = threadIdx.x % 64, wv = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int j = l % 16, h = l / 16;
  const QuantShape &s = a.s;
  const int K = s.n_in;
  const uint8_t *base = a.packed + (size_t)matrix * s.stride;
  const uint8_t *q[NT];
  const S *scale[NT];
  const uint8_t *zero[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {   // tiles past the last one compute a copy of it, never stored
    const int t = blockIdx.x * NT + n;
    const size_t tile = t < s.tiles ? t : s.tiles - 1;
    q[n] = base + tile * s.blocks * 1024 + l * 16;
    scale[n] = (const S *)(base + s.scale_at) + tile * s.groups * kTileN + 4 * h;
    zero[n] = base + s.zero_at + tile * s.groups * kTileN + 4 * h;
  }
  const T *rows[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {   // lanes past the last row compute a copy of it, never stored
    const int64_t r = r0 + 16 * m + j;
    rows[m] = (const T *)a.x + (r < r1 ? r : r1 - 1) * K;
  }
  typename M::frag ones;
#pragma unroll
  for (int i = 0; i < 8; ++i) ones[i] = 1.f;
  f32x4 acc[MT][NT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[m][n] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int b = wv; b < s.blocks; b += a.n_waves) {
    uint4 d[NT];
    f32x4 sc[NT][NG], ze[NT][NG];
#pragma unroll
    for (int n = 0; n < NT; ++n) d[n] = *reinterpret_cast<const uint4 *>(q[n] + (size_t)b * 1024);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int g = 0; g < NG; ++g) sc[n][g] = load_scales(scale[n] + ((size_t)b * NG + g) * kTileN);
    if (s.has_zeros) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          const uint32_t z = *reinterpret_cast<const uint32_t *>(zero[n] + ((size_t)b * NG + g) * kTileN);
#pragma unroll
          for (int i = 0; i < 4; ++i) ze[n][g][i] = (float)((z >> (8 * i)) & 255u);
        }
    } else {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int g = 0; g < NG; ++g) ze[n][g] = f32x4{8.f, 8.f, 8.f, 8.f};
    }
    const bool whole = (b + 1) * kBlockK <= K;
    f32x4 part[MT][NT], xs[MT];
#pragma unroll
    for (int st = 0; st < 4; ++st) {
      if (st % (G / 32) == 0) {
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          xs[m] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int n = 0; n < NT; ++n) part[m][n] = f32x4{0.f, 0.f, 0.f, 0.f};
        }
      }
      typename M::frag w[NT];
#pragma unroll
      for (int n = 0; n < NT; ++n) w[n] = M::weights(st == 0 ? d[n].x : st == 1 ? d[n].y : st == 2 ? d[n].z : d[n].w);
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        typename M::frag x[P];
        row_parts<T>(load_row<T>(rows[m], b * kBlockK + 32 * st + 8 * h, K, whole), x);
#pragma unroll
        for (int p = 0; p < P; ++p) {
          xs[m] = M::mul(ones, x[p], xs[m]);
#pragma unroll
          for (int n = 0; n < NT; ++n) part[m][n] = M::mul(w[n], x[p], part[m][n]);
        }
      }
      if (st % (G / 32) == G / 32 - 1) {
        constexpr int kSteps = G / 32;
        const int g = st / kSteps;
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              acc[m][n][i] = fmaf(sc[n][g][i], fmaf(-ze[n][g][i], xs[m][i], part[m][n][i]), acc[m][n][i]);
      }
    }
  }
  constexpr int MN = MT * NT;
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n) sums[(wv * MN + m * NT + n) * 64 + l] = acc[m][n];
  __syncthreads();
  // lane (j, h) of a tile pair holds outputs 4 h .. 4 h + 3 of row j
  for (int c = wv; c < MN; c += a.n_waves) {
    const int m = c / NT, n = c % NT;
    const int64_t r = r0 + 16 * m + j;
    const int o = (blockIdx.x * NT + n) * kTileN + 4 * h;
    if (r >= r1 || o >= s.n_out) continue;
    f32x4 v = sums[c * 64 + l];
    for (int w = 1; w < a.n_waves; ++w) {
      const f32x4 u = sums[(w * MN + c) * 64 + l];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] += u[i];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (o + i >= s.n_out) break;
      if (a.bias) v[i] += a.bias[(size_t)matrix * s.n_out + o + i];
      if (a.relu) v[i] = v[i] < 0.f ? 0.f : v[i];   // NaN stays
      if (a.out_f32) ((float *)a.y)[r * s.n_out + o + i] = v[i];
      else ((T *)a.y)[r * s.n_out + o + i] = (T)v[i];
    }
  }
}

template <class T, class S, int G, int MT, int NT>
void launch_linear(LinearArgs a, hipStream_t stream) {
  a.n_waves = a.s.blocks < kMaxWaves ? a.s.blocks : kMaxWaves;
  a.n_units = a.offsets ? (a.n_rows + 16 * MT - 1) / (16 * MT) + a.n_matrices : (a.n_rows + 16 * MT - 1) / (16 * MT);
  const int64_t y = a.n_units < 32768 ? a.n_units : 32768, z = (a.n_units + y - 1) / y;
  const dim3 grid((unsigned)((a.s.tiles + NT - 1) / NT), (unsigned)y, (unsigned)z);
  k_linear<T, S, G, MT, NT><<<grid, 64 * a.n_waves, (size_t)a.n_waves * MT * NT * 1024, stream>>>(a);
}

template <class F>
void with_group(int32_t group, F f) {
  if (group == 32) f(std::integral_constant<int, 32>{});
  else if (group == 64) f(std::integral_constant<int, 64>{});
  else f(std::integral_constant<int, 128>{});
}

int check_weights(const char *who, const svt_quant_weights *w) {
  if (!w) return report(SVT_EINVAL, "%s: NULL weights", who);
  if (w->n_matrices < 1 || w->n_matrices > SVT_MAX_EXPERTS)
    return report(SVT_EINVAL, "%s: n_matrices %d out of [1, %d]", who, w->n_matrices, SVT_MAX_EXPERTS);
  if (w->n_out < 1 || w->n_out > kMaxOut) return report(SVT_EINVAL, "%s: n_out %d out of [1, %d]", who, w->n_out, kMaxOut);
  if (w->n_in < 1 || w->n_in > kMaxIn) return report(SVT_EINVAL, "%s: n_in %d out of [1, %d]", who, w->n_in, kMaxIn);
  if (w->group != 32 && w->group != 64 && w->group != 128)
    return report(SVT_EUNSUPPORTED, "%s: group %d not in {32, 64, 128}", who, w->group);
  if (!elem_size(w->scale_type)) return report(SVT_EINVAL, "%s: unknown scale type %d", who, w->scale_type);
  if (w->has_zeros != 0 && w->has_zeros != 1) return report(SVT_EINVAL, "%s: has_zeros %d is not 0 or 1", who, w->has_zeros);
  return SVT_OK;
}

}  // namespace

}  // namespace svt

using namespace svt;

extern "C" size_t svt_quant_pack_size(const svt_quant_weights *w) {
  (void)report(SVT_OK, "%s", "");
  if (check_weights("svt_quant_pack_size", w) != SVT_OK) return 0;
  return quant_shape(*w).stride * w->n_matrices;
}

extern "C" int svt_quant_pack(const svt_quant_weights *w, const uint8_t *nibbles, const void *scales,
                              const uint8_t *zeros, void *hip_stream) {
  const char *who = "svt_quant_pack";
  (void)report(SVT_OK, "%s", "");
  const int rc = check_weights(who, w);
  if (rc != SVT_OK) return rc;
  if (!w->packed || !nibbles || !scales || (w->has_zeros && !zeros))
    return report(SVT_EINVAL, "%s: NULL packed, nibbles, scales or zeros", who);
  if (!w->has_zeros && zeros) return report(SVT_EINVAL, "%s: zeros given, but has_zeros is 0", who);
  const QuantShape s = quant_shape(*w);
  const size_t need = s.stride * w->n_matrices;
  if (w->packed_bytes < need)
    return report(SVT_EINVAL, "%s: packed buffer of %zu bytes, needs %zu", who, w->packed_bytes, need);
  const int b = elem_size(w->scale_type), src_groups = (w->n_in + w->group - 1) / w->group;
  if (misaligned(w->packed, 256) || misaligned(scales, b))
    return report(SVT_EINVAL, "%s: misaligned packed buffer (256 bytes) or scales", who);
  const size_t rows = (size_t)w->n_matrices * w->n_out;
  if (overlap(w->packed, need, nibbles, rows * ((w->n_in + 1) / 2)) ||
      overlap(w->packed, need, scales, rows * src_groups * b) || overlap(w->packed, need, zeros, rows * src_groups))
    return report(SVT_EINVAL, "%s: the packed buffer overlaps an input", who);
  hipStream_t st = (hipStream_t)hip_stream;
  auto grid = [](int64_t n) {
    const int64_t g = (n + kPackThreads - 1) / kPackThreads;
    return (unsigned)(g < 65536 ? g : 65536);
  };
  const int64_t pieces = (int64_t)w->n_matrices * s.tiles * s.blocks * 64;
  k_pack_q<<<grid(pieces), kPackThreads, 0, st>>>(s, pieces, nibbles, (uint8_t *)w->packed);
  const int64_t values = (int64_t)w->n_matrices * s.tiles * s.groups * kTileN;
  if (b == 4)
    k_pack_groups<uint32_t><<<grid(values), kPackThreads, 0, st>>>(s, values, src_groups, s.scale_at,
                                                                  (const uint32_t *)scales, (uint8_t *)w->packed);
  else
    k_pack_groups<uint16_t><<<grid(values), kPackThreads, 0, st>>>(s, values, src_groups, s.scale_at,
                                                                  (const uint16_t *)scales, (uint8_t *)w->packed);
  if (w->has_zeros)
    k_pack_groups<uint8_t><<<grid(values), kPackThreads, 0, st>>>(s, values, src_groups, s.zero_at, zeros,
                                                                 (uint8_t *)w->packed);
  return launched(who);
}

extern "C" int svt_quant_linear(int32_t n_rows, int32_t dtype, const void *x, const svt_quant_weights *w,
                                const int32_t *offsets, const float *bias, int32_t activation, int32_t out_dtype,
                                void *y, void *hip_stream) {
  const char *who = "svt_quant_linear";
  (void)report(SVT_OK, "%s", "");
  const int rc = check_weights(who, w);
  if (rc != SVT_OK) return rc;
  if (n_rows < 0) return report(SVT_EINVAL, "%s: n_rows %d < 0", who, n_rows);
  if (!elem_size(dtype)) return report(SVT_EINVAL, "%s: unknown element type %d", who, dtype);
  if (out_dtype != dtype && out_dtype != SVT_F32)
    return report(SVT_EINVAL, "%s: output type %d is neither the rows' nor float32", who, out_dtype);
  if (activation != SVT_ACT_NONE && activation != SVT_ACT_RELU)
    return report(SVT_EINVAL, "%s: unknown activation %d", who, activation);
  if (!offsets && w->n_matrices != 1)
    return report(SVT_EINVAL, "%s: %d matrices need offsets", who, w->n_matrices);
  if (n_rows == 0) return SVT_OK;
  if (!x || !y || !w->packed) return report(SVT_EINVAL, "%s: NULL rows, packed weights or output", who);
  const QuantShape s = quant_shape(*w);
  const size_t need = s.stride * w->n_matrices;
  if (w->packed_bytes < need)
    return report(SVT_EINVAL, "%s: packed buffer of %zu bytes, needs %zu", who, w->packed_bytes, need);
  const int bx = elem_size(dtype), by = elem_size(out_dtype);
  if (misaligned(x, bx) || misaligned(y, by) || misaligned(w->packed, 256) || misaligned(offsets, 4) || misaligned(bias, 4))
    return report(SVT_EINVAL, "%s: misaligned rows, packed weights (256 bytes), offsets, bias or output", who);
  const size_t ny = (size_t)n_rows * w->n_out * by;
  if (overlap(y, ny, x, (size_t)n_rows * w->n_in * bx) || overlap(y, ny, w->packed, need) ||
      overlap(y, ny, offsets, offsets ? ((size_t)w->n_matrices + 1) * 4 : 0) ||
      overlap(y, ny, bias, (size_t)w->n_matrices * w->n_out * 4))
    return report(SVT_EINVAL, "%s: the output overlaps an input", who);
  const LinearArgs a{s, n_rows, w->n_matrices, 1, 0, (const uint8_t *)w->packed, offsets, bias,
                     activation == SVT_ACT_RELU, out_dtype == SVT_F32, x, y};
  with_type(dtype, [&](auto tx) {
    with_type(w->scale_type, [&](auto ts) {
      with_group(w->group, [&](auto g) {
        using T = decltype(tx);
        using S = decltype(ts);
        constexpr int G = decltype(g)::value;
        launch_linear<T, S, G, 1, 1>(a, (hipStream_t)hip_stream);
      });
    });
  });
  return launched(who);
}

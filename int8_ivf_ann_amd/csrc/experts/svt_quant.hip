// svt_quant.hip - products with 4-bit weights and group scales: packing, argument checks and entry points (the
// kernel and the packed layout: svt_linear.h).

#include "svt_linear.h"

namespace svt {

extern template int linear_rows<float>(const char *, LinearArgs, int32_t, void *);
extern template int linear_rows<f16>(const char *, LinearArgs, int32_t, void *);
extern template int linear_rows<bf16>(const char *, LinearArgs, int32_t, void *);

namespace {

// ---- pack ----------------------------------------------------------------------------------------

constexpr int kPackThreads = 256;

__global__ __launch_bounds__(kPackThreads) void k_pack_q(QuantShape s, int64_t n_pieces, const uint8_t *nibbles,
                                                         uint8_t *packed) {
  const int64_t row_bytes = (s.n_in + 1) / 2;
  const int64_t per_matrix = (int64_t)s.tiles * s.blocks * 64;
  for (int64_t p = (int64_t)blockIdx.x * kPackThreads + threadIdx.x; p < n_pieces; p += (int64_t)gridDim.x * kPackThreads) {
    const int64_t m = p / per_matrix, r = p % per_matrix, bt = r / 64;
    const int lane = (int)(r % 64), block = (int)(bt / s.tiles);
    const int n = (int)(bt % s.tiles) * kTileN + lane % 16;
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
    *reinterpret_cast<uint4 *>(packed + m * s.stride + bt * s.record + lane * 16) = out;
  }
}

// scales (at kGroupsAt) or, ZEROS, zero points (at zeros_at)
template <class T, bool ZEROS>
__global__ __launch_bounds__(kPackThreads) void k_pack_groups(QuantShape s, int64_t n_values, int src_groups,
                                                              const T *src, uint8_t *packed) {
  const int ng = kBlockK / s.group;
  const int64_t per_matrix = (int64_t)s.tiles * s.blocks * kTileN * ng;
  for (int64_t p = (int64_t)blockIdx.x * kPackThreads + threadIdx.x; p < n_values; p += (int64_t)gridDim.x * kPackThreads) {
    const int64_t m = p / per_matrix, r = p % per_matrix, bt = r / (kTileN * ng);
    const int in = (int)(r % (kTileN * ng));   // zero points: output * ng + g; scales: (h * ng + g) * 4 + i
    const int gi = ZEROS ? in % ng : in / 4 % ng, o = ZEROS ? in / ng : in / (4 * ng) * 4 + in % 4;
    const int g = (int)(bt / s.tiles) * ng + gi, n = (int)(bt % s.tiles) * kTileN + o;
    const T v = (n < s.n_out && g < src_groups) ? src[(m * s.n_out + n) * src_groups + g] : T(0);
    reinterpret_cast<T *>(packed + m * s.stride + bt * s.record + (ZEROS ? s.zeros_at : kGroupsAt))[in] = v;
  }
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
  auto grid = [](int64_t n) {
    const int64_t g = (n + kPackThreads - 1) / kPackThreads;
    return (unsigned)(g < 65536 ? g : 65536);
  };
  const int64_t pieces = (int64_t)w->n_matrices * s.tiles * s.blocks * 64;
  int done = launch(who, k_pack_q, grid(pieces), kPackThreads, 0, hip_stream, s, pieces, nibbles, (uint8_t *)w->packed);
  const int64_t values = (int64_t)w->n_matrices * s.tiles * s.blocks * kTileN * (kBlockK / s.group);
  auto groups = [&](auto *src, auto zero_points) {
    using S = std::remove_const_t<std::remove_pointer_t<decltype(src)>>;
    return launch(who, k_pack_groups<S, decltype(zero_points)::value>, grid(values), kPackThreads, 0, hip_stream, s,
                  values, src_groups, src, (uint8_t *)w->packed);
  };
  if (done == SVT_OK)
    done = b == 4 ? groups((const uint32_t *)scales, std::false_type{}) : groups((const uint16_t *)scales, std::false_type{});
  if (done == SVT_OK && w->has_zeros) done = groups(zeros, std::true_type{});
  return done;
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
  LinearArgs a{};
  a.s = s;
  a.n_rows = n_rows;
  a.n_matrices = w->n_matrices;
  a.packed = (const uint8_t *)w->packed;
  a.offsets = offsets;
  a.bias = bias;
  a.relu = activation == SVT_ACT_RELU;
  a.out_f32 = out_dtype == SVT_F32;
  a.wide_store = w->n_out % 4 == 0 && !misaligned(y, 4 * by);
  a.x = x;
  a.y = y;
  return with_type(dtype, [&](auto tx) { return linear_rows<decltype(tx)>(who, a, w->scale_type, hip_stream); });
}

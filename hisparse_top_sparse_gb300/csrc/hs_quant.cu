// Latent rows into the q8 row format as they are written, and q8 rows back
// (the format: hs_q8.cuh). "vllm 分析(十二) HiSparse 下篇", section c4a kv cache
// 写入, quantises a cache's entries where they are stored; hs_backup_rows and
// hs_swap_apply_plan move such rows as bytes.
//
// Both kernels move each byte once and do a few operations per value, so HBM
// bounds them (the host link, when one side is host memory). A warp takes a
// row: lane l holds VEC = 16 / sizeof(T) consecutive dims of every pass, so
// that each 16-byte access of the wide side and each VEC-byte access of the
// codes is contiguous over the warp; a group of 32 dims is 32 / VEC
// neighbouring lanes, whose largest magnitude and scale byte take shuffles
// only. A warp has two rows in flight in bf16, one in f32 (its registers hold
// no more), 32 warps on an SM, and loads its next slots meanwhile. Measured,
// scattered slots: 262144 bf16 rows quantised and read back 165 us, 86 % of the
// measured copy rate for the bytes both move (slots not loaded ahead 178, one
// row in flight 180, 40 warps 193); 131072 rows read back to bf16 40 us (89 %),
// 131072 f32 rows there and back 128 us.

#include "hs_q8.cuh"
#include "hs_rows.cuh"

namespace {

template <typename T>
struct Lay {
  static constexpr int VEC = 16 / (int)sizeof(T);         // dims per lane and pass
  static constexpr int GL = Q8_GROUP / VEC;                // lanes per scale group
  static constexpr int PASSES = HS_VALUE_DIM / (32 * VEC);
  static constexpr int ROPE_LANES = (HS_LATENT_DIM - HS_VALUE_DIM) / VEC;
  static constexpr int ROWS = sizeof(T) == 2 ? 2 : 1;      // rows of one warp in flight
};

template <typename T>
__global__ void __launch_bounds__(QT_THREADS, QT_BLOCKS) k_quant_rows(
    const char *__restrict__ src, int64_t src_stride, int64_t src_rows, char *__restrict__ dst,
    int64_t dst_rows, const int32_t *__restrict__ src_slots, const int32_t *__restrict__ dst_slots,
    int32_t n, uint32_t *status) {
  using L = Lay<T>;
  const int lane = threadIdx.x & 31;
  const int64_t warp = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const int64_t n_warps = ((int64_t)gridDim.x * blockDim.x) >> 5;
  bool bad = false;
  Slots<L::ROWS> next(src_slots, dst_slots, warp, n_warps, n);
  for (int64_t base = warp; base < n; base += n_warps * L::ROWS) {
    char *d[L::ROWS];
    uint4 w[L::ROWS][L::PASSES], rope[L::ROWS];
    const Slots<L::ROWS> here = next;
    next = Slots<L::ROWS>(src_slots, dst_slots, base + n_warps * L::ROWS, n_warps, n);
#pragma unroll
    for (int u = 0; u < L::ROWS; ++u) {
      d[u] = nullptr;
      const int64_t s = row_of(here.s[u], src_rows, bad), t = row_of(here.d[u], dst_rows, bad);
      if (s >= 0 && t >= 0) {
        d[u] = dst + t * HS_Q8_ROW_BYTES;
        const uint4 *p = reinterpret_cast<const uint4 *>(src + s * src_stride) + lane;
#pragma unroll
        for (int k = 0; k < L::PASSES; ++k) w[u][k] = __ldcs(p + 32 * k);
        if (lane < L::ROPE_LANES) rope[u] = __ldcs(p + 32 * L::PASSES);
      }
    }
#pragma unroll
    for (int u = 0; u < L::ROWS; ++u) {
      if (!d[u]) continue;                        // the same for the whole warp
      uint32_t sc[4] = {0, 0, 0, 0};
#pragma unroll
      for (int k = 0; k < L::PASSES; ++k) {
        float f[L::VEC];
        unpack<T>(w[u][k], f);
        float amax = 0.f;
#pragma unroll
        for (int j = 0; j < L::VEC; ++j) amax = fmaxf(amax, fabsf(f[j]));   // a NaN is passed over
#pragma unroll
        for (int o = 1; o < L::GL; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        const uint32_t e = q8_exponent(amax);
        const float inv = q8_inv_scale(e);
        uint32_t c[L::VEC / 4];
#pragma unroll
        for (int j = 0; j < L::VEC / 4; ++j)
          c[j] = q8_encode2(f[4 * j] * inv, f[4 * j + 1] * inv) |
                 (q8_encode2(f[4 * j + 2] * inv, f[4 * j + 3] * inv) << 16);
        char *at = d[u] + (32 * k + lane) * L::VEC;
        if constexpr (L::VEC == 8)
          *reinterpret_cast<uint2 *>(at) = make_uint2(c[0], c[1]);
        else
          *reinterpret_cast<uint32_t *>(at) = c[0];
        // the bytes of four neighbouring groups into one word
        uint32_t b = e << (8 * ((lane / L::GL) & 3));
        b |= __shfl_xor_sync(0xffffffffu, b, L::GL);
        b |= __shfl_xor_sync(0xffffffffu, b, 2 * L::GL);
        if constexpr (L::VEC == 8) {
          sc[2 * k] = b;
          sc[2 * k + 1] = __shfl_sync(0xffffffffu, b, 16);
        } else {
          sc[k] = b;
        }
      }
      if (lane < L::ROPE_LANES) {
        char *at = d[u] + Q8_ROPE_OFF + lane * (2 * L::VEC);
        if constexpr (L::VEC == 8) {
          *reinterpret_cast<uint4 *>(at) = rope[u];
        } else {
          float f[L::VEC];
          unpack<T>(rope[u], f);
          const __nv_bfloat162 a = __floats2bfloat162_rn(f[0], f[1]), b = __floats2bfloat162_rn(f[2], f[3]);
          *reinterpret_cast<uint2 *>(at) = make_uint2(*reinterpret_cast<const uint32_t *>(&a),
                                                      *reinterpret_cast<const uint32_t *>(&b));
        }
      }
      if (lane == 0) *reinterpret_cast<uint4 *>(d[u] + Q8_SCALE_OFF) = make_uint4(sc[0], sc[1], sc[2], sc[3]);
    }
  }
  if (bad && status) atomicOr(status, HS_STATUS_INDEX);
}

template <typename T>
__global__ void __launch_bounds__(QT_THREADS, QT_BLOCKS) k_dequant_rows(
    const char *__restrict__ src, int64_t src_rows, char *__restrict__ dst, int64_t dst_stride,
    int64_t dst_rows, const int32_t *__restrict__ src_slots, const int32_t *__restrict__ dst_slots,
    int32_t n, uint32_t *status) {
  using L = Lay<T>;
  using Code = typename std::conditional<L::VEC == 8, uint2, uint32_t>::type;
  const int lane = threadIdx.x & 31;
  const int64_t warp = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const int64_t n_warps = ((int64_t)gridDim.x * blockDim.x) >> 5;
  bool bad = false;
  Slots<L::ROWS> next(src_slots, dst_slots, warp, n_warps, n);
  for (int64_t base = warp; base < n; base += n_warps * L::ROWS) {
    char *d[L::ROWS];
    Code c[L::ROWS][L::PASSES], rope_lo[L::ROWS], rope_hi[L::ROWS];
    uint32_t e[L::ROWS][L::PASSES];
    const Slots<L::ROWS> here = next;
    next = Slots<L::ROWS>(src_slots, dst_slots, base + n_warps * L::ROWS, n_warps, n);
#pragma unroll
    for (int u = 0; u < L::ROWS; ++u) {
      d[u] = nullptr;
      const int64_t s = row_of(here.s[u], src_rows, bad), t = row_of(here.d[u], dst_rows, bad);
      if (s >= 0 && t >= 0) {
        d[u] = dst + t * dst_stride;
        const char *row = src + s * HS_Q8_ROW_BYTES;
        const Code *p = reinterpret_cast<const Code *>(row) + lane;
#pragma unroll
        for (int k = 0; k < L::PASSES; ++k) {
          c[u][k] = __ldg(p + 32 * k);
          e[u][k] = __ldg(reinterpret_cast<const unsigned char *>(row) + Q8_SCALE_OFF +
                          (32 * k + lane) / L::GL);
        }
        if (lane < L::ROPE_LANES) {             // VEC bf16 dims per lane: two Code words
          const Code *rp = reinterpret_cast<const Code *>(row + Q8_ROPE_OFF) + 2 * lane;
          rope_lo[u] = __ldg(rp);
          rope_hi[u] = __ldg(rp + 1);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < L::ROWS; ++u) {
      if (!d[u]) continue;
      uint4 *out = reinterpret_cast<uint4 *>(d[u]) + lane;
#pragma unroll
      for (int k = 0; k < L::PASSES; ++k) {
        if constexpr (L::VEC == 8) {
          const uint64_t s = q8_scale2(e[u][k]);
          const uint2 a = q8_decode4_bf16(c[u][k].x, s), b = q8_decode4_bf16(c[u][k].y, s);
          __stcs(out + 32 * k, make_uint4(a.x, a.y, b.x, b.y));
        } else {
          const float s = q8_scale(e[u][k]);
          const float2 a = q8_decode2(c[u][k], 0, s), b = q8_decode2(c[u][k], 2, s);
          __stcs(out + 32 * k, make_uint4(__float_as_uint(a.x), __float_as_uint(a.y),
                                          __float_as_uint(b.x), __float_as_uint(b.y)));
        }
      }
      if (lane < L::ROPE_LANES) {
        if constexpr (L::VEC == 8)
          __stcs(out + 32 * L::PASSES, make_uint4(rope_lo[u].x, rope_lo[u].y, rope_hi[u].x, rope_hi[u].y));
        else
          __stcs(out + 32 * L::PASSES,
                 make_uint4(rope_lo[u] << 16, rope_lo[u] & 0xFFFF0000u, rope_hi[u] << 16,
                            rope_hi[u] & 0xFFFF0000u));
      }
    }
  }
  if (bad && status) atomicOr(status, HS_STATUS_INDEX);
}

}  // namespace

extern "C" int hs_quant_rows(const void *src, int32_t src_dtype, int64_t src_stride, int64_t src_rows,
                             void *dst, int64_t dst_rows, const int32_t *src_slots,
                             const int32_t *dst_slots, int32_t n, uint32_t *status,
                             hs_stream_t stream) {
  const void *s = nullptr, *d = nullptr;
  int rc = hs_check_rows(src, src_dtype, src_stride, src_rows, dst, dst_rows, src_slots, dst_slots,
                      status, n, &s, &d);
  if (rc || n == 0) return rc;
  int blocks = 0;
  if ((rc = hs_row_blocks(n, &blocks))) return rc;
  const char *sp = reinterpret_cast<const char *>(s);
  char *dp = reinterpret_cast<char *>(const_cast<void *>(d));
  if (src_dtype == HS_LOGITS_F32)
    k_quant_rows<float><<<blocks, QT_THREADS, 0, stream>>>(sp, src_stride * 4, src_rows, dp, dst_rows,
                                                           src_slots, dst_slots, n, status);
  else
    k_quant_rows<__nv_bfloat16><<<blocks, QT_THREADS, 0, stream>>>(
        sp, src_stride * 2, src_rows, dp, dst_rows, src_slots, dst_slots, n, status);
  HS_LAUNCH_CHECK("k_quant_rows");
  return HS_OK;
}

extern "C" int hs_dequant_rows(const void *src, int64_t src_rows, void *dst, int32_t dst_dtype,
                               int64_t dst_stride, int64_t dst_rows, const int32_t *src_slots,
                               const int32_t *dst_slots, int32_t n, uint32_t *status,
                               hs_stream_t stream) {
  const void *s = nullptr, *d = nullptr;
  int rc = hs_check_rows(dst, dst_dtype, dst_stride, dst_rows, src, src_rows, src_slots, dst_slots,
                      status, n, &d, &s);
  if (rc || n == 0) return rc;
  int blocks = 0;
  if ((rc = hs_row_blocks(n, &blocks))) return rc;
  const char *sp = reinterpret_cast<const char *>(s);
  char *dp = reinterpret_cast<char *>(const_cast<void *>(d));
  if (dst_dtype == HS_LOGITS_F32)
    k_dequant_rows<float><<<blocks, QT_THREADS, 0, stream>>>(sp, src_rows, dp, dst_stride * 4, dst_rows,
                                                             src_slots, dst_slots, n, status);
  else
    k_dequant_rows<__nv_bfloat16><<<blocks, QT_THREADS, 0, stream>>>(
        sp, src_rows, dp, dst_stride * 2, dst_rows, src_slots, dst_slots, n, status);
  HS_LAUNCH_CHECK("k_dequant_rows");
  return HS_OK;
}

// Latent rows into the q4 row format as they are written, and q4 rows back (the
// format: hs_q4.cuh; q8 rows: hs_quant.cu, whose plan this is). The pages name an
// FP4 cache ("vllm 分析(十二) HiSparse 下篇", section c4a kv cache 写入: use_fp4_cache,
// quant_block, scale_dim, token_stride) without its layout.
//
// A warp takes a row: lane l holds VEC = 16 / sizeof(T) consecutive dims of every
// pass, so the wide side moves in contiguous 16-byte accesses and the codes in
// contiguous words; a group of 16 dims is 16 / VEC neighbouring lanes, whose
// largest magnitude takes shuffles only. Measured: 262144 bf16 rows quantised into
// scattered slots 76 us, 79 % of the measured copy rate for the bytes moved, read back
// 69.5, 87 %; 131072 f32 rows 62 and 62; 4 rows 1.9 and 1.6. Reading back is bound by
// HBM; quantising by it and by the ALU pipe, busy for 59 % of the cycles (93 us with
// maxima value by value, a rounded reciprocal a group and codes put together by
// shifts). Two bf16 rows of a warp in flight and four blocks an SM (64 registers, one
// word of the bf16 kernel spilled): three blocks 81 us, three rows 81, five blocks spill
// more.

#include "hs_q4.cuh"
#include "hs_rows.cuh"

namespace {

template <typename T>
struct Lay {
  static constexpr int VEC = 16 / (int)sizeof(T);         // dims per lane and pass
  static constexpr int GL = Q4_GROUP / VEC;                // lanes per scale group
  static constexpr int PASSES = HS_VALUE_DIM / (32 * VEC);
  static constexpr int ROPE_LANES = (HS_LATENT_DIM - HS_VALUE_DIM) / VEC;
  static constexpr int ROWS = sizeof(T) == 2 ? 2 : 1;      // rows of one warp in flight
};

__device__ __forceinline__ uint32_t pair_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&v);
}

// The bits of the largest magnitude of a scale group, this lane's 16 bytes and its
// neighbours' (as whole numbers: infinities and NaNs come out on top).
template <typename T>
__device__ __forceinline__ uint32_t group_amax(const uint4 w) {
  if constexpr (sizeof(T) == 2) {
    constexpr uint32_t M = 0x7fff7fffu;           // both halves at once
    uint32_t a = __vmaxs2(__vimax3_s16x2(w.x & M, w.y & M, w.z & M), w.w & M);
#pragma unroll
    for (int o = 1; o < Lay<T>::GL; o <<= 1) a = __vmaxs2(a, __shfl_xor_sync(0xffffffffu, a, o));
    return max(a << 16, a & 0xffff0000u);
  } else {
    constexpr uint32_t M = 0x7fffffffu;
    uint32_t a = max(max(w.x & M, w.y & M), max(w.z & M, w.w & M));
#pragma unroll
    for (int o = 1; o < Lay<T>::GL; o <<= 1) a = max(a, __shfl_xor_sync(0xffffffffu, a, o));
    return a;
  }
}

template <typename T>
__global__ void __launch_bounds__(QT_THREADS, QT_BLOCKS) k_quant_rows_q4(
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
        d[u] = dst + t * HS_Q4_ROW_BYTES;
        const uint4 *p = reinterpret_cast<const uint4 *>(src + s * src_stride) + lane;
#pragma unroll
        for (int k = 0; k < L::PASSES; ++k) w[u][k] = __ldcs(p + 32 * k);
        if (lane < L::ROPE_LANES) rope[u] = __ldcs(p + 32 * L::PASSES);
      }
    }
#pragma unroll
    for (int u = 0; u < L::ROWS; ++u) {
      if (!d[u]) continue;                        // the same for the whole warp
#pragma unroll
      for (int k = 0; k < L::PASSES; ++k) {
        float f[L::VEC];
        unpack<T>(w[u][k], f);
        const uint32_t byte = q4_scale_byte(group_amax<T>(w[u][k]));
        const float scale = q4_scale(byte), minus_inv = -q4_reciprocal(scale);
        const uint64_t s = q4_pair(scale, scale), inv = q4_pair(minus_inv, minus_inv);
        // the word of eight dims: bytes (0, 2), (4, 6), (1, 3), (5, 7)
        if constexpr (L::VEC == 8) {
          const uint32_t c = q4_codes(q4_minus_over(f[0], f[2], s, inv), q4_minus_over(f[4], f[6], s, inv),
                                      q4_minus_over(f[1], f[3], s, inv), q4_minus_over(f[5], f[7], s, inv));
          *reinterpret_cast<uint32_t *>(d[u] + (32 * k + lane) * 4) = c ^ Q4_SIGNS;
        } else {
          // half of it each in two neighbouring lanes
          const float2 zero = make_float2(0.f, 0.f);
          uint32_t c = q4_codes(q4_minus_over(f[0], f[2], s, inv), zero, q4_minus_over(f[1], f[3], s, inv), zero)
                       << (8 * (lane & 1));
          c |= __shfl_xor_sync(0xffffffffu, c, 1);
          if (!(lane & 1)) *reinterpret_cast<uint32_t *>(d[u] + (32 * k + lane) * 2) = c ^ Q4_SIGNS;
        }
        if (lane % L::GL == 0) d[u][Q4_SCALE_OFF + (32 * k + lane) / L::GL] = (char)byte;
      }
      if (lane < L::ROPE_LANES) {
        char *at = d[u] + Q4_ROPE_OFF + lane * (2 * L::VEC);
        if constexpr (L::VEC == 8) {
          *reinterpret_cast<uint4 *>(at) = rope[u];
        } else {
          float f[L::VEC];
          unpack<T>(rope[u], f);
          *reinterpret_cast<uint2 *>(at) = make_uint2(pair_bf16(f[0], f[1]), pair_bf16(f[2], f[3]));
        }
      }
    }
  }
  if (bad && status) atomicOr(status, HS_STATUS_INDEX);
}

template <typename T>
__global__ void __launch_bounds__(QT_THREADS, QT_BLOCKS) k_dequant_rows_q4(
    const char *__restrict__ src, int64_t src_rows, char *__restrict__ dst, int64_t dst_stride,
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
    uint32_t c[L::ROWS][L::PASSES], e[L::ROWS][L::PASSES];
    uint4 rope[L::ROWS];
    const Slots<L::ROWS> here = next;
    next = Slots<L::ROWS>(src_slots, dst_slots, base + n_warps * L::ROWS, n_warps, n);
#pragma unroll
    for (int u = 0; u < L::ROWS; ++u) {
      d[u] = nullptr;
      const int64_t s = row_of(here.s[u], src_rows, bad), t = row_of(here.d[u], dst_rows, bad);
      if (s >= 0 && t >= 0) {
        d[u] = dst + t * dst_stride;
        const char *row = src + s * HS_Q4_ROW_BYTES;
#pragma unroll
        for (int k = 0; k < L::PASSES; ++k) {
          // the word that holds this lane's dims (in f32 half of it, shared by two lanes)
          c[u][k] = __ldg(reinterpret_cast<const uint32_t *>(row) + (32 * k + lane) * L::VEC / 8);
          e[u][k] = __ldg(reinterpret_cast<const unsigned char *>(row) + Q4_SCALE_OFF + (32 * k + lane) / L::GL);
        }
        if (lane < L::ROPE_LANES) {
          if constexpr (L::VEC == 8) {
            rope[u] = __ldg(reinterpret_cast<const uint4 *>(row + Q4_ROPE_OFF) + lane);
          } else {
            const uint2 r = __ldg(reinterpret_cast<const uint2 *>(row + Q4_ROPE_OFF) + lane);
            rope[u] = make_uint4(r.x << 16, r.x & 0xFFFF0000u, r.y << 16, r.y & 0xFFFF0000u);
          }
        }
      }
    }
#pragma unroll
    for (int u = 0; u < L::ROWS; ++u) {
      if (!d[u]) continue;
      uint4 *out = reinterpret_cast<uint4 *>(d[u]) + lane;
#pragma unroll
      for (int k = 0; k < L::PASSES; ++k) {
        const uint32_t s = q4_scale2(e[u][k]);
        if constexpr (L::VEC == 8) {
          const uint32_t w = c[u][k];
          __stcs(out + 32 * k, make_uint4(q4_mul(q4_decode2<0>(w, s), Q4_UP2), q4_mul(q4_decode2<1>(w, s), Q4_UP2),
                                          q4_mul(q4_decode2<2>(w, s), Q4_UP2), q4_mul(q4_decode2<3>(w, s), Q4_UP2)));
        } else {
          const uint32_t w = c[u][k] >> (8 * (lane & 1));
          const uint32_t a = q4_mul(q4_decode2<0>(w, s), Q4_UP2), b = q4_mul(q4_decode2<1>(w, s), Q4_UP2);
          __stcs(out + 32 * k, make_uint4(a << 16, a & 0xFFFF0000u, b << 16, b & 0xFFFF0000u));
        }
      }
      if (lane < L::ROPE_LANES) __stcs(out + 32 * L::PASSES, rope[u]);
    }
  }
  if (bad && status) atomicOr(status, HS_STATUS_INDEX);
}

}  // namespace

extern "C" int hs_quant_rows_q4(const void *src, int32_t src_dtype, int64_t src_stride, int64_t src_rows,
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
    k_quant_rows_q4<float><<<blocks, QT_THREADS, 0, stream>>>(sp, src_stride * 4, src_rows, dp, dst_rows,
                                                              src_slots, dst_slots, n, status);
  else
    k_quant_rows_q4<__nv_bfloat16><<<blocks, QT_THREADS, 0, stream>>>(
        sp, src_stride * 2, src_rows, dp, dst_rows, src_slots, dst_slots, n, status);
  HS_LAUNCH_CHECK("k_quant_rows_q4");
  return HS_OK;
}

extern "C" int hs_dequant_rows_q4(const void *src, int64_t src_rows, void *dst, int32_t dst_dtype,
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
    k_dequant_rows_q4<float><<<blocks, QT_THREADS, 0, stream>>>(sp, src_rows, dp, dst_stride * 4, dst_rows,
                                                                src_slots, dst_slots, n, status);
  else
    k_dequant_rows_q4<__nv_bfloat16><<<blocks, QT_THREADS, 0, stream>>>(
        sp, src_rows, dp, dst_stride * 2, dst_rows, src_slots, dst_slots, n, status);
  HS_LAUNCH_CHECK("k_dequant_rows_q4");
  return HS_OK;
}

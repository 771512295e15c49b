// What the calls that move latent rows between row formats share (hs_quant.cu:
// q8 rows, hs_quant4.cu: q4 rows): the lists of slots, the checks, the launch.
#pragma once

#include <type_traits>

#include "hs_internal.cuh"

constexpr int QT_THREADS = 256;
constexpr int QT_BLOCKS = 4;    // blocks per SM, at most and at least

// The values of 16 bytes, in f32.
template <typename T>
__device__ __forceinline__ void unpack(const uint4 w, float (&f)[16 / sizeof(T)]) {
  const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
  if constexpr (std::is_same<T, float>::value) {
#pragma unroll
    for (int k = 0; k < 4; ++k) f[k] = __uint_as_float(ws[k]);
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      f[2 * k] = __uint_as_float(ws[k] << 16);
      f[2 * k + 1] = __uint_as_float(ws[k] & 0xFFFF0000u);
    }
  }
}

// The slots of a warp's next rows, loaded while the rows before them are on
// their way: entries base, base + step, ...; without a list entry i is row i;
// -1 past the last.
template <int ROWS>
struct Slots {
  int32_t s[ROWS], d[ROWS];
  __device__ __forceinline__ Slots(const int32_t *src_slots, const int32_t *dst_slots, int64_t base,
                                   int64_t step, int32_t n) {
#pragma unroll
    for (int u = 0; u < ROWS; ++u) {
      const int64_t i = base + u * step;
      s[u] = i >= n ? -1 : src_slots ? __ldg(src_slots + i) : (int32_t)i;
      d[u] = i >= n ? -1 : dst_slots ? __ldg(dst_slots + i) : (int32_t)i;
    }
  }
};

// -1: no entry; a slot at or past `rows` gives -1 and sets bad.
__device__ __forceinline__ int64_t row_of(int32_t s, int64_t rows, bool &bad) {
  if (s >= rows) {
    bad = true;
    return -1;
  }
  return s;
}

// Checks shared by both directions; wide: the bf16 / f32 side, cache: the other.
static inline int hs_check_rows(const void *wide, int32_t dtype, int64_t wide_stride, int64_t wide_rows, const void *cache,
               int64_t cache_rows, const int32_t *src_slots, const int32_t *dst_slots,
               const uint32_t *status, int32_t n, const void **wide_dev, const void **cache_dev) {
  if (dtype != HS_LOGITS_F32 && dtype != HS_LOGITS_BF16)
    return hs_set_error(HS_ERR_INVALID_ARG, "row dtype %d", dtype);
  const int64_t elem = dtype == HS_LOGITS_F32 ? 4 : 2;
  if (n < 0 || wide_rows < 0 || cache_rows < 0 || wide_stride < HS_LATENT_DIM ||
      wide_stride > (int64_t)1 << 30 || (wide_stride * elem) % 16)
    return hs_set_error(HS_ERR_INVALID_ARG,
                        "bad sizes n=%d rows=%lld/%lld stride=%lld (elements: at least 576, a "
                        "multiple of 16 bytes)",
                        n, (long long)wide_rows, (long long)cache_rows, (long long)wide_stride);
  if (n == 0) return HS_OK;
  if (!wide || !cache || (((uintptr_t)wide | (uintptr_t)cache) & 15))
    return hs_set_error(HS_ERR_INVALID_ARG, "src and dst must be 16-byte aligned and not NULL");
  if (((uintptr_t)src_slots | (uintptr_t)dst_slots | (uintptr_t)status) & 3)
    return hs_set_error(HS_ERR_INVALID_ARG, "slot lists and status must be 4-byte aligned");
  int rc = hs_device_alias(wide, wide_dev, "the bf16 / f32 rows");
  if (rc) return rc;
  return hs_device_alias(cache, cache_dev, "the quantised rows");
}

// Blocks for n rows: a warp per row, up to QT_BLOCKS on every SM.
static inline int hs_row_blocks(int32_t n, int *blocks) {
  int sms = 0;
  int rc = hs_sm_count(&sms);
  if (rc) return rc;
  const int64_t want = ((int64_t)n + QT_THREADS / 32 - 1) / (QT_THREADS / 32);
  *blocks = (int)(want < (int64_t)sms * QT_BLOCKS ? want : (int64_t)sms * QT_BLOCKS);
  return HS_OK;
}

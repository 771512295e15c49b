// Rotary positions: rows (queries, keys, latent rows) rotated pair by pair by
// angles proportional to their positions, on the way from a projection into q or
// a cache, or in place. The pages' caches hold 64 rotated dims in each latent row
// (HS_LATENT_DIM = 512 + 64) and the attention rotates nothing.
//
// The angle of a pair at position p is p * w. In f32 an angle of 10^5 radians is
// off by up to 0.004; in 64-bit whole fractions of a turn (w / 2 pi * 2^64, kept in
// `freqs`) the product wraps as the angle does and is exact modulo a turn at any
// position, for one integer multiplication a pair; its top 32 bits go to
// sincospif.
//
// A thread takes one unit of a head: as many pairs as 16-byte accesses hold
// (interleaved: 16 bytes; half: 16 bytes of each half), or 16 bytes of the dims
// beside the rotated part, which it copies. It computes the unit's cosines and
// sines once and applies them to every STEP-th head of its row.

#include "hs_internal.cuh"

namespace {

constexpr int RT = 256;               // threads of a block, at most

struct RopeArgs {
  const char *src;
  char *dst;
  int64_t src_row, src_head, dst_row, dst_head;       // bytes
  int64_t src_rows, dst_rows;
  const int32_t *src_slots, *dst_slots, *positions;
  const int64_t *freqs;
  uint32_t *status;
  int32_t n, heads, step;             // a thread's heads are h, h + step, ...
  int32_t half;                       // pairs of a head
  int32_t off;                        // bytes before the rotated part
  int32_t rot_units, units;           // units of a head: rotated, and all
  int32_t chunks, per_block;          // blocks of an entry, or (chunks 1) entries of a block
  float factor, sign;
};

// the elements of one access and their values
template <typename T, bool VECTOR>
struct Access {
  static constexpr int N = VECTOR ? 16 / (int)sizeof(T) : 1;
  static __device__ __forceinline__ void load(const char *p, float (&f)[N]) {
    if constexpr (!VECTOR) {
      f[0] = (float)*reinterpret_cast<const T *>(p);
    } else {
      const uint4 w = __ldcs(reinterpret_cast<const uint4 *>(p));
      const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if constexpr (sizeof(T) == 4) {
          f[k] = __uint_as_float(ws[k]);
        } else {
          f[2 * k] = __uint_as_float(ws[k] << 16);
          f[2 * k + 1] = __uint_as_float(ws[k] & 0xFFFF0000u);
        }
      }
    }
  }
  static __device__ __forceinline__ void store(char *p, const float (&f)[N]) {
    if constexpr (!VECTOR) {
      *reinterpret_cast<T *>(p) = (T)f[0];
    } else {
      uint32_t ws[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if constexpr (sizeof(T) == 4) {
          ws[k] = __float_as_uint(f[k]);
        } else {
          const __nv_bfloat162 v = __floats2bfloat162_rn(f[2 * k], f[2 * k + 1]);
          ws[k] = *reinterpret_cast<const uint32_t *>(&v);
        }
      }
      *reinterpret_cast<uint4 *>(p) = make_uint4(ws[0], ws[1], ws[2], ws[3]);
    }
  }
};

template <typename T, bool HALF, bool VECTOR>
__global__ void __launch_bounds__(RT) k_rope_rows(const __grid_constant__ RopeArgs a) {
  using A = Access<T, VECTOR>;
  constexpr int N = A::N;
  constexpr bool TWO = HALF || !VECTOR;           // a unit's pairs lie in two accesses
  constexpr int PAIRS = TWO ? N : N / 2;
  int64_t i;                                      // the entry
  int w;                                          // this thread's place in it
  const int width = a.units * a.step;
  if (a.chunks > 1) {
    i = blockIdx.x / (unsigned)a.chunks;
    w = (int)(blockIdx.x % (unsigned)a.chunks) * RT + (int)threadIdx.x;
    if (w >= width) return;
  } else {
    const int e = (int)threadIdx.x / width;
    i = (int64_t)blockIdx.x * a.per_block + e;
    w = (int)threadIdx.x - e * width;
    if (e >= a.per_block || i >= a.n) return;
  }
  const int64_t s = a.src_slots ? a.src_slots[i] : i, d = a.dst_slots ? a.dst_slots[i] : i;
  if (s >= a.src_rows || d >= a.dst_rows) {
    if (a.status && w == 0) atomicOr(a.status, HS_STATUS_INDEX);
    return;
  }
  if (s < 0 || d < 0) return;
  const int unit = w % a.units;
  int h = w / a.units;
  const char *src = a.src + s * a.src_row + (int64_t)h * a.src_head;
  char *dst = a.dst + d * a.dst_row + (int64_t)h * a.dst_head;
  const int64_t src_step = a.step * a.src_head, dst_step = a.step * a.dst_head;
  if (unit < a.rot_units) {
    const uint64_t p = (uint64_t)(int64_t)a.positions[i];
    float c[PAIRS], sn[PAIRS];
#pragma unroll
    for (int k = 0; k < PAIRS; ++k) {
      // the angle in half turns, within [-1, 1)
      const uint64_t turn = p * (uint64_t)a.freqs[unit * PAIRS + k];
      sincospif((float)(int32_t)(turn >> 32) * 0x1p-31f, &sn[k], &c[k]);
      c[k] *= a.factor;
      sn[k] *= a.sign;
    }
    // the unit's first access, and its second
    const int at = a.off + unit * (HALF ? N : 2 * PAIRS) * (int)sizeof(T);
    const int second = HALF ? a.half * (int)sizeof(T) : (int)sizeof(T);
#pragma unroll 4
    for (; h < a.heads; h += a.step, src += src_step, dst += dst_step) {
      float f[N];
      A::load(src + at, f);
      if constexpr (TWO) {
        float g[N];
        A::load(src + at + second, g);
#pragma unroll
        for (int k = 0; k < PAIRS; ++k) {
          const float x = f[k], y = g[k];
          f[k] = x * c[k] - y * sn[k];
          g[k] = y * c[k] + x * sn[k];
        }
        A::store(dst + at, f);
        A::store(dst + at + second, g);
      } else {
#pragma unroll
        for (int k = 0; k < PAIRS; ++k) {
          const float x = f[2 * k], y = f[2 * k + 1];
          f[2 * k] = x * c[k] - y * sn[k];
          f[2 * k + 1] = y * c[k] + x * sn[k];
        }
        A::store(dst + at, f);
      }
    }
  } else {
    // a unit beside the rotated part, moved as it is
    const int bytes = VECTOR ? 16 : (int)sizeof(T);
    int at = (unit - a.rot_units) * bytes;
    if (at >= a.off) at += 2 * a.half * (int)sizeof(T);
#pragma unroll 4
    for (; h < a.heads; h += a.step, src += src_step, dst += dst_step) {
      if constexpr (VECTOR)
        *reinterpret_cast<uint4 *>(dst + at) = __ldcs(reinterpret_cast<const uint4 *>(src + at));
      else
        *reinterpret_cast<T *>(dst + at) = *reinterpret_cast<const T *>(src + at);
    }
  }
}

template <typename T>
int launch(const RopeArgs &a, bool half, bool vector, unsigned blocks, int threads, cudaStream_t stream) {
  if (half) {
    if (vector)
      k_rope_rows<T, true, true><<<blocks, threads, 0, stream>>>(a);
    else
      k_rope_rows<T, true, false><<<blocks, threads, 0, stream>>>(a);
  } else {
    if (vector)
      k_rope_rows<T, false, true><<<blocks, threads, 0, stream>>>(a);
    else
      k_rope_rows<T, false, false><<<blocks, threads, 0, stream>>>(a);
  }
  HS_LAUNCH_CHECK("k_rope_rows");
  return HS_OK;
}

}  // namespace

extern "C" int hs_rope_rows(const void *src, int64_t src_row_stride, int64_t src_head_stride, int64_t src_rows,
                            void *dst, int64_t dst_row_stride, int64_t dst_head_stride, int64_t dst_rows,
                            int32_t dtype, const int32_t *src_slots, const int32_t *dst_slots,
                            const int32_t *positions, int32_t n, int32_t heads, int32_t head_dim,
                            int32_t rot_off, int32_t rot_dim, int32_t layout, const int64_t *freqs,
                            float factor, int32_t inverse, uint32_t *status, hs_stream_t stream) {
  if (dtype != HS_LOGITS_F32 && dtype != HS_LOGITS_BF16)
    return hs_set_error(HS_ERR_INVALID_ARG, "row dtype %d", dtype);
  if (layout != HS_ROPE_INTERLEAVED && layout != HS_ROPE_HALF)
    return hs_set_error(HS_ERR_INVALID_ARG, "rotary layout %d", layout);
  if (n < 0 || src_rows < 0 || dst_rows < 0 || heads < 1 || heads > 65535 || head_dim < 2 || head_dim > 65536 ||
      rot_dim < 2 || rot_dim % 2 || rot_off < 0 || rot_dim > head_dim || rot_off > head_dim - rot_dim)
    return hs_set_error(HS_ERR_INVALID_ARG,
                        "bad sizes n=%d rows=%lld/%lld heads=%d (1..65535) head_dim=%d (2..65536), dims %d + %d "
                        "(an even number, within the head) rotated",
                        n, (long long)src_rows, (long long)dst_rows, heads, head_dim, rot_off, rot_dim);
  const int64_t most = (int64_t)1 << 40, elem = dtype == HS_LOGITS_F32 ? 4 : 2;
  if (src_row_stride < 0 || src_head_stride < 0 || dst_row_stride < 0 || dst_head_stride < 0 ||
      src_row_stride > most || src_head_stride > most || dst_row_stride > most || dst_head_stride > most)
    return hs_set_error(HS_ERR_INVALID_ARG, "strides must be in 0..2^40 elements");
  if ((int64_t)heads * head_dim > 1 << 30)
    return hs_set_error(HS_ERR_UNSUPPORTED, "heads * head_dim past 2^30");
  // no two heads or rows of the destination share an element: the heads of a row
  // lie within its stride, or the rows of a head within the head's
  const auto within = [&](int64_t inner, int64_t count, int64_t outer, int64_t outers) {
    return (count <= 1 || inner >= head_dim) && (outers <= 1 || outer >= (count - 1) * inner + head_dim);
  };
  if (!within(dst_head_stride, heads, dst_row_stride, dst_rows) &&
      !within(dst_row_stride, dst_rows, dst_head_stride, heads))
    return hs_set_error(HS_ERR_INVALID_ARG, "rows or heads of dst overlap (strides %lld and %lld)",
                        (long long)dst_row_stride, (long long)dst_head_stride);
  if (!(factor == factor) || isinf(factor)) return hs_set_error(HS_ERR_INVALID_ARG, "factor is not finite");
  if (n == 0) return HS_OK;
  if (!src || !dst || !positions || !freqs)
    return hs_set_error(HS_ERR_INVALID_ARG, "NULL src/dst/positions/freqs");
  if ((((uintptr_t)src | (uintptr_t)dst) & (elem - 1)) || ((uintptr_t)freqs & 7) ||
      (((uintptr_t)src_slots | (uintptr_t)dst_slots | (uintptr_t)positions | (uintptr_t)status) & 3))
    return hs_set_error(HS_ERR_INVALID_ARG, "arrays must be aligned to their elements");
  const void *s = nullptr, *d = nullptr;
  int rc = hs_device_alias(src, &s, "src", (int)elem);
  if (rc || (rc = hs_device_alias(dst, &d, "dst", (int)elem))) return rc;

  // In place nothing beside the rotated part moves.
  const bool same = s == d && src_row_stride == dst_row_stride && src_slots == dst_slots &&
                    (heads == 1 || src_head_stride == dst_head_stride);
  RopeArgs a = {};
  a.src = reinterpret_cast<const char *>(s);
  a.dst = reinterpret_cast<char *>(const_cast<void *>(d));
  a.src_row = src_row_stride * elem;
  a.src_head = heads > 1 ? src_head_stride * elem : 0;
  a.dst_row = dst_row_stride * elem;
  a.dst_head = heads > 1 ? dst_head_stride * elem : 0;
  a.src_rows = src_rows;
  a.dst_rows = dst_rows;
  a.src_slots = src_slots;
  a.dst_slots = dst_slots;
  a.positions = positions;
  a.freqs = freqs;
  a.status = status;
  a.n = n;
  a.heads = heads;
  a.half = rot_dim / 2;
  a.off = (int32_t)(rot_off * elem);
  a.factor = factor;
  a.sign = inverse ? -factor : factor;
  // 16-byte accesses where everything that a unit's place is made of allows them
  const bool half = layout == HS_ROPE_HALF;
  const uint64_t parts = (uint64_t)(uintptr_t)s | (uint64_t)(uintptr_t)d | (uint64_t)a.src_row | (uint64_t)a.src_head |
                         (uint64_t)a.dst_row | (uint64_t)a.dst_head | (uint64_t)a.off |
                         (uint64_t)((half ? a.half : rot_dim) * elem) | (uint64_t)(same ? 0 : head_dim * elem);
  const bool vector = parts % 16 == 0;
  const int per = vector ? (int)(16 / elem) : 1;
  a.rot_units = !vector || half ? a.half / per : rot_dim / per;
  a.units = a.rot_units + (same ? 0 : (head_dim - rot_dim) / per);
  // Heads of a thread: one while that leaves threads for every SM, up to eight
  // (whose cosines and sines it then computes once).
  int sms = 0;
  if ((rc = hs_sm_count(&sms))) return rc;
  int64_t each = (int64_t)n * heads * a.units / ((int64_t)sms * 2048);
  each = each < 1 ? 1 : each > 8 ? 8 : each;
  a.step = (int32_t)((heads + each - 1) / each);
  const int64_t width = (int64_t)a.units * a.step;
  a.chunks = (int32_t)((width + RT - 1) / RT);
  a.per_block = width <= RT ? (int32_t)(RT / width) : 1;
  if (a.per_block > n) a.per_block = n;
  const int threads = a.chunks > 1 ? RT : (int)((width * a.per_block + 31) / 32 * 32);
  const int64_t blocks = a.chunks > 1 ? (int64_t)n * a.chunks : ((int64_t)n + a.per_block - 1) / a.per_block;
  if (blocks > INT32_MAX) return hs_set_error(HS_ERR_UNSUPPORTED, "n * heads * head_dim too large");
  return dtype == HS_LOGITS_F32 ? launch<float>(a, half, vector, (unsigned)blocks, threads, stream)
                                : launch<__nv_bfloat16>(a, half, vector, (unsigned)blocks, threads, stream);
}

extern "C" int hs_rope_freqs(int32_t rot_dim, double base, int32_t scaling, double scale, double context,
                             double fast, double slow, int64_t *freqs, float *factor) {
  if (rot_dim < 2 || rot_dim % 2 || rot_dim > 65536)
    return hs_set_error(HS_ERR_INVALID_ARG, "rot_dim %d is not even in 2..65536", rot_dim);
  if (scaling < HS_ROPE_PLAIN || scaling > HS_ROPE_YARN)
    return hs_set_error(HS_ERR_INVALID_ARG, "frequency scaling %d", scaling);
  if (!freqs || !factor) return hs_set_error(HS_ERR_INVALID_ARG, "NULL freqs or factor");
  if (!(base > 1.0) || !(base <= 1e300)) return hs_set_error(HS_ERR_INVALID_ARG, "base must be above 1");
  if (scaling != HS_ROPE_PLAIN && (!(scale >= 1.0) || !(scale <= 1e9)))
    return hs_set_error(HS_ERR_INVALID_ARG, "scale must be in [1, 10^9]");
  if (scaling == HS_ROPE_NTK && rot_dim == 2)
    return hs_set_error(HS_ERR_INVALID_ARG, "one pair has no base to scale");
  const double two_pi = 6.283185307179586476925286766559;
  *factor = 1.f;
  double low = 0., high = 0.;
  if (scaling == HS_ROPE_YARN) {
    if (!(context > 0.) || !(context <= 1e18) || !(slow > 0.) || !(fast >= slow) || !(fast <= 1e18))
      return hs_set_error(HS_ERR_INVALID_ARG, "yarn wants a context above 0 and 0 < slow <= fast");
    // the pair that turns r times over the context
    auto pair = [&](double r) { return rot_dim * log(context / (r * two_pi)) / (2. * log(base)); };
    low = fmax(floor(pair(fast)), 0.);
    high = fmin(ceil(pair(slow)), rot_dim - 1.);
    if (high - low < 0.001) high = low + 0.001;
    *factor = (float)(0.1 * log(scale) + 1.);
  }
  if (scaling == HS_ROPE_NTK) base *= pow(scale, (double)rot_dim / (rot_dim - 2));
  for (int i = 0; i < rot_dim / 2; ++i) {
    double w = pow(base, -2. * i / rot_dim);
    if (scaling == HS_ROPE_LINEAR) w /= scale;
    if (scaling == HS_ROPE_YARN) {
      const double ramp = fmin(fmax((i - low) / (high - low), 0.), 1.);
      w = w / scale * ramp + w * (1. - ramp);
    }
    freqs[i] = (int64_t)llround(w / two_pi * 18446744073709551616.);
  }
  return HS_OK;
}

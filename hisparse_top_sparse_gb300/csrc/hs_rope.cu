// Rotary positions: rows (queries, keys, latent rows) rotated pair by pair by
// angles proportional to their positions, on the way from a projection into q or
// a cache, or in place. The pages' caches hold 64 rotated dims in each latent row
// (HS_LATENT_DIM = 512 + 64) and the attention rotates nothing.
//
// The angle of a pair at position p is p * w. In f32 an angle of 10^5 radians is
// off by up to 0.004; in 64-bit whole fractions of a turn (w / 2 pi * 2^64, kept in
// `freqs`) the product wraps as the angle does and is exact modulo a turn at any
// position, for one integer multiplication a pair; the sine and the cosine are
// taken of its top 32 bits.
//
// A thread takes one unit of a head: as many pairs as 16-byte accesses hold
// (interleaved: 16 bytes; half: 16 bytes of each half), or 16 bytes of the dims
// beside the rotated part, which it copies. HBM bounds large calls, so a thread has
// several loads in flight (src may be dst, and the compiler would keep each load behind
// the store before it): of four heads of a row, whose cosines and sines it computes
// once, or, where heads are few, of eight rows (the rotated units then a row each).

#include <type_traits>

#include "hs_internal.cuh"

namespace {

constexpr int RT = 256;               // threads of a block, at most
// A thread has HEAD_BATCH heads of a row in flight, of at most most_heads(), or copies
// dims of ROW_BATCH rows. Measured: 65535 rows of 576 dims, 2 / 4 / 8 rows in flight
// 36 / 29 / 26.5 us (the floor is 22.3); 8192 rows x 128 heads x 64 dims, interleaved,
// 47.4 us (the floor is 39.5). The numbers of heads and blocks were chosen when every
// thread ended with a fence that is gone: interleaved, five blocks an SM, at most 8 / 16
// / 32 heads 52 / 48.5 / 49.5 us; half, three blocks (16 bytes of either half take
// registers), 8 heads 50, four blocks and 16 heads 57.
constexpr int HEAD_BATCH = 4, ROW_BATCH = 8;
constexpr int most_heads(bool half) { return half ? 8 : 16; }

struct RopeArgs {
  const char *src;
  char *dst;
  int64_t src_row, src_head, dst_row, dst_head;       // bytes
  int64_t src_rows, dst_rows;
  const int32_t *src_slots, *dst_slots, *positions;
  const int64_t *freqs;
  uint32_t *status;
  int32_t n, heads, step;             // a thread's heads are h, h + step, ... (ROWS: h alone)
  int32_t half;                       // pairs of a head
  int32_t off;                        // bytes before the rotated part
  int32_t rot_units, copy_units;      // units of a head
  // blocks of an entry (ROWS: of ROW_BATCH entries), and, where that is one, entries (or
  // batches of them) of a block
  int32_t chunks, per_block;
  float factor, sign;
};

// one access: 16 bytes, or one element
template <typename T, bool VECTOR>
struct Access {
  using Raw = typename std::conditional<VECTOR, uint4, T>::type;
  static constexpr int BYTES = (int)sizeof(Raw), N = BYTES / (int)sizeof(T);
  static __device__ __forceinline__ Raw load(const char *p) {
    if constexpr (VECTOR)
      return __ldcs(reinterpret_cast<const uint4 *>(p));
    else
      return *reinterpret_cast<const T *>(p);
  }
  static __device__ __forceinline__ void store(char *p, const Raw &v) { *reinterpret_cast<Raw *>(p) = v; }
  static __device__ __forceinline__ void unpack(const Raw &v, float (&f)[N]) {
    if constexpr (!VECTOR) {
      f[0] = (float)v;
    } else {
      const uint32_t ws[4] = {v.x, v.y, v.z, v.w};
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
  static __device__ __forceinline__ Raw pack(const float (&f)[N]) {
    if constexpr (!VECTOR) {
      return (T)f[0];
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
      return make_uint4(ws[0], ws[1], ws[2], ws[3]);
    }
  }
};

// Sine and cosine of a 32-bit fraction of a turn. The nearest quarter turn leaves
// exactly, in whole numbers; what is left, at most pi / 4, goes through the Taylor
// series (of 9th and 10th degree: cut off below 2^-29 and 2^-33), and the quarter
// swaps and signs the two. Off by at most 2^-22: the angle's rounding to f32 and its
// product with 2 pi 2^-32 (pi / 4 * 2^-23 together), and the series' roundings.
__device__ __forceinline__ void sincos_turn(uint32_t turn, float &sine, float &cosine) {
  const uint32_t quarter = (turn + 0x20000000u) >> 30;
  const float x = (float)(int32_t)(turn - (quarter << 30)) * (6.283185307179586f * 0x1p-32f), y = x * x;
  float s = fmaf(y, 1.f / 362880.f, -1.f / 5040.f);
  s = fmaf(y, s, 1.f / 120.f);
  s = fmaf(y, s, -1.f / 6.f);
  s = fmaf(x * y, s, x);
  float c = fmaf(y, -1.f / 3628800.f, 1.f / 40320.f);
  c = fmaf(y, c, -1.f / 720.f);
  c = fmaf(y, c, 1.f / 24.f);
  c = fmaf(y, c, -0.5f);
  c = fmaf(y, c, 1.f);
  const bool odd = quarter & 1;
  sine = __uint_as_float(__float_as_uint(odd ? c : s) ^ (quarter & 2) << 30);
  cosine = __uint_as_float(__float_as_uint(odd ? s : c) ^ ((quarter + 1) & 2) << 30);
}

template <typename T, bool HALF, bool VECTOR, bool ROWS>
__global__ void __launch_bounds__(RT, HALF || ROWS ? 3 : 5) k_rope_rows(const __grid_constant__ RopeArgs a) {
  using A = Access<T, VECTOR>;
  using Raw = typename A::Raw;
  constexpr int N = A::N;
  constexpr bool TWO = HALF || !VECTOR;           // a unit's pairs lie in two accesses
  constexpr int PAIRS = TWO ? N : N / 2;
  constexpr int BATCH = ROWS ? ROW_BATCH : HEAD_BATCH, SET = ROWS ? BATCH : 1;
  // The rotated units of a block's entries come first, then, from the next warp on,
  // the others: a warp with both would spend the cosines' time on the latter too.
  int w = (int)threadIdx.x;
  int64_t i = blockIdx.x;                         // the block's first entry
  if (a.chunks > 1) {
    w += (int)(blockIdx.x % (unsigned)a.chunks) * RT;
    i = blockIdx.x / (unsigned)a.chunks;
  }
  i *= a.per_block * SET;
  const int turning = a.rot_units * a.step * a.per_block * SET;
  const bool rotated = w < turning;
  if (!rotated) {
    w -= (turning + 31) & ~31;
    if (w < 0 || w >= a.copy_units * a.step * a.per_block) return;
  }
  const int units = rotated ? a.rot_units : a.copy_units;
  const int unit = w % units;
  w /= units;
  int h = w % a.step;                             // the (first) head
  i += w / a.step;
  auto slots = [&](int64_t e, int64_t &s, int64_t &d) {
    s = d = -1;
    if (e < a.n) {
      s = a.src_slots ? a.src_slots[e] : e;
      d = a.dst_slots ? a.dst_slots[e] : e;
    }
    if (s < a.src_rows && d < a.dst_rows) return true;
    s = -1;
    return false;
  };
  if (rotated) {
    if (i >= a.n) return;
    int64_t s, d;
    if (!slots(i, s, d) && a.status && unit == 0 && h == 0) atomicOr(a.status, HS_STATUS_INDEX);
    if (s < 0 || d < 0) return;
    // the unit's first access, and (TWO) its second
    const int at = a.off + unit * (HALF || !TWO ? 1 : 2) * A::BYTES;
    const int second = HALF ? a.half * (int)sizeof(T) : (int)sizeof(T);
    const char *p = a.src + s * a.src_row + (int64_t)h * a.src_head + at;
    char *q = a.dst + d * a.dst_row + (int64_t)h * a.dst_head + at;
    const int64_t src_step = a.step * a.src_head, dst_step = a.step * a.dst_head;
    const uint64_t position = (uint64_t)(int64_t)a.positions[i];
    float c[PAIRS], sn[PAIRS];
    auto angles = [&]() {
#pragma unroll
      for (int k = 0; k < PAIRS; ++k) {
        const uint64_t turn = position * (uint64_t)a.freqs[unit * PAIRS + k];
        sincos_turn((uint32_t)(turn >> 32), sn[k], c[k]);
        c[k] *= a.factor;
        sn[k] *= a.sign;
      }
    };
    // (which product of a sum is fused is written down: left to the compiler it differed
    // between the variants, and a row's last bits with its alignment)
    auto turn = [&](Raw &x, Raw &y) {
      float f[N];
      A::unpack(x, f);
      if constexpr (TWO) {
        float g[N];
        A::unpack(y, g);
#pragma unroll
        for (int k = 0; k < PAIRS; ++k) {
          const float u = f[k], v = g[k];
          f[k] = fmaf(u, c[k], -(v * sn[k]));
          g[k] = fmaf(u, sn[k], v * c[k]);
        }
        y = A::pack(g);
      } else {
#pragma unroll
        for (int k = 0; k < PAIRS; ++k) {
          const float u = f[2 * k], v = f[2 * k + 1];
          f[2 * k] = fmaf(u, c[k], -(v * sn[k]));
          f[2 * k + 1] = fmaf(u, sn[k], v * c[k]);
        }
      }
      x = A::pack(f);
    };
    if constexpr (ROWS) {
      Raw x = A::load(p), y;
      if (TWO) y = A::load(p + second);
      angles();
      turn(x, y);
      if (TWO) A::store(q + second, y);
      A::store(q, x);
    } else {
      bool fresh = true;
      for (; h < a.heads; h += BATCH * a.step, p += BATCH * src_step, q += BATCH * dst_step) {
        Raw x[BATCH], y[BATCH];
#pragma unroll
        for (int r = 0; r < BATCH; ++r)
          if (h + r * a.step < a.heads) {
            x[r] = A::load(p + r * src_step);
            if (TWO) y[r] = A::load(p + r * src_step + second);
          }
        if (fresh) angles();                      // (while the first loads are on their way)
        fresh = false;
#pragma unroll
        for (int r = 0; r < BATCH; ++r)
          if (h + r * a.step < a.heads) {
            turn(x[r], y[r]);
            if (TWO) A::store(q + r * dst_step + second, y[r]);
            A::store(q + r * dst_step, x[r]);
          }
      }
    }
  } else {
    // beside the rotated part, moved as it is
    int at = unit * A::BYTES;
    if (at >= a.off) at += 2 * a.half * (int)sizeof(T);
    const char *p[BATCH];
    char *q[BATCH];
    Raw x[BATCH];
    if constexpr (ROWS) {
#pragma unroll
      for (int r = 0; r < BATCH; ++r) {
        int64_t s, d;
        slots(i + (int64_t)r * a.per_block, s, d);
        p[r] = s >= 0 && d >= 0 ? a.src + s * a.src_row + (int64_t)h * a.src_head + at : nullptr;
        q[r] = a.dst + d * a.dst_row + (int64_t)h * a.dst_head + at;
      }
    } else {
      int64_t s, d;
      slots(i, s, d);
      if (s < 0 || d < 0) return;
      p[0] = a.src + s * a.src_row + at;
      q[0] = a.dst + d * a.dst_row + at;
    }
    if constexpr (ROWS) {
#pragma unroll
      for (int r = 0; r < BATCH; ++r)
        if (p[r]) x[r] = A::load(p[r]);
#pragma unroll
      for (int r = 0; r < BATCH; ++r)
        if (p[r]) A::store(q[r], x[r]);
    } else {
      for (; h < a.heads; h += BATCH * a.step) {
#pragma unroll
        for (int r = 0; r < BATCH; ++r)
          if (h + r * a.step < a.heads) x[r] = A::load(p[0] + (int64_t)(h + r * a.step) * a.src_head);
#pragma unroll
        for (int r = 0; r < BATCH; ++r)
          if (h + r * a.step < a.heads) A::store(q[0] + (int64_t)(h + r * a.step) * a.dst_head, x[r]);
      }
    }
  }
}

template <typename T, bool HALF, bool VECTOR>
int launch(const RopeArgs &a, bool rows, unsigned blocks, int threads, cudaStream_t stream) {
  if (rows)
    k_rope_rows<T, HALF, VECTOR, true><<<blocks, threads, 0, stream>>>(a);
  else
    k_rope_rows<T, HALF, VECTOR, false><<<blocks, threads, 0, stream>>>(a);
  HS_LAUNCH_CHECK("k_rope_rows");
  return HS_OK;
}
template <typename T>
int launch(const RopeArgs &a, bool half, bool vector, bool rows, unsigned blocks, int threads, cudaStream_t stream) {
  if (half)
    return vector ? launch<T, true, true>(a, rows, blocks, threads, stream)
                  : launch<T, true, false>(a, rows, blocks, threads, stream);
  return vector ? launch<T, false, true>(a, rows, blocks, threads, stream)
                : launch<T, false, false>(a, rows, blocks, threads, stream);
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
    // (in floating point: the product of any count and stride has a place there)
    return (count <= 1 || inner >= head_dim) &&
           (outers <= 1 || (double)outer >= ((double)count - 1.) * (double)inner + head_dim);
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
  if (rc) return rc;
  if (src == dst)
    d = s;
  else if ((rc = hs_device_alias(dst, &d, "dst", (int)elem)))
    return rc;

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
  a.copy_units = same ? 0 : (head_dim - rot_dim) / per;
  // Units of a thread: one up to 512 threads an SM, then up to most_heads() heads of a
  // row or, where there are fewer heads than a batch, ROW_BATCH rows (with one unit up
  // to 2048 threads an SM 8191 rows of 576 dims took 10.7 us, now 4.7, and 512 rows of
  // 128 heads 9.1, now 5).
  int sms = 0;
  if ((rc = hs_sm_count(&sms))) return rc;
  const int64_t full = (int64_t)n * heads * (a.rot_units + a.copy_units) / ((int64_t)sms * 512);
  const int64_t each = full < 1 ? 1 : full > most_heads(half) ? most_heads(half) : full;
  const bool rows = heads < HEAD_BATCH && full > 0;
  a.step = rows ? heads : (int32_t)((heads + each - 1) / each);
  const int set = rows ? ROW_BATCH : 1;
  const auto threads_of = [&](int64_t sets) {
    return (sets * set * a.rot_units * a.step + 31) / 32 * 32 + sets * a.copy_units * a.step;
  };
  const int64_t sets = ((int64_t)n + set - 1) / set;       // entries, or batches of them
  a.chunks = (int32_t)((threads_of(1) + RT - 1) / RT);
  a.per_block = 1;
  while (a.chunks == 1 && a.per_block < sets && threads_of(a.per_block + 1) <= RT) ++a.per_block;
  const int threads = a.chunks > 1 ? RT : (int)((threads_of(a.per_block) + 31) / 32 * 32);
  const int64_t blocks = (sets + a.per_block - 1) / a.per_block * a.chunks;
  if (blocks > INT32_MAX) return hs_set_error(HS_ERR_UNSUPPORTED, "n * heads * head_dim too large");
  return dtype == HS_LOGITS_F32 ? launch<float>(a, half, vector, rows, (unsigned)blocks, threads, stream)
                                : launch<__nv_bfloat16>(a, half, vector, rows, (unsigned)blocks, threads, stream);
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

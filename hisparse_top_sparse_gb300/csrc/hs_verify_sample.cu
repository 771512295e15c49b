// Verification of drafted tokens by sampling, from given random numbers: the
// acceptance rule of speculative sampling in place of the greedy one of
// hs_verify.cu ("投机解码的 KV 流转：prefill 阶段 DFlash 也要吃下整个 prompt",
// section ④, checks the drafts greedily), and the same commit.
//
// For a request with temperature T > 0, target logits l_i, draft
// probabilities q_i, drafts x_i and given numbers u_i in [0, 1) and E_v > 0:
//   p_i(v) = exp((l_i(v) - M_i) / T) / S_i, M_i = max_v l_i(v), S_i the sum;
//   draft i is accepted while u_i q_i(x_i) < p_i(x_i); m drafts are accepted;
//   the next token is argmax_v w(v) / E_v, where w = max(p_m - q_m, 0) after a
//   refusal and w = p_d past the last draft. With E_v exponentially
//   distributed, that is v with probability w(v) / sum w: a race whose winner
//   needs one pass and no running sum over the vocabulary, so that the order
//   of additions cannot move the answer. (p is off by about (|l - M| / T + 8)
//   2^-22 of itself: the exponent's argument is rounded four times in f32, the
//   exponential and the sum add the rest, the ratio's approximate reciprocal
//   2^-23. After a refusal w = p - q is off by as much as p, which is more of
//   itself where p and q are near each other. Two tokens closer than that may
//   change places.)
//
// One cluster of 1 to 16 blocks per request takes the request's rows in order,
// one or a few at a time, and stops at the first refusal: the logits behind it,
// and the draft probabilities of every row but the last, are never read. HBM
// bounds it: each logits row is streamed once for (M, S), and the row that
// yields the token a second time, beside q and E, mostly from L2. M and S
// come in one pass (a thread rescales its sum when a batch of its values
// brings a new maximum). The sums are f32, each of a thread's V / 256 terms (505
// at V = 129280) or, with more blocks, fewer, in batches of 16 or 32 that are
// summed first, then joined as a tree in a fixed order: results do not depend on
// scheduling. A thread copies its values ahead into places of its own in
// shared memory (cp.async), so no barrier stands between loading and using.
//
// The blocks of a cluster exchange (M, S) and the race's winner through
// distributed shared memory, every warp joining all warps' figures in the
// same order; the request's drafts, numbers and temperature are read once by
// the first block and pushed to the others. So every warp takes the same
// decisions from the same bits, and the barriers match even if a caller
// overwrites the inputs during the call (what it then gets is unspecified).
//
// Measured (bf16 logits, draft probabilities given): 256 requests x 3 drafts,
// V = 129280: 70 us, 82 % of what the 385 MB it has to move take at the
// measured copy rate (V = 129281: 80 us); 128 x 3: 43 us; 64 x 3: 26 us; 1 x 3:
// 9.6 us and 2 x 3, V = 1024 f32: 6.4 us, latency.

#include <float.h>

#include <atomic>
#include <type_traits>

#include "hs_commit.cuh"

namespace {

constexpr int NT = 256;             // threads per block
constexpr int MIN_BLOCKS = 3;       // blocks per SM, at least (80 registers, nothing spilled)
constexpr int WARPS = NT / 32;
constexpr int RING = 12;            // 16-byte places of a thread's ring of copies in flight
constexpr int WARP_RING = 489;      // 16-byte places of a warp's ring in the race: 3 to 7 windows
constexpr int BATCH = 4;            // vectors of a row taken together
constexpr int NB = 8;               // values of a thread in flight where rows are not aligned
static_assert(WARP_RING * WARPS >= RING * NT, "row_stat's places");
constexpr size_t RING_BYTES = (size_t)WARP_RING * WARPS * 16;
constexpr int MAX_CLUSTER = 16;
constexpr int MAX_DRAFTS = 255;
constexpr float LOG2E = 1.4426950408889634f;

// How the rows of logits, draft probabilities and noise lie: each on 16 bytes;
// anywhere in arrays on 16 bytes; anywhere.
enum Rows { ROWS_ON_16, ARRAYS_ON_16, ROWS_ANYWHERE };

struct SampleArgs {
  const void *logits;
  int32_t d, V;
  const float *temperature;
  const int32_t *drafts;
  const float *probs, *uniforms, *noise;
  int32_t *accept_len, *next_token;
  float *logprob;
  uint32_t *status;
  uint32_t log_rows;       // 2^log_rows rows side by side in a cluster, at most its blocks
  Rows rows;
};

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;\n" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;\n" : "=r"(r));
  return r;
}
// the cluster barrier: writes before a thread's arrival are seen by every
// thread that has waited
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}
// 4 / 8 bytes into block `rank`'s shared memory, at the place p has in this
// block's
__device__ __forceinline__ uint32_t remote(const void *p, uint32_t rank) {
  uint32_t a = (uint32_t)__cvta_generic_to_shared(p);
  asm volatile("mapa.shared::cluster.u32 %0, %0, %1;\n" : "+r"(a) : "r"(rank));
  return a;
}
__device__ __forceinline__ void push(const void *p, uint32_t rank, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;\n" ::"r"(remote(p, rank)), "r"(v) : "memory");
}
__device__ __forceinline__ void push2(const void *p, uint32_t rank, uint32_t a, uint32_t b) {
  asm volatile("st.shared::cluster.v2.u32 [%0], {%1, %2};\n" ::"r"(remote(p, rank)), "r"(a), "r"(b)
               : "memory");
}
// a thread's 16-byte copies into its own ring places
__device__ __forceinline__ void copy16(uint4 *dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"((uint32_t)__cvta_generic_to_shared(dst)),
               "l"(src)
               : "memory");
}
// its first `bytes`, zeros behind them
__device__ __forceinline__ void copy16(uint4 *dst, const void *src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"((uint32_t)__cvta_generic_to_shared(dst)),
               "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory");
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}
// A logit as it counts: NaN as -inf (a masked token), +inf as the type's
// largest finite value, so that no difference of two logits is undefined but
// that of two masked ones, which never meet (a row's maximum is finite or the
// row is empty).
template <int DTYPE>
__device__ __forceinline__ float clean(float x) {
  return fminf(fmaxf(x, -INFINITY), DTYPE == HS_LOGITS_F32 ? FLT_MAX : __uint_as_float(0x7f7f0000u));
}

// what is read once and given to every block (volatile: a second reading might
// find something else)
__device__ __forceinline__ uint32_t once(const void *p) {
  uint32_t v;
  asm volatile("ld.global.b32 %0, [%1];\n" : "=r"(v) : "l"(p));
  return v;
}
template <int DTYPE>
__device__ __forceinline__ float logit_once(const void *row, int64_t i) {
  if (DTYPE == HS_LOGITS_F32) return clean<DTYPE>(__uint_as_float(once(reinterpret_cast<const float *>(row) + i)));
  unsigned short u;
  asm volatile("ld.global.u16 %0, [%1];\n" : "=h"(u) : "l"(reinterpret_cast<const unsigned short *>(row) + i));
  return clean<DTYPE>(__uint_as_float((uint32_t)u << 16));
}

template <int DTYPE>
__device__ __forceinline__ float raw_logit_at(const void *row, int64_t i) {
  if (DTYPE == HS_LOGITS_F32) return __ldg(reinterpret_cast<const float *>(row) + i);
  return __uint_as_float((uint32_t)__ldg(reinterpret_cast<const unsigned short *>(row) + i) << 16);
}
template <int DTYPE>
__device__ __forceinline__ float logit_at(const void *row, int64_t i) {
  return clean<DTYPE>(raw_logit_at<DTYPE>(row, i));
}

// (a, b) packed for the two-at-a-time f32 instructions
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};\n" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float &a, float &b) {
  asm("mov.b64 {%0, %1}, %2;\n" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
// part `rank` of `total` things among 2^log_n
__device__ __forceinline__ int32_t part_of(int32_t total, uint32_t rank, uint32_t log_n) {
  return (int32_t)(((int64_t)total * rank) >> log_n);
}

// Running (maximum, sum of exp2((x - max) * c)) of one thread, and the batch
// at which the maximum was first reached.
struct Stat {
  float m, s;
  int32_t at;
};
__device__ __forceinline__ void join(float &m, float &s, float om, float os, float c) {
  const float t = fmaxf(m, om);
  if (t == -INFINITY) return;                  // both empty
  s = s * ex2((m - t) * c) + os * ex2((om - t) * c);
  m = t;
}

// One slice of a row: the 16-byte vectors [lo, hi) of its aligned body, taken
// by all threads of the block, and the fewer than 2 PER values outside the
// body, all the first slice's.
template <int DTYPE>
struct Slice {
  static constexpr int PER = DTYPE == HS_LOGITS_F32 ? 4 : 8;
  const uint4 *body;
  int32_t lo, hi, head, tail, rest;

  __device__ __forceinline__ Slice(const char *row, int32_t V, uint32_t rank, uint32_t log_n) {
    constexpr int elem = DTYPE == HS_LOGITS_F32 ? 4 : 2;
    head = (int)(((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15) / elem);
    if (head > V) head = V;
    const int32_t vecs = (V - head) / PER;
    body = reinterpret_cast<const uint4 *>(row + (int64_t)head * elem);
    lo = part_of(vecs, rank, log_n);
    hi = part_of(vecs, rank + 1, log_n);
    tail = head + vecs * PER;
    rest = rank == 0 ? head + (V - tail) : 0;
  }
  __device__ __forceinline__ int32_t rest_index(int32_t j) const {
    return j < head ? j : tail + (j - head);
  }
};

// the values of a vector as they count
template <int DTYPE>
__device__ __forceinline__ uint4 clean16(uint4 w) {
  uint32_t *x = reinterpret_cast<uint32_t *>(&w);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (DTYPE == HS_LOGITS_F32) {
      x[j] = __float_as_uint(clean<DTYPE>(__uint_as_float(x[j])));
    } else {
      __nv_bfloat162 &h = reinterpret_cast<__nv_bfloat162 &>(x[j]);
      const uint32_t lowest = 0xff80ff80u, most = 0x7f7f7f7fu;
      h = __hmin2(__hmax2(h, reinterpret_cast<const __nv_bfloat162 &>(lowest)),
                  reinterpret_cast<const __nv_bfloat162 &>(most));
    }
  }
  return w;
}
template <int DTYPE>
__device__ __forceinline__ uint4 masked16() {
  const uint32_t none = DTYPE == HS_LOGITS_F32 ? 0xff800000u : 0xff80ff80u;
  return make_uint4(none, none, none, none);
}
// value j of a vector
template <int DTYPE>
__device__ __forceinline__ float value(const uint4 &w, int j) {
  const uint32_t x[4] = {w.x, w.y, w.z, w.w};
  if (DTYPE == HS_LOGITS_F32) return __uint_as_float(x[j & 3]);
  return __uint_as_float((j & 1) ? x[j >> 1] & 0xFFFF0000u : x[j >> 1] << 16);
}

template <int DTYPE>
__device__ __forceinline__ float batch_max(const uint4 (&w)[BATCH]) {
  if (DTYPE == HS_LOGITS_F32) {
    float t = -INFINITY;
#pragma unroll
    for (int u = 0; u < BATCH; ++u)
      t = fmaxf(t, fmaxf(fmaxf(__uint_as_float(w[u].x), __uint_as_float(w[u].y)),
                         fmaxf(__uint_as_float(w[u].z), __uint_as_float(w[u].w))));
    return t;
  }
  const __nv_bfloat162 *h = reinterpret_cast<const __nv_bfloat162 *>(w);
  __nv_bfloat162 t = h[0];
#pragma unroll
  for (int u = 1; u < 4 * BATCH; ++u) t = __hmax2(t, h[u]);
  return fmaxf(__low2float(t), __high2float(t));
}

// A batch into the running statistics.
template <int DTYPE>
__device__ __forceinline__ void take_batch(Stat &st, const uint4 (&w)[BATCH], int32_t k, float c) {
  const float t = batch_max<DTYPE>(w);
  if (t > st.m) {
    st.s *= ex2((st.m - t) * c);
    st.m = t;
    st.at = k;
  }
  if (st.m == -INFINITY) return;
  const uint64_t nm = pack2(-st.m, -st.m), cc = pack2(c, c);
  uint64_t acc[2] = {0, 0};                  // four partial sums
#pragma unroll
  for (int u = 0; u < BATCH; ++u) {
#pragma unroll
    for (int j = 0; j < Slice<DTYPE>::PER; j += 2) {
      float a, b;
      unpack2(mul2(add2(pack2(value<DTYPE>(w[u], j), value<DTYPE>(w[u], j + 1)), nm), cc), a, b);
      acc[(j >> 1) & 1] = add2(acc[(j >> 1) & 1], pack2(ex2(a), ex2(b)));
    }
  }
  float a, b;
  unpack2(add2(acc[0], acc[1]), a, b);
  st.s += a + b;
}

// The slice's statistics: batches of BATCH vectors through this thread's own
// ring places (its column of `ring`), RING / BATCH of them in flight; no
// thread reads another's, so nothing but the copies is waited for. The values
// are taken as they are: a NaN or +inf among them makes the sum NaN, and the
// thread then goes through its part once more, cleaning each value.
// `meanwhile` runs while the first copies are on their way.
template <int DTYPE, typename F>
__device__ __forceinline__ Stat row_stat(const Slice<DTYPE> &sl, const void *row, float c, uint4 *ring,
                                         const F &meanwhile) {
  constexpr int DEPTH = RING / BATCH, STEP = BATCH * NT;
  Stat st = {-INFINITY, 0.f, -1};
  const int32_t k0 = sl.lo + (int)threadIdx.x;
  const int32_t full = sl.hi - (BATCH - 1) * NT;        // batches before it are whole
  auto issue = [&](int32_t k, int place) {
    uint4 *to = ring + place * STEP;
    if (k < full) {
#pragma unroll
      for (int u = 0; u < BATCH; ++u) copy16(to + u * NT, sl.body + k + u * NT);
    } else {
#pragma unroll
      for (int u = 0; u < BATCH - 1; ++u)
        if (k + u * NT < sl.hi) copy16(to + u * NT, sl.body + k + u * NT);
    }
    copy_commit();
  };
#pragma unroll
  for (int p = 0; p < DEPTH; ++p) issue(k0 + p * STEP, p);
  static_assert(2 * Slice<DTYPE>::PER <= NT, "a value outside the body per thread");
  const float rest = (int)threadIdx.x < sl.rest ? logit_at<DTYPE>(row, sl.rest_index(threadIdx.x)) : -INFINITY;
  meanwhile();
  int place = 0;
  for (int32_t k = k0; k < sl.hi; k += STEP) {
    copy_wait<DEPTH - 1>();
    uint4 w[BATCH];
    const uint4 *from = ring + place * STEP;
#pragma unroll
    for (int u = 0; u < BATCH; ++u) w[u] = from[u * NT];
    if (k >= full) {
#pragma unroll
      for (int u = 1; u < BATCH; ++u)
        if (k + u * NT >= sl.hi) w[u] = masked16<DTYPE>();
    }
    issue(k + DEPTH * STEP, place);
    place = place + 1 == DEPTH ? 0 : place + 1;
    take_batch<DTYPE>(st, w, k, c);
  }
  copy_wait<0>();
  if (st.s != st.s) {
    st = {-INFINITY, 0.f, -1};
#pragma unroll 1
    for (int32_t k = k0; k < sl.hi; k += STEP) {
      uint4 w[BATCH];
#pragma unroll
      for (int u = 0; u < BATCH; ++u)
        w[u] = k + u * NT < sl.hi ? clean16<DTYPE>(__ldg(sl.body + k + u * NT)) : masked16<DTYPE>();
      take_batch<DTYPE>(st, w, k, c);
    }
  }
  join(st.m, st.s, rest, rest == -INFINITY ? 0.f : 1.f, c);
  return st;
}

// The lowest index of this thread's values equal to `top` (its own maximum,
// first reached in the batch st.at), or INT32_MAX.
template <int DTYPE>
__device__ __forceinline__ int32_t row_first(const Slice<DTYPE> &sl, const void *row, const Stat &st,
                                             float top) {
  int32_t best = INT32_MAX;
  if (st.m != top) return best;
  if (st.at >= 0) {
#pragma unroll 1
    for (int u = 0; u < BATCH; ++u) {
      const int32_t k = st.at + u * NT;
      if (k >= sl.hi) break;
      const uint4 w = clean16<DTYPE>(__ldg(sl.body + k));
#pragma unroll
      for (int j = 0; j < Slice<DTYPE>::PER; ++j)
        if (value<DTYPE>(w, j) == top) best = min(best, sl.head + k * Slice<DTYPE>::PER + j);
    }
  }
  const int32_t j = threadIdx.x;
  if (j < sl.rest && logit_at<DTYPE>(row, sl.rest_index(j)) == top) best = min(best, sl.rest_index(j));
  return best;
}

struct Shared {
  // the first block's reading of the request, pushed to every block
  float temperature;
  float draft_logit[MAX_DRAFTS], draft_bar[MAX_DRAFTS];     // l_i(x_i); u_i q_i(x_i)
  int32_t draft[MAX_DRAFTS];
  // a pair from every warp of the cluster, at two alternating places
  uint2 pair[2][MAX_CLUSTER * WARPS];
};

// Joins a (float, word) pair of every thread of the cluster by `op`, apart
// for each of the G = 2^log_g rows (row g the blocks of ranks g n / G and up).
// Each warp joins its own threads' pairs and pushes the result to every block;
// behind the cluster's barrier every warp joins all warps' pairs, in the same
// order everywhere (`behind` runs first: it may set op from what the first block
// has pushed). On return lane g * 32 / G holds row g's. A place of `pair`
// is written again two calls later, behind the barrier of the call between,
// by when it has been read.
struct Nothing {
  __device__ __forceinline__ void operator()() const {}
};
template <typename Op, typename F = Nothing>
__device__ __forceinline__ void cluster_join(Shared &sh, float &a, uint32_t &b, uint32_t rank,
                                             uint32_t n, uint32_t log_g, int &turn, const Op &op,
                                             const F &behind = F{}) {
  const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  op.across(a, b, 32);
  uint2 *pairs = sh.pair[turn];
  if (n == 1) {
    if (lane == 0) pairs[warp] = make_uint2(__float_as_uint(a), b);
    __syncthreads();
  } else {
    if (lane < n) push2(pairs + rank * WARPS + warp, lane, __float_as_uint(a), b);
    cluster_arrive();
    cluster_wait();
  }
  turn ^= 1;
  behind();
  op.empty(a, b);
  // 32 / G lanes for the pairs of each row
  const uint32_t lanes = 32u >> log_g, count = (n >> log_g) * WARPS, row = lane / lanes;
  for (uint32_t k = lane & (lanes - 1); k < count; k += lanes) {
    const uint2 p = pairs[row * count + k];
    op.two(a, b, __uint_as_float(p.x), p.y);
  }
  op.across(a, b, lanes);
}

// (maximum, sum of exp2((x - maximum) c))
struct StatOp {
  float c;
  __device__ __forceinline__ void empty(float &m, uint32_t &s) const {
    m = -INFINITY;
    s = 0u;
  }
  __device__ __forceinline__ void two(float &m, uint32_t &s, float om, uint32_t os) const {
    float t = __uint_as_float(s);
    join(m, t, om, __uint_as_float(os), c);
    s = __float_as_uint(t);
  }
  // over groups of `width` lanes: the maximum first, then each sum on it
  __device__ __forceinline__ void across(float &m, uint32_t &s, uint32_t width) const {
    float top = m, t = __uint_as_float(s);
    for (uint32_t o = 1; o < width; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (m != -INFINITY) t *= ex2((m - top) * c);
    for (uint32_t o = 1; o < width; o <<= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    m = top;
    s = __float_as_uint(t);
  }
};
// the lowest index
struct MinOp {
  __device__ __forceinline__ void empty(float &, uint32_t &i) const { i = INT32_MAX; }
  __device__ __forceinline__ void two(float &, uint32_t &i, float, uint32_t oi) const { i = min(i, oi); }
  __device__ __forceinline__ void across(float &, uint32_t &i, uint32_t width) const {
    for (uint32_t o = 1; o < width; o <<= 1) i = min(i, __shfl_xor_sync(0xffffffffu, i, o));
  }
};
// the largest value, the lowest index of it
struct BestOp {
  __device__ __forceinline__ void empty(float &v, uint32_t &i) const {
    v = 0.f;
    i = INT32_MAX;
  }
  __device__ __forceinline__ void two(float &v, uint32_t &i, float ov, uint32_t oi) const {
    if (ov > v || (ov == v && oi < i)) {
      v = ov;
      i = oi;
    }
  }
  __device__ __forceinline__ void across(float &v, uint32_t &i, uint32_t width) const {
    for (uint32_t o = 1; o < width; o <<= 1) {
      const float ov = __shfl_xor_sync(0xffffffffu, v, o);
      const uint32_t oi = __shfl_xor_sync(0xffffffffu, i, o);
      two(v, i, ov, oi);
    }
  }
};

// What the race needs of its row.
struct RaceRow {
  float top, c, inv;       // p(v) = exp2((l(v) - top) c) inv
  int32_t barred;          // a token without weight, or -1
};

// w(v) / E(v) of the pair of values l2 (their draft probabilities minus, their
// E): one multiplication by an approximate reciprocal, as exact as p itself. A
// NaN never wins; neither does a weight of 0 or less.
__device__ __forceinline__ void ratio2(uint64_t l2, uint64_t minus_q, float e0, float e1, uint64_t nm,
                                       uint64_t cc, uint64_t ii, float &r0, float &r1) {
  float a, b, f, g;
  unpack2(mul2(add2(l2, nm), cc), a, b);
  const uint64_t p = fma2(pack2(ex2(a), ex2(b)), ii, minus_q);
  asm("rcp.approx.ftz.f32 %0, %1;\n" : "=f"(f) : "f"(e0));
  asm("rcp.approx.ftz.f32 %0, %1;\n" : "=f"(g) : "f"(e1));
  unpack2(mul2(p, pack2(f, g)), r0, r1);
}

// The race over the row that yields the token: this thread's largest ratio and
// its index (INT32_MAX: none above 0). A thread looks for the place of a
// group's largest ratio only when it reaches the best of its warp so far.
struct Race {
  float best;
  uint32_t at;
  float bar;               // the warp's best so far

  // (the whole warp; `big` is the largest of r, or 0 to take none)
  template <int N, typename At>
  __device__ __forceinline__ void group(const float (&r)[N], float big, const At &index) {
    if (big >= bar && big > best) {
      best = big;
#pragma unroll
      for (int j = N - 1; j >= 0; --j)
        if (r[j] == big) at = (uint32_t)index(j);      // indices ascend: the lowest of equals stays
    }
    bar = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(best)));
  }
};

template <int DTYPE, Rows ROWS, bool HAS_Q>
__device__ __forceinline__ Race race(const char *row, const float *q, const float *E, int32_t V,
                                     uint32_t rank, uint32_t log_n, const RaceRow &rr, uint4 *ring) {
  Race ra = {0.f, INT32_MAX, 0.f};
  const uint64_t nm = pack2(-rr.top, -rr.top), cc = pack2(rr.c, rr.c), ii = pack2(rr.inv, rr.inv);
  // the block's values: whole vectors of logits
  constexpr int PER = Slice<DTYPE>::PER;
  const int32_t vecs = (V + PER - 1) / PER, lo = part_of(vecs, rank, log_n) * PER,
                hi = min(part_of(vecs, rank + 1, log_n) * PER, V);
  if (ROWS != ROWS_ANYWHERE) {
    // A warp takes UNIT values at a time and copies for each array the 16-byte
    // vectors that hold them, so that every copy of a warp is one contiguous
    // piece (where each lane copied eight values' worth of E and q side by side,
    // the copies touched each 32-byte sector twice: 94 us against 82 on 256 x 3
    // drafts). Where the rows start on 16 bytes a lane takes groups of four
    // values, a vector of E and q each; else the values lie somewhere in the
    // copied windows, each array's its own way on, and a lane takes every 32nd (256
    // x 3 drafts, V = 129281: 80 us, by loads without copies 122; V = 129280 the
    // same way 72.9 against 70).
    constexpr int ELEM = 16 / PER, UNIT = 32 * PER;
    constexpr int LV = 32 + 1, EV = UNIT / 4 + 1, STAGE = LV + (HAS_Q ? 2 : 1) * EV, DEPTH = WARP_RING / STAGE;
    const int32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint4 *mine = ring + warp * WARP_RING;
    // lane l's vector of each array's first window (its other vectors of a window
    // are 32 further on; the last one is lane 0's, 1's and 2's), and how far the
    // lane's first value lies in the window
    const int32_t first = lo + warp * UNIT;
    const char *ls = row + (int64_t)first * ELEM, *ew = reinterpret_cast<const char *>(E + first),
               *qw = HAS_Q ? reinterpret_cast<const char *>(q + first) : ew;
    const int l_at = (int)(reinterpret_cast<uintptr_t>(ls) & 15) / ELEM + lane,
              e_at = (int)(reinterpret_cast<uintptr_t>(ew) & 15) / 4 + lane,
              q_at = (int)(reinterpret_cast<uintptr_t>(qw) & 15) / 4 + lane;
    ls += 16 * lane - ELEM * (l_at - lane);
    ew += 16 * lane - 4 * (e_at - lane);
    qw += 16 * lane - 4 * (q_at - lane);
    const char *last = lane == 0 ? ls + 512 : (lane == 1 ? ew : qw) + 4 * UNIT - 16 * lane;
    const int last_at = lane == 0 ? 32 : LV + lane * EV - 1, last_step = WARPS * UNIT * (lane == 0 ? ELEM : 4);
    auto issue = [&](int32_t v0, int place) {
      uint4 *to = mine + place * STAGE;
      if (v0 + UNIT + PER <= V && v0 < hi) {
        copy16(to + lane, ls);
#pragma unroll
        for (int k = 0; k < UNIT / 128; ++k) {
          copy16(to + LV + 32 * k + lane, ew + 512 * k);
          if (HAS_Q) copy16(to + LV + EV + 32 * k + lane, qw + 512 * k);
        }
        if (ROWS != ROWS_ON_16 && lane < (HAS_Q ? 3 : 2)) copy16(to + last_at, last);
      } else if (v0 < hi) {                     // no byte past the row's end
        auto part = [&](uint4 *at, const char *from, const void *end) {
          const int64_t left = reinterpret_cast<const char *>(end) - from;
          if (left > 0) copy16(at, from, left < 16 ? (int)left : 16);
        };
        part(to + lane, ls, row + (int64_t)V * ELEM);
#pragma unroll
        for (int k = 0; k < UNIT / 128; ++k) {
          part(to + LV + 32 * k + lane, ew + 512 * k, E + V);
          if (HAS_Q) part(to + LV + EV + 32 * k + lane, qw + 512 * k, q + V);
        }
        if (ROWS != ROWS_ON_16 && lane < (HAS_Q ? 3 : 2))
          part(to + last_at, last, lane == 0 ? row + (int64_t)V * ELEM : reinterpret_cast<const char *>((lane == 1 ? E : q) + V));
      }
      copy_commit();
      ls += WARPS * UNIT * ELEM;
      ew += WARPS * UNIT * 4;
      qw += WARPS * UNIT * 4;
      last += last_step;
    };
#pragma unroll 1
    for (int p = 0; p < DEPTH; ++p) issue(first + p * WARPS * UNIT, p);
    int place = 0;
    for (int32_t v0 = first; v0 < hi; v0 += WARPS * UNIT) {       // the whole warp
      copy_wait<DEPTH - 1>();
      __syncwarp();
      const uint4 *from = mine + place * STAGE;
      const float *es = reinterpret_cast<const float *>(from + LV) + e_at;
      const float *qs = reinterpret_cast<const float *>(from + LV + EV) + q_at;
      float r[PER], e[PER], w[PER], big = 0.f;
      auto value_at = [&](int o) {
        return ROWS == ROWS_ON_16 ? v0 + 128 * (o / 4) + 4 * lane + (o & 3) : v0 + 32 * o + lane;
      };
#pragma unroll
      for (int o = 0; o < PER; ++o) {
        if (ROWS == ROWS_ON_16) {
          if (o & 3) continue;
          // (a bf16 lane's logits are the halves of two others' copies)
          const uint2 half = reinterpret_cast<const uint2 *>(from)[32 * (o / 4) + lane];
          const uint4 x = DTYPE == HS_LOGITS_F32 ? from[lane] : make_uint4(half.x, half.y, 0, 0);
          const uint4 e4 = from[LV + 32 * (o / 4) + lane];
          const uint4 w4 = HAS_Q ? from[LV + EV + 32 * (o / 4) + lane] : make_uint4(0, 0, 0, 0);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            r[o + i] = value<DTYPE>(x, i);
            e[o + i] = value<HS_LOGITS_F32>(e4, i);
            w[o + i] = value<HS_LOGITS_F32>(w4, i);
          }
          continue;
        }
        r[o] = DTYPE == HS_LOGITS_F32
                   ? reinterpret_cast<const float *>(from)[l_at + 32 * o]
                   : __uint_as_float((uint32_t)reinterpret_cast<const unsigned short *>(from)[l_at + 32 * o] << 16);
        e[o] = es[32 * o];
        w[o] = HAS_Q ? qs[32 * o] : 0.f;
      }
#pragma unroll
      for (int o = 0; o < PER; o += 2) {
        ratio2(pack2(r[o], r[o + 1]), pack2(-w[o], -w[o + 1]), e[o], e[o + 1], nm, cc, ii, r[o], r[o + 1]);
        big = fmaxf(big, fmaxf(r[o], r[o + 1]));
      }
      const bool cut = v0 + UNIT > hi;             // (the places past hi: what they held)
      if (cut || (rr.barred >= v0 && rr.barred < v0 + UNIT)) {
        big = 0.f;
#pragma unroll
        for (int o = 0; o < PER; ++o) {
          const int32_t v = value_at(o);
          if (v >= hi || v == rr.barred) r[o] = 0.f;
          big = fmaxf(big, r[o]);
        }
      }
      __syncwarp();
      issue(v0 + DEPTH * WARPS * UNIT, place);
      place = place + 1 == DEPTH ? 0 : place + 1;
      ra.template group<PER>(r, big, value_at);
    }
    copy_wait<0>();
  } else {
    for (int32_t k0 = lo; k0 < hi; k0 += NB * NT) {
      float r[NB], e[NB], w[NB], big = 0.f;
#pragma unroll
      for (int u = 0; u < NB; ++u) {
        const int32_t v = k0 + u * NT + (int)threadIdx.x;
        r[u] = -INFINITY;
        e[u] = 1.f;
        w[u] = 0.f;
        if (v < hi) {
          r[u] = raw_logit_at<DTYPE>(row, v);
          e[u] = __ldcs(E + v);
          if (HAS_Q) w[u] = __ldcs(q + v);
        }
      }
#pragma unroll
      for (int u = 0; u < NB; u += 2) {
        ratio2(pack2(r[u], r[u + 1]), pack2(-w[u], -w[u + 1]), e[u], e[u + 1], nm, cc, ii, r[u], r[u + 1]);
        big = fmaxf(big, fmaxf(r[u], r[u + 1]));
      }
      const int32_t v0 = k0 + (int)threadIdx.x;
      if (rr.barred >= 0) {
#pragma unroll
        for (int u = 0; u < NB; ++u)
          if (v0 + u * NT == rr.barred) r[u] = 0.f;
        big = 0.f;
#pragma unroll
        for (int u = 0; u < NB; ++u) big = fmaxf(big, r[u]);
      }
      ra.template group<NB>(r, big, [&](int u) { return v0 + u * NT; });
    }
  }
  return ra;
}

// The race for every noise and logit. ratio2 gives 0 for a noise whose reciprocal
// is below the normal floats, and infinity for one above them and for a logit
// of +inf: a race whose winner is infinite, or one that a noise past E_MAX could
// have won (no ratio reaches SMALL), is run again here, over noise within
// [E_MIN, E_MAX] and logits as they count, each ratio times scale^2. Where both
// races are exact their ratios are the same bits.
constexpr float E_MIN = 0x1p-126f, E_MAX = 0x1p126f, SMALL = 0x1p-125f;
template <int DTYPE>
__device__ __noinline__ Race careful_race(const char *row, const float *q, const float *E, int32_t V, uint32_t rank,
                                          uint32_t log_n, const RaceRow rr, float scale) {
  Race ra = {0.f, INT32_MAX, 0.f};
  const int32_t lo = part_of(V, rank, log_n), hi = part_of(V, rank + 1, log_n);
#pragma unroll 1
  for (int32_t k = lo; k < hi; k += NT) {
    const int32_t v = k + (int)threadIdx.x;
    float r[1] = {0.f};
    if (v < hi && v != rr.barred) {
      const float w = fmaf(ex2((logit_at<DTYPE>(row, v) - rr.top) * rr.c), rr.inv, q ? -q[v] : 0.f);
      float f;
      asm("rcp.approx.ftz.f32 %0, %1;\n" : "=f"(f) : "f"(fminf(fmaxf(E[v], E_MIN), E_MAX)));
      r[0] = fmaxf((w * scale) * (f * scale), 0.f);
    }
    ra.template group<1>(r, r[0], [&](int) { return v; });
  }
  return ra;
}

template <int DTYPE, bool COMMIT>
__global__ void __launch_bounds__(NT, MIN_BLOCKS) k_verify_sample(const __grid_constant__ SampleArgs sa,
                                                                  const __grid_constant__ CommitArgs ca) {
  extern __shared__ uint4 ring_base[];
  __shared__ Shared sh;
  const uint32_t rank = cluster_rank(), n = cluster_size();
  if (n > 1) cluster_arrive();       // waited for before the first push: every block runs by then
  const int b = (int)(blockIdx.x / n);
  const int32_t d = sa.d, V = sa.V;
  const int tid = threadIdx.x;
  const int64_t row_bytes = (int64_t)V * (DTYPE == HS_LOGITS_F32 ? 4 : 2);
  const char *rows = reinterpret_cast<const char *>(sa.logits) + (int64_t)b * (d + 1) * row_bytes;

  // What decides is read once, by the first block, and pushed to the others
  // before the first exchange; this reading of the temperature only scales
  // the first rows' sums.
  static_assert(MAX_DRAFTS <= NT, "a thread per draft");
  int32_t x = -1;
  float x_logit = -INFINITY, x_bar = 0.f;
  const float t_read = __uint_as_float(once(sa.temperature + b));
  // within the normal floats: products with it are never 0 * inf
  auto scale_of = [](float t) { return fminf(fmaxf(LOG2E / (t > 0.f ? t : 1.f), FLT_MIN), FLT_MAX); };
  float c = scale_of(t_read);

  // Rows m0 .. m0 + G - 1 at a time, n / G blocks a row.
  const uint32_t log_n = 31 - __clz(n), log_g = sa.log_rows, G = 1u << log_g, per_row = n >> log_g;
  int turn = 0, m = 0;
  float top = -INFINITY, sum = 0.f, T = 1.f;
  uint32_t first = INT32_MAX;
  bool greedy = false, done = false;
  for (int m0 = 0; !done; m0 += (int)G) {
    const int mine = m0 + (int)(rank >> (log_n - log_g));
    const char *row = rows + (mine <= d ? mine : d) * row_bytes;
    const Slice<DTYPE> sl(row, mine <= d ? V : 0, rank & (per_row - 1), log_n - log_g);
    const Stat st = row_stat<DTYPE>(sl, row, c, ring_base + tid, [&]() {
      if (m0 != 0 || rank != 0 || tid >= d) return;
      const int64_t k = (int64_t)b * d + tid;
      x = (int32_t)once(sa.drafts + k);
      const bool ok = x >= 0 && x < V;         // any other token is refused
      if (!ok) {
        x = -1;
        if (sa.status) atomicOr(sa.status, HS_STATUS_INDEX);
      }
      x_logit = ok ? logit_once<DTYPE>(rows + tid * row_bytes, x) : -INFINITY;
      x_bar = __uint_as_float(once(sa.uniforms + k)) *
              (sa.probs && ok ? __uint_as_float(once(sa.probs + k * V + x)) : 1.f);
    });
    if (m0 == 0) {
      if (n > 1) cluster_wait();
      if (rank == 0) {
        for (uint32_t r = 0; r < n; ++r) {
          if (tid < d) {
            push(sh.draft + tid, r, (uint32_t)x);
            push(sh.draft_logit + tid, r, __float_as_uint(x_logit));
            push(sh.draft_bar + tid, r, __float_as_uint(x_bar));
          }
          if (tid == 0) push(&sh.temperature, r, __float_as_uint(t_read));
        }
      }
    }
    float tops = st.m;
    uint32_t sums = __float_as_uint(st.s);
    StatOp op{c};
    cluster_join(sh, tops, sums, rank, n, log_g, turn, op, [&]() {
      if (m0 != 0) return;
      // from here on by the pushed temperature, the join of all warps' sums too
      const float t = sh.temperature;
      greedy = !(t > 0.f);
      T = greedy ? 1.f : t;
      op.c = c = scale_of(t);
    });
    uint32_t firsts = INT32_MAX;
    if (greedy) {
      const float own = __shfl_sync(0xffffffffu, tops, (rank >> (log_n - log_g)) * (32 >> log_g));
      if (own != -INFINITY) firsts = (uint32_t)row_first<DTYPE>(sl, row, st, own);
      float unused = 0.f;
      cluster_join(sh, unused, firsts, rank, n, log_g, turn, MinOp{});
    }
    for (uint32_t g = 0; g < G && !done; ++g) {
      top = __shfl_sync(0xffffffffu, tops, g * (32 >> log_g));
      sum = __uint_as_float(__shfl_sync(0xffffffffu, sums, g * (32 >> log_g)));
      first = __shfl_sync(0xffffffffu, firsts, g * (32 >> log_g));
      const float lx = m < d ? sh.draft_logit[m] : -INFINITY;
      // (an empty row accepts nothing: lx is -inf too)
      const bool take = greedy ? m < d && first != INT32_MAX && sh.draft[m] == (int32_t)first
                               : lx != -INFINITY && sh.draft_bar[m] < ex2((lx - top) * c) / sum;
      if (take) {
        if (sa.logprob && rank == 0 && tid == 0)
          sa.logprob[(int64_t)b * (d + 1) + m] = (lx - top) / T - logf(sum);
        ++m;
      } else {
        done = true;
      }
    }
  }

  const char *row = rows + m * row_bytes;
  int32_t token = -1;
  if (greedy) {
    token = first == INT32_MAX ? -1 : (int32_t)first;
  } else if (top != -INFINITY) {
    const float inv = 1.f / sum;
    const float *E = sa.noise + (int64_t)b * V;
    const float *q = sa.probs && m < d ? sa.probs + ((int64_t)b * d + m) * V : nullptr;
    int32_t barred = !sa.probs && m < d ? sh.draft[m] : -1;   // a sure draft's own token
    float scale = 0.f;                                        // (0: the race proper)
    for (;;) {
      const RaceRow rr = {top, c, inv, barred};
      Race ra;
      if (scale > 0.f) {
        ra = careful_race<DTYPE>(row, q, E, V, rank, log_n, rr, scale);
      } else {
        switch (sa.rows) {
          case ROWS_ON_16:
            ra = q ? race<DTYPE, ROWS_ON_16, true>(row, q, E, V, rank, log_n, rr, ring_base)
                   : race<DTYPE, ROWS_ON_16, false>(row, q, E, V, rank, log_n, rr, ring_base);
            break;
          case ARRAYS_ON_16:
            ra = q ? race<DTYPE, ARRAYS_ON_16, true>(row, q, E, V, rank, log_n, rr, ring_base)
                   : race<DTYPE, ARRAYS_ON_16, false>(row, q, E, V, rank, log_n, rr, ring_base);
            break;
          default:
            ra = q ? race<DTYPE, ROWS_ANYWHERE, true>(row, q, E, V, rank, log_n, rr, ring_base)
                   : race<DTYPE, ROWS_ANYWHERE, false>(row, q, E, V, rank, log_n, rr, ring_base);
        }
      }
      cluster_join(sh, ra.best, ra.at, rank, n, 0, turn, BestOp{});
      if (scale == 0.f && ra.best == INFINITY) {
        scale = 1.f;
        continue;
      }
      if (scale < 2.f && ra.best < SMALL) {                   // (times 2^126: none vanishes)
        scale = 0x1p63f;
        continue;
      }
      if (ra.at != INT32_MAX) {
        token = (int32_t)ra.at;
        break;
      }
      if (!q && barred < 0) break;
      // nothing left of the target past the draft's probabilities (they are
      // equal, up to rounding): the target's own
      q = nullptr;
      barred = -1;
      scale = 0.f;
    }
  }

  if (rank == 0) {
    if (tid == 0) {
      sa.accept_len[b] = m;
      sa.next_token[b] = token;
      if (sa.logprob)
        sa.logprob[(int64_t)b * (d + 1) + m] =
            token < 0 ? -INFINITY : (logit_at<DTYPE>(row, token) - top) / T - logf(sum);
    }
    if (sa.logprob)
      for (int i = m + 1 + tid; i <= d; i += NT) sa.logprob[(int64_t)b * (d + 1) + i] = 0.f;
    if (COMMIT) commit_rows(b, m, ca);
  }
}

int check_sample(const void *logits, int32_t dtype, int32_t B, int32_t d, int32_t V,
                 const float *temperature, const int32_t *drafts, const float *probs,
                 const float *uniforms, const float *noise, const int32_t *accept_len,
                 const int32_t *next_token, const float *logprob, const uint32_t *status) {
  if (B < 1 || d < 0 || d > MAX_DRAFTS || V < 1 || V > 1 << 30)
    return hs_set_error(HS_ERR_INVALID_ARG, "bad sizes B=%d d=%d (0..%d) V=%d (1..2^30)", B, d,
                        MAX_DRAFTS, V);
  if (dtype != HS_LOGITS_F32 && dtype != HS_LOGITS_BF16)
    return hs_set_error(HS_ERR_INVALID_ARG, "logits_dtype %d", dtype);
  if (!logits || !temperature || (d > 0 && (!drafts || !uniforms)) || !noise || !accept_len || !next_token)
    return hs_set_error(HS_ERR_INVALID_ARG, "NULL argument");
  const uintptr_t elem = dtype == HS_LOGITS_F32 ? 4 : 2;
  if ((uintptr_t)logits % elem ||
      (((uintptr_t)temperature | (uintptr_t)drafts | (uintptr_t)probs | (uintptr_t)uniforms |
        (uintptr_t)noise | (uintptr_t)accept_len | (uintptr_t)next_token | (uintptr_t)logprob |
        (uintptr_t)status) & 3))
    return hs_set_error(HS_ERR_INVALID_ARG, "an array is not aligned to its elements");
  return HS_OK;
}

// Blocks per request and rows side by side.
//
// A cluster that takes its rows one after the other reads no row behind the
// refusal, but each row costs a few microseconds of latency (the first loads,
// the joins). So while all blocks run at once, up to four rows are taken side
// by side as long as one row of every request is less than 18 MB, some three
// microseconds of HBM (2 x 3 drafts, V = 1024: 6.5 us against 11 one by one; 33 x
// 5, V = 50257: 13.3 against 21; 96 x 3, V = 50257: 20.3 against 21.7 two by two;
// 64 x 7, V = 65000 f32, 16.6 MB: 30.9 against 33.1), else two (110 x 3, V =
// 129280: 36.7 us against 41.7 by fours). The blocks of a request double, to
// eight, while all blocks run at once and a part of a row keeps 2048 values, and
// to sixteen while each has an SM of its own (1 x 3, V = 129280: 9.5 us against
// 11.2). Not past that: 256 x 3, V = 129280 takes 70 us with one block, 84 with
// two, 77 with four.
int cluster_shape(int32_t B, int32_t d, int32_t V, int32_t elem, int *n, int *g) {
  int sms = 0;
  int rc = hs_sm_count(&sms);
  if (rc) return rc;
  const int64_t at_once = (int64_t)sms * MIN_BLOCKS;
  const int most = d >= 2 ? 4 : d + 1;           // rows side by side
  int k = 1;
  while (k < MAX_CLUSTER && (int64_t)B * 2 * k <= (k < 8 ? at_once : (int64_t)sms) &&
         (k < most || (int64_t)V * most / (2 * k) >= 2048))
    k *= 2;
  int r = (int64_t)B * k > at_once ? 1 : (int64_t)B * V * elem < 18000000 ? most : 2;
  if (r > most) r = most;
  if (r > k) r = k;
  *n = k;
  *g = r;
  return HS_OK;
}

template <bool COMMIT>
int launch(SampleArgs &sa, int32_t dtype, int32_t B, const CommitArgs &ca, cudaStream_t stream) {
  int n = 1, g = 1;
  int rc = cluster_shape(B, sa.d, sa.V, dtype == HS_LOGITS_F32 ? 4 : 2, &n, &g);
  if (rc) return rc;
  if ((int64_t)B * n > INT32_MAX) return hs_set_error(HS_ERR_UNSUPPORTED, "B too large");
  sa.log_rows = 31 - __builtin_clz((unsigned)g);
  const bool arrays = (((uintptr_t)sa.logits | (uintptr_t)sa.probs | (uintptr_t)sa.noise) & 15) == 0;
  sa.rows = !arrays ? ROWS_ANYWHERE : sa.V % (dtype == HS_LOGITS_F32 ? 4 : 8) == 0 ? ROWS_ON_16 : ARRAYS_ON_16;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(B * n));
  cfg.blockDim = dim3(NT);
  cfg.dynamicSmemBytes = RING_BYTES;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = n;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int dev = 0;
  HS_CUDA_TRY(cudaGetDevice(&dev));
  static std::atomic<bool> attr_done[64];
  if (dev >= 64 || !attr_done[dev]) {
    HS_CUDA_TRY(cudaFuncSetAttribute(k_verify_sample<HS_LOGITS_F32, COMMIT>,
                                     cudaFuncAttributeMaxDynamicSharedMemorySize, (int)RING_BYTES));
    HS_CUDA_TRY(cudaFuncSetAttribute(k_verify_sample<HS_LOGITS_BF16, COMMIT>,
                                     cudaFuncAttributeMaxDynamicSharedMemorySize, (int)RING_BYTES));
    // clusters of 16 blocks
    HS_CUDA_TRY(cudaFuncSetAttribute(k_verify_sample<HS_LOGITS_F32, COMMIT>,
                                     cudaFuncAttributeNonPortableClusterSizeAllowed, 1));
    HS_CUDA_TRY(cudaFuncSetAttribute(k_verify_sample<HS_LOGITS_BF16, COMMIT>,
                                     cudaFuncAttributeNonPortableClusterSizeAllowed, 1));
    if (dev < 64) attr_done[dev] = true;
  }
  if (dtype == HS_LOGITS_F32)
    HS_CUDA_TRY(cudaLaunchKernelEx(&cfg, k_verify_sample<HS_LOGITS_F32, COMMIT>, sa, ca));
  else
    HS_CUDA_TRY(cudaLaunchKernelEx(&cfg, k_verify_sample<HS_LOGITS_BF16, COMMIT>, sa, ca));
  HS_LAUNCH_CHECK("k_verify_sample");
  return HS_OK;
}

}  // namespace

extern "C" int hs_verify_sample(const void *logits, int32_t logits_dtype, int32_t B, int32_t d,
                                int32_t V, const float *temperature, const int32_t *draft_tokens,
                                const float *draft_probs, const float *uniforms, const float *noise,
                                int32_t *accept_len, int32_t *next_token, float *logprob,
                                uint32_t *status, hs_stream_t stream) {
  int rc = check_sample(logits, logits_dtype, B, d, V, temperature, draft_tokens, draft_probs,
                        uniforms, noise, accept_len, next_token, logprob, status);
  if (rc) return rc;
  SampleArgs sa = {logits,   d,     V,          temperature, draft_tokens, draft_probs,
                         uniforms, noise, accept_len, next_token,  logprob,      status, 0, ROWS_ANYWHERE};
  return launch<false>(sa, logits_dtype, B, CommitArgs{}, stream);
}

extern "C" int hs_verify_sample_finalize(hs_buffer *buf, const void *logits, int32_t logits_dtype,
                                         int32_t B, int32_t d, int32_t V, const float *temperature,
                                         const int32_t *draft_tokens, const float *draft_probs,
                                         const float *uniforms, const float *noise,
                                         const void *step_kv, const int32_t *req_ids, int32_t *kv_len,
                                         int32_t *accept_len, int32_t *next_token, float *logprob,
                                         hs_stream_t stream) {
  int rc = hs_check_buffer(buf);
  if (rc) return rc;
  rc = check_sample(logits, logits_dtype, B, d, V, temperature, draft_tokens, draft_probs, uniforms,
                    noise, accept_len, next_token, logprob, nullptr);
  if (rc) return rc;
  if (B > buf->max_reqs || d + 1 > buf->n_step)
    return hs_set_error(HS_ERR_INVALID_ARG, "bad sizes B=%d (1..%d) d=%d (d+1<=%d)", B, buf->max_reqs,
                        d, buf->n_step);
  if (!step_kv || !kv_len) return hs_set_error(HS_ERR_INVALID_ARG, "NULL argument");
  if (((uintptr_t)step_kv & 15) || (((uintptr_t)req_ids | (uintptr_t)kv_len) & 3))
    return hs_set_error(HS_ERR_INVALID_ARG, "step_kv must be 16-byte aligned, req_ids and kv_len to 4");
  // A commit is told from a repeated one by the host's clock, which a
  // replayed graph does not advance: its second run would commit nothing.
  cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
  HS_CUDA_TRY(cudaStreamIsCapturing(stream, &cap));
  if (cap != cudaStreamCaptureStatusNone)
    return hs_set_error(HS_ERR_UNSUPPORTED, "hs_verify_sample_finalize cannot be captured in a graph");
  buf->clock += 1;
  SampleArgs sa = {logits,   d,     V,          temperature, draft_tokens, draft_probs,
                         uniforms, noise, accept_len, next_token,  logprob,      buf->status, 0, ROWS_ANYWHERE};
  return launch<true>(sa, logits_dtype, B, commit_args(buf, d, step_kv, req_ids, kv_len), stream);
}

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
//   of additions cannot move the answer.
//
// One cluster of 1 to 8 blocks per request takes the request's rows one after
// the other and stops at the first refusal: the logits of later inputs, and
// the draft probabilities and noise of every row but the last one, are never
// read. HBM bounds it: each logits row is streamed once for (M, S), and the
// row that yields the token a second time, beside q and E, mostly from L2.
// M and S come in one pass (a thread rescales its sum when a batch of its
// values brings a new maximum). The sums are f32, each of a thread's few
// hundred terms, then joined as a tree in a fixed order: results do not
// depend on scheduling.
//
// The blocks of a cluster exchange (M, S) and the race's winner through
// distributed shared memory, each pulling all blocks' figures and joining
// them in the same order; the request's drafts, numbers and temperature are
// read once by the first block and pulled by the others. So every block takes
// the same decisions from the same bits, and the barriers match even if a
// caller overwrites the inputs during the call.

#include <float.h>

#include "hs_commit.cuh"

namespace {

constexpr int NT = 512;             // threads per block
constexpr int NB = 8;               // 16-byte loads of a thread in flight
constexpr int MAX_CLUSTER = 8;
constexpr int MAX_DRAFTS = 255;
constexpr float LOG2E = 1.4426950408889634f;

struct SampleArgs {
  const void *logits;
  int32_t d, V;
  const float *temperature;
  const int32_t *drafts;
  const float *probs, *uniforms, *noise;
  int32_t *accept_len, *next_token;
  float *logprob;
  uint32_t *status;
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
// every thread of the cluster: writes before it are seen by reads after it
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;\n" ::
                   : "memory");
}
// a word of block `rank`'s shared memory, at the place p has in this block's
__device__ __forceinline__ uint32_t pull(const void *p, uint32_t rank) {
  uint32_t a = (uint32_t)__cvta_generic_to_shared(p), v;
  asm volatile("mapa.shared::cluster.u32 %0, %0, %1;\n" : "+r"(a) : "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];\n" : "=r"(v) : "r"(a) : "memory");
  return v;
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

template <int DTYPE>
__device__ __forceinline__ float logit_at(const void *row, int64_t i) {
  if (DTYPE == HS_LOGITS_F32) return clean<DTYPE>(__ldg(reinterpret_cast<const float *>(row) + i));
  const uint32_t u = __ldg(reinterpret_cast<const unsigned short *>(row) + i);
  return clean<DTYPE>(__uint_as_float(u << 16));
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

// One slice of a row: its 16-byte vectors [lo, hi) by all threads of the
// block, batch k of a thread being vectors k .. k + (NB - 1) NT.
template <int DTYPE>
struct Slice {
  const uint4 *body;
  int32_t lo, hi, head, V;     // `head` unaligned values before the body
  static constexpr int PER = DTYPE == HS_LOGITS_F32 ? 4 : 8;

  __device__ __forceinline__ Slice(const char *row, int32_t V_, uint32_t rank, uint32_t n) {
    constexpr int elem = DTYPE == HS_LOGITS_F32 ? 4 : 2;
    V = V_;
    head = (int)(((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15) / elem);
    if (head > V) head = V;
    const int32_t vecs = (V - head) / PER;
    body = reinterpret_cast<const uint4 *>(row + (int64_t)head * elem);
    lo = (int32_t)((int64_t)vecs * rank / n);
    hi = (int32_t)((int64_t)vecs * (rank + 1) / n);
    if (rank == 0) rest = head + (V - head - vecs * PER); else rest = 0;
    tail0 = head + vecs * PER;
  }
  // the values outside the body (fewer than 2 PER), all the first block's
  int32_t rest, tail0;
  __device__ __forceinline__ int32_t rest_index(int32_t j) const {
    return j < head ? j : tail0 + (j - head);
  }
  __device__ __forceinline__ void load(int32_t k, uint4 (&w)[NB]) const {
    const uint32_t none = DTYPE == HS_LOGITS_F32 ? 0xff800000u : 0xff80ff80u;
#pragma unroll
    for (int u = 0; u < NB; ++u)
      w[u] = k + u * NT < hi ? __ldg(body + k + u * NT) : make_uint4(none, none, none, none);
#pragma unroll
    for (int u = 0; u < NB; ++u) {
      uint32_t *x = reinterpret_cast<uint32_t *>(&w[u]);
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
    }
  }
};

template <int DTYPE>
__device__ __forceinline__ float batch_max(const uint4 (&w)[NB]) {
  if (DTYPE == HS_LOGITS_F32) {
    float t = -INFINITY;
#pragma unroll
    for (int u = 0; u < NB; ++u)
      t = fmaxf(t, fmaxf(fmaxf(__uint_as_float(w[u].x), __uint_as_float(w[u].y)),
                         fmaxf(__uint_as_float(w[u].z), __uint_as_float(w[u].w))));
    return t;
  }
  const __nv_bfloat162 *h = reinterpret_cast<const __nv_bfloat162 *>(w);
  __nv_bfloat162 t = h[0];
#pragma unroll
  for (int u = 1; u < 4 * NB; ++u) t = __hmax2(t, h[u]);
  return fmaxf(__low2float(t), __high2float(t));
}

template <int DTYPE>
__device__ __forceinline__ Stat row_stat(const Slice<DTYPE> &sl, const void *row, float c) {
  Stat st = {-INFINITY, 0.f, -1};
  const uint64_t cc = pack2(c, c);
  for (int32_t k = sl.lo + (int)threadIdx.x; k < sl.hi; k += NB * NT) {
    uint4 w[NB];
    sl.load(k, w);
    const float t = batch_max<DTYPE>(w);
    if (t > st.m) {
      st.s *= ex2((st.m - t) * c);
      st.m = t;
      st.at = k;
    }
    if (st.m == -INFINITY) continue;
    const uint64_t nm = pack2(-st.m, -st.m);
    uint64_t acc[4] = {0, 0, 0, 0};            // eight partial sums
#pragma unroll
    for (int u = 0; u < NB; ++u) {
      const uint32_t x[4] = {w[u].x, w[u].y, w[u].z, w[u].w};
#pragma unroll
      for (int j = 0; j < 4; j += DTYPE == HS_LOGITS_F32 ? 2 : 1) {
        const uint64_t v = DTYPE == HS_LOGITS_F32
                               ? pack2(__uint_as_float(x[j]), __uint_as_float(x[j + 1]))
                               : pack2(__uint_as_float(x[j] << 16), __uint_as_float(x[j] & 0xFFFF0000u));
        float a, b;
        unpack2(mul2(add2(v, nm), cc), a, b);
        acc[j] = add2(acc[j], pack2(ex2(a), ex2(b)));
      }
    }
    float a, b;
    unpack2(add2(add2(acc[0], acc[1]), add2(acc[2], acc[3])), a, b);
    st.s += a + b;
  }
  for (int32_t j = threadIdx.x; j < sl.rest; j += NT) {
    const float x = logit_at<DTYPE>(row, sl.rest_index(j));
    join(st.m, st.s, x, x == -INFINITY ? 0.f : 1.f, c);
  }
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
    uint4 w[NB];
    sl.load(st.at, w);
#pragma unroll
    for (int u = 0; u < NB; ++u) {
      const uint32_t x[4] = {w[u].x, w[u].y, w[u].z, w[u].w};
      const int32_t i0 = sl.head + (st.at + u * NT) * Slice<DTYPE>::PER;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (DTYPE == HS_LOGITS_F32) {
          if (__uint_as_float(x[j]) == top) best = min(best, i0 + j);
        } else {
          if (__uint_as_float(x[j] << 16) == top) best = min(best, i0 + 2 * j);
          if (__uint_as_float(x[j] & 0xFFFF0000u) == top) best = min(best, i0 + 2 * j + 1);
        }
      }
    }
  }
  for (int32_t j = threadIdx.x; j < sl.rest; j += NT)
    if (logit_at<DTYPE>(row, sl.rest_index(j)) == top) best = min(best, sl.rest_index(j));
  return best;
}

struct Shared {
  // of the first block, pulled by the others at the start
  float temperature;
  float draft_logit[MAX_DRAFTS], draft_bar[MAX_DRAFTS];     // l_i(x_i); u_i q_i(x_i)
  int32_t draft[MAX_DRAFTS];
  // per warp, per block (two alternating places) and per cluster
  float wa[NT / 32];
  uint32_t wb[NT / 32];
  uint32_t part[2][2];
  float a;
  uint32_t b;
};

// Joins a pair of words of every thread of the cluster: within the warps and
// the block by `op` on (float, word), over the blocks in rank order. Every
// thread gets the result. `turn` alternates between the two exchange places;
// the barrier inside keeps a place from being written while it is read.
template <typename Op>
__device__ __forceinline__ void cluster_join(Shared &sh, float &a, uint32_t &b, uint32_t n, int &turn,
                                             const Op &op) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    const float oa = __shfl_xor_sync(0xffffffffu, a, o);
    const uint32_t ob = __shfl_xor_sync(0xffffffffu, b, o);
    op(a, b, oa, ob);
  }
  if (lane == 0) {
    sh.wa[warp] = a;
    sh.wb[warp] = b;
  }
  __syncthreads();
  if (warp == 0) {
    a = sh.wa[lane & (NT / 32 - 1)];
    b = sh.wb[lane & (NT / 32 - 1)];
#pragma unroll
    for (int o = NT / 64; o; o >>= 1) {
      const float oa = __shfl_xor_sync(0xffffffffu, a, o);
      const uint32_t ob = __shfl_xor_sync(0xffffffffu, b, o);
      op(a, b, oa, ob);
    }
    if (lane == 0) {
      sh.part[turn][0] = __float_as_uint(a);
      sh.part[turn][1] = b;
      sh.a = a;
      sh.b = b;
    }
  }
  if (n == 1) {
    __syncthreads();
  } else {
    cluster_sync();
    if (warp == 0) {
      const uint32_t from = (uint32_t)lane < n ? lane : 0;
      const uint32_t pa = pull(&sh.part[turn][0], from), pb = pull(&sh.part[turn][1], from);
      a = __uint_as_float(__shfl_sync(0xffffffffu, pa, 0));
      b = __shfl_sync(0xffffffffu, pb, 0);
      for (uint32_t r = 1; r < n; ++r)
        op(a, b, __uint_as_float(__shfl_sync(0xffffffffu, pa, r)), __shfl_sync(0xffffffffu, pb, r));
      if (lane == 0) {
        sh.a = a;
        sh.b = b;
      }
    }
    __syncthreads();
  }
  a = sh.a;
  b = sh.b;
  turn ^= 1;
  __syncthreads();      // wa, wb, a and b may be written again
}

template <int DTYPE, bool COMMIT>
__global__ void __launch_bounds__(NT) k_verify_sample(const __grid_constant__ SampleArgs sa,
                                                      const __grid_constant__ CommitArgs ca) {
  __shared__ Shared sh;
  const uint32_t rank = cluster_rank(), n = cluster_size();
  const int b = (int)(blockIdx.x / n);
  const int32_t d = sa.d, V = sa.V;
  const int tid = threadIdx.x;
  const int64_t row_bytes = (int64_t)V * (DTYPE == HS_LOGITS_F32 ? 4 : 2);
  const char *rows = reinterpret_cast<const char *>(sa.logits) + (int64_t)b * (d + 1) * row_bytes;

  if (rank == 0) {
    bool bad = false;
    for (int i = tid; i < d; i += NT) {
      const int64_t k = (int64_t)b * d + i;
      const int32_t x = __ldg(sa.drafts + k);
      const bool ok = x >= 0 && x < V;         // any other token is refused
      bad |= !ok;
      sh.draft[i] = ok ? x : -1;
      sh.draft_logit[i] = ok ? logit_at<DTYPE>(rows + i * row_bytes, x) : -INFINITY;
      sh.draft_bar[i] = __ldg(sa.uniforms + k) * (sa.probs && ok ? __ldg(sa.probs + k * V + x) : 1.f);
    }
    if (tid == 0) sh.temperature = __ldg(sa.temperature + b);
    if (bad && sa.status) atomicOr(sa.status, HS_STATUS_INDEX);
  }
  if (n > 1) {
    cluster_sync();
    if (rank != 0) {
      for (int i = tid; i < d; i += NT) {
        sh.draft[i] = (int32_t)pull(&sh.draft[i], 0);
        sh.draft_logit[i] = __uint_as_float(pull(&sh.draft_logit[i], 0));
        sh.draft_bar[i] = __uint_as_float(pull(&sh.draft_bar[i], 0));
      }
      if (tid == 0) sh.temperature = __uint_as_float(pull(&sh.temperature, 0));
    }
  }
  __syncthreads();
  const bool greedy = !(sh.temperature > 0.f);
  const float T = greedy ? 1.f : sh.temperature;
  // within the normal floats: products with it are never 0 * inf
  const float c = fminf(fmaxf(LOG2E / T, FLT_MIN), FLT_MAX);

  int turn = 0, m = 0;
  float top, sum;
  int32_t token = -1;
  for (;; ++m) {
    const char *row = rows + m * row_bytes;
    const Slice<DTYPE> sl(row, V, rank, n);
    const Stat st = row_stat<DTYPE>(sl, row, c);
    top = st.m;
    uint32_t s_bits = __float_as_uint(st.s);
    cluster_join(sh, top, s_bits, n, turn, [c](float &am, uint32_t &as, float bm, uint32_t bs) {
      float s = __uint_as_float(as);
      join(am, s, bm, __uint_as_float(bs), c);
      as = __float_as_uint(s);
    });
    sum = __uint_as_float(s_bits);
    if (greedy) {
      float unused = 0.f;
      uint32_t first = top == -INFINITY ? INT32_MAX : (uint32_t)row_first<DTYPE>(sl, row, st, top);
      cluster_join(sh, unused, first, n, turn,
                   [](float &, uint32_t &ai, float, uint32_t bi) { ai = min(ai, bi); });
      token = first == INT32_MAX ? -1 : (int32_t)first;
    }
    if (m == d) break;
    const float lx = sh.draft_logit[m];
    // an empty row (top = -inf) accepts nothing
    bool take;
    if (greedy)
      take = token >= 0 && sh.draft[m] == token;
    else
      take = lx != -INFINITY && sh.draft_bar[m] < ex2((lx - top) * c) / sum;
    if (!take) break;
    if (sa.logprob && rank == 0 && tid == 0)
      sa.logprob[(int64_t)b * (d + 1) + m] = (lx - top) / T - logf(sum);
  }

  const char *row = rows + m * row_bytes;
  if (!greedy && top != -INFINITY) {
    const float inv = 1.f / sum;
    const float *E = sa.noise + (int64_t)b * V;
    const float *q = sa.probs && m < d ? sa.probs + ((int64_t)b * d + m) * V : nullptr;
    int32_t barred = !sa.probs && m < d ? sh.draft[m] : -1;   // a sure draft's own token
    const int32_t lo = (int32_t)((int64_t)V * rank / n), hi = (int32_t)((int64_t)V * (rank + 1) / n);
    uint32_t winner;
    for (int again = 0; again < 2; ++again) {
      float best = -1.f;
      winner = INT32_MAX;
      for (int32_t v0 = lo + tid; v0 < hi; v0 += NB * NT) {
        float x[NB], e[NB], w[NB];
#pragma unroll
        for (int u = 0; u < NB; ++u) {
          const int32_t v = v0 + u * NT;
          x[u] = -INFINITY;
          e[u] = 1.f;
          w[u] = 0.f;
          if (v < hi) {
            x[u] = logit_at<DTYPE>(row, v);
            e[u] = __ldcs(E + v);
            if (q) w[u] = __ldcs(q + v);
          }
        }
#pragma unroll
        for (int u = 0; u < NB; ++u) {
          const int32_t v = v0 + u * NT;
          const float p = ex2((x[u] - top) * c) * inv - w[u];
          const float r = p / e[u];
          if (p > 0.f && v != barred && r > best) {    // a thread's indices ascend: the lowest stays
            best = r;
            winner = (uint32_t)v;
          }
        }
      }
      cluster_join(sh, best, winner, n, turn, [](float &av, uint32_t &ai, float bv, uint32_t bi) {
        if (bv > av || (bv == av && bi < ai)) {
          av = bv;
          ai = bi;
        }
      });
      // nothing left of the target past the draft's probabilities (they are
      // equal, up to rounding): the target's own
      if (winner != INT32_MAX || (!q && barred < 0)) break;
      q = nullptr;
      barred = -1;
    }
    token = winner == INT32_MAX ? -1 : (int32_t)winner;
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
  if (n > 1) cluster_sync();      // no block leaves while another may read its shared memory
}

int check_sample(const void *logits, int32_t dtype, int32_t B, int32_t d, int32_t V,
                 const float *temperature, const int32_t *drafts, const float *probs,
                 const float *uniforms, const float *noise, const int32_t *accept_len,
                 const int32_t *next_token) {
  if (B < 1 || d < 0 || d > MAX_DRAFTS || V < 1 || V > 1 << 30)
    return hs_set_error(HS_ERR_INVALID_ARG, "bad sizes B=%d d=%d (0..%d) V=%d (1..2^30)", B, d,
                        MAX_DRAFTS, V);
  if (dtype != HS_LOGITS_F32 && dtype != HS_LOGITS_BF16)
    return hs_set_error(HS_ERR_INVALID_ARG, "logits_dtype %d", dtype);
  if (!logits || !temperature || (d > 0 && (!drafts || !uniforms)) || !noise || !accept_len || !next_token)
    return hs_set_error(HS_ERR_INVALID_ARG, "NULL argument");
  const uintptr_t elem = dtype == HS_LOGITS_F32 ? 4 : 2;
  if ((uintptr_t)logits % elem || (((uintptr_t)temperature | (uintptr_t)probs | (uintptr_t)uniforms |
                                    (uintptr_t)noise) & 3))
    return hs_set_error(HS_ERR_INVALID_ARG, "an array is not aligned to its elements");
  return HS_OK;
}

// Blocks per request: enough to give every SM one, while a block's part of a
// row stays at least 2048 values.
int cluster_blocks(int32_t B, int32_t V, int *n) {
  int dev = 0, sms = 0;
  HS_CUDA_TRY(cudaGetDevice(&dev));
  HS_CUDA_TRY(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev));
  int k = 1;
  while (k < MAX_CLUSTER && (int64_t)B * k < sms && V / (2 * k) >= 2048) k *= 2;
  *n = k;
  return HS_OK;
}

template <bool COMMIT>
int launch(const SampleArgs &sa, int32_t dtype, int32_t B, const CommitArgs &ca, cudaStream_t stream) {
  int n = 1;
  int rc = cluster_blocks(B, sa.V, &n);
  if (rc) return rc;
  if ((int64_t)B * n > INT32_MAX) return hs_set_error(HS_ERR_UNSUPPORTED, "B too large");
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(B * n));
  cfg.blockDim = dim3(NT);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = n;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
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
                        uniforms, noise, accept_len, next_token);
  if (rc) return rc;
  const SampleArgs sa = {logits,   d,     V,          temperature, draft_tokens, draft_probs,
                         uniforms, noise, accept_len, next_token,  logprob,      status};
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
                    noise, accept_len, next_token);
  if (rc) return rc;
  if (B > buf->max_reqs || d + 1 > buf->n_step)
    return hs_set_error(HS_ERR_INVALID_ARG, "bad sizes B=%d (1..%d) d=%d (d+1<=%d)", B, buf->max_reqs,
                        d, buf->n_step);
  if (!step_kv || !kv_len) return hs_set_error(HS_ERR_INVALID_ARG, "NULL argument");
  if ((uintptr_t)step_kv & 15)
    return hs_set_error(HS_ERR_INVALID_ARG, "step_kv must be 16-byte aligned");
  // A commit is told from a repeated one by the host's clock, which a
  // replayed graph does not advance: its second run would commit nothing.
  cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
  HS_CUDA_TRY(cudaStreamIsCapturing(stream, &cap));
  if (cap != cudaStreamCaptureStatusNone)
    return hs_set_error(HS_ERR_UNSUPPORTED, "hs_verify_sample_finalize cannot be captured in a graph");
  buf->clock += 1;
  const SampleArgs sa = {logits,   d,     V,          temperature, draft_tokens, draft_probs,
                         uniforms, noise, accept_len, next_token,  logprob,      buf->status};
  return launch<true>(sa, logits_dtype, B, commit_args(buf, d, step_kv, req_ids, kv_len), stream);
}

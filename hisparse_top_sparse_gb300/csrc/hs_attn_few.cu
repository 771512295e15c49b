// a6 over a q8 cache for up to 16 heads (a query's heads divided over several
// devices, or a small model): the formulas of hs_attn.cu, another shape.
//
// With 128 heads a row's products are what k_attn_pair is built around; with 16
// they are an eighth, HBM's 656 bytes a key stay, and a cluster that holds two
// SMs for a row waits for itself. Here a block of eight warps takes a row (or a
// part of its keys), two blocks an SM. Per tile of 32 keys:
//   * warp w takes dims [64 w, 64 w + 64) of every key: its lanes read 16 codes
//     of a key each (lane 4 k + j: key k of eight, codes 16 j ..), decoded once
//     into registers that are at the same time the B operand of Q K^T (mma.sync
//     m16n8k16; the order of the dims inside a contraction is free, Q's is the
//     same) and, transposed eight by eight by movmatrix, that of P V. Nothing
//     decoded goes through shared memory;
//   * the eight partial S (16 heads x 32 keys), and two of the rope dims, meet
//     in shared memory; warp w adds those of heads 2 w and 2 w + 1, takes their
//     maximum and sum (f32; 16 lanes a head) and writes P (bf16, the values'
//     type, as in k_attn_pair: mma.sync takes one type). A head's reference moves only when a score passes it by more
//     than 30 (of the exponent of two), so P stays below 2^30;
//   * each warp scales its 64 dims of O (f32 registers) when a reference moved
//     and adds P V.
// Raw rows come by cp.async, three tiles in flight, in places of 704 bytes (of
// 656 used), which spreads a warp's reads over the banks.
//
// Measured, 16 heads (k_attn_pair, its heads padded to 128, in brackets): 8 rows
// of 64 keys 5.0 us (7.3), 300 rows of one key 5.0 (31), 256 rows of 300 keys 24
// (52), 128 rows of 2048 keys 67 (90), 512 rows 236 (312). What bounds the long
// ones is sixteen warps an SM, each a chain of a tile's reading, decoding,
// products and meetings: an instruction issues on 40 % of the cycles, no pipe is
// busy for half of them, and fewer instructions is what has helped (sums two at
// a time, the keys' validity from the copying warp: 74 before). Tried: sixteen
// warps of 32 dims 101 us on 128 rows (twice the partial sums, 64 registers);
// rows by one bulk copy each 92; two tiles in flight 81, four 76; the maximum
// of every tile 76 (of 74).
//
// tcgen05 would want 128 rows of something: heads padded eightfold, or keys and
// dims in that place, and then every decoded tile through shared memory;
// mma.sync needs neither.

#include <atomic>
#include <math.h>

#include "hs_q8.cuh"

namespace {

constexpr int NT = 256, WARPS = NT / 32;
constexpr int HEADS = HS_ATTN_FEW_HEADS;       // a matrix instruction's rows
constexpr int KEYS = 32;                       // keys of a tile
constexpr int STAGES = 3;                      // tiles of raw rows on their way
constexpr int ROW_STRIDE = 704;
constexpr int STAGE_BYTES = KEYS * ROW_STRIDE;
constexpr int PARTIALS = WARPS + 2;            // 512 dims by warps, the rope dims in halves
constexpr int S_STRIDE = 40;                   // floats from head to head
constexpr int P_STRIDE = 40;                   // bf16 values from head to head
constexpr int S_OFF = STAGES * STAGE_BYTES;
constexpr int P_OFF = S_OFF + PARTIALS * HEADS * S_STRIDE * 4;
constexpr int ALPHA_OFF = P_OFF + HEADS * P_STRIDE * 2;
constexpr float REF_SLACK = 30.f;
// which keys have a row: a byte for each warp's four, of STAGES + 1 tiles (a
// tile's bits are read after the place of its raw rows has been given away)
constexpr int VALID_OFF = ALPHA_OFF + HEADS * 4, VALID_TILES = STAGES + 1;
constexpr int SMEM = VALID_OFF + VALID_TILES * WARPS;
static_assert(HEADS == 16 && 2 * WARPS == HEADS && HS_VALUE_DIM == 64 * WARPS, "layout");
static_assert(2 * (SMEM + 1024) <= 228 * 1024, "two blocks on an SM");

struct FewArgs {
  const __nv_bfloat16 *q;
  const char *kv;
  int64_t n_kv;
  const int32_t *idx;
  int32_t R, H, K, n, keys;         // n parts of `keys` keys a row
  float scale_log2;
  __nv_bfloat16 *out;
  float *lse, *part_o, *part_lse;
};

__device__ __forceinline__ uint32_t smem_addr(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void cp16(uint32_t dst, const void *src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}
// d (16 x 8, f32) += a (16 x 16) b (16 x 8)
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transposed(uint32_t a) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(d) : "r"(a));
  return d;
}
// two f32 sums
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  asm("add.rn.f32x2 %0, %0, %1;\n" : "+l"(a) : "l"(b));
  return a;
}
__device__ __forceinline__ uint32_t pack(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&v);
}

__global__ void __launch_bounds__(NT, 2) k_attn_few(const __grid_constant__ FewArgs a) {
  extern __shared__ __align__(16) unsigned char sm[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, j = lane & 3;           // a fragment's row / column of four
  const int part = (int)(blockIdx.x % (unsigned)a.n), r = (int)(blockIdx.x / (unsigned)a.n);
  const int K = min(a.keys, a.K - part * a.keys), T = (K + KEYS - 1) / KEYS;
  const int32_t *idx = a.idx + (int64_t)r * a.K + (int64_t)part * a.keys;
  // a programmatic dependent launch (its inputs may be written until here, so
  // none is read by the non-coherent path)
  asm volatile("griddepcontrol.wait;\n" ::: "memory");

  // (volatile, so that it is loaded here, a tile before its use, and compared
  // only there: the compiler would load it where it is used)
  auto index = [&](int t, int key) -> int32_t {
    const int k = t * KEYS + key;
    int32_t i = -1;
    if (k < K) asm volatile("ld.global.b32 %0, [%1];\n" : "=r"(i) : "l"(idx + k));
    return i;
  };
  // warp w copies keys 4 w .. 4 w + 3 of a tile; lane k < 4 holds the index of the
  // k-th, read a turn before
  int32_t id = index(0, 4 * warp + j);
  // (a copy of no bytes has an address all the same: row 0, of an empty cache q)
  const char *kv = (a.n_kv > 0 ? a.kv : reinterpret_cast<const char *>(a.q)) + 16 * lane;
  auto copy = [&](int t, int stage) {
    if (t < T) {
      const uint32_t to = smem_addr(sm) + stage * STAGE_BYTES + 4 * warp * ROW_STRIDE + 16 * lane;
      const bool valid = id >= 0 && id < a.n_kv;
      const uint32_t have = __ballot_sync(0xffffffffu, valid);
      if (lane == 0) sm[VALID_OFF + (t % VALID_TILES) * WARPS + warp] = have & 15u;
      if (!valid) id = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const char *row = kv + (int64_t)__shfl_sync(0xffffffffu, id, k) * HS_Q8_ROW_BYTES;
        const bool v = (have >> k) & 1u;
        cp16(to + k * ROW_STRIDE, row, v);
        if (lane < HS_Q8_ROW_BYTES / 16 - 32) cp16(to + k * ROW_STRIDE + 512, row + 512, v);
      }
      id = index(t + 1, 4 * warp + j);
    }
    asm volatile("cp.async.commit_group;\n" ::: "memory");
  };
#pragma unroll 1
  for (int t = 0; t < STAGES; ++t) copy(t, t);

  // Q of the warp's 64 dims (four contractions of 16) and of the rope dims
  // [16 j + 8 half, + 8) of every column (two): heads g and g + 8
  uint32_t qa[4][4], qr[2][4];
  const int half = warp >> 2;
#pragma unroll
  for (int hh = 0; hh < 2; ++hh) {
    uint4 w0 = make_uint4(0, 0, 0, 0), w1 = w0, w2 = w0;
    if (g + 8 * hh < a.H) {
      const __nv_bfloat16 *row = a.q + ((int64_t)r * a.H + g + 8 * hh) * HS_LATENT_DIM;
      w0 = *reinterpret_cast<const uint4 *>(row + 64 * warp + 16 * j);
      w1 = *reinterpret_cast<const uint4 *>(row + 64 * warp + 16 * j + 8);
      w2 = *reinterpret_cast<const uint4 *>(row + HS_VALUE_DIM + 16 * j + 8 * half);
    }
    qa[0][hh] = w0.x, qa[0][2 + hh] = w0.y, qa[1][hh] = w0.z, qa[1][2 + hh] = w0.w;
    qa[2][hh] = w1.x, qa[2][2 + hh] = w1.y, qa[3][hh] = w1.z, qa[3][2 + hh] = w1.w;
    qr[0][hh] = w2.x, qr[0][2 + hh] = w2.y, qr[1][hh] = w2.z, qr[1][2 + hh] = w2.w;
  }

  // O of heads g and g + 8: o[s][i] columns 2 j, 2 j + 1 are dims 16 j + 4 s + 2 i, + 1
  float o[4][2][4];
#pragma unroll
  for (int k = 0; k < 32; ++k) o[k >> 3][(k >> 2) & 1][k & 3] = 0.f;
  float *s_part = reinterpret_cast<float *>(sm + S_OFF);
  float *s_alpha = reinterpret_cast<float *>(sm + ALPHA_OFF);
  // softmax: this lane's head and its keys 2 c, 2 c + 1 of a tile
  const int head = 2 * warp + (lane >> 4), c = lane & 15;
  float m = -INFINITY, l = 0.f;

  asm volatile("cp.async.wait_group %0;\n" ::"n"(STAGES - 1) : "memory");
  __syncthreads();
  for (int t = 0, stage = 0; t < T; ++t) {
    const unsigned char *raw = sm + stage * STAGE_BYTES;
    uint32_t kf[4][4][2];
    uint4 code[4];
    uint32_t byte[4];
#pragma unroll
    for (int nt = 0; nt < 4; ++nt) {
      const unsigned char *row = raw + (8 * nt + g) * ROW_STRIDE;
      code[nt] = *reinterpret_cast<const uint4 *>(row + 64 * warp + 16 * j);
      byte[nt] = row[Q8_SCALE_OFF + 2 * warp + (j >> 1)];
    }
#pragma unroll
    for (int nt = 0; nt < 4; ++nt) {
      const uint4 w = code[nt];
      const uint64_t sc = q8_scale2(byte[nt]);
      const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
      float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint2 d = q8_decode4_bf16(ws[k], sc);
        kf[nt][k][0] = d.x;
        kf[nt][k][1] = d.y;
        mma(s, qa[k][0], qa[k][1], qa[k][2], qa[k][3], d.x, d.y);
      }
      float *to = s_part + (warp * HEADS + g) * S_STRIDE + 8 * nt + 2 * j;
      *reinterpret_cast<float2 *>(to) = make_float2(s[0], s[1]);
      *reinterpret_cast<float2 *>(to + 8 * S_STRIDE) = make_float2(s[2], s[3]);
    }
    {
      // the rope dims of eight keys, half of each row's
      const int nt = warp & 3;
      const uint4 w = *reinterpret_cast<const uint4 *>(raw + (8 * nt + g) * ROW_STRIDE + Q8_ROPE_OFF +
                                                       2 * (16 * j + 8 * half));
      float s[4] = {0.f, 0.f, 0.f, 0.f};
      mma(s, qr[0][0], qr[0][1], qr[0][2], qr[0][3], w.x, w.y);
      mma(s, qr[1][0], qr[1][1], qr[1][2], qr[1][3], w.z, w.w);
      float *to = s_part + ((WARPS + half) * HEADS + g) * S_STRIDE + 8 * nt + 2 * j;
      *reinterpret_cast<float2 *>(to) = make_float2(s[0], s[1]);
      *reinterpret_cast<float2 *>(to + 8 * S_STRIDE) = make_float2(s[2], s[3]);
    }
    __syncthreads();                 // the partial sums are in place, the raw tile is free
    copy(t + STAGES, stage);
    stage = stage + 1 == STAGES ? 0 : stage + 1;
    bool moved = false;              // (the whole warp)
    {
      uint64_t sum = 0;
#pragma unroll
      for (int p = 0; p < PARTIALS; ++p)
        sum = add2(sum, *reinterpret_cast<const uint64_t *>(s_part + (p * HEADS + head) * S_STRIDE + 2 * c));
      float s0, s1;
      asm("mov.b64 {%0, %1}, %2;\n" : "=f"(s0), "=f"(s1) : "l"(sum));
      const uint32_t have = sm[VALID_OFF + (t % VALID_TILES) * WARPS + (c >> 1)] >> (2 * (c & 1));
      s0 = have & 1u ? s0 * a.scale_log2 : -INFINITY;
      s1 = have & 2u ? s1 * a.scale_log2 : -INFINITY;
      float top = fmaxf(s0, s1), alpha = 1.f;
      moved = __any_sync(0xffffffffu, top > m + REF_SLACK);
      if (moved) {
#pragma unroll
        for (int d = 1; d < 16; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
        top = fmaxf(top, m);
        alpha = top == -INFINITY ? 1.f : ex2(m - top);
        m = top;
        l *= alpha;
      }
      const float ref = m == -INFINITY ? 0.f : m;          // no key yet
      s0 = ex2(s0 - ref);
      s1 = ex2(s1 - ref);
      l += s0 + s1;
      *reinterpret_cast<uint32_t *>(sm + P_OFF + (head * P_STRIDE + 2 * c) * 2) = pack(s0, s1);
      if (c == 0) s_alpha[head] = alpha;
    }
    asm volatile("cp.async.wait_group %0;\n" ::"n"(STAGES - 1) : "memory");
    moved = __syncthreads_or(moved);       // P and the next raw tile are in place
    {
      if (moved) {
        const float a0 = s_alpha[g], a1 = s_alpha[g + 8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          o[k >> 1][k & 1][0] *= a0;
          o[k >> 1][k & 1][1] *= a0;
          o[k >> 1][k & 1][2] *= a1;
          o[k >> 1][k & 1][3] *= a1;
        }
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const uint32_t *p = reinterpret_cast<const uint32_t *>(sm + P_OFF) + g * (P_STRIDE / 2) + 8 * u + j;
        const uint32_t p0 = p[0], p1 = p[8 * (P_STRIDE / 2)], p2 = p[4], p3 = p[8 * (P_STRIDE / 2) + 4];
#pragma unroll
        for (int k = 0; k < 8; ++k)
          mma(o[k >> 1][k & 1], p0, p1, p2, p3, transposed(kf[2 * u][k >> 1][k & 1]),
              transposed(kf[2 * u + 1][k >> 1][k & 1]));
      }
    }
  }
  asm volatile("cp.async.wait_group 0;\n" ::: "memory");

  // O / l; the log-sum-exp
#pragma unroll
  for (int d = 1; d < 16; d <<= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
  __syncthreads();                   // alpha has been read
  if (c == 0) {
    s_alpha[head] = l == 0.f ? 0.f : 1.f / l;
    float *to = a.n > 1 ? a.part_lse + (int64_t)part * a.R * a.H : a.lse;
    if (to && head < a.H)
      to[(int64_t)r * a.H + head] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994530942f;
  }
  __syncthreads();
#pragma unroll
  for (int hh = 0; hh < 2; ++hh) {
    const int h = g + 8 * hh;
    if (h >= a.H) continue;
    const float inv = s_alpha[h];
    float f[16];
#pragma unroll
    for (int k = 0; k < 16; ++k) f[k] = o[k >> 2][(k >> 1) & 1][2 * hh + (k & 1)] * inv;
    const int dim = 64 * warp + 16 * j;
    if (a.n > 1) {
      float4 *to = reinterpret_cast<float4 *>(a.part_o + (((int64_t)part * a.R + r) * a.H + h) * HS_VALUE_DIM + dim);
#pragma unroll
      for (int k = 0; k < 4; ++k) to[k] = make_float4(f[4 * k], f[4 * k + 1], f[4 * k + 2], f[4 * k + 3]);
    } else {
      uint4 *to = reinterpret_cast<uint4 *>(a.out + ((int64_t)r * a.H + h) * HS_VALUE_DIM + dim);
#pragma unroll
      for (int k = 0; k < 2; ++k)
        to[k] = make_uint4(pack(f[8 * k], f[8 * k + 1]), pack(f[8 * k + 2], f[8 * k + 3]),
                           pack(f[8 * k + 4], f[8 * k + 5]), pack(f[8 * k + 6], f[8 * k + 7]));
    }
  }
}

}  // namespace

int hs_attn_few_places(int *places) {
  int sms = 0;
  int rc = hs_sm_count(&sms);
  *places = 2 * sms;
  return rc;
}

int hs_attn_few_launch(const void *q, const void *kv, int64_t n_kv, const int32_t *idx, int32_t R, int32_t H,
                       int32_t K, float scale, void *out, float *lse, int32_t n, int32_t keys, float *part_o,
                       float *part_lse, cudaStream_t stream) {
  if ((int64_t)R * n > INT32_MAX) return hs_set_error(HS_ERR_UNSUPPORTED, "R too large");
  int dev = 0;
  HS_CUDA_TRY(cudaGetDevice(&dev));
  static std::atomic<bool> attr_done[64];
  if (dev >= 64 || !attr_done[dev]) {
    HS_CUDA_TRY(cudaFuncSetAttribute(k_attn_few, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM));
    if (dev < 64) attr_done[dev] = true;
  }
  FewArgs a = {reinterpret_cast<const __nv_bfloat16 *>(q), reinterpret_cast<const char *>(kv), n_kv, idx, R, H, K, n,
               keys, scale * 1.4426950408889634f, reinterpret_cast<__nv_bfloat16 *>(out), lse, part_o, part_lse};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(R * n));
  cfg.blockDim = dim3(NT);
  cfg.dynamicSmemBytes = SMEM;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  HS_CUDA_TRY(cudaLaunchKernelEx(&cfg, k_attn_few, a));
  HS_LAUNCH_CHECK("k_attn_few");
  return HS_OK;
}

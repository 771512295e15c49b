// a7-a8: greedy verify of [anchor, drafts] and commit of the accepted prefix.
//
// "投机解码的 KV 流转：prefill 阶段 DFlash 也要吃下整个 prompt", section ④: the
// target runs once over the anchor and the d drafts; the logits at input i
// check draft i+1, the first mismatch yields the correction token, and when
// every draft passes the last input's logits yield one more token. Only the
// KV of the agreeing prefix (anchor + accepted drafts) is kept; the token
// picked last has no KV until the next round, where it is the anchor at
// position L (section ⑥ and the closing table).
//
// One launch, k_verify: a block per (request, input) row takes the streaming
// argmax over the vocabulary (16-byte loads, ties to the lowest index); the
// last of a request's rows to finish then, with the whole block, takes the
// accepted length and next token and commits: host-pool write of the kept
// rows through the mapped pool, LRU slot choice (the first slots of the
// request's (ts, slot) order, a ring whose head then moves past them, so the
// commit writes as many order entries as it keeps rows), hot-slot write,
// kv_len update.

#include <float.h>

#include "hs_commit.cuh"

namespace {

// The acceptance: the drafts, every row's argmax and the results.
struct AcceptArgs {
  const int32_t *drafts;
  int32_t *pred, n_step;
  int32_t *accept_len, *next_token;
};

// Acceptance and commit of batch request b, by a whole block (HS_ARGMAX_THREADS
// threads): longest agreeing prefix m and next token, then commit_rows.
__device__ __forceinline__ void commit_request(const int b, const AcceptArgs &aa,
                                               const CommitArgs &ca) {
  int m = 0;
  if (threadIdx.x == 0) {
    const int32_t *p = aa.pred + (int64_t)b * aa.n_step;   // rows written by other blocks
    while (m < ca.d && aa.drafts[(int64_t)b * ca.d + m] == __ldcg(p + m)) ++m;
    aa.accept_len[b] = m;
    aa.next_token[b] = __ldcg(p + m);
  }
  commit_rows(b, m, ca);
}

// Block per logits row: its argmax into pred; the request's last row to finish
// (a count per request, put back to 0) then commits the request with the
// whole block.
template <int DTYPE>
__global__ void __launch_bounds__(HS_ARGMAX_THREADS) k_verify(const void *__restrict__ logits,
                                                             int32_t V, int32_t *row_count,
                                                             const __grid_constant__ AcceptArgs aa,
                                                             const __grid_constant__ CommitArgs ca) {
  __shared__ int s_last;
  const int64_t row = blockIdx.x;
  const int rows_per_req = ca.d + 1;
  const int64_t elem = (DTYPE == HS_LOGITS_F32) ? 4 : 2;
  const int32_t best = hs_row_argmax<DTYPE>(
      reinterpret_cast<const char *>(logits) + row * (int64_t)V * elem, V);
  const int b = (int)(row / rows_per_req);
  if (threadIdx.x == 0) {
    aa.pred[(int64_t)b * aa.n_step + row % rows_per_req] = best;
    __threadfence();
    s_last = atomicAdd(&row_count[b], 1) == ca.d;
    if (s_last) {
      __threadfence();   // every row of request b has its pred
      row_count[b] = 0;
    }
  }
  __syncthreads();
  if (s_last) commit_request(b, aa, ca);
}

}  // namespace

extern "C" int hs_verify_finalize(hs_buffer *buf, const void *logits, int32_t logits_dtype,
                                  int32_t B, int32_t d, int32_t V, const int32_t *draft_tokens,
                                  const void *step_kv, const int32_t *req_ids, int32_t *kv_len,
                                  int32_t *accept_len, int32_t *next_token, hs_stream_t stream) {
  int rc = hs_check_buffer(buf);
  if (rc) return rc;
  if (B < 1 || B > buf->max_reqs || d < 0 || d + 1 > buf->n_step || V < 1)
    return hs_set_error(HS_ERR_INVALID_ARG, "bad sizes B=%d (1..%d) d=%d (d+1<=%d) V=%d", B,
                        buf->max_reqs, d, buf->n_step, V);
  if (logits_dtype != HS_LOGITS_F32 && logits_dtype != HS_LOGITS_BF16)
    return hs_set_error(HS_ERR_INVALID_ARG, "logits_dtype %d", logits_dtype);
  if (!logits || (d > 0 && !draft_tokens) || !step_kv || !kv_len || !accept_len || !next_token)
    return hs_set_error(HS_ERR_INVALID_ARG, "NULL argument");
  if ((uintptr_t)step_kv & 15)
    return hs_set_error(HS_ERR_INVALID_ARG, "step_kv must be 16-byte aligned");
  buf->clock += 1;
  const int rows = B * (d + 1);
  const CommitArgs ca = commit_args(buf, d, step_kv, req_ids, kv_len);
  const AcceptArgs aa = {draft_tokens, buf->pred, buf->n_step, accept_len, next_token};
  if (logits_dtype == HS_LOGITS_F32)
    k_verify<HS_LOGITS_F32><<<rows, HS_ARGMAX_THREADS, 0, stream>>>(logits, V, buf->row_count, aa, ca);
  else
    k_verify<HS_LOGITS_BF16><<<rows, HS_ARGMAX_THREADS, 0, stream>>>(logits, V, buf->row_count, aa, ca);
  HS_LAUNCH_CHECK("k_verify");
  return HS_OK;
}

// The commit of a verified request, shared by the greedy and the sampled verify.
#pragma once

#include "hs_internal.cuh"

struct CommitArgs {
  int32_t d;
  const uint4 *step_kv;
  const int32_t *req_ids;
  int32_t *kv_len;
  int32_t max_reqs, S, S_tot, max_ctx, block_size, hbt_stride;
  const int32_t *hbt;
  int64_t pool_rows;
  uint4 *pool, *hot;
  int32_t *token_slot, *slot_token;
  int64_t *slot_ts;
  int32_t *lru_order, *lru_head;
  uint32_t *verify_claim;
  uint32_t *status;
  int64_t now;
};

// Commit of batch request b with m accepted drafts (the block's thread 0 knows
// m), by a whole block of at least HS_MAX_STEP threads: the m + 1 kept step
// rows go to the host pool and to the first m + 1 slots of the LRU order
// (nothing protected), which take the current time and move to the order's
// end; the maps and kv_len follow.
__device__ __forceinline__ void commit_rows(const int b, const int m, const CommitArgs &ca) {
  const int32_t d = ca.d;
  const uint4 *step_kv = ca.step_kv;
  const int32_t *req_ids = ca.req_ids;
  int32_t *kv_len = ca.kv_len;
  const int32_t max_reqs = ca.max_reqs, S = ca.S, S_tot = ca.S_tot,
                max_ctx = ca.max_ctx, block_size = ca.block_size, hbt_stride = ca.hbt_stride;
  const int32_t *hbt = ca.hbt;
  const int64_t pool_rows = ca.pool_rows;
  uint4 *pool = ca.pool, *hot = ca.hot;
  int32_t *token_slot = ca.token_slot, *slot_token = ca.slot_token, *lru_order = ca.lru_order;
  int64_t *slot_ts = ca.slot_ts;
  uint32_t *status = ca.status;
  const int64_t now = ca.now;
  __shared__ int sm_m, sm_L, sm_ok;
  __shared__ int32_t chosen[HS_MAX_STEP];
  const int32_t req = req_ids ? req_ids[b] : b;
  if (threadIdx.x == 0) {
    int ok = 1;
    int L = 0;
    if (req < 0 || req >= max_reqs) {
      ok = 0;
      atomicOr(status, HS_STATUS_INDEX);
    } else if (atomicExch(ca.verify_claim + req, (uint32_t)now) == (uint32_t)now) {
      // the request appears twice in req_ids: only its first claimant commits
      ok = 0;
      atomicOr(status, HS_STATUS_INDEX);
    } else {
      L = kv_len[req];
      if ((int64_t)L + m + 1 > max_ctx || m + 1 > S) {
        ok = 0;
        atomicOr(status, HS_STATUS_CAPACITY);
      }
    }
    sm_m = m; sm_L = L; sm_ok = ok;
  }
  __syncthreads();
  if (!sm_ok) return;
  const int n = sm_m + 1, L = sm_L;
  const int64_t sbase = (int64_t)req * S;

  // The victims are the first n slots of the LRU order (ascending (ts, slot),
  // nothing protected). They take the current time, so the new order is the
  // rest of the order followed by the victims in slot order. The order is a
  // ring from lru_head[req]: the victims' ring positions take them back in
  // slot order and the head moves past them (n entries written, not S).
  int32_t *lru = lru_order + sbase;
  const int head = ca.lru_head[req];
  if ((int)threadIdx.x < n) {
    int p = head + (int)threadIdx.x;
    if (p >= S) p -= S;
    chosen[threadIdx.x] = lru[p];
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    int32_t sorted[HS_MAX_STEP];
    for (int k = 0; k < n; ++k) {               // insertion sort of at most 16 slots
      int32_t v = chosen[k];
      int j = k;
      while (j > 0 && sorted[j - 1] > v) { sorted[j] = sorted[j - 1]; --j; }
      sorted[j] = v;
    }
    for (int k = 0; k < n; ++k) {
      int p = head + k;
      if (p >= S) p -= S;
      lru[p] = sorted[k];
    }
    ca.lru_head[req] = head + n >= S ? head + n - S : head + n;
  }

  // map updates (one thread per kept position)
  const int64_t cbase = (int64_t)req * max_ctx;
  if (threadIdx.x < n) {
    const int k = threadIdx.x;
    const int32_t s = chosen[k], t = L + k;
    const int32_t old = slot_token[sbase + s];
    if (old >= 0 && old < max_ctx) token_slot[cbase + old] = -1;
    slot_token[sbase + s] = t;
    token_slot[cbase + t] = s;
    slot_ts[sbase + s] = now;
  }
  // row copies: kept step rows -> host pool rows and hot slots
  const int32_t *hbt_row = hbt + (int64_t)req * hbt_stride;
  for (int e = threadIdx.x; e < n * HS_ROW_VEC16; e += blockDim.x) {
    const int k = e / HS_ROW_VEC16, c = e % HS_ROW_VEC16;
    const int32_t t = L + k;
    const uint4 v = step_kv[((int64_t)b * (d + 1) + k) * HS_ROW_VEC16 + c];
    const int32_t hb = hbt_row[t / block_size];
    const int64_t hr = (int64_t)hb * block_size + t % block_size;
    if (hb >= 0 && hr < pool_rows) pool[hr * HS_ROW_VEC16 + c] = v;
    else if (c == 0) atomicOr(status, HS_STATUS_INDEX);
    hot[((int64_t)req * S_tot + chosen[k]) * HS_ROW_VEC16 + c] = v;
  }
  if (threadIdx.x == 0) kv_len[req] = L + n;
}

// The buffer's side of the commit arguments (the caller has advanced the clock).
inline CommitArgs commit_args(const hs_buffer *buf, int32_t d, const void *step_kv,
                              const int32_t *req_ids, int32_t *kv_len) {
  CommitArgs ca;
  ca.d = d;
  ca.step_kv = reinterpret_cast<const uint4 *>(step_kv); ca.req_ids = req_ids;
  ca.kv_len = kv_len;
  ca.max_reqs = buf->max_reqs; ca.S = buf->S; ca.S_tot = buf->S_tot;
  ca.max_ctx = buf->max_ctx; ca.block_size = buf->block_size; ca.hbt_stride = buf->hbt_stride;
  ca.hbt = buf->hbt; ca.pool_rows = buf->host_pool_rows;
  ca.pool = reinterpret_cast<uint4 *>(const_cast<__nv_bfloat16 *>(buf->host_pool));
  ca.hot = reinterpret_cast<uint4 *>(buf->hot_kv);
  ca.token_slot = buf->token_slot; ca.slot_token = buf->slot_token; ca.slot_ts = buf->slot_ts;
  ca.lru_order = buf->lru_order; ca.lru_head = buf->lru_head;
  ca.verify_claim = buf->verify_claim; ca.status = buf->status;
  ca.now = buf->clock;
  return ca;
}

// The paged K/V cache: argument blocks and launchers of the append (rotation
// and store of a step's rows) and of the attention that reads the pages.
//
// Pages are [num_pages, page_size, nkv, hd]; token t of request b lives in
// page table[b, t >> ps_log2] at row t & (page_size - 1). A prefix that every
// request shares has a page list of its own and is not part of the tables.
#pragma once
#include "common.cuh"

namespace pe {

// Rows of a paged step. Request b's rows start at off[b] + b * extra and
// number off[b+1] - off[b] + extra: its new rows, then `extra` masked rows
// (a draft step's K - 1; 0 elsewhere). Row j is token kv_len[b] + j of the
// request's own table and sees the tokens up to itself.
struct PagedRows {
  int B, T;               // requests; rows the row arrays have room for
  const int* off;         // device [B+1], ascending
  int extra;
  int min_new;            // new rows a request has at least (a draft step: its anchor)
  const int* kv_len;      // device [B]: own tokens cached before this step
  const int* table;       // device [B, max_pages]
  int max_pages, ps_log2, num_pages;
};
struct PagedReq {
  int first, n_new, base, n, kv;   // off[b], new rows, first row, rows, cached tokens
};
__device__ __forceinline__ int pr_base(const PagedRows& p, int b) { return p.off[b] + b * p.extra; }
// Whether request b is well formed: its rows inside [0, T], its tokens inside
// its page table.
// (lo, hi, kv: off[b], off[b+1], kv_len[b])
__device__ __forceinline__ bool pr_check(const PagedRows& p, int b, int lo, int hi, int kv, PagedReq* q) {
  q->first = lo;
  q->n_new = hi - lo;
  q->base = lo + b * p.extra;
  q->n = hi - lo + p.extra;
  q->kv = kv;
  return lo >= 0 && hi <= p.T && lo <= hi && hi - lo >= p.min_new &&
         (long long)q->base + q->n <= p.T && kv >= 0 &&
         (long long)kv + q->n <= ((long long)p.max_pages << p.ps_log2);
}
__device__ __forceinline__ bool pr_request(const PagedRows& p, int b, PagedReq* q) {
  return pr_check(p, b, p.off[b], p.off[b + 1], p.kv_len[b], q);
}
// The request whose rows hold row r is the largest b with base(b) <= r (0 when
// there is none).
// Request of row r, its lengths, and *ok whether it is well formed. By a whole
// warp: one round of loads for up to 32 requests, two for up to 1024.
__device__ __forceinline__ int pr_lookup(const PagedRows& p, int r, PagedReq* q, bool* ok) {
  const int lane = threadIdx.x & 31;
  int first = 0, len = p.B;   // the answer is in [first, first + len)
  while (len > 32) {
    const int step = (len + 31) / 32, b = first + lane * step;
    const unsigned m = __ballot_sync(0xffffffffu, lane * step < len && pr_base(p, b) <= r);
    const int k = m ? 31 - __clz(m) : 0;
    len = min(step, len - k * step);
    first += k * step;
  }
  int lo = 0, hi = 0, kv = 0;
  if (lane < len) {
    lo = p.off[first + lane];
    hi = p.off[first + lane + 1];
    kv = p.kv_len[first + lane];
  }
  const unsigned m = __ballot_sync(0xffffffffu, lane < len && lo + (first + lane) * p.extra <= r);
  const int k = m ? 31 - __clz(m) : 0;
  lo = __shfl_sync(0xffffffffu, lo, k);
  hi = __shfl_sync(0xffffffffu, hi, k);
  kv = __shfl_sync(0xffffffffu, kv, k);
  *ok = pr_check(p, first + k, lo, hi, kv, q);
  return first + k;
}

// Append: rows of a fused q/k/v projection, rotated and stored.
struct KvAppendArgs {
  PagedRows rows;
  int nq, nkv, hd;
  const void* in;          // [*, (nq + 2 nkv) * hd] rows of the projection
  long long in_ld;
  int in_compact;          // 1: only new rows have a projection row (index off[b] + j)
  const float* mask_row;   // projection row of every masked row, or NULL
  const int* positions;    // per new row (index off[b] + j); masked row d after the last at +d
  const float *rcos, *rsin;
  int max_pos;
  void* q;                 // [T, nq, hd] or NULL
  void *k_pages, *v_pages;
  // draft layer 0: seed of the residual stream (h NULL: none)
  float* h;
  int H;
  const float *resid, *mask_resid;   // [new rows, H], [H]
  int* status;
};
cudaError_t launch_kv_append(int dtype, int in_dtype, const KvAppendArgs& a, cudaStream_t st);

// Attention of the rows over [shared prefix, own tokens].
struct PagedAttnArgs {
  PagedRows rows;
  int nq, nkv, hd;
  const void* q;           // [T, nq, hd]
  const void *k_pages, *v_pages;
  const int* prefix_pages; // device [ceil(prefix / page_size)] or NULL
  int prefix;              // tokens of the shared prefix
  float scale;
  void* out;               // [T, nq, hd]
  float* lse;              // [T, nq] or NULL
  void* ws;                // paged_attn_ws_bytes
  int* status;
};
size_t paged_attn_ws_bytes(int dtype, int T, int B, int nq, int nkv, int hd, int prefix);
cudaError_t launch_paged_attn(int dtype, const PagedAttnArgs& a, int probe_op, cudaStream_t st);
// its bf16 form on the tensor cores
size_t paged_attn_tc_ws_bytes(int T, int B, int nq, int nkv, int hd, int prefix);
cudaError_t launch_paged_attn_tc(const PagedAttnArgs& a, int probe_op, cudaStream_t st);
// its fp32 form (up to 64 query heads to a key head)
size_t paged_attn_f32_ws_bytes(int T, int B, int nq, int nkv, int hd, int prefix);
cudaError_t launch_paged_attn_f32(const PagedAttnArgs& a, int probe_op, cudaStream_t st);

}  // namespace pe

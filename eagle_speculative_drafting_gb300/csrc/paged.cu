// Paged K/V cache: the append and the attention over pages.
#include <math.h>

#include "paged_plan.cuh"

namespace pe {

// -------------------------------------------------------------------------
// Append. Row r = (b, j): q and k heads rotate by the row's position
//   u'_i = u_i cos - u_{i+half} sin,  u'_{i+half} = u_{i+half} cos + u_i sin
// in fp32 and round once to the cache's type; k and v go to token
// kv_len[b] + j of the request's pages.
//
// Bound by memory: a block of 128 threads per row, a thread 16 bytes of a
// head's lower and upper half, the same of every head it takes, so that its
// cosines and sines stay in registers. A row's loads (JB heads per thread at
// once, all of them in the usual shapes) go out before the chain of lookups
// that finds its request, page and table row.
// Measured: 12 prompts of 500 to 4000 rows, 32/8 heads of 128 from a bf16
// projection, 112 us at 6.5 TB/s (0.95 of the measured copy); a step of 4 to
// 512 rows 6.4 to 6.9 us, which is what the call and the launch take.
// -------------------------------------------------------------------------
template <typename TI> struct Chunk;   // 16 bytes of the projection as floats
template <> struct Chunk<float> {
  static constexpr int N = 4;
  float4 v;
  __device__ __forceinline__ void load(const float* p) { v = __ldcs(reinterpret_cast<const float4*>(p)); }
  __device__ __forceinline__ void get(float (&x)[4]) const {
    x[0] = v.x;
    x[1] = v.y;
    x[2] = v.z;
    x[3] = v.w;
  }
};
template <> struct Chunk<bf16> {
  static constexpr int N = 8;
  uint4 v;
  __device__ __forceinline__ void load(const bf16* p) { v = __ldcs(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]));
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
};
template <int N>
__device__ __forceinline__ void put(float* p, const float (&x)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 4) *reinterpret_cast<float4*>(p + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
}
template <int N>
__device__ __forceinline__ void put(bf16* p, const float (&x)[N]) {
  uint32_t w[N / 2];
#pragma unroll
  for (int i = 0; i < N / 2; ++i) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&v);
  }
  if constexpr (N == 8) *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  else *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
}

template <typename T, typename TI, int HD>
__global__ void __launch_bounds__(128) kv_append_kernel(KvAppendArgs a) {
  constexpr int HALF = HD / 2, N = Chunk<TI>::N, TPH = HALF / N, HPB = 128 / TPH, JB = sizeof(TI) == 4 ? 6 : 3;
  pdl_trigger();
  pdl_wait();
  const int r = blockIdx.x, i0 = (threadIdx.x % TPH) * N, h0 = threadIdx.x / TPH;
  const int rot = a.nq + a.nkv, heads = rot + a.nkv;
  const int skip = a.q ? 0 : a.nq;   // without q its columns are not read
  Chunk<TI> lo[JB], hi[JB];
  auto fetch = [&](const TI* in, int h) {
#pragma unroll
    for (int i = 0; i < JB; ++i)
      if (h + i * HPB < heads) {
        lo[i].load(in + (h + i * HPB) * HD + i0);
        hi[i].load(in + (h + i * HPB) * HD + i0 + HALF);
      }
  };
  const TI* base = static_cast<const TI*>(a.in);
  if (!a.in_compact) fetch(base + (long long)r * a.in_ld, skip + h0);
  PagedReq q;
  bool ok;
  const int b = pr_lookup(a.rows, r, &q, &ok);
  const int j = r - q.base;
  if (!ok || j < 0 || j >= q.n) {
    // a row of a malformed request is flagged; one behind the last is left alone
    if (threadIdx.x == 0 && !ok && j >= 0) set_status(a.status, PEAGLE_DEV_BOUNDS);
    return;
  }
  const int jn = min(j, q.n_new - 1);
  const int pos = a.positions[q.first + jn] + (j - jn);
  const int tok = q.kv + j;
  const int page = a.rows.table[(size_t)b * a.rows.max_pages + (tok >> a.rows.ps_log2)];
  if (pos < 0 || pos >= a.max_pos || page < 0 || page >= a.rows.num_pages) {
    if (threadIdx.x == 0) set_status(a.status, PEAGLE_DEV_BOUNDS);
    return;
  }
  const bool masked = a.mask_row && j >= q.n_new;
  const TI* in = masked ? reinterpret_cast<const TI*>(a.mask_row)
                        : base + (long long)(a.in_compact ? q.first + jn : r) * a.in_ld;
  if (a.in_compact) fetch(in, skip + h0);
  float cs[N], sn[N];
#pragma unroll
  for (int i = 0; i < N; i += 4) {
    *reinterpret_cast<float4*>(cs + i) = *reinterpret_cast<const float4*>(a.rcos + (size_t)pos * HALF + i0 + i);
    *reinterpret_cast<float4*>(sn + i) = *reinterpret_cast<const float4*>(a.rsin + (size_t)pos * HALF + i0 + i);
  }
  const size_t slot = ((size_t)page << a.rows.ps_log2) + (tok & ((1 << a.rows.ps_log2) - 1));
  T* Q = static_cast<T*>(a.q) + (size_t)r * a.nq * HD;
  T* Kp = static_cast<T*>(a.k_pages) + slot * a.nkv * HD;
  T* Vp = static_cast<T*>(a.v_pages) + slot * a.nkv * HD;
  for (int h = skip + h0; h < heads; h += JB * HPB) {
#pragma unroll
    for (int i = 0; i < JB; ++i) {
      const int hd = h + i * HPB;
      if (hd >= heads) break;
      T* dst = hd < a.nq ? Q + hd * HD : hd < rot ? Kp + (hd - a.nq) * HD : Vp + (hd - rot) * HD;
      float x[N], y[N];
      lo[i].get(x);
      hi[i].get(y);
      if (hd < rot) {
#pragma unroll
        for (int e = 0; e < N; ++e) {
          const float u = x[e] * cs[e] - y[e] * sn[e], v = y[e] * cs[e] + x[e] * sn[e];
          x[e] = u;
          y[e] = v;
        }
      }
      put<N>(dst + i0, x);
      put<N>(dst + i0 + HALF, y);
    }
    if (h + JB * HPB < heads) fetch(in, h + JB * HPB);
  }
  if (a.h) {
    const float* src = masked ? a.mask_resid : a.resid + (size_t)(q.first + jn) * a.H;
    for (int e = threadIdx.x; e < a.H; e += blockDim.x) a.h[(size_t)r * a.H + e] = src[e];
  }
}

template <typename T, typename TI>
static void append_hd(const KvAppendArgs& a, cudaStream_t st) {
  if (a.hd == 128) launch_pdl(kv_append_kernel<T, TI, 128>, a.rows.T, 128, 0, st, a);
  else launch_pdl(kv_append_kernel<T, TI, 64>, a.rows.T, 128, 0, st, a);
}
cudaError_t launch_kv_append(int dtype, int in_dtype, const KvAppendArgs& a, cudaStream_t st) {
  if (a.rows.T <= 0 || a.rows.B <= 0) return cudaSuccess;
  if (dtype == PEAGLE_F32) append_hd<float, float>(a, st);
  else if (in_dtype == PEAGLE_F32) append_hd<bf16, float>(a, st);
  else append_hd<bf16, bf16>(a, st);
  note_launch();
  return cudaGetLastError();
}

// fp32 with more query heads to a key head than a query tile of the tiled
// kernel holds: a warp per (row, head).
constexpr int kF32Heads = 64;
// Attention of row r, head h, by one warp: lane owns dims [lane*E, lane*E+E),
// the keys go by one at a time with a running maximum m, sum l and weighted
// value sum o.
template <typename T, int E>
__device__ __forceinline__ void paged_row_simt(const PagedAttnArgs& a, int b, const PagedReq& q, int r, int h) {
  const int lane = threadIdx.x & 31, hd = 32 * E, g = h / (a.nq / a.nkv);
  const T* Q = static_cast<const T*>(a.q) + ((size_t)r * a.nq + h) * hd + lane * E;
  const T* K = static_cast<const T*>(a.k_pages);
  const T* V = static_cast<const T*>(a.v_pages);
  const int sh = a.rows.ps_log2, mask = (1 << sh) - 1;
  float x[E], o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    x[e] = to_f(Q[e]);
    o[e] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  bool bad = false;
  auto keys = [&](const int* pages, int count) {
    for (int t = 0; t < count; ++t) {
      const int page = pages[t >> sh];
      if (page < 0 || page >= a.rows.num_pages) {
        bad = true;
        continue;
      }
      const size_t at = ((((size_t)page << sh) + (t & mask)) * a.nkv + g) * hd + lane * E;
      float s = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) s = fmaf(x[e], to_f(K[at + e]), s);
      s = warp_sum(s) * a.scale;
      const float mn = fmaxf(m, s);
      const float c = m == -INFINITY ? 0.f : expf(m - mn);
      const float p = s == -INFINITY ? 0.f : expf(s - mn);   // (no -inf - -inf before a finite score)
      l = l * c + p;
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = o[e] * c + p * to_f(V[at + e]);
      m = mn;
    }
  };
  keys(a.prefix_pages, a.prefix);
  keys(a.rows.table + (size_t)b * a.rows.max_pages, q.kv + (r - q.base) + 1);
  if (bad && lane == 0) set_status(a.status, PEAGLE_DEV_BOUNDS);
  T* out = static_cast<T*>(a.out) + ((size_t)r * a.nq + h) * hd + lane * E;
#pragma unroll
  for (int e = 0; e < E; ++e) out[e] = from_f<T>(o[e] / l);
  if (a.lse && lane == 0) a.lse[(size_t)r * a.nq + h] = m + logf(l);
}
template <typename T, int E>
__global__ void __launch_bounds__(128) paged_attn_simt(PagedAttnArgs a) {
  pdl_trigger();
  pdl_wait();
  const int r = blockIdx.x, w = threadIdx.x >> 5, nw = blockDim.x >> 5;
  PagedReq q;
  if (r == 0 && blockIdx.y == 0)   // (a malformed request need not have a row)
    for (int b = threadIdx.x; b < a.rows.B; b += blockDim.x)
      if (!pr_request(a.rows, b, &q)) set_status(a.status, PEAGLE_DEV_BOUNDS);
  bool ok;
  const int b = pr_lookup(a.rows, r, &q, &ok);
  if (!ok || r < q.base || r >= q.base + q.n) {
    if (threadIdx.x == 0 && !ok && r >= q.base) set_status(a.status, PEAGLE_DEV_BOUNDS);
    return;
  }
  for (int h = blockIdx.y * nw + w; h < a.nq; h += gridDim.y * nw) paged_row_simt<T, E>(a, b, q, r, h);
}

size_t paged_attn_ws_bytes(int dtype, int T, int B, int nq, int nkv, int hd, int prefix) {
  if (dtype == PEAGLE_BF16) return paged_attn_tc_ws_bytes(T, B, nq, nkv, hd, prefix);
  return nq / nkv <= kF32Heads ? paged_attn_f32_ws_bytes(T, B, nq, nkv, hd, prefix) : 0;
}

cudaError_t launch_paged_attn(int dtype, const PagedAttnArgs& a, int probe_op, cudaStream_t st) {
  if (a.rows.T <= 0 || a.rows.B <= 0) return cudaSuccess;
  if (dtype == PEAGLE_BF16) return launch_paged_attn_tc(a, probe_op, st);
  if (a.nq / a.nkv <= kF32Heads) return launch_paged_attn_f32(a, probe_op, st);
  const dim3 grid(a.rows.T, (a.nq + 3) / 4);
  probe_start(probe_op, st);
  if (a.hd == 128) launch_pdl(paged_attn_simt<float, 4>, grid, 128, 0, st, a);
  else launch_pdl(paged_attn_simt<float, 2>, grid, 128, 0, st, a);
  note_launch();
  probe_stop(probe_op, st);
  return cudaGetLastError();
}

}  // namespace pe

// Paged attention in fp32 on the CUDA cores.
//
// Two CTAs per SM take equal shares of the line of key tiles (paged_plan.cuh).
// A tile is 64 query rows (rows x heads of one key head) against 64 keys;
// thread (ty, tx) of 16 x 16 holds 4 query rows x 4 keys of the scores and
// 4 rows x hd/16 dims of the output in registers. K and V tiles come page by
// page with cp.async: the next K as soon as the scores are done, the next V
// as soon as the product is, so that one is always on its way. Score and
// value loops read float4s from shared memory, 12 wavefronts for 64 (128)
// FMAs, so a full tile is bound by the FMA pipes; a warp whose 8 query rows
// are not there skips the arithmetic, which leaves a decode step bound by
// the latency of its loads. Each tile's 64 cache slots are looked up once, two
// tiles ahead, into shared memory.
// Measured: prompts of 500 to 900 rows, 8 heads of 128, 218 us, 28 TFLOP/s (of
// about 75 by the FMA pipes; what is missing are barriers and the softmax
// between the products); 32 requests of 4 to 8 rows x 4 heads to a key head,
// 1000 to 4000 keys, 377 us; a step of 9 requests over 30 to 900 keys behind
// 300 shared ones 21 us, one tile to a CTA and the joining kernel.
// Rows' maxima meet by shuffles in the 16 threads that share them; the sum is
// kept per thread and added up once a unit.
#include <limits.h>

#include "mma.cuh"
#include "paged_plan.cuh"

namespace pe {

namespace pf {
constexpr int TQ = 64, TK = 64, THREADS = 256;
template <int HD>
struct Cfg {
  static constexpr int LDP = TK;   // (two CTAs of hd = 128 just fit)
  static constexpr int SMEM = (TQ * HD + 2 * TK * HD + TQ * LDP) * 4;
};
// float offset of 16-byte chunk c of a tile row, swizzled so that 8 rows'
// same chunk lies in 8 different bank groups
template <int HD>
__device__ __forceinline__ int at(int row, int c) {
  return row * HD + ((c ^ (row & 7)) << 2);
}
// d += a * b on two packed floats: one issue slot for two FMAs
__device__ __forceinline__ void fma2(float& dx, float& dy, float ax, float ay, float bx, float by) {
  asm("{\n .reg .b64 d, a, b;\n mov.b64 d, {%0, %1};\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n"
      " fma.rn.f32x2 d, a, b, d;\n mov.b64 {%0, %1}, d;\n}"
      : "+f"(dx), "+f"(dy)
      : "f"(ax), "f"(ay), "f"(bx), "f"(by));
}
}  // namespace pf

template <int HD>
__global__ void __launch_bounds__(pf::THREADS, 2) paged_attn_f32(PagedAttnArgs a, PagedPlan p) {
  using namespace pf;
  constexpr int LDP = Cfg<HD>::LDP, C4 = HD / 4, NO = HD / 64;   // chunks of a row; output float4s per thread and row
  extern __shared__ __align__(16) float smf[];
  float* sQ = smf;                 // [TQ][HD] swizzled
  float* sK = sQ + TQ * HD;        // [TK][HD] swizzled
  float* sV = sK + TK * HD;        // [TK][HD] swizzled
  float* sP = sV + TK * HD;        // [TQ][LDP]
  __shared__ long long sLL[THREADS / 32 + 1];
  __shared__ int sStart, sOdd, sSlot[2][TK];
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, tx = tid & 15, ty = tid >> 4;
  const int B = a.rows.B, cta = blockIdx.x, nkv = a.nkv, T = a.rows.T;
  const float* Q = static_cast<const float*>(a.q);

  // ---- the line: every CTA adds up all requests' costs
  const long long prefix_line = nkv * pp_prefix(p, T);
  const int per = (B + THREADS - 1) / THREADS, b_lo = min(tid * per, B), b_hi = min(b_lo + per, B);
  long long mine = 0;
  for (int b = b_lo; b < b_hi; ++b) {
    PagedReq q;
    if (pr_request(a.rows, b, &q)) mine += nkv * pp_request(p, q.n, q.kv);
    else if (cta == 0) set_status(a.status, PEAGLE_DEV_BOUNDS);
  }
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) sLL[warp] = incl;
  if (tid == 0) sStart = B;
  __syncthreads();
  long long cum = prefix_line + incl - mine, total = prefix_line;
  for (int i = 0; i < THREADS / 32; ++i) {
    if (i < warp) cum += sLL[i];
    total += sLL[i];
  }
  const long long part = pp_part(total, p.ncta), x0 = cta * part, x1 = min(x0 + part, total);
  if (x0 >= total) return;
  for (int b = b_lo; b < b_hi; ++b) {
    PagedReq q;
    const long long c = per == 1 ? mine : pr_request(a.rows, b, &q) ? nkv * pp_request(p, q.n, q.kv) : 0;
    if (cum <= x0 && x0 < cum + c) {
      sStart = b;
      sLL[THREADS / 32] = cum;
    }
    cum += c;
  }
  if (tid == 0 && x0 < prefix_line) {
    sStart = 0;
    sLL[THREADS / 32] = prefix_line;
  }
  __syncthreads();

  const float sl2 = a.scale * 1.4426950408889634f;
  const int sh = a.rows.ps_log2, slot_mask = (1 << sh) - 1;
  bool first_unit = true;
  int jr[4];   // rows of the unit that this thread's query rows belong to
#pragma unroll
  for (int i = 0; i < 4; ++i) jr[i] = (ty * 4 + i) / p.G;

  // one piece of a unit: rows row0.. of request b (or of the whole batch)
  // against tiles [t0, t0 + nt) of the list that has pt tiles of the prefix
  auto piece = [&](bool prefix_unit, int b, int g, int row0, int rows, int t0, int nt, bool begins, bool whole, int pt,
                   int vis0, int own, unsigned ctas) {
    const int live = rows * p.G;
    if (first_unit && tid == 0) p.cid[cta] = begins ? 0 : piece_id(row0, g, prefix_unit);
    first_unit = false;
    const int* own_pages = a.rows.table + (size_t)b * a.rows.max_pages;
    // Slot of key k of tile t, -1 where there is none (its row reads as
    // zeros). Tile t's 64 are in sSlot[t & 1]; those of the tile after next
    // are looked up while a tile is at work.
    auto look_up = [&](int t, int k) {   // page of the key, -1: behind the last
      const bool pre = t < pt;
      const int tok = (pre ? t : t - pt) * TK + k;
      return tok < (pre ? a.prefix : own) ? (pre ? a.prefix_pages : own_pages)[tok >> sh] : INT_MIN;
    };
    auto put_slot = [&](int t, int k, int page) {
      const int tok = (t < pt ? t : t - pt) * TK + k;
      const bool in = page >= 0 && page < a.rows.num_pages;
      if (!in && page != INT_MIN) set_status(a.status, PEAGLE_DEV_BOUNDS);
      sSlot[t & 1][k] = in ? (page << sh) + (tok & slot_mask) : -1;
    };
    auto load = [&](const void* src, float* dst, int t) {
      const float* base = static_cast<const float*>(src);
#pragma unroll 4
      for (int e = tid; e < TK * C4; e += THREADS) {
        const int k = e / C4, c = e % C4, slot = sSlot[t & 1][k];
        const size_t from = ((size_t)max(slot, 0) * nkv + g) * HD + c * 4;
        mm::cp16(mm::sa(dst + at<HD>(k, c)), base + from, slot >= 0 ? 16 : 0);
      }
      mm::cp_commit();
    };
    __syncthreads();   // the last piece is done with the tiles
    if (tid == 0) sOdd = 0;
    int page = 0;
    const int ahead = t0 + (tid >> 6);   // of 128 threads, the first two tiles
    if (tid < 2 * TK && ahead < t0 + nt) page = look_up(ahead, tid & (TK - 1));
    for (int e = tid; e < TQ * C4; e += THREADS) {
      const int i = e / C4, c = e % C4, r = row0 + i / p.G, h = g * p.G + i % p.G;
      mm::cp16(mm::sa(sQ + at<HD>(i, c)), Q + (i < live ? ((size_t)r * a.nq + h) * HD + c * 4 : 0), i < live ? 16 : 0);
    }
    if (tid < 2 * TK && ahead < t0 + nt) put_slot(ahead, tid & (TK - 1), page);
    __syncthreads();
    load(a.k_pages, sK, t0);
    load(a.v_pages, sV, t0);
    float m[4], l[4];
    float4 o[4][NO];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      m[i] = -INFINITY;
      l[i] = 0.f;
#pragma unroll
      for (int j = 0; j < NO; ++j) o[i][j] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    const bool wlive = warp * 8 < live;
    for (int t = t0; t < t0 + nt; ++t) {
      const bool pre = t < pt, more = t + 1 < t0 + nt;
      const int key0 = (pre ? t : t - pt) * TK;
      const bool next2 = t + 2 < t0 + nt && tid < TK;
      if (next2) page = look_up(t + 2, tid);
      mm::cp_wait<1>();
      __syncthreads();
      float s[4][4], s1[4][4];   // of a row's even and odd dims
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[i][j] = s1[i][j] = 0.f;
      if (wlive) {
#pragma unroll 4
        for (int c = 0; c < C4; ++c) {
          float4 x[4], y[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const float4*>(sQ + at<HD>(ty * 4 + i, c));
#pragma unroll
          for (int j = 0; j < 4; ++j) y[j] = *reinterpret_cast<const float4*>(sK + at<HD>(tx + 16 * j, c));
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              fma2(s[i][j], s1[i][j], x[i].x, x[i].y, y[j].x, y[j].y);
              fma2(s[i][j], s1[i][j], x[i].z, x[i].w, y[j].z, y[j].w);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int lim = (pre ? a.prefix : vis0 + jr[i]) - key0;   // keys of the tile that the row sees
          float mx = -INFINITY;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            s[i][j] = tx + 16 * j < lim ? (s[i][j] + s1[i][j]) * sl2 : -INFINITY;
            mx = fmaxf(mx, s[i][j]);
          }
#pragma unroll
          for (int w = 1; w < 16; w <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
          const float mn = fmaxf(m[i], mx);
          const float corr = m[i] == -INFINITY ? 0.f : exp2f(m[i] - mn);
          l[i] *= corr;
#pragma unroll
          for (int j = 0; j < NO; ++j) {
            o[i][j].x *= corr;
            o[i][j].y *= corr;
            o[i][j].z *= corr;
            o[i][j].w *= corr;
          }
          m[i] = mn;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            // nothing seen yet: every weight is 0 (a NaN score stays)
            const float w = mn == -INFINITY ? (s[i][j] != s[i][j] ? s[i][j] : 0.f) : exp2f(s[i][j] - mn);
            l[i] += w;
            sP[(ty * 4 + i) * LDP + tx + 16 * j] = w;
          }
        }
      }
      __syncthreads();   // K is read, P is written
      if (more) load(a.k_pages, sK, t + 1);
      else mm::cp_commit();
      mm::cp_wait<1>();
      // a token that some rows see and others do not may hold anything in V:
      // its odd elements are taken out, each by the thread that copied them
      if (!pre && key0 + TK > vis0) {
        for (int e = tid; e < TK * C4; e += THREADS) {
          const int k = e / C4, c = e % C4;
          if (key0 + k >= vis0 && key0 + k < own) {
            float4* at_v = reinterpret_cast<float4*>(sV + at<HD>(k, c));
            const float4 v = *at_v;
            const bool x = fabsf(v.x) < INFINITY, y = fabsf(v.y) < INFINITY, z = fabsf(v.z) < INFINITY, w = fabsf(v.w) < INFINITY;
            if (!(x && y && z && w)) {
              *at_v = make_float4(x ? v.x : 0.f, y ? v.y : 0.f, z ? v.z : 0.f, w ? v.w : 0.f);
              sOdd = 1;
            }
          }
        }
      }
      __syncthreads();
      if (wlive) {
#pragma unroll 2
        for (int k = 0; k < TK; k += 4) {
          float4 w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) w[i] = *reinterpret_cast<const float4*>(sP + (ty * 4 + i) * LDP + k);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
#pragma unroll
            for (int j = 0; j < NO; ++j) {
              const float4 v = *reinterpret_cast<const float4*>(sV + at<HD>(k + kk, tx + 16 * j));
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float wi = kk == 0 ? w[i].x : kk == 1 ? w[i].y : kk == 2 ? w[i].z : w[i].w;
                fma2(o[i][j].x, o[i][j].y, wi, wi, v.x, v.y);
                fma2(o[i][j].z, o[i][j].w, wi, wi, v.z, v.w);
              }
            }
          }
        }
      }
      __syncthreads();   // V and P are read
      if (more) load(a.v_pages, sV, t + 1);
      else mm::cp_commit();
      if (next2) put_slot(t + 2, tid, page);
    }
    const bool odd = sOdd != 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int w = 1; w < 16; w <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], w);
      const int qi = ty * 4 + i;
      if (qi >= live) continue;
      const size_t rh = (size_t)(row0 + jr[i]) * a.nq + g * p.G + (qi - jr[i] * p.G);
      const size_t at_c = (size_t)cta * p.RP * p.G + qi;
      const bool direct = whole && !odd;
      float* dst = direct ? static_cast<float*>(a.out) + rh * HD
                          : !begins ? p.co + at_c * HD : (prefix_unit ? p.qo : p.po) + rh * HD;
      const float f = direct ? 1.f / l[i] : 1.f;
#pragma unroll
      for (int j = 0; j < NO; ++j)
        *reinterpret_cast<float4*>(dst + (tx + 16 * j) * 4) =
            make_float4(o[i][j].x * f, o[i][j].y * f, o[i][j].z * f, o[i][j].w * f);
      if (tx == 0) {
        if (!begins) p.cml[at_c] = make_float2(m[i], pp_odd(l[i], odd));
        else (prefix_unit ? p.qml : p.pml)[rh] = Piece{direct ? __uint_as_float(kPieceDone) : m[i], pp_odd(l[i], odd), ctas, qi};
        if (direct && a.lse) a.lse[rh] = (m[i] + log2f(l[i])) * 0.6931471805599453f;
      }
    }
  };
  // where a unit whose last tile starts at x ends
  auto span = [&](long long x) { return (unsigned)cta | (unsigned)(x < x1 ? 0 : pp_cta(x, part) - cta) << 16; };

  if (x0 < prefix_line) {
    const long long per_g = pp_prefix(p, T);
    const int blocks = (T + p.RP - 1) / p.RP;
    for (int g = pp_cta(x0, per_g); g < nkv && g * per_g < x1; ++g)
      for (int k = 0; k < blocks; ++k) {
        const long long u0 = g * per_g + k * pp_unit(p, p.pt, p.w2);
        if (u0 >= x1) break;
        const int rows = min(p.RP, T - k * p.RP), w = pp_weight(p, rows);
        const int lo = pp_before(p, x0, u0, w, p.pt), hi = pp_before(p, x1, u0, w, p.pt);
        if (hi > lo)
          piece(true, 0, g, k * p.RP, rows, lo, hi - lo, lo == 0, false, p.pt, 0, 0, span(pp_tile(p, u0, w, p.pt - 1)));
      }
  }
  long long u0 = sLL[THREADS / 32];
  for (int b = sStart; b < B && u0 < x1; ++b) {
    PagedReq q;
    if (!pr_request(a.rows, b, &q) || q.n == 0) continue;
    const long long cb = pp_request(p, q.n, q.kv);
    for (int g = 0; g < nkv && u0 < x1; ++g) {
      if (u0 + cb <= x0) {
        u0 += cb;
        continue;
      }
      for (int j = 0; j < q.n; j += p.RP) {
        const int rows = min(p.RP, q.n - j), w = pp_weight(p, rows), tiles = pp_tiles(p, q.kv, j + rows - 1);
        const int lo = pp_before(p, x0, u0, w, tiles), hi = pp_before(p, x1, u0, w, tiles);
        const long long last = pp_tile(p, u0, w, tiles - 1);
        u0 += pp_unit(p, tiles, w);
        if (hi > lo)
          piece(false, b, g, q.base + j, rows, lo, hi - lo, lo == 0, !p.shared && lo == 0 && hi == tiles,
                p.shared ? 0 : p.pt, q.kv + j + 1, q.kv + j + rows, span(last));
      }
    }
  }
  if (first_unit && tid == 0) p.cid[cta] = 0;
}

static PagedPlan f32_plan(int T, int B, int nq, int nkv, int prefix) {
  PagedPlan p{};
  p.G = nq / nkv;
  p.RT = pf::TQ / p.G;
  p.RP = p.RT;
  p.tk_log2 = 6;
  p.pt = (prefix + pf::TK - 1) / pf::TK;
  p.w1 = p.w2 = 10;
  p.o1 = p.o2 = 5;
  p.shared = pp_pack(p, T, B, prefix);
  p.ncta = 2 * num_sms();
  return p;
}

size_t paged_attn_f32_ws_bytes(int T, int B, int nq, int nkv, int hd, int prefix) {
  PagedPlan p = f32_plan(T, B, nq, nkv, prefix);
  return pp_layout(p, T, nq, hd, nullptr);
}

template <int HD>
static cudaError_t launch_f32(const PagedAttnArgs& a, const PagedPlan& p, int probe_op, cudaStream_t st) {
  constexpr int smem = pf::Cfg<HD>::SMEM;
  static std::atomic<unsigned long long> attr{0};
  cudaError_t e = once_per_device(
      attr, [] { return cudaFuncSetAttribute(paged_attn_f32<HD>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem); });
  if (e != cudaSuccess) return e;
  probe_start(probe_op, st);
  launch_pdl(paged_attn_f32<HD>, dim3(p.ncta), pf::THREADS, smem, st, a, p);
  note_launch();
  probe_stop(probe_op, st);
  launch_combine<float, HD>(a, p, st);
  return cudaGetLastError();
}

cudaError_t launch_paged_attn_f32(const PagedAttnArgs& a, int probe_op, cudaStream_t st) {
  PagedPlan p = f32_plan(a.rows.T, a.rows.B, a.nq, a.nkv, a.prefix);
  pp_layout(p, a.rows.T, a.nq, a.hd, static_cast<char*>(a.ws));
  return a.hd == 128 ? launch_f32<128>(a, p, probe_op, st) : launch_f32<64>(a, p, probe_op, st);
}

}  // namespace pe

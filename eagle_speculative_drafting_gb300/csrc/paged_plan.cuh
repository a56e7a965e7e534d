// How the work of the paged attention is cut, shared by the kernel that
// computes the pieces and the one that joins them.
//
// A unit is one key head's queries of a block of consecutive rows, against
// one list of keys, which goes by in tiles of TK keys. With `shared`, the
// rows of all requests are packed into blocks against the prefix
// ("prefix units") and each request's own rows into blocks against its own
// tokens; otherwise a request's blocks take the prefix's tiles first, then
// their own. All units' tiles lie on one line of costs (prefix units first:
// key head outermost, so that the blocks that read the same keys run at the
// same time; then request by request), and CTA c takes the tiles that start
// in its n-th of the line: every CTA has the same cost whatever the lengths
// are, and a unit has at most one piece per CTA.
#pragma once
#include <math.h>

#include <type_traits>

#include "paged.cuh"

namespace pe {

// A row's part of a unit's first piece: maximum (log2 units) and sum, whose
// sign bit is set when the piece met infinite or NaN elements of V that only
// some of the unit's rows see (pp_odd); the CTA that has it and how many CTAs
// after it may have more of the unit; the row's place in the unit.
struct __align__(16) Piece {
  float m, l;
  unsigned ctas;   // first | following << 16
  int qi;
};
// a unit's name, for the pieces that continue it
__device__ __forceinline__ unsigned long long piece_id(int row0, int g, int prefix) {
  return 1 + (((unsigned long long)row0 << 12 | g) << 1 | prefix);
}

struct PagedPlan {
  int RT;          // rows of one query tile (RT * G <= the tile's query rows)
  int RP;          // rows of a unit: two query tiles
  int pt;          // key tiles of the prefix
  int shared;
  int w1, w2;      // cost of a key tile against one query tile, against two
  int o1, o2;      // cost of such a unit beside its tiles
  int tk_log2;
  int G, ncta;
  // workspace
  Piece *pml, *qml;    // first pieces by (row, head): of request units, of prefix units
  float *po, *qo;      // their outputs, unnormalised [T*nq][hd]
  float2* cml;         // pieces that continue a unit begun by an earlier CTA: maximum and sum,
  float* co;           // output [ncta][RP*G][hd]
  unsigned long long* cid;   // [ncta] which unit CTA c's piece continues (0: none)
};
// Mark in the place of a first piece's maximum: the row is finished (a NaN
// payload no maximum has).
constexpr unsigned kPieceDone = 0x7fc0d0e5u;
// Odd elements. A V element of a token that some rows of a unit see and others
// do not takes part in the unit's product with weight 0 for the latter, and
// 0 * inf or 0 * NaN is NaN. Such elements are taken out of the tile; the
// joining kernel adds them to the rows that see their token (a weight is
// positive: what it multiplies them by changes nothing). The sum's sign bit
// says that there are some.
__device__ __forceinline__ float pp_odd(float l, bool odd) {
  return odd ? __uint_as_float(__float_as_uint(l) | 0x80000000u) : l;
}
__device__ __forceinline__ bool pp_is_odd(float l) { return __float_as_uint(l) >> 31; }

__host__ __device__ __forceinline__ int pp_weight(const PagedPlan& p, int rows) { return rows > p.RT ? p.w2 : p.w1; }
// cost of a unit, and where its tile i starts when the unit starts at u0
// (its own cost comes with its first tile)
__host__ __device__ __forceinline__ long long pp_unit(const PagedPlan& p, int tiles, int w) {
  return (w == p.w2 ? p.o2 : p.o1) + (long long)tiles * w;
}
__device__ __forceinline__ long long pp_tile(const PagedPlan& p, long long u0, int w, int i) {
  return i > 0 ? u0 + pp_unit(p, i, w) : u0;
}
// key tiles of the block of a request whose last row is row `last`
__device__ __forceinline__ int pp_tiles(const PagedPlan& p, int kv, int last) {
  return (p.shared ? 0 : p.pt) + (int)(((long long)kv + last + (1 << p.tk_log2)) >> p.tk_log2);
}
// cost of a request's blocks [0, blocks) for one key head
__device__ __forceinline__ long long pp_blocks(const PagedPlan& p, int n, int kv, int blocks) {
  long long c = 0;
  for (int k = 0; k < blocks; ++k) {
    const int rows = min(p.RP, n - k * p.RP);
    c += pp_unit(p, pp_tiles(p, kv, k * p.RP + rows - 1), pp_weight(p, rows));
  }
  return c;
}
__device__ __forceinline__ long long pp_request(const PagedPlan& p, int n, int kv) {
  return pp_blocks(p, n, kv, (n + p.RP - 1) / p.RP);
}
// how much of that is the units' own
__device__ __forceinline__ long long pp_own(const PagedPlan& p, int n) {
  const int full = n / p.RP, rest = n - full * p.RP;
  return (long long)full * (p.RP > p.RT ? p.o2 : p.o1) + (rest > p.RT ? p.o2 : rest > 0 ? p.o1 : 0);
}
// prefix units: cost of one key head's
__device__ __forceinline__ long long pp_prefix(const PagedPlan& p, int T) {
  if (!p.shared) return 0;
  const int blocks = (T + p.RP - 1) / p.RP;
  return (blocks - 1) * pp_unit(p, p.pt, p.w2) + pp_unit(p, p.pt, pp_weight(p, T - (blocks - 1) * p.RP));
}
// The parts: CTA c of n has [c * part, (c + 1) * part) of the line (where there
// are fewer tiles than CTAs, a part may hold no tile's start). A division
// of 64-bit integers costs as much as a load from memory; the float one is
// scaled up by more than its roundings, so that n parts cover the line, and
// every CTA gets the same result.
__device__ __forceinline__ long long pp_part(long long total, int n) {
  return (long long)(__fdiv_rn(__fmul_rn((float)total, 1.0000005f), (float)n)) + 1;
}
// tiles of a unit that start before x
__device__ __forceinline__ int pp_before(const PagedPlan& p, long long x, long long u0, int w, int tiles) {
  if (x <= u0) return 0;
  const long long y = x - u0 - pp_unit(p, 1, w);   // from where tile 1 starts
  if (y <= 0) return min(1, tiles);
  return y >= (long long)tiles * w ? tiles : min(tiles, 1 + ((int)y + w - 1) / w);
}
// the part that x lies in
__device__ __forceinline__ int pp_cta(long long x, long long part) {
  int c = (int)((float)x / (float)part);
  while ((c + 1) * part <= x) ++c;
  while (c > 0 && c * part > x) --c;
  return c;
}

// -------------------------------------------------------------------------
// Joins the pieces of every (row, head) that the attention kernel did not
// finish: with M the largest of their maxima, out = sum_i o_i 2^(m_i - M) /
// sum_i l_i 2^(m_i - M). LPI lanes take one of them, 32 / LPI side by side in
// a warp. It is bound by the latency of three loads in a row (the first
// pieces' records, the names of the CTAs that may continue them, their
// values), so the first pieces' values are loaded ahead of the lookups and
// further ones several at a time. The blocks an SM holds are given so that the
// compiler spends the registers this takes, 64 to 80: left alone it packs most
// forms into 40 to 48 and the loads go one after the other (one request of 4
// rows 17.2 us with the attention, 15.5 so).
// -------------------------------------------------------------------------
template <typename T, int HD, int LPI>
__global__ void __launch_bounds__(128, HD == 128 && LPI == 8 ? 7 : 6) paged_combine(PagedAttnArgs a, PagedPlan p) {
  pdl_trigger();
  pdl_wait();
  constexpr int IPW = 32 / LPI, E = HD / LPI;   // items of a warp, dims of a lane
  typedef typename std::conditional<E % 4 == 0, float4, float2>::type Vec;
  constexpr int VN = sizeof(Vec) / 4, NV = E / VN, NB = LPI == 32 ? 8 : 2;   // pieces in flight beyond the first
  const int lane = threadIdx.x & 31, sub = lane / LPI, li = lane % LPI;
  const unsigned group = 0xffffffffu >> (32 - LPI) << (sub * LPI);
  const size_t end = (size_t)a.rows.T * a.nq, e0 = ((size_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5)) * IPW;
  if (e0 >= end) return;
  const size_t rh = e0 + sub < end ? e0 + sub : e0;
  const Piece none{-INFINITY, 0.f, 0u, 0};
  Piece P = p.pml[rh];
  bool open = e0 + sub < end && __float_as_uint(P.m) != kPieceDone;
  if (!__any_sync(0xffffffffu, open)) return;
  auto load = [&](const float* from, Vec (&v)[NV]) {
#pragma unroll
    for (int k = 0; k < NV; ++k) v[k] = reinterpret_cast<const Vec*>(from)[li + LPI * k];
  };
  // the first pieces, ahead of the lookups that say whether the row is one
  const Piece Q = p.shared ? p.qml[rh] : none;
  Vec vp[NV] = {}, vq[NV] = {};
  if (open) load(p.po + rh * HD, vp);
  if (open && p.shared) load(p.qo + rh * HD, vq);
  int r = (int)(e0 / a.nq), h = (int)(e0 % a.nq) + (int)(rh - e0);
  while (h >= a.nq) {
    h -= a.nq;
    ++r;
  }
  const int g = h / p.G;
  PagedReq q{};
  int b = 0;
  for (int k = 0, seen = -1; k < IPW; ++k) {   // (mostly one row)
    const int rk = __shfl_sync(0xffffffffu, r, k * LPI);
    if (rk != seen) {
      PagedReq x;
      bool ok;
      const int bk = pr_lookup(a.rows, rk, &x, &ok);
      if (r == rk) {
        q = x;
        b = bk;
        open = open && ok && r >= x.base && r < x.base + x.n;
      }
      seen = rk;
    }
  }
  bool odd = pp_is_odd(P.l);   // (a prefix's tokens are seen by all)
  P.l = fabsf(P.l);
  // a piece that saw nothing has no sum (or a NaN one, which stays)
  auto weight = [](float m, float l, float M) { return l != l ? l : (m == -INFINITY ? 0.f : exp2f(m - M)); };
  float M = fmaxf(P.m, Q.m);
  const float fp = weight(P.m, P.l, M), fq = weight(Q.m, Q.l, M);
  float l = P.l * fp + Q.l * fq, o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const float x = reinterpret_cast<const float*>(&vp[e / VN])[e % VN], y = reinterpret_cast<const float*>(&vq[e / VN])[e % VN];
    o[e] = x * fp + (p.shared ? y * fq : 0.f);
  }
  // pieces of later CTAs: the request unit's, then the prefix unit's (the
  // bounds only matter after a wait ran out and left a record unwritten)
  const int cn = open ? min((int)(P.ctas >> 16), p.ncta) : 0, dn = open ? min((int)(Q.ctas >> 16), p.ncta) : 0;
  for (int i0 = 0; __any_sync(0xffffffffu, i0 < cn + dn); i0 += LPI) {
    const int i = i0 + li;
    const bool own = i < cn;
    const Piece& F = own ? P : Q;
    int at = -1;
    float mi = -INFINITY, sum = 0.f;
    if (i < cn + dn) {
      // (a CTA's part may hold no tile's start; its slot is loaded along)
      const int c = min((int)(F.ctas & 0xffffu) + 1 + (own ? i : i - cn), p.ncta - 1);
      const int to = c * p.RP * p.G + min(max(F.qi, 0), p.RP * p.G - 1);
      const unsigned long long id = p.cid[c];
      const float2 v = p.cml[to];
      if (id == piece_id(r - F.qi / p.G, g, !own)) {
        at = to;
        mi = v.x;
        sum = v.y;
      }
    }
    odd |= (__ballot_sync(0xffffffffu, pp_is_odd(sum)) & group) != 0;
    sum = fabsf(sum);
    float top = mi;
#pragma unroll
    for (int w = 1; w < LPI; w <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
    const float Mn = fmaxf(M, top);
    const float fo = M == -INFINITY ? 0.f : exp2f(M - Mn);
    const float f = weight(mi, sum, Mn);
    sum *= f;
#pragma unroll
    for (int w = 1; w < LPI; w <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
    l = l * fo + sum;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] *= fo;
    M = Mn;
    unsigned live = __ballot_sync(0xffffffffu, at >= 0) & group;
    while (__any_sync(0xffffffffu, live != 0)) {
      Vec v[NB][NV] = {};
      float w[NB];
#pragma unroll
      for (int z = 0; z < NB; ++z) {
        const int src = live ? __ffs(live) - 1 : lane;
        const int from = __shfl_sync(0xffffffffu, at, src);
        w[z] = __shfl_sync(0xffffffffu, f, src);
        if (live) load(p.co + (size_t)from * HD, v[z]);
        else w[z] = 0.f;
        live &= live - 1;
      }
#pragma unroll
      for (int z = 0; z < NB; ++z)
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] += reinterpret_cast<const float*>(&v[z][e / VN])[e % VN] * w[z];
    }
  }
  if (open && odd) {   // the unit's tokens behind its first row's, up to this row's own
    const int last = q.kv + (r - q.base), back = min(max(P.qi, 0), p.RP * p.G - 1) / p.G;
    for (int t = max(last - back + 1, q.kv); t <= last; ++t) {
      const int page = a.rows.table[(size_t)b * a.rows.max_pages + (t >> a.rows.ps_log2)];
      if (page < 0 || page >= a.rows.num_pages) continue;
      const size_t slot = ((size_t)page << a.rows.ps_log2) + (t & ((1 << a.rows.ps_log2) - 1));
      const T* v = static_cast<const T*>(a.v_pages) + (slot * a.nkv + g) * HD;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float x = to_f(v[(li + LPI * (e / VN)) * VN + e % VN]);
        if (!(fabsf(x) < INFINITY)) o[e] += x;
      }
    }
  }
  if (open) {
    const float inv = 1.f / l;
    T* out = static_cast<T*>(a.out) + rh * HD;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      T t[VN];
#pragma unroll
      for (int e = 0; e < VN; ++e) t[e] = from_f<T>(o[k * VN + e] * inv);
      typedef typename std::conditional<sizeof t == 16, uint4, typename std::conditional<sizeof t == 8, uint2, uint32_t>::type>::type Raw;
      reinterpret_cast<Raw*>(out)[li + LPI * k] = *reinterpret_cast<const Raw*>(t);
    }
    if (a.lse && li == 0) a.lse[rh] = (M + log2f(l)) * 0.6931471805599453f;
  }
}

template <typename T, int HD>
inline void launch_combine(const PagedAttnArgs& a, const PagedPlan& p, cudaStream_t st) {
  // About one wave of warps (40 to an SM): a warp each, eight pieces in flight
  // (one request of 4 rows, 17 pieces to a row: 15.6 us with the attention, 16
  // lanes 19.7, eight 23.9; 2000 items 26.4, 27.1, 28.6). More: eight lanes,
  // whose warps wait for four at once (16384 items of two or three pieces: 81.1
  // us, 16 lanes 82.2, a warp each 89.6; 114000, a third of them open: 192.6,
  // 194.8, 217.8).
  const size_t items = (size_t)a.rows.T * a.nq;
  if (items <= (size_t)num_sms() * 40)
    launch_pdl(paged_combine<T, HD, 32>, dim3((unsigned)((items + 3) / 4)), 128, 0, st, a, p);
  else
    launch_pdl(paged_combine<T, HD, 8>, dim3((unsigned)((items + 15) / 16)), 128, 0, st, a, p);
  note_launch();
}

// ---- host side of the plan
// Whether rows are packed against the prefix. Query tiles of a key head when
// they are, and request by request (taken as equally long): packing saves the
// prefix's tiles of the difference, and pays with pieces of every row to
// write and join, about the traffic of four key tiles for each query tile.
inline int pp_pack(const PagedPlan& p, int T, int B, int prefix) {
  const long long packed = (T + p.RT - 1) / p.RT;
  const long long apart = (long long)B * (((T + B - 1) / B + p.RT - 1) / p.RT);
  return prefix > 0 && (apart - packed) * p.pt > 4 * packed;
}
// Sets the plan's workspace pointers (base NULL: only measures).
inline size_t pp_layout(PagedPlan& p, int T, int nq, int hd, char* base) {
  size_t off = 0;
  auto take = [&](size_t bytes) {
    char* q = base ? base + off : nullptr;
    off += (bytes + 255) & ~size_t(255);
    return q;
  };
  const size_t th = (size_t)T * nq, cr = (size_t)p.ncta * p.RP * p.G;
  p.cid = reinterpret_cast<unsigned long long*>(take((size_t)p.ncta * 8));
  p.pml = reinterpret_cast<Piece*>(take(th * sizeof(Piece)));
  p.cml = reinterpret_cast<float2*>(take(cr * 8));
  p.co = reinterpret_cast<float*>(take(cr * hd * 4));
  p.po = reinterpret_cast<float*>(take(th * hd * 4));
  if (p.shared) {
    p.qml = reinterpret_cast<Piece*>(take(th * sizeof(Piece)));
    p.qo = reinterpret_cast<float*>(take(th * hd * 4));
  }
  return off;
}

}  // namespace pe

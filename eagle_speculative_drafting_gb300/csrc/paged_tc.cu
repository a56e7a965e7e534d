// Paged attention on the 5th-generation tensor cores (bf16).
//
// Per query row i with scores s_ij = scale q_i k_j: a running maximum m_i,
// l_i = sum_j 2^(s_ij log2 e - m_i) and o_i = sum_j 2^(s_ij log2 e - m_i) v_j
// in one pass over the key tiles; out = o_i / l_i, lse = (m_i + log2 l_i) ln 2.
//
// One persistent CTA per SM takes an equal share of the line of key tiles
// (paged_plan.cuh), 512 threads:
//   warps 0-3   add up the line and find where the CTA's part begins; then
//   warp 0      scheduler: walks the CTA's part of the line, hands out units
//               (a block of rows of one key head, a range of key tiles)
//               through a small ring in shared memory and loads their Q,
//               rows x heads of a key head as one box;
//   warps 12-15 K/V producers, two for K and two for V: per tile of 128 keys
//               one TMA box per page and 64 columns, into a ring of stages
//               that K and V share. Four warps, because a box costs its warp
//               70 cycles to issue whatever its size (16-token pages: 16
//               boxes a stage), and warps issue side by side; page numbers
//               come from the tables 32 at a time, a load ahead;
//   warp 2      issues tcgen05.mma: S = Q K^T (128 query rows x 128 keys)
//               and O += P V, P read from TMEM, V as it is stored (its keys
//               are the contracted index: no transposed copy). A stream's
//               PV and its next scores go out together, the streams in turn:
//               side by side they would end together, and then both groups'
//               softmax would run at the same time and the tensor cores wait
//               for both;
//   warps 4-7, 8-11   two softmax groups, one thread per query row: scores
//               out of TMEM, running maximum and sum, P back over the scores.
// There are two streams of score and output tiles in TMEM, A and B, one per
// softmax group, so that one group's exponentials run under the other's
// products. A unit of more than 128 query rows gives each stream its own 128
// rows and both read every key tile: K and V cross the L2 once for 256 rows.
// A unit of at most 128 rows gives the streams alternate key tiles of the
// same rows, joined at the end: a batch's single steps are bound by reading
// K and V, and what counts there is that a tile's latency hides under the
// other's.
// Products of one thread run in the order of issue, so the scores of a
// stream's next tile may be issued right behind the product that reads its
// P; the commit behind a score product covers the stream's earlier products,
// so a thread that has seen its scores may rescale O without a further wait.
// The reference maximum of a row is only raised (and O rescaled) when a tile
// exceeds it by more than 2^8; in between, weights relative to the older
// maximum stay below 256. P is rounded to bf16 for the product (relative
// 2^-8 of each weight); sums and maxima are fp32.
// Keys behind the last token of a unit may hold anything: their scores are
// dropped and their V rows zeroed in shared memory (0 * NaN). A token that
// some rows of a unit see and others do not may be NaN or infinite in V too;
// such elements are zeroed as well, and the joining kernel adds them to the
// rows that see them (paged_plan.cuh).
// Every wait is bounded; on expiry the kernel sets PEAGLE_DEV_TIMEOUT,
// drains what it issued and returns.
//
// What bounds it, and what it measured (bf16, head_dim 128; measured copy
// 6.78 TB/s, library product 1.92 PFLOP/s):
//   64 requests x 8 rows, own contexts of 512 to 8192 tokens, 32/8 heads: the
//     bytes of K and V, 197 to 203 us at 6.1 to 6.3 TB/s;
//   48 requests, 529 rows behind 40000 shared tokens: the softmax of a stream
//     (two query tiles against a key tile take 2800 to 3100 cycles, their four
//     products 2048), 303 to 318 us at 1.1 to 1.2 PFLOP/s;
//   one request, 4 rows, 2048 tokens: latency, 15.5 us, of which the joining
//     kernel is 5.7 and fetching instructions about 4.
// Tried and slower: two threads per row (16 softmax warps; 360 against 318 us
// at 40000 shared tokens), P in shared memory, 64-key score tiles (a product
// with N = 64 takes as long as one with N = 128), rows copied in the query tile.
#include "paged_plan.cuh"
#include "tc.cuh"

namespace pe {

namespace pt {
constexpr int TK = 128, THREADS = 512, SERVICE = 128, NU = 4, NODD = 2 * NU;
constexpr int BOX = 128 * 128;        // 128 rows x 64 bf16 columns
constexpr float kRescale = 8.f;       // log2 headroom before the reference maximum moves
// register shares of the scheduler's and issuer's warps, of the softmax groups
// and of the producers: 80 * 128 + 192 * 256 + 48 * 128 = 65536, the launch's
// 128 * 512
constexpr int kRegLaunch = 128, kRegService = 80, kRegSoftmax = 192, kRegProducer = 48;
static_assert(kRegService * 128 + kRegSoftmax * 256 + kRegProducer * 128 <= kRegLaunch * THREADS, "register shares");
enum { U_TWO = 1, U_DIRECT = 2, U_FIRST = 4, U_PREFIX = 8, U_END = 16 };

struct Unit {
  int flags, b, g, row0, rows;   // rows: of the unit (both query tiles)
  int t0, nt;                    // key tiles [t0, t0 + nt) of the unit's list
  int pt;                        // how many of the list are the prefix's
  int vis0;                      // own tokens the first row sees
  int own;                       // own tokens the last row sees
  unsigned ctas;                 // of a first piece: this CTA | how many more CTAs the unit may cross << 16
  int pad[5];
};

template <int HD>
struct Cfg {
  static constexpr int NH = HD / 64;              // 64-column boxes per row
  static constexpr int TB = NH * BOX;             // a Q, K or V tile
  static constexpr int NS = HD == 128 ? 5 : 10;   // K/V ring stages
  static constexpr int SMEM = (2 + NS) * TB + NU * sizeof(Unit) + 4 * 128 * 4 + 704;
};
// one lane of a converged warp, always the same
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(r));
  return r != 0;
}
__device__ __forceinline__ int kpos(int t) { return t == 0 ? 0 : 2 * t - 1; }
__device__ __forceinline__ int vpos(int t, int nt) { return t < nt - 1 ? 2 * t + 2 : 2 * nt - 1; }

// a * b + c on two packed floats
__device__ __forceinline__ void fma2(float& x, float& y, float b, float c) {
  asm("{\n .reg .b64 p, q, r;\n mov.b64 p, {%0, %1};\n mov.b64 q, {%2, %2};\n mov.b64 r, {%3, %3};\n"
      " fma.rn.f32x2 p, p, q, r;\n mov.b64 {%0, %1}, p;\n}"
      : "+f"(x), "+f"(y)
      : "f"(b), "f"(c));
}
__device__ __forceinline__ void add2(float& x, float& y, float a, float b) {
  asm("{\n .reg .b64 p, q;\n mov.b64 p, {%0, %1};\n mov.b64 q, {%2, %3};\n add.rn.f32x2 p, p, q;\n"
      " mov.b64 {%0, %1}, p;\n}"
      : "+f"(x), "+f"(y)
      : "f"(a), "f"(b));
}
}  // namespace pt

template <int HD>
__global__ void __launch_bounds__(pt::THREADS, 1)
    paged_attn_tc(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                  const __grid_constant__ CUtensorMap tmV, PagedAttnArgs a, PagedPlan p, unsigned long long wait_ns) {
  using namespace pt;
  using C = Cfg<HD>;
  constexpr int NS = C::NS, TB = C::TB, NH = C::NH;
  extern __shared__ __align__(1024) uint8_t smem[];   // no slack to align by hand: the tiles fill it
  uint8_t* sQ = smem;                 // [2][TB]
  uint8_t* sKV = sQ + 2 * TB;         // [NS][TB]
  Unit* sU = reinterpret_cast<Unit*>(sKV + NS * TB);            // [NU]
  float* sM = reinterpret_cast<float*>(sU + NU);                // [2 streams][128] row maxima
  float* sL = sM + 256;                                         // [2][128] row sums
  uint64_t* ufull = reinterpret_cast<uint64_t*>(sL + 256);      // [NU]
  uint64_t* uempty = ufull + NU;      // [NU]
  uint64_t* kvfull = uempty + NU;     // [NS]
  uint64_t* kvempty = kvfull + NS;    // [NS]
  uint64_t* qfull = kvempty + NS;     // [2]
  uint64_t* qempty = qfull + 2;       // [2]
  uint64_t* sfull = qempty + 2;       // [2] a stream's scores are in TMEM
  uint64_t* pfull = sfull + 2;        // [2 streams][2 halves] its P of 64 keys is, and its O is rescaled
  uint64_t* odone = pfull + 4;        // [2] every product of a stream's part of a unit has completed
  uint64_t* exch = odone + 2;         // [2] both groups wrote their maxima and sums; both have read O
  uint64_t* drain = exch + 2;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tslot + 1);
  volatile int* sIssued = abort_flag + 1;   // [5] ring positions the producers filled, Q copies issued
  // [NODD] in slot u % NODD 1 + unit u when it met odd elements of V. Warps
  // are at different units at a time: one that has still to look at unit u's
  // mark has signed uempty for no later unit, so no unit behind u + NU is
  // handed out and NODD > NU slots never meet.
  volatile int* sOdd = sIssued + 5;
  int* sStart = const_cast<int*>(sOdd + NODD);   // [4] request the CTA begins with; its rows, cached tokens, first row
  long long* sLL = reinterpret_cast<long long*>((reinterpret_cast<uintptr_t>(sStart + 4) + 7) & ~uintptr_t(7));  // [2 * SERVICE / 32 + 1]

  const int cta = blockIdx.x, nkv = a.nkv;
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < NU; ++i) {
      tc::mbar_init(&ufull[i], 1);
      tc::mbar_init(&uempty[i], 13);   // four producers, the issuer, eight softmax warps
    }
    for (int i = 0; i < NS; ++i) {
      tc::mbar_init(&kvfull[i], 4);
      tc::mbar_init(&kvempty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&qfull[i], 1);
      tc::mbar_init(&qempty[i], 1);
      tc::mbar_init(&sfull[i], 1);
      tc::mbar_init(&pfull[i], 4);
      tc::mbar_init(&pfull[2 + i], 4);
      tc::mbar_init(&odone[i], 1);
      tc::mbar_init(&exch[i], 8);
    }
    for (int i = 0; i < NODD; ++i) sOdd[i] = 0;
    for (int i = 0; i < 5; ++i) sIssued[i] = 0;
    tc::mbar_init(drain, 1);
    *abort_flag = 0;
    sStart[0] = a.rows.B;
    sStart[1] = 0;
    tc::fence_mbar_init();
    tc::prefetch_map(&tmQ);
    tc::prefetch_map(&tmK);
    tc::prefetch_map(&tmV);
  }
  pdl_trigger();
  pdl_wait();   // rows, lengths, tables, q and pages come from earlier kernels
  // all of TMEM, so not before the predecessor is done with its part of it
  if (warp == 2) tc::tmem_alloc(tslot, 512);
  tc::fence_before();

  __syncthreads();
  tc::fence_after();
  const uint32_t tbase = *tslot;

  auto wait = [&](uint64_t* bar, uint32_t par) -> bool {
    if (tc::mbar_test_wait(bar, par)) return true;
    if (*abort_flag) return false;
    if (wait_ns != 0 && tc::mbar_wait_for(bar, par, wait_ns)) return true;   // (0: one try)
    if (!*abort_flag) {
      *abort_flag = 1;
      set_status(a.status, PEAGLE_DEV_TIMEOUT);
    }
    return false;
  };

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegService));
    auto bar_service = [] { asm volatile("bar.sync 1, %0;" ::"n"(SERVICE) : "memory"); };
    // ---- the line: every CTA adds up all requests' costs
    const int B = a.rows.B;
    const int per = (B + SERVICE - 1) / SERVICE, b_lo = min(tid * per, B), b_hi = min(b_lo + per, B);
    long long mine = 0, bare = 0;   // without the units' own cost
    PagedReq q;
    for (int b = b_lo; b < b_hi; ++b) {
      if (pr_request(a.rows, b, &q)) {
        const long long c = pp_request(p, q.n, q.kv);
        mine += nkv * c;
        bare += nkv * (c - pp_own(p, q.n));
      } else if (cta == 0) {
        set_status(a.status, PEAGLE_DEV_BOUNDS);
      }
    }
    long long incl = mine, incl_b = bare;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, incl, o), z = __shfl_up_sync(0xffffffffu, incl_b, o);
      if (lane >= o) {
        incl += y;
        incl_b += z;
      }
    }
    if (lane == 31) {
      sLL[warp] = incl;
      sLL[SERVICE / 32 + warp] = incl_b;
    }
    bar_service();
    long long at = incl - mine, at_b = incl_b - bare, total = 0, total_b = 0;
    for (int i = 0; i < SERVICE / 32; ++i) {
      const long long x = sLL[i], y = sLL[SERVICE / 32 + i];
      at += i < warp ? x : 0;
      at_b += i < warp ? y : 0;
      total += x;
      total_b += y;
    }
    long long prefix_line = nkv * pp_prefix(p, a.rows.T);
    const long long prefix_b = prefix_line - (p.shared ? nkv * pp_own(p, a.rows.T) : 0);
    // no more tiles than CTAs: one each, wherever units begin
    const bool few = total_b + prefix_b <= (long long)p.ncta * p.w1;
    if (few) {
      p.o1 = p.o2 = 0;
      at = at_b;
      total = total_b;
      mine = bare;
      prefix_line = prefix_b;
    }
    at += prefix_line;
    total += prefix_line;
    const long long part = pp_part(total, p.ncta), x0 = cta * part, x1 = min(x0 + part, total);
    const bool working = x0 < total;
    for (int b = b_lo; b < b_hi; ++b) {
      // (up to a request per thread, what the first pass found is at hand)
      const long long c = per == 1 ? mine : pr_request(a.rows, b, &q) ? nkv * pp_request(p, q.n, q.kv) : 0;
      // the request whose tiles x0 falls among; behind prefix units the first
      if (working && (x0 < prefix_line ? b == 0 : at <= x0 && x0 < at + c)) {
        sStart[0] = b;
        sStart[1] = c > 0 ? q.n : 0;
        sStart[2] = q.kv;
        sStart[3] = q.base;
        sLL[2 * (SERVICE / 32)] = at;
      }
      at += c;
    }
    bar_service();
    if (warp == 0) {
      // ---------------------------------------------------------- scheduler
      int u = 0, qpos = 0;
      auto push = [&](const Unit& d) -> bool {
        if (!__all_sync(0xffffffffu, wait(&uempty[u % NU], ((u / NU) & 1) ^ 1))) return false;
        if (lane == 0) {
          sU[u % NU] = d;
          tc::mbar_arrive(&ufull[u % NU]);
          // the CTA's first unit may be one that another began
          if (u == 0) p.cid[cta] = (d.flags & (U_FIRST | U_END)) ? 0 : piece_id(d.row0, d.g, (d.flags & U_PREFIX) != 0);
        }
        __syncwarp();
        ++u;
        for (int X = 0; X < ((d.flags & U_END) ? 0 : (d.flags & U_TWO) ? 2 : 1); ++X) {
          const int s = qpos & 1;
          if (!__all_sync(0xffffffffu, wait(&qempty[s], ((qpos >> 1) & 1) ^ 1))) return false;
          if (lane == 0) {
            tc::mbar_expect_tx(&qfull[s], (uint32_t)(p.RT * p.G) * 128 * NH);
            for (int hf = 0; hf < NH; ++hf)
              tc::tma_load_3d(sQ + s * TB + hf * BOX, &tmQ, hf * 64, d.g * p.G, d.row0 + X * p.RT, &qfull[s]);
          }
          __syncwarp();
          ++qpos;
        }
        return true;
      };
      // where a unit whose last tile starts at x ends
      auto span = [&](long long x) { return (unsigned)cta | (unsigned)(x < x1 ? 0 : pp_cta(x, part) - cta) << 16; };
      bool go = working;
      const int T = a.rows.T;
      if (x0 < prefix_line) {
        const long long per_g = pp_prefix(p, T);
        const int blocks = (T + p.RP - 1) / p.RP;
        for (int g = pp_cta(x0, per_g); go && g < nkv && g * per_g < x1; ++g)
          for (int k = 0; go && k < blocks; ++k) {
            const long long u0 = g * per_g + k * pp_unit(p, p.pt, p.w2);
            if (u0 >= x1) break;
            const int rows = min(p.RP, T - k * p.RP), w = pp_weight(p, rows);
            const int lo = pp_before(p, x0, u0, w, p.pt), hi = pp_before(p, x1, u0, w, p.pt);
            if (hi <= lo) continue;
            Unit d{};
            d.flags = U_PREFIX | (rows > p.RT ? U_TWO : 0) | (lo == 0 ? U_FIRST : 0);
            d.g = g;
            d.row0 = k * p.RP;
            d.rows = rows;
            d.t0 = lo;
            d.nt = hi - lo;
            d.pt = p.pt;
            d.ctas = span(pp_tile(p, u0, w, p.pt - 1));
            go = push(d);
          }
      }
      // a request's units, key head by key head
      long long u0 = sLL[2 * (SERVICE / 32)];
      auto request = [&](int b, int n, int kv, int base, long long cb) {
        for (int g = 0; go && g < nkv && u0 < x1; ++g) {
          if (u0 + cb <= x0) {
            u0 += cb;
            continue;
          }
          for (int j = 0; go && j < n; j += p.RP) {
            const int rows = min(p.RP, n - j), w = pp_weight(p, rows), tiles = pp_tiles(p, kv, j + rows - 1);
            const int lo = pp_before(p, x0, u0, w, tiles), hi = pp_before(p, x1, u0, w, tiles);
            const long long last = pp_tile(p, u0, w, tiles - 1);
            u0 += pp_unit(p, tiles, w);
            if (hi <= lo) continue;
            Unit d{};
            d.flags = (rows > p.RT ? U_TWO : 0) | (lo == 0 ? U_FIRST : 0) |
                      (!p.shared && lo == 0 && hi == tiles ? U_DIRECT : 0);
            d.b = b;
            d.g = g;
            d.row0 = base + j;
            d.rows = rows;
            d.t0 = lo;
            d.nt = hi - lo;
            d.pt = p.shared ? 0 : p.pt;
            d.vis0 = kv + j + 1;
            d.own = kv + j + rows;
            d.ctas = span(last);
            go = push(d);
          }
        }
      };
      // the first one's lengths were found above, the next 32's are loaded
      // while its units go out, and so on
      int b0 = sStart[0] + 1, lo = 0, hi = 0, kv = -1;
      auto fetch = [&]() {
        if (b0 + lane < B) {
          lo = a.rows.off[b0 + lane];
          hi = a.rows.off[b0 + lane + 1];
          kv = a.rows.kv_len[b0 + lane];
        }
      };
      fetch();
      if (go && u0 < x1 && sStart[1] > 0)
        request(sStart[0], sStart[1], sStart[2], sStart[3], pp_request(p, sStart[1], sStart[2]));
      while (go && b0 < B && u0 < x1) {
        PagedReq r{};
        const bool valid = b0 + lane < B && pr_check(a.rows, b0 + lane, lo, hi, kv, &r);
        const long long cost = valid ? pp_request(p, r.n, r.kv) : 0;
        const int first = b0;
        b0 += 32;
        fetch();
        for (int i = 0; go && i < 32 && first + i < B && u0 < x1; ++i) {
          const long long cb = __shfl_sync(0xffffffffu, cost, i);
          const int n = __shfl_sync(0xffffffffu, r.n, i), k = __shfl_sync(0xffffffffu, r.kv, i);
          const int base = __shfl_sync(0xffffffffu, r.base, i);
          if (cb > 0) request(first + i, n, k, base, cb);
        }
      }
      if (go || !working) {
        Unit d{};
        d.flags = U_END;
        push(d);
      }
      if (lane == 0) sIssued[4] = qpos;
    } else if (warp == 2) {
      // -------------------------------------------------------- MMA issuer
      // The whole warp walks the units and waits; one lane issues. What the
      // operands are made of is uniform (broadcast from lane 0), so that the
      // descriptors live in uniform registers: issuing eight products from a
      // single lane's own values took 900 cycles, more than their execution.
      constexpr uint32_t idS = tc::idesc_bf16(128, 128), idO = tc::idesc_bf16(128, HD) | tc::kIdescBmn;
      auto uni = [](uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); };
      auto waitw = [&](uint64_t* bar, uint32_t par) -> bool { return __all_sync(0xffffffffu, wait(bar, par)); };
      const uint32_t tb = uni(tbase);
      const uint64_t dk0 = tc::sw128_desc(tc::smem_u32(sKV)), dv0 = tc::sw128_desc_mn(tc::smem_u32(sKV), BOX);
      const uint64_t dq0 = tc::sw128_desc(tc::smem_u32(sQ));
      int base = 0, qpos = 0, pc0 = 0, pc1 = 0;
      for (int u = 0;; ++u) {
        if (!waitw(&ufull[u % NU], (u / NU) & 1)) break;
        const int flags = uni(sU[u % NU].flags), nt = uni(sU[u % NU].nt);
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&uempty[u % NU]);
        if (flags & U_END) break;
        const bool two = flags & U_TWO;
        const int q = qpos, step = two ? 1 : 2;
        bool ok = waitw(&qfull[q & 1], (q >> 1) & 1);
        if (two) ok = ok && waitw(&qfull[(q + 1) & 1], ((q + 1) >> 1) & 1);
        qpos += two ? 2 : 1;
        // S = Q K^T of a stream's tile t (descriptors count 16-byte units)
        auto scores = [&](int X, int t, int s, bool free) {
          tc::fence_after();
          if (elect_one()) {
            const uint64_t dq = dq0 + ((two ? q + X : q) & 1) * (TB >> 4), dk = dk0 + s * (TB >> 4);
#pragma unroll
            for (int kk = 0; kk < HD / 16; ++kk)
              tc::mma_bf16(tb + X * 128, dq + (kk >> 2) * (BOX >> 4) + (kk & 3) * 2,
                           dk + (kk >> 2) * (BOX >> 4) + (kk & 3) * 2, idS, kk > 0 ? 1u : 0u);
            tc::mma_commit(&sfull[X]);
            if (free) {
              tc::mma_commit(&kvempty[s]);
              if (t == nt - 1) {   // the unit's last
                tc::mma_commit(&qempty[q & 1]);
                if (two) tc::mma_commit(&qempty[(q + 1) & 1]);
              }
            }
          }
          __syncwarp();
        };
        // O += P V of a stream's tile t, the first 64 keys while its softmax
        // is at the others
        auto values = [&](int X, int t, int s, bool free, int pc) -> bool {
          const uint64_t dv = dv0 + s * (TB >> 4);
          const uint32_t more = t >= step ? 1u : 0u;
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            if (!waitw(&pfull[X * 2 + hf], pc & 1)) return false;
            tc::fence_after();
            if (elect_one()) {
#pragma unroll
              for (int kk = hf * (TK / 32); kk < (hf + 1) * (TK / 32); ++kk)
                tc::mma_bf16_tmem_a(tb + 256 + X * 128, tb + X * 128 + kk * 8, dv + kk * (2048 >> 4), idO,
                                    kk > 0 ? 1u : more);
              if (hf == 1) {
                if (free) tc::mma_commit(&kvempty[s]);
                if (t + step > nt - 1) tc::mma_commit(&odone[X]);   // the stream's last of the unit
              }
            }
            __syncwarp();
          }
          return true;
        };
        for (int i = 0; ok && i <= nt; ++i) {
          const int kp = base + kpos(i), sk = kp % NS, vp = base + vpos(i - 1, nt), sv = vp % NS;
          if (i < nt) ok = waitw(&kvfull[sk], (kp / NS) & 1);
          if (i > 0 && two) ok = ok && waitw(&kvfull[sv], (vp / NS) & 1);
          if (!ok) break;
          if (two) {
            if (i > 0) ok = values(0, i - 1, sv, false, pc0++);
            if (!ok) break;
            if (i < nt) scores(0, i, sk, false);
            if (i > 0) ok = values(1, i - 1, sv, true, pc1++);
            if (!ok) break;
            if (i < nt) scores(1, i, sk, true);
          } else {
            if (i < nt) scores(i & 1, i, sk, true);
            if (i > 0) {
              const bool B = !(i & 1);   // tile i - 1 is stream B's
              ok = waitw(&kvfull[sv], (vp / NS) & 1) && values(B, i - 1, sv, true, B ? pc1++ : pc0++);
            }
          }
        }
        if (!ok) break;
        base += 2 * nt;
      }
    }
  } else if (warp >= 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegProducer));
    // -------------------------------------------------------- K/V producers
    const int which = (warp - 12) >> 1, part = warp & 1;   // K or V, which boxes of a stage
    const CUtensorMap* map = which ? &tmV : &tmK;
    const int sh = a.rows.ps_log2, ps = 1 << sh, bx = min(ps, TK), np = TK / bx;
    // this lane's box: page pg of the tile, 64 columns half (a stage's boxes
    // alternate between the two warps)
    const int box = lane * 2 + part, pg = box / NH, half = box % NH;
    const bool mine_box = box < np * NH;
    const int oob = max(a.rows.num_pages << sh, 1);   // a row behind the last: reads zeros
    const uint32_t bytes = (uint32_t)((np * NH + 1 - part) / 2 * bx) * 128;
    const uint32_t dst = half * BOX + pg * bx * 128;
    int base = 0, issued = 0;   // ring position; the last one filled, + 1
    bool ok = true;
    for (int u = 0; ok; ++u) {
      if (!__all_sync(0xffffffffu, wait(&ufull[u % NU], (u / NU) & 1))) break;
      const int flags = sU[u % NU].flags, t0 = sU[u % NU].t0, nt = sU[u % NU].nt, upt = sU[u % NU].pt;
      const int own = sU[u % NU].own, xcol = sU[u % NU].g * HD + half * 64;
      const int* own_pages = a.rows.table + (size_t)sU[u % NU].b * a.rows.max_pages;
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&uempty[u % NU]);
      if (flags & U_END) break;
      // 32 page numbers of the tile's list from entry `first` on, one a lane,
      // and the 32 behind them
      const int* list = nullptr;
      int of_prefix = -1, first = 0, cur = 0, nxt = 0, last = 0;
      auto entry = [&](int i) { return i <= last ? list[i] : -1; };
      // all four pass every stage in the ring's order (K of a tile, then V of
      // the tile before it) and sign it, with their boxes or without: a
      // parity wait tells only two phases apart, so none may miss one
      for (int i = 0; i < 2 * nt; ++i) {
        const bool is_v = (i & 1) == 0 ? i > 0 : i == 2 * nt - 1;
        const int pos = base + i, s = pos % NS;
        int y = oob;
        const bool mine_now = is_v == (which == 1);
        if (mine_now) {
          const int t = is_v ? (i == 2 * nt - 1 ? nt - 1 : i / 2 - 1) : (i + 1) / 2;
          const bool pre = t0 + t < upt;
          const int key0 = (pre ? t0 + t : t0 + t - upt) * TK, end = pre ? a.prefix : own;
          const int p0 = key0 >> sh;
          if (of_prefix != (int)pre) {
            of_prefix = pre;
            list = pre ? a.prefix_pages : own_pages;
            last = (end - 1) >> sh;
            first = p0;
            cur = entry(first + lane);
            nxt = entry(first + 32 + lane);
          } else if (p0 >= first + 32) {
            first += 32;
            cur = nxt;
            nxt = entry(first + 32 + lane);
          }
          // (a tile's pages are at most 16, a power of two: never across the 32)
          const int page = __shfl_sync(0xffffffffu, cur, (p0 - first + pg) & 31);
          if (mine_box && key0 + pg * bx < end) {
            if (page >= 0 && page < a.rows.num_pages) y = (page << sh) + ((key0 + pg * bx) & (ps - 1));
            else set_status(a.status, PEAGLE_DEV_BOUNDS);
          }
        }
        ok = __all_sync(0xffffffffu, wait(&kvempty[s], ((pos / NS) & 1) ^ 1));
        if (!ok) break;
        if (lane == 0) {
          if (mine_now) tc::mbar_expect_tx(&kvfull[s], bytes);
          else tc::mbar_arrive(&kvfull[s]);
        }
        __syncwarp();
        if (mine_now && mine_box) tc::tma_load_2d(sKV + s * TB + dst, map, xcol, y, &kvfull[s]);
        issued = pos + 1;
      }
      base += 2 * nt;
    }
    if (lane == 0) sIssued[warp - 12] = issued;
  } else {
    // ------------------------------------------------------------- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegSoftmax));
    const int X = (warp - 4) >> 2, quad = warp & 3;
    const int row = quad * 32 + lane, wtid = tid - 128 - X * 128;   // query row = TMEM lane; thread of the group
    const uint32_t tl = (uint32_t)(quad * 32) << 16;
    const uint32_t tS = tbase + tl + X * 128, tO = tbase + tl + 256;
    const float sl2 = a.scale * 1.4426950408889634f;
    auto waitw = [&](uint64_t* bar, uint32_t par) -> bool { return __all_sync(0xffffffffu, wait(bar, par)); };
    const int jr = row / p.G, hh = row % p.G;   // row of the query tile, head of the group
    int cnt = 0, base = 0, ex0 = 0, ex1 = 0, oX = 0, oY = 0;   // tiles, ring position, phases of exch and odone (own, other)
    bool owed = false;   // the other group may still be reading O from the last unit
    // Before the first unit a tile of nothing goes through (dry: no waits, no
    // stores): its instructions are fetched while the scheduler and the first
    // loads are at work, instead of when the first scores are there.
    for (int u = -1;; ++u) {
      const bool dry = u < 0;
      if (!dry && !waitw(&ufull[u % NU], (u / NU) & 1)) break;
      Unit d = sU[max(u, 0) % NU];
      __syncwarp();
      if (dry) {
        d.flags = 0;
        d.nt = 2;
        d.t0 = d.pt = 0;
        d.rows = p.RT;
        d.own = 2 * TK;   // (no key to zero)
        d.vis0 = TK / 2;
      } else {
        if (lane == 0) tc::mbar_arrive(&uempty[u % NU]);
        if (d.flags & U_END) break;
      }
      const bool two = d.flags & U_TWO;
      const int nX = two ? d.nt : (X == 0 ? (d.nt + 1) / 2 : d.nt / 2);
      // this thread's query row: row j of the unit, head hh of the group
      const int jX = two && X == 1 ? p.RT : 0;                        // the stream's first row
      const int rowsX = two ? (X == 0 ? p.RT : d.rows - p.RT) : d.rows;
      const bool wlive = quad * 32 < rowsX * p.G, live = row < rowsX * p.G;
      const int j = jX + jr;
      const int vis = d.vis0 + j;
      float m_ref = -INFINITY, l = 0.f;
      bool ok = true;
      for (int i = 0; i < nX; ++i) {
        const int tloc = two ? i : 2 * i + X, t = d.t0 + tloc;
        if (!dry) {
          ok = waitw(&sfull[X], cnt & 1);
          if (!ok) break;
          ++cnt;
        }
        tc::fence_after();
        const bool pre = t < d.pt;
        const int key0 = (pre ? t : t - d.pt) * TK;
        // keys behind the unit's last token, and tokens some of the unit's rows
        // do not see: look at their V (of two query tiles, the first stream does:
        // its product of a key tile is issued before the second's)
        const int valid = (pre ? a.prefix : d.own) - key0;
        const int hide = pre ? TK : d.vis0 - key0;   // first key that the unit's first row does not see
        if ((valid < TK || hide < TK) && !(two && X == 1)) {
          const int pos = base + vpos(tloc, d.nt), s = pos % NS;
          if (!dry) {
            ok = waitw(&kvfull[s], (pos / NS) & 1);
            if (!ok) break;
          }
          uint4* v = reinterpret_cast<uint4*>(sKV + s * TB + wtid * 128);
          if (wtid >= valid) {
#pragma unroll 1
            for (int hf = 0; hf < NH; ++hf)
#pragma unroll
              for (int c = 0; c < 8; ++c) v[hf * (BOX / 16) + (c ^ (wtid & 7))] = make_uint4(0, 0, 0, 0);
          } else if (wtid >= hide) {
            // 0 * x stays 0 unless x is infinite or NaN
            __nv_bfloat162 z = __floats2bfloat162_rn(0.f, 0.f), acc = z;
#pragma unroll 1
            for (int hf = 0; hf < NH; ++hf)
#pragma unroll
              for (int c = 0; c < 8; ++c) {   // (in any order: no need to undo the swizzle)
                const uint4 x = v[hf * (BOX / 16) + (c ^ (wtid & 7))];
                acc = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&x.x), z, acc);
                acc = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&x.y), z, acc);
                acc = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&x.z), z, acc);
                acc = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&x.w), z, acc);
              }
            const float2 bad = __bfloat1622float2(acc);
            if ((bad.x != 0.f || bad.y != 0.f) && !dry) {
              sOdd[u % NODD] = u + 1;
              uint16_t* e = reinterpret_cast<uint16_t*>(v);   // (in any order, as above)
#pragma unroll 1
              for (int k = 0; k < NH * 64; ++k) {
                uint16_t* x = e + (k >> 6) * (BOX / 2) + (k & 63);
                if ((*x & 0x7f80) == 0x7f80) *x = 0;
              }
            }
          }
          tc::fence_proxy_async();
        }
        if (owed) {   // this tile's P lets a product overwrite O
          ok = waitw(&exch[1], ex1 & 1);
          if (!ok) break;
          ++ex1;
          owed = false;
        }
        // P of a half is in TMEM: the product of its 64 keys may start
        auto signal = [&](int hf) {
          tc::tmem_st_wait();
          tc::fence_before();
          __syncwarp();
          if (lane == 0 && !dry) tc::mbar_arrive(&pfull[X * 2 + hf]);
        };
        if (!wlive) {
          signal(0);
        } else {
          uint32_t r[128];
          float* sv = reinterpret_cast<float*>(r);
          // columns this row does not see, in a pass of its own: it is rare, and
          // with the selects in the main path that is half again as long, which
          // the first tiles of a launch spend on fetching instructions
          const int lim = (pre ? a.prefix : vis) - key0;
          if (__any_sync(0xffffffffu, lim < TK)) {
#pragma unroll 1
            for (int c = 0; c < TK; c += 32) {
              uint32_t o[32];
              tc::tmem_ld32_nowait(tS + c, o);
              tc::tmem_ld_wait32(o);
#pragma unroll
              for (int k = 0; k < 32; ++k) o[k] = c + k < lim ? o[k] : 0xff800000u;
              if (!dry) tc::tmem_st32_nowait(tS + c, o);
            }
            tc::tmem_st_wait();
          }
#pragma unroll
          for (int c = 0; c < 4; ++c) tc::tmem_ld32_nowait(tS + c * 32, r + c * 32);
#pragma unroll
          for (int c = 0; c < 4; ++c) tc::tmem_ld_wait32(r + c * 32);
          float pm[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) pm[k] = fmaxf(sv[k], sv[k + 4]);
#pragma unroll
          for (int c = 8; c < TK; c += 8)
#pragma unroll
            for (int k = 0; k < 4; ++k) pm[k] = fmaxf(fmaxf(sv[c + k], sv[c + k + 4]), pm[k]);
          const float mx = fmaxf(fmaxf(pm[0], pm[1]), fmaxf(pm[2], pm[3])) * sl2;
          const bool raise = mx > m_ref + kRescale;   // false while everything is masked
          // (0 when the old maximum lies 2^126 or more below: what was summed
          // under it vanishes from O as it does from l)
          const float corr = !raise ? 1.f : (m_ref == -INFINITY ? 0.f : tc::ex2_approx(m_ref - mx));
          if (i > 0 && __any_sync(0xffffffffu, raise && m_ref != -INFINITY)) {
#pragma unroll 1
            for (int c = 0; c < HD / 32; ++c) {
              uint32_t o[32];
              tc::tmem_ld32_nowait(tO + X * 128 + c * 32, o);
              tc::tmem_ld_wait32(o);
#pragma unroll
              for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * corr);
              tc::tmem_st32_nowait(tO + X * 128 + c * 32, o);
            }
          }
          if (raise) {
            l *= corr;
            m_ref = mx;
          }
          const float shift = m_ref == -INFINITY ? -INFINITY : -m_ref;   // nothing seen yet: every weight is 0
          float ps[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) ps[k] = 0.f;
#pragma unroll
          for (int c = 0; c < TK; c += 2) {
            float p0 = sv[c], p1 = sv[c + 1];
            fma2(p0, p1, sl2, shift);
            p0 = tc::ex2_approx(p0);
            p1 = tc::ex2_approx(p1);
            add2(ps[(c & 6)], ps[(c & 6) + 1], p0, p1);
            const __nv_bfloat162 pp = __floats2bfloat162_rn(p0, p1);
            r[c / 2] = *reinterpret_cast<const uint32_t*>(&pp);
            if (c == 62 && !dry) tc::tmem_st32_nowait(tS, r);
            if (c == 78) signal(0);   // (its stores have had 16 exponentials' time)
          }
          if (!dry) tc::tmem_st32_nowait(tS + 32, r + 32);
          l += ((ps[0] + ps[1]) + (ps[2] + ps[3])) + ((ps[4] + ps[5]) + (ps[6] + ps[7]));
        }
        signal(1);
      }
      if (!ok) break;
      if (dry) continue;
      // ---- the unit's result: a stream's own rows, or the join of both
      // streams' parts of the same rows, each group half of the columns
      const bool join = !two && d.nt > 1;
      float fA = 1.f, fB = 0.f, m = m_ref, lt = l;
      if (join) {
        if (owed) {
          if (!waitw(&exch[1], ex1 & 1)) break;
          ++ex1;
        }
        sM[X * 128 + row] = m_ref;
        sL[X * 128 + row] = l;
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&exch[0]);
        // (also keeps the groups in step: neither may miss a phase of odone,
        // and a stream without tiles in a unit has none)
        if (!waitw(&exch[0], ex0 & 1) || !waitw(&odone[X ^ 1], oY & 1)) break;
        ++ex0;
        const float mA = sM[row], mB = sM[128 + row], lA = sL[row], lB = sL[128 + row];
        m = fmaxf(mA, mB);
        // a stream that saw nothing has no sum (or a NaN one, which stays)
        fA = lA != lA ? lA : (mA == -INFINITY ? 0.f : tc::ex2_approx(mA - m));
        fB = lB != lB ? lB : (mB == -INFINITY ? 0.f : tc::ex2_approx(mB - m));
        lt = lA * fA + lB * fB;
      }
      if (nX > 0 && !waitw(&odone[X], oX & 1)) break;
      tc::fence_after();
      if (two || X == 0 || join) {
        const bool odd = sOdd[u % NODD] == u + 1;
        const bool direct = (d.flags & U_DIRECT) && !odd;
        if (wlive) {
          const size_t rh = (size_t)(d.row0 + j) * a.nq + d.g * p.G + hh;
          const int qi = j * p.G + hh;
          const size_t at_c = (size_t)cta * p.RP * p.G + qi;
          float* po = !(d.flags & U_FIRST) ? p.co + at_c * HD : ((d.flags & U_PREFIX) ? p.qo : p.po) + rh * HD;
          const float inv = 1.f / lt;
          if (live && (two || X == 0)) {
            if (!(d.flags & U_FIRST)) {
              p.cml[at_c] = make_float2(m, pp_odd(lt, odd));
            } else {
              Piece pc;
              pc.m = direct ? __uint_as_float(kPieceDone) : m;
              pc.l = pp_odd(lt, odd);
              pc.ctas = d.ctas;
              pc.qi = qi;
              ((d.flags & U_PREFIX) ? p.qml : p.pml)[rh] = pc;
            }
            if (direct && a.lse) a.lse[rh] = (m + log2f(lt)) * 0.6931471805599453f;
          }
          const int c_lo = join ? X * (HD / 2) : 0, c_n = join ? HD / 2 : HD;
          const uint32_t t0 = tO + (two ? X * 128 : 0);
#pragma unroll 1
          for (int c = c_lo; c < c_lo + c_n; c += 32) {
            uint32_t o[32];
            tc::tmem_ld32_nowait(t0 + c, o);
            if (join) {
              uint32_t ob[32];
              tc::tmem_ld32_nowait(tO + 128 + c, ob);
              tc::tmem_ld_wait32(o);
              tc::tmem_ld_wait32(ob);
#pragma unroll
              for (int k = 0; k < 32; ++k)
                o[k] = __float_as_uint(__uint_as_float(o[k]) * fA + __uint_as_float(ob[k]) * fB);
            } else {
              tc::tmem_ld_wait32(o);
            }
            if (!live) continue;
            if (direct) {
              uint4* dst = reinterpret_cast<uint4*>(static_cast<bf16*>(a.out) + rh * HD + c);
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                uint32_t w[4];
#pragma unroll
                for (int z = 0; z < 4; ++z) {
                  const __nv_bfloat162 pp = __floats2bfloat162_rn(__uint_as_float(o[k * 8 + z * 2]) * inv,
                                                                  __uint_as_float(o[k * 8 + z * 2 + 1]) * inv);
                  w[z] = *reinterpret_cast<const uint32_t*>(&pp);
                }
                dst[k] = make_uint4(w[0], w[1], w[2], w[3]);
              }
            } else {
              uint4* dst = reinterpret_cast<uint4*>(po + c);
#pragma unroll
              for (int k = 0; k < 8; ++k) dst[k] = make_uint4(o[k * 4], o[k * 4 + 1], o[k * 4 + 2], o[k * 4 + 3]);
            }
          }
        }
      }
      if (join) {
        tc::fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&exch[1]);
        owed = true;   // until this group's next P, or the next join
      }
      oX += nX > 0;
      oY += two || X == 1 || d.nt > 1;
      base += 2 * d.nt;
    }
  }
  tc::fence_before();
  __syncthreads();   // every role has stopped issuing
  if (*abort_flag) {
    if (tid == 32) {
      // sign the stages that some producers filled and others did not come
      // to, then every stage's phase ends with its last copy
      const int n = max(max(sIssued[0], sIssued[1]), max(sIssued[2], sIssued[3]));
      for (int w = 0; w < 4; ++w)
        for (int i = sIssued[w]; i < n; ++i) tc::mbar_arrive(&kvfull[i % NS]);
      for (int i = max(0, n - NS); i < n; ++i) tc::mbar_wait(&kvfull[i % NS], (i / NS) & 1);
    } else if (tid == 0) {
      const int n = sIssued[4];
      for (int i = max(0, n - 2); i < n; ++i) tc::mbar_wait(&qfull[i & 1], (i >> 1) & 1);
    } else if (warp == 2) {   // the issuer's products
      __syncwarp();
      if (elect_one()) {
        tc::mma_commit(drain);
        tc::mbar_wait(drain, 0);
      }
      __syncwarp();
    }
    tc::fence_before();
    __syncthreads();
  }
  if (warp == 2) {
    tc::fence_after();
    tc::tmem_dealloc(tbase, 512);
  }
}

// -------------------------------------------------------------------------
static PagedPlan tc_plan(int T, int B, int nq, int nkv, int prefix) {
  PagedPlan p{};
  p.G = nq / nkv;
  p.RT = 128 / p.G;
  p.RP = 2 * p.RT;
  p.tk_log2 = 7;
  p.pt = (prefix + pt::TK - 1) / pt::TK;
  // measured, in units of 100 cycles: a tile of 128 keys against one query
  // tile, against two, and what such units cost beside their tiles. (o1 = 60
  // to 70 gains 5% behind 40000 shared tokens and costs 2 to 5% behind 2048
  // and 4096, where units are short and their loads meet)
  p.w1 = 19;
  p.w2 = 31;
  p.o1 = 50;
  p.o2 = 100;
  p.shared = pp_pack(p, T, B, prefix);
  p.ncta = num_sms();
  return p;
}

size_t paged_attn_tc_ws_bytes(int T, int B, int nq, int nkv, int hd, int prefix) {
  PagedPlan p = tc_plan(T, B, nq, nkv, prefix);
  return pp_layout(p, T, nq, hd, nullptr);
}

template <int HD>
static cudaError_t launch_tc(const PagedAttnArgs& a, const PagedPlan& p, int probe_op, cudaStream_t st) {
  using C = pt::Cfg<HD>;
  static_assert(C::SMEM <= 227 * 1024, "shared memory of one CTA");
  const int slots = a.rows.num_pages << a.rows.ps_log2, bx = 1 << (a.rows.ps_log2 < 7 ? a.rows.ps_log2 : 7);
  CUtensorMap mq, mk, mv;
  if (!make_tma_heads(&mq, a.q, a.rows.T, a.nq, HD, p.G, p.RT) ||
      !make_tma_2d(&mk, a.k_pages, slots > 0 ? slots : 1, a.nkv * HD, a.nkv * HD, bx) ||
      !make_tma_2d(&mv, a.v_pages, slots > 0 ? slots : 1, a.nkv * HD, a.nkv * HD, bx)) {
    set_error("paged attention: cuTensorMapEncodeTiled failed");
    return cudaErrorInvalidValue;
  }
  static std::atomic<unsigned long long> attr{0};
  cudaError_t e = once_per_device(attr, [] {
    // the register shares must fit what the launch gives, or the kernel's
    // warps would wait for registers that nobody returns
    cudaFuncAttributes fa;
    cudaError_t r = cudaFuncGetAttributes(&fa, paged_attn_tc<HD>);
    if (r != cudaSuccess) return r;
    if (fa.numRegs < pt::kRegLaunch) return cudaErrorLaunchOutOfResources;
    return cudaFuncSetAttribute(paged_attn_tc<HD>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  });
  if (e != cudaSuccess) return e;
  probe_start(probe_op, st);
  launch_pdl(paged_attn_tc<HD>, dim3(p.ncta), pt::THREADS, C::SMEM, st, mq, mk, mv, a, p, wait_limit_ns());
  note_launch();
  probe_stop(probe_op, st);
  launch_combine<bf16, HD>(a, p, st);
  return cudaGetLastError();
}

cudaError_t launch_paged_attn_tc(const PagedAttnArgs& a, int probe_op, cudaStream_t st) {
  PagedPlan p = tc_plan(a.rows.T, a.rows.B, a.nq, a.nkv, a.prefix);
  pp_layout(p, a.rows.T, a.nq, a.hd, static_cast<char*>(a.ws));
  return a.hd == 128 ? launch_tc<128>(a, p, probe_op, st) : launch_tc<64>(a, p, probe_op, st);
}

}  // namespace pe

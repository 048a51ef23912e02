// Attention of the newest tokens over a paged K/V cache (decoding), sm_100a.
//
// For every row (sequence b, new token t, q-head h), over its keys j:
//   o = sum_j p_j v_j / sum_j p_j,   p_j = exp2(s_j - m),   s_j = sigma log2(e) q.k_j,
// kept as (m, l = sum p, O = sum p v) so that shares of the keys computed apart can be
// joined: with M = max m_i,  l = sum_i 2^(m_i - M) l_i,  O = sum_i 2^(m_i - M) O_i.
//
// What bounds it: up to 16 rows (G * q_len) per kv-head a step reads every cached K and V row
// once and does 4 d flops per row and key with it, one a byte and row in BF16 and two in FP8, far
// under the tensor cores' 250; so it is the cache's bytes over the memory bandwidth.  More rows
// are more units, and each reads K and V again (figures below).  The kernel is built to keep
// TMA loads in flight and to give every SM the same number of bytes:
//   - The work is a line of 64-token tiles (one K page and one V page of one kv-head),
//     sequence after sequence; every CTA of one resident round takes an equal share, the
//     lengths being read on the device.  A unit (the up to 16 rows that read one kv-head
//     of one sequence) whose tiles fall to several CTAs leaves one partial each, joined by
//     decode_finish; a unit inside one CTA is written out directly.
//   - Gangs of up to eight CTAs walk the line together, each with another kv-head of the same
//     pages: pieces of 128 bytes, one head at a time, cost DRAM a third of its rate (one FP8
//     sequence of 128K tokens, then with two CTAs per SM: 69 us, 48 us in gangs).
//   - One producer warp loads tiles into a ring of three: 96 KB per CTA and two CTAs per SM, or
//     (d 64, FP8) 48 KB and three.  It looks pages up 32 at a time, a batch ahead.
//   - Four consumer warps each take 16 tokens of every tile with running statistics of
//     their own, so that nothing in the loop waits for another warp; they are joined in
//     shared memory at a unit's end.  m16n8k16 matrix instructions with the rows as M: a
//     128-row tcgen05 tile would hold 4 rows here, and its softmax would still be
//     one thread per row.
//   - FP8: K and V codes are widened to f16 in registers, which is exact, and P is rounded
//     to f16 (2^-11), not to e4m3.  f16's normal range ends at 2^-14, and a long tail of small
//     weights has to count; so p is taken as 2^(s - m + kLift): its largest entry is at least 2^7,
//     and at most 2^15 by the running maximum's slack, and what is below the normal range is off
//     by 2^-32 of the largest weight at most.  BF16: P is rounded to bf16 (2^-8), the type
//     of V, which the matrix instruction wants in both; it has float32's range.
//     The sums l are those of the unrounded p.
// Measured on one B200, whole calls: four ragged BF16 sequences of up to 128K tokens, 32 q- and
// 8 kv-heads of 128, 214 to 219 us (all of the copy rate); 48 of up to 4K with four new tokens
// each, 78 us (80 %: the start, and 1 us to join the warps of a unit); four of 128K with 4 / 16 /
// 20 / 32 / 64 rows per kv-head, BF16 314 / 327 / 635 / 631 / 1232 us (a reading's bytes at the copy
// rate: 328), FP8 195 / 191 / 387 / 370 / 763 to 810 (164); one FP8 sequence of 128K,
// 52 to 54 us (77 %: twelve consumer warps of 128 registers an SM and their chains of dependent steps;
// the scheduler issues in 45 % of the cycles, the ALU with the 64 conversions per warp and
// tile is 44 % busy, the matrix pipe 37 %.  The e4m3 form of the product for S: 55.7.  V's codes
// shifted into place instead of converted: 55.9, and 59 to 63 with the test for NaN codes that
// it needs.  Tokens as the 128 rows of tcgen05: 67 to 86).
// Waits are bounded; on expiry the CTA raises its abort flag, records STEM_ERR_TIMEOUT and
// runs through the rest of its units without computing.
#include <string.h>

#include <type_traits>

#include "stem_internal.cuh"

namespace stem {
namespace {

constexpr int kThreads = 160;       // four consumer warps, one producer warp
constexpr int kFinishThreads = 256;
constexpr int kTile = STEM_PAGE_SIZE;
static_assert(kTile == 64, "a tile is one page: four warps of 16 tokens");

template <int D, bool FP8>
struct Cfg {
  static constexpr int ES = FP8 ? 1 : 2;
  static constexpr int CH = 128 / ES;               // elements of a 128-byte swizzle row
  static constexpr int DCH = D * ES / 128;          // such rows per token
  static constexpr int CHUNK = kTile * 128;         // one box: 64 tokens of 128 bytes
  static constexpr int TILE = kTile * D * ES;
  static constexpr int STAGE = 2 * TILE;            // K and V
  // Two CTAs per SM where a tile is 32 KB, three where it is 16 KB: the same bytes in flight,
  // and per byte twice the work, which is latency and wants more warps
  static constexpr int CTAS = STAGE == 32 * 1024 ? 2 : 3;
  static constexpr int NST = 3;
  static constexpr float kLift = FP8 ? kLiftF16 : 0.f;
  static constexpr int MROWS = 512 / D;             // rows joined in one round
  static constexpr int MSTRIDE = D + 8;             // floats: the rows' banks apart
  static constexpr int MERGE = 4 * MROWS * MSTRIDE * 4;  // of four warps
  static constexpr int OFF_MERGE = NST * STAGE;
  static constexpr int OFF_ML = OFF_MERGE + MERGE;  // float2 [4][16]
  static constexpr int OFF_BAR = OFF_ML + 512;
  static constexpr int QSTRIDE = D * 2 + 16;        // a Q row in 16 bits; the rows' banks apart
  static constexpr bool Q_IN_MERGE = CTAS == 2;     // no room of its own: a barrier before the joining
  static constexpr int OFF_Q = Q_IN_MERGE ? OFF_MERGE : OFF_BAR + 512;
  static constexpr int QPIECES = D * ES / 128;      // 16-byte pieces of the unit's Q a thread loads
  static constexpr int OFF_CUM = OFF_BAR + 512 + (Q_IN_MERGE ? 0 : kDecodeRows * QSTRIDE);  // the line: int [STEM_MAX_DECODE_SEQS + 1]
  static constexpr int SMEM = OFF_CUM + (STEM_MAX_DECODE_SEQS + 1) * 4 + 1024;  // 1024: alignment
  static_assert(DCH >= 1 && NST >= 3 && NST <= 16, "ring");
  static_assert(CTAS * (SMEM + 1024) <= 228 * 1024, "resident CTAs");
};

struct DecodeParams {
  CUtensorMap tk, tv;        // [slots * 64, Hkv, d]: box (CH, 1, 64)
  DecodeArgs a;
  int rt, prt;               // 16-row tiles of a unit's rows: own, prefix (0: no prefix)
  int prefix_pages, prefix_span;  // pages of the prefix, its length on the line
  int gang;                  // CTAs that walk together, each with another kv-head of the same pages
  int gangs, head_groups;    // ctas / gang, Hkv / gang
  PrefixPlan pre;            // gangs > 0: the prefix is prefix_kernel's, ahead of this one; prt is 0 then
  uint32_t g_magic;          // ceil(2^32 / G): x / G = umulhi(x, g_magic) for G > 1 (see div_g)
};

// x / G without a division: g_magic exceeds 2^32 / G by less than 1, so the product is off by
// less than x / 2^32, which does not reach the next multiple of 1 / G for x < 2^32 / G (rows
// number 2^24 at most, and G = 256 is exact).
__device__ __forceinline__ int div_g(const DecodeParams& p, int x) {
  return p.a.G == 1 ? x : static_cast<int>(__umulhi(static_cast<uint32_t>(x), p.g_magic));
}

__device__ __forceinline__ int clamp_len(const DecodeArgs& a, int b) {
  return min(max(__ldg(a.kv_lens + b), 0), a.max_kv_len);
}
__device__ __forceinline__ int pages_of(int len) { return (len + kTile - 1) / kTile; }

__device__ __forceinline__ int span_of(int pages) { return pages > 0 ? pages + kDecodeUnitCost : 0; }

// Each sequence's first place on the line into cum[0..B] (shared), T threads' worth of
// sequences at a time; returns the line's length.  `look` sees every length as it came.
template <int T, typename F>
__device__ __forceinline__ int line_places(const DecodeParams& p, int* cum, int* sums, F look) {
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int units = p.head_groups * p.rt;
  int run = p.prefix_span;
  for (int b0 = 0; b0 < p.a.B; b0 += T) {
    const int b = b0 + tid;
    int x = 0;
    if (b < p.a.B) {
      const int raw = __ldg(p.a.kv_lens + b);
      look(raw);
      x = span_of(pages_of(min(max(raw, 0), p.a.max_kv_len))) * units;
    }
    int inc = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    if (b0 > 0) __syncthreads();
    if (lane == 31) sums[warp] = inc;
    __syncthreads();
    int before = run, sum = 0;
#pragma unroll
    for (int w = 0; w < T / 32; ++w) {
      const int v = sums[w];
      before += w < warp ? v : 0;
      sum += v;
    }
    if (b < p.a.B) cum[b] = before + inc - x;
    run += sum;
  }
  if (tid == 0) cum[p.a.B] = run;
  __syncthreads();
  return run;
}

// One CTA's share of one unit.
struct Seg {
  bool own;
  int b, kvh, rtile;
  int unit;            // index on the line of one gang member
  int p0, p1, pages, len;
};

// The sequence with cum[b] <= pos < cum[b + 1].
__device__ __forceinline__ int find_seq(const DecodeParams& p, const int* cum, int pos) {
  int lo = 0, hi = p.a.B - 1;
  while (lo < hi) {
    const int mid = (lo + hi) / 2;
    if (pos >= cum[mid + 1]) lo = mid + 1;
    else hi = mid;
  }
  return lo;
}

// Walks the units of [t, end) in line order: the prefix's (head group, row tile), then
// sequence after sequence (head group, row tile); a gang's member `rank` takes the head
// group's head of that number.  b, base, span: the sequence it stands in, its first place and
// its units' length (base = -1: none yet).
struct Walk {
  int t, end, b, rank, base, span, len;
  __device__ __forceinline__ bool next(const DecodeParams& p, const int* cum, Seg* s) {
    while (t < end) {
      int at;  // place inside the unit, the empty tiles first
      if (t < p.prefix_span) {
        const int length = p.prefix_pages + kDecodeUnitCost, u = t / length;
        s->own = false;
        s->unit = u;
        s->kvh = u / p.prt * p.gang + rank;
        s->rtile = u % p.prt;
        s->b = 0;
        s->pages = p.prefix_pages;
        s->len = p.a.prefix_len;
        at = t - u * length;
      } else {
        const int units = p.head_groups * p.rt;
        if (base < 0) b = find_seq(p, cum, t);
        if (base < 0 || t >= cum[b + 1]) {
          while (t >= cum[b + 1]) ++b;
          base = cum[b];
          span = (cum[b + 1] - base) / units;
          len = clamp_len(p.a, b);
        }
        const int u = (t - base) / span;
        s->own = true;
        const int hg = p.rt == 1 ? u : u / p.rt;
        s->unit = p.head_groups * (p.prt + b * p.rt) + u;
        s->kvh = hg * p.gang + rank;
        s->rtile = u - hg * p.rt;
        s->b = b;
        s->pages = span - kDecodeUnitCost;
        s->len = len;
        at = t - base - u * span;
      }
      const int stop = min(s->pages + kDecodeUnitCost, at + (end - t));
      t += stop - at;
      s->p0 = max(0, at - kDecodeUnitCost);
      s->p1 = stop - kDecodeUnitCost;
      if (s->p1 > s->p0) return true;
    }
    return false;
  }
};

// A load that stays where it is written (before the barriers that follow).
__device__ __forceinline__ uint4 ld_early(const uint4* at) {
  uint4 r;
  asm volatile("ld.global.nc.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(at));
  return r;
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
template <bool F16>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (F16)
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t e4m3x2_to_h2(uint32_t v) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(v)));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ void consumer_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

// 16-bit masks of a fragment register that holds tokens j and j + 1: the halves whose
// token is at or behind `limit` become zero (masked V rows may hold NaN).
__device__ __forceinline__ uint32_t keep_below(int j, int limit) {
  return (j < limit ? 0xFFFFu : 0u) | (j + 1 < limit ? 0xFFFF0000u : 0u);
}

template <int D, bool FP8, bool SCORES>
__global__ void __launch_bounds__(kThreads, Cfg<D, FP8>::CTAS) decode_kernel(const __grid_constant__ DecodeParams p) {
  using C = Cfg<D, FP8>;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem =
      reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sring = smem_u32(smem);
  float* merge = reinterpret_cast<float*>(smem + C::OFF_MERGE);
  float2* ml = reinterpret_cast<float2*>(smem + C::OFF_ML);
  const uint32_t bars = smem_u32(smem + C::OFF_BAR);
  auto full = [&](int s) { return bars + 8 * s; };
  auto empty = [&](int s) { return bars + 128 + 8 * s; };
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_BAR + 256);
  int* warp_sums = reinterpret_cast<int*>(smem + C::OFF_BAR + 288);   // [5]
  const DecodeArgs& a = p.a;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const unsigned all = 0xffffffffu;

  if (tid == 0) {
    for (int s = 0; s < C::NST; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 4);
    }
    *abort_flag = 0;
    mbar_fence_init();
    tma_prefetch_map(&p.tk);
    tma_prefetch_map(&p.tv);
  }
  // Nothing of the caller's, nor the workspace, is touched before the step's first kernel has
  // waited: this one, or prefix_kernel, whose CTAs let this launch go after their wait.
  const bool second = p.pre.gangs > 0;
  if (!second) pdl_wait();
  pdl_trigger();  // not earlier: decode_finish relies on that wait
  int* cum = reinterpret_cast<int*>(smem + C::OFF_CUM);
  const int run = line_places<kThreads>(p, cum, warp_sums, [&](int raw) {
    if (blockIdx.x == 0 && (raw < 0 || raw > a.max_kv_len)) atomicOr(a.status, kStatusBounds);
  });
  const int gang_no = static_cast<int>(blockIdx.x) / p.gang, rank = static_cast<int>(blockIdx.x) % p.gang;
  const int per = (run + p.gangs - 1) / p.gangs;
  const int t0 = min(run, gang_no * per), t1 = min(run, t0 + per);
  if (warp == 4) {
    // ------------------------------------------------------------ producer
    // 32 places of the line at a time, a lane each: which unit and page it is, and the page's
    // slot, looked up one batch ahead so that short units wait for no lookup.
    struct Place {
      int kvh, slot;
      bool tile;
    };
    auto look = [&](int pos) {
      Place q{0, 0, false};
      if (pos >= t1) return q;
      const int32_t* table = a.prefix_table;
      int at;
      if (pos < p.prefix_span) {
        const int length = p.prefix_pages + kDecodeUnitCost, u = pos / length;
        q.kvh = u / p.prt * p.gang + rank;
        at = pos - u * length;
      } else {
        const int lo = find_seq(p, cum, pos);
        const int base = cum[lo], span = (cum[lo + 1] - base) / (p.head_groups * p.rt), u = (pos - base) / span;
        q.kvh = (p.rt == 1 ? u : u / p.rt) * p.gang + rank;
        at = pos - base - u * span;
        table = a.table + static_cast<long long>(lo) * a.max_pages;
      }
      q.tile = at >= kDecodeUnitCost;
      if (q.tile) q.slot = __ldg(table + at - kDecodeUnitCost);
      return q;
    };
    uint32_t it = 0;
    bool alive = true;
    Place ahead = look(t0 + lane);
    for (int x = t0; x < t1 && alive; x += 32) {
      const Place now = ahead;
      bool looked = false;
      int issued = 0;
      int mine = now.slot;
      if (mine < 0 || mine >= a.num_slots) {
        atomicOr(a.status, kStatusBounds);
        mine = 0;
      }
      for (unsigned todo = __ballot_sync(all, now.tile); todo; todo &= todo - 1, ++it) {
        const int l = __ffs(todo) - 1;
        const int row = __shfl_sync(all, mine, l) * kTile, kvh = __shfl_sync(all, now.kvh, l);
        const int st = it % C::NST;
        const bool ok = mbar_wait(empty(st), ((it / C::NST) & 1) ^ 1, abort_flag, a.status);
        if (!__all_sync(all, ok)) {
          alive = false;
          break;
        }
        if (lane == 0) {
          mbar_arrive_expect_tx(full(st), C::STAGE);
          const uint32_t dst = sring + st * C::STAGE;
#pragma unroll
          for (int c = 0; c < C::DCH; ++c) {
            tma_load_3d(dst + c * C::CHUNK, &p.tk, full(st), c * C::CH, kvh, row);
            tma_load_3d(dst + C::TILE + c * C::CHUNK, &p.tv, full(st), c * C::CH, kvh, row);
          }
        }
        if (++issued == C::NST) {  // the ring is filled before the look ahead
          ahead = look(x + 32 + lane);
          looked = true;
        }
      }
      if (!looked) ahead = look(x + 32 + lane);
    }
    if (!alive)  // let the copies already issued land before the CTA can exit
      for (uint32_t q = it > C::NST ? it - C::NST : 0; q < it; ++q)
        for (int spin = 0; spin < 1000000 && !mbar_try_wait(full(q % C::NST), (q / C::NST) & 1); ++spin) {}
    return;
  }

  // -------------------------------------------------------------- consumers
  const int r0 = lane / 4, qd = lane % 4, mi = lane / 8;
  const int G = a.G;
  // this lane's row of the ldmatrix groups of a warp's 16 tokens, and its swizzled chunks
  const uint32_t k_row = static_cast<uint32_t>(warp * 16 + (FP8 ? (mi & 1) : (mi >> 1)) * 8 + (lane & 7)) * 128;
  const uint32_t v_row = static_cast<uint32_t>(warp * 16 + (mi & 1) * 8 + (lane & 7)) * 128;
  const int k_sub = FP8 ? mi >> 1 : mi & 1, v_sub = mi >> 1;
  const int sw = lane & 7;
  // A unit's Q, 16 rows in 16 bits, lies in shared memory: as fragments it took 32 registers.
  // FP8: in the order in which e4m3x2_to_h2 gives K's codes, a word's low pairs of a group of
  // 16, then its high pairs.
  unsigned char* sq = smem + C::OFF_Q;
  const uint32_t q_frag = smem_u32(sq) + ((lane & 7) + (mi & 1) * 8) * C::QSTRIDE + (mi >> 1) * 16;
  constexpr int PPR = D * C::ES / 16;  // pieces of a row
  uint4 qn[C::QPIECES];
  auto load_q = [&](const Seg& g) {
    const int first = g.rtile * kDecodeRows;
    const int nrows = min(kDecodeRows, (g.own ? a.n * G : a.B * a.n * G) - first);
    const int base = (g.own ? g.b * a.n * G : 0) + first;
#pragma unroll
    for (int k = 0; k < C::QPIECES; ++k) {
      const int x = tid + 128 * k, r = x / PPR, row = base + r, tok = div_g(p, row);
      const long long at = (static_cast<long long>(tok) * a.Hq + g.kvh * G + row - tok * G) * PPR + x % PPR;
      qn[k] = make_uint4(0, 0, 0, 0);
      if (r < nrows) qn[k] = ld_early(static_cast<const uint4*>(a.q) + at);
    }
  };
  auto store_q = [&]() {
#pragma unroll
    for (int k = 0; k < C::QPIECES; ++k) {
      const int x = tid + 128 * k;
      unsigned char* to = sq + x / PPR * C::QSTRIDE + x % PPR * (FP8 ? 32 : 16);
      if (FP8) {
        const uint4 v = qn[k];
        *reinterpret_cast<uint4*>(to) = make_uint4(e4m3x2_to_h2(v.x & 0xFFFFu), e4m3x2_to_h2(v.y & 0xFFFFu),
                                                   e4m3x2_to_h2(v.z & 0xFFFFu), e4m3x2_to_h2(v.w & 0xFFFFu));
        *reinterpret_cast<uint4*>(to + 16) =
            make_uint4(e4m3x2_to_h2(v.x >> 16), e4m3x2_to_h2(v.y >> 16), e4m3x2_to_h2(v.z >> 16), e4m3x2_to_h2(v.w >> 16));
      } else {
        *reinterpret_cast<uint4*>(to) = qn[k];
      }
    }
    consumer_sync();
  };
  Walk walk{t0, t1, 0, rank, -1, 0, 0};
  Seg sg;
  bool have = walk.next(p, cum, &sg);
  if (have) {
    load_q(sg);
    store_q();
  }
  uint32_t it = 0;
  while (have) {
    const int rows_all = sg.own ? a.n * G : a.B * a.n * G;
    const int first = sg.rtile * kDecodeRows;
    const int nrows = min(kDecodeRows, rows_all - first);
    const int row_base = (sg.own ? sg.b * a.n * G : 0) + first;
    // keys that the unit's first and last row, and this thread's two rows, see
    auto limit_of = [&](int r) {
      if (!sg.own) return sg.len;
      return max(0, sg.len - a.n + div_g(p, first + r) + 1);
    };
    const bool upper_rows = nrows > 8;
    const int lim_lo = limit_of(0), lim_hi = limit_of(nrows - 1);
    const int lim0 = limit_of(min(r0, nrows - 1)), lim1 = limit_of(min(r0 + 8, nrows - 1));
    float* srow = nullptr;
    if (SCORES && sg.own)
      srow = a.scores + (static_cast<long long>(sg.b * a.Hkv + sg.kvh) * rows_all + first) * a.score_stride;
    float acc[D / 8][4];
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[i][e] = 0.f;
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;

    for (int pg = sg.p0; pg < sg.p1; ++pg, ++it) {
      const int st = it % C::NST;
      if (mbar_wait(full(st), (it / C::NST) & 1, abort_flag, a.status)) {
        const uint32_t kt = sring + st * C::STAGE, vt = kt + C::TILE;
        const int s0 = pg * kTile + warp * 16;     // this warp's first token
        // S = Q K^T for 16 tokens
        // (two accumulators each, for half the chain of dependent products)
        float s[2][4], s_odd[2][4];
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[j][e] = s_odd[j][e] = 0.f;
        if (FP8) {
#pragma unroll
          for (int k = 0; k < D / 16; k += 2) {
            uint32_t r[4], q[2][4];
            ldsm4(r, kt + k_row + (((k + k_sub) ^ sw) << 4));
            ldsm4(q[0], q_frag + k * 32);
            ldsm4(q[1], q_frag + k * 32 + 32);
#pragma unroll
            for (int kk = 0; kk < 2; ++kk)
#pragma unroll
              for (int j = 0; j < 2; ++j)
                mma16816<true>(kk ? s_odd[j] : s[j], q[kk], e4m3x2_to_h2(r[2 * kk + j] & 0xFFFFu), e4m3x2_to_h2(r[2 * kk + j] >> 16));
          }
        } else {
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const int c = 2 * k + k_sub;
            uint32_t r[4], q[4];
            ldsm4(r, kt + (c >> 3) * C::CHUNK + k_row + (((c & 7) ^ sw) << 4));
            ldsm4(q, q_frag + k * 32);
            mma16816<false>(k & 1 ? s_odd[0] : s[0], q, r[0], r[1]);
            mma16816<false>(k & 1 ? s_odd[1] : s[1], q, r[2], r[3]);
          }
        }
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[j][e] = (s[j][e] + s_odd[j][e]) * a.scale_log2;
        const bool edge = s0 + 16 > lim_lo;
        if (edge) {
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (s0 + j * 8 + qd * 2 + (e & 1) >= (e < 2 ? lim0 : lim1)) s[j][e] = -INFINITY;
        }
        if (SCORES && sg.own) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float* at = srow + s0 + j * 8 + qd * 2;
            if (r0 < nrows) *reinterpret_cast<float2*>(at + r0 * a.score_stride) = make_float2(s[j][0], s[j][1]);
            if (r0 + 8 < nrows)
              *reinterpret_cast<float2*>(at + (r0 + 8) * a.score_stride) = make_float2(s[j][2], s[j][3]);
          }
        }
        // running maximum (raised lazily, when it grows by more than 2^8: p <= 2^8 until then);
        // the upper eight rows only where the unit has them
        float x0 = fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[1][0], s[1][1])), x1 = -INFINITY;
        x0 = fmaxf(x0, __shfl_xor_sync(all, x0, 1));
        x0 = fmaxf(x0, __shfl_xor_sync(all, x0, 2));
        if (upper_rows) {
          x1 = fmaxf(fmaxf(s[0][2], s[0][3]), fmaxf(s[1][2], s[1][3]));
          x1 = fmaxf(x1, __shfl_xor_sync(all, x1, 1));
          x1 = fmaxf(x1, __shfl_xor_sync(all, x1, 2));
        }
        if (__any_sync(all, x0 > m0 + 8.0f || x1 > m1 + 8.0f)) {
          // each row by its own scores alone: a prefix's rows are several sequences'
          const float n0 = x0 > m0 + 8.0f ? x0 : m0, n1 = x1 > m1 + 8.0f ? x1 : m1;
          const float a0 = n0 == m0 ? 1.0f : ex2_approx(m0 - n0), a1 = n1 == m1 ? 1.0f : ex2_approx(m1 - n1);
          m0 = n0;
          m1 = n1;
          l0 *= a0;
          l1 *= a1;
#pragma unroll
          for (int i = 0; i < D / 8; ++i) {
            acc[i][0] *= a0;
            acc[i][1] *= a0;
            acc[i][2] *= a1;
            acc[i][3] *= a1;
          }
        }
        const float u0 = m0 == -INFINITY ? 0.f : m0 - C::kLift;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          s[j][0] = ex2_approx(s[j][0] - u0);
          s[j][1] = ex2_approx(s[j][1] - u0);
        }
        l0 += (s[0][0] + s[0][1]) + (s[1][0] + s[1][1]);
        if (upper_rows) {
          const float u1 = m1 == -INFINITY ? 0.f : m1 - C::kLift;
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            s[j][2] = ex2_approx(s[j][2] - u1);
            s[j][3] = ex2_approx(s[j][3] - u1);
          }
          l1 += (s[0][2] + s[0][3]) + (s[1][2] + s[1][3]);
        } else {
          s[0][2] = s[0][3] = s[1][2] = s[1][3] = 0.f;
        }
        uint32_t pf[4];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          pf[2 * j] = FP8 ? pack_f16x2(s[j][0], s[j][1]) : pack_bf16x2(s[j][0], s[j][1]);
          pf[2 * j + 1] = FP8 ? pack_f16x2(s[j][2], s[j][3]) : pack_bf16x2(s[j][2], s[j][3]);
        }
        // O += P V with V's tokens at or behind `limit` taken as zero; ONLY: into the rows
        // flagged in w0 / w1 alone
        auto pv = [&](auto only, bool cut, int limit, bool w0, bool w1) {
          constexpr bool ONLY = decltype(only)::value;
          auto mm = [&](float(&c)[4], uint32_t b0, uint32_t b1) {
            if constexpr (!ONLY) {
              mma16816<FP8>(c, pf, b0, b1);
            } else {
              float x[4] = {0.f, 0.f, 0.f, 0.f};
              mma16816<FP8>(x, pf, b0, b1);
              c[0] += w0 ? x[0] : 0.f;
              c[1] += w0 ? x[1] : 0.f;
              c[2] += w1 ? x[2] : 0.f;
              c[3] += w1 ? x[3] : 0.f;
            }
          };
          const uint32_t z0 = cut ? keep_below(s0 + qd * 2, limit) : 0xFFFFFFFFu;
          const uint32_t z1 = cut ? keep_below(s0 + qd * 2 + 8, limit) : 0xFFFFFFFFu;
          if (FP8) {
#pragma unroll
            for (int c = 0; c < D / 16; c += 2) {
              uint32_t r[4];
              ldsm4_t(r, vt + v_row + (((c + v_sub) ^ sw) << 4));
#pragma unroll
              for (int cc = 0; cc < 2; ++cc) {
                const uint32_t x = r[2 * cc] & z0, y = r[2 * cc + 1] & z1;
                const uint32_t xl = e4m3x2_to_h2(x & 0xFFFFu), xh = e4m3x2_to_h2(x >> 16);
                const uint32_t yl = e4m3x2_to_h2(y & 0xFFFFu), yh = e4m3x2_to_h2(y >> 16);
                mm(acc[2 * (c + cc)], __byte_perm(xl, xh, 0x5410), __byte_perm(yl, yh, 0x5410));
                mm(acc[2 * (c + cc) + 1], __byte_perm(xl, xh, 0x7632), __byte_perm(yl, yh, 0x7632));
              }
            }
          } else {
#pragma unroll
            for (int c = 0; c < D / 8; c += 2) {
              uint32_t r[4];
              const int cv = c + v_sub;
              ldsm4_t(r, vt + (cv >> 3) * C::CHUNK + v_row + (((cv & 7) ^ sw) << 4));
              mm(acc[c], r[0] & z0, r[1] & z1);
              mm(acc[c + 1], r[2] & z0, r[3] & z1);
            }
          }
        };
        if (!edge) {
          pv(std::false_type{}, false, 0, true, true);
        } else if (lim_lo == lim_hi || lim_hi <= s0) {
          pv(std::false_type{}, true, lim_hi, true, true);
        } else {
          // The rows' limits differ inside these 16 tokens (drafted tokens): one product per
          // new token, taken by its rows alone, so that a row is never touched by a V row
          // that it does not see (0 * NaN).
          const int ta = div_g(p, first), tb = div_g(p, first + nrows - 1);
          const int mine0 = div_g(p, first + min(r0, nrows - 1)), mine1 = div_g(p, first + min(r0 + 8, nrows - 1));
          for (int t = ta; t <= tb; ++t)
            pv(std::true_type{}, true, max(0, sg.len - a.n + t + 1), mine0 == t, mine1 == t);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(empty(st));
    }

    // the next unit's Q on its way while this one is joined
    const Seg was = sg;
    have = walk.next(p, cum, &sg);
    if (have) load_q(sg);

    // join the four warps' shares
    if (C::Q_IN_MERGE) consumer_sync();
    l0 += __shfl_xor_sync(all, l0, 1);
    l1 += __shfl_xor_sync(all, l1, 1);
    l0 += __shfl_xor_sync(all, l0, 2);
    l1 += __shfl_xor_sync(all, l1, 2);
    if (qd == 0) {
      ml[warp * 16 + r0] = make_float2(m0 - C::kLift, l0);
      ml[warp * 16 + r0 + 8] = make_float2(m1 - C::kLift, l1);
    }
    const bool direct = was.own && was.p0 == 0 && was.p1 == was.pages && a.prefix_len == 0;
    const long long slot = static_cast<long long>(gang_no + was.unit) * p.gang + rank;
    // rounds of 4 rows x 128 columns (d 64: 8 rows x 64): few rows, few barriers
    constexpr int RPR = C::MROWS;
#pragma unroll 1
    for (int round = 0; round * RPR < nrows; ++round) {
      const bool upper = round * RPR >= 8;
      if (r0 / RPR == round % (8 / RPR)) {
        float* mine = merge + (warp * RPR + r0 % RPR) * C::MSTRIDE;
#pragma unroll
        for (int x = 0; x < D / 8; x += 2) {
          const float e0 = upper ? acc[x][2] : acc[x][0], e1 = upper ? acc[x][3] : acc[x][1];
          const float f0 = upper ? acc[x + 1][2] : acc[x + 1][0], f1 = upper ? acc[x + 1][3] : acc[x + 1][1];
          if (FP8) {
            *reinterpret_cast<float4*>(mine + x * 8 + qd * 4) = make_float4(e0, f0, e1, f1);
          } else {
            *reinterpret_cast<float2*>(mine + x * 8 + qd * 2) = make_float2(e0, e1);
            *reinterpret_cast<float2*>(mine + x * 8 + 8 + qd * 2) = make_float2(f0, f1);
          }
        }
      }
      consumer_sync();
      const int rr = tid / (D / 4), r = round * RPR + rr, col = tid % (D / 4) * 4;  // RPR rows x groups of 4 columns
      if (r < nrows) {
        float M = -INFINITY;
        float2 v[4];
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          v[w] = ml[w * 16 + r];
          M = fmaxf(M, v[w].x);
        }
        float L = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const float f = v[w].x == -INFINITY ? 0.f : ex2_approx(v[w].x - M);
          const float4 x = *reinterpret_cast<const float4*>(merge + (w * RPR + rr) * C::MSTRIDE + col);
          L += f * v[w].y;
          o.x += f * x.x;
          o.y += f * x.y;
          o.z += f * x.z;
          o.w += f * x.w;
        }
        if (direct) {
          const int g = row_base + r;
          const int tok = div_g(p, g);
          const int h = was.kvh * G + g - tok * G;
          const float inv = M == -INFINITY && L == 0.f ? 0.f : 1.0f / L;  // nothing seen: o = 0
          *reinterpret_cast<uint2*>(static_cast<unsigned char*>(a.out) + ((static_cast<long long>(tok) * a.Hq + h) * D + col) * 2) =
              make_uint2(pack_bf16x2(o.x * inv * a.v_scale, o.y * inv * a.v_scale),
                         pack_bf16x2(o.z * inv * a.v_scale, o.w * inv * a.v_scale));
          if (a.lse != nullptr && col == 0)
            a.lse[static_cast<long long>(h) * a.B * a.n + tok] =
                L == 0.f ? -INFINITY : (M + log2f(L)) * 0.69314718055994531f;
        } else {
          *reinterpret_cast<float4*>(a.part_o + (slot * a.part_rows + r) * D + col) = o;
        }
        if (col == 0 && (!direct || SCORES)) a.part_ml[slot * kDecodeRows + r] = make_float2(M, L);
      }
      consumer_sync();
    }
    if (have) store_q();
  }
  // decode_finish takes this launch's end for prefix_kernel's too: one CTA that stays for it is
  // enough, and the others leave their places to the CTAs still to come
  if (second && blockIdx.x == gridDim.x - 1) pdl_wait();
}

// The partials of one row: number i's (m, l) at ml[i * ml_step], its output at o[i * o_step].
struct Pieces {
  const float2* ml;
  const float* o;
  int ml_step, o_step, n;
};
// Pieces of a unit whose tiles are first .. first + tiles - 1 on a line of which every CTA
// takes `per`; its slots start at (share + unit) * gang + rank, each of `rows` output rows.
__device__ __forceinline__ Pieces pieces_of(const float2* ml, const float* o, int ml_rows, int rows, int d, int first,
                                            int tiles, int unit, int gang, int rank, int per, int row) {
  const unsigned c0 = static_cast<unsigned>(first) / static_cast<unsigned>(per);
  const unsigned c1 = static_cast<unsigned>(first + tiles - 1) / static_cast<unsigned>(per);
  const long long slot = static_cast<long long>(c0 + unit) * gang + rank;
  return Pieces{ml + slot * ml_rows + row, o + (slot * rows + row) * d, gang * ml_rows, gang * rows * d,
                tiles == 0 ? 0 : static_cast<int>(c1 - c0) + 1};
}
// kvh = hg * gang + rank
__device__ __forceinline__ Pieces own_pieces(const DecodeParams& p, int per, int b, int base, int pages, int hg,
                                             int rank, int rr) {
  const DecodeArgs& a = p.a;
  const int u = hg * p.rt + rr / kDecodeRows;
  return pieces_of(a.part_ml, a.part_o, kDecodeRows, a.part_rows, a.d,
                   base + u * (pages + kDecodeUnitCost) + kDecodeUnitCost, pages,
                   p.head_groups * (p.prt + b * p.rt) + u, p.gang, rank, per, rr % kDecodeRows);
}
// tok: token of the batch; g: q-head of the group
__device__ __forceinline__ Pieces prefix_pieces(const DecodeParams& p, int per, int hg, int rank, int tok, int g) {
  const DecodeArgs& a = p.a;
  const PrefixPlan& q = p.pre;
  if (q.gangs > 0) {
    const unsigned tile = static_cast<unsigned>(tok) / static_cast<unsigned>(q.slot_tokens);
    const int u = hg * q.pairs + static_cast<int>(tile / 2);
    return pieces_of(a.prefix_ml, a.prefix_o, 256, 256, a.d, u * (q.tiles + kPrefixUnitCost) + kPrefixUnitCost, q.tiles,
                     u, q.gang, rank, q.per,
                     static_cast<int>(tile % 2) * 128 + (tok - static_cast<int>(tile) * q.slot_tokens) * a.G + g);
  }
  if (p.prt == 0) return Pieces{nullptr, nullptr, 0, 0, 0};
  const int row = tok * a.G + g, u = hg * p.prt + row / kDecodeRows;
  return pieces_of(a.part_ml, a.part_o, kDecodeRows, a.part_rows, a.d,
                   u * (p.prefix_pages + kDecodeUnitCost) + kDecodeUnitCost, p.prefix_pages, u, p.gang, rank, per,
                   row % kDecodeRows);
}
// Pages of a sequence from its length on the line.
__device__ __forceinline__ int pages_on_line(const DecodeParams& p, int length) {
  return length > 0 ? length / (p.head_groups * p.rt) - kDecodeUnitCost : 0;
}

__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
  for (int o = 16; o; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}
__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// A row's partials, the own ones first.
struct RowPieces {
  Pieces own, pre;
  __device__ __forceinline__ int count() const { return own.n + pre.n; }
  __device__ __forceinline__ float2 stats(int i) const {
    return i < own.n ? own.ml[i * own.ml_step] : pre.ml[(i - own.n) * pre.ml_step];
  }
  __device__ __forceinline__ const float* out(int i) const {
    return i < own.n ? own.o + static_cast<long long>(i) * own.o_step
                     : pre.o + static_cast<long long>(i - own.n) * pre.o_step;
  }
};
__device__ __forceinline__ RowPieces row_pieces(const DecodeParams& p, int per, int b, int base, int pages, int kvh,
                                                int t, int g) {
  const int hg = p.head_groups == 1 ? 0 : kvh / p.gang, rank = kvh - hg * p.gang;
  return RowPieces{own_pieces(p, per, b, base, pages, hg, rank, t * p.a.G + g),
                   prefix_pieces(p, per, hg, rank, b * p.a.n + t, g)};
}

// 2^(m - M), for a partial whose scores were all -inf 0 (and 1 where its sum is NaN: the
// NaN has to arrive).
__device__ __forceinline__ float piece_factor(float2 v, float M) {
  return v.x == -INFINITY ? (v.y == 0.f ? 0.f : 1.f) : ex2_approx(v.x - M);
}

// Maximum and sum over a row's partials (all lanes get both).
__device__ __forceinline__ float2 row_stats(const RowPieces& q) {
  const int lane = threadIdx.x % 32, n = q.count();
  float2 v = make_float2(-INFINITY, 0.f);
  if (lane < n) v = q.stats(lane);
  float M = v.x;
  for (int i = lane + 32; i < n; i += 32) M = fmaxf(M, q.stats(i).x);
  M = warp_max(M);
  float L = piece_factor(v, M) * v.y;
  for (int i = lane + 32; i < n; i += 32) {
    v = q.stats(i);
    L += piece_factor(v, M) * v.y;
  }
  return make_float2(M, warp_sum(L));
}

template <int E>
__device__ __forceinline__ void load_share(float (&x)[E], const float* src) {
  if constexpr (E == 4) {
    const float4 v = *reinterpret_cast<const float4*>(src);
    x[0] = v.x;
    x[1] = v.y;
    x[2] = v.z;
    x[3] = v.w;
  } else {
    const float2 v = *reinterpret_cast<const float2*>(src);
    x[0] = v.x;
    x[1] = v.y;
  }
}

// Joins the partials of rows whose keys fell to several CTAs (blocks below row_blocks, WPR
// warps per row: 8, a block for one row, or 1) and adds up the softmax weights (the other blocks, from the stored scores).
// What follows pdl_wait is latency, so where each row's partials lie is worked out before
// it, from the lengths (what decode_kernel lets go starts after the step's first wait, when all that
// came before it in the stream is complete), and all loads after it are independent.  Every
// block waits, those with nothing to join too: what follows in the stream takes this launch's
// end for decode_kernel's.
template <int D, bool SCORES, int WPR>
__global__ void __launch_bounds__(kFinishThreads, 3) decode_finish(const __grid_constant__ DecodeParams p, int row_blocks) {
  const DecodeArgs& a = p.a;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, G = a.G, R = a.n * G;
  constexpr int E = D / 32, RPB = kFinishThreads / 32 / WPR;  // columns of a lane, rows of a block
  constexpr int PF = 8;                         // partials a warp loads at once
  __shared__ int cum[STEM_MAX_DECODE_SEQS + 1];
  __shared__ int sums[kFinishThreads / 32];
  __shared__ float lse2[256];
  __shared__ float shares[WPR > 1 ? kFinishThreads * E : 1];
  __shared__ int where;
  pdl_trigger();
  const int total = line_places<kFinishThreads>(p, cum, sums, [](int) {});
  const int per = max(1, (total + p.gangs - 1) / p.gangs);

  if (static_cast<int>(blockIdx.x) < row_blocks) {
    const int w = warp % WPR;
    const unsigned rows = static_cast<unsigned>(a.B) * a.n * a.Hq;  // token-major, then head
    bool waited = false;
    for (unsigned row = blockIdx.x * RPB + warp / WPR; row < rows; row += row_blocks * RPB) {
      const int tok = static_cast<int>(row / static_cast<unsigned>(a.Hq)), h = static_cast<int>(row) - tok * a.Hq;
      const int b = a.n == 1 ? tok : tok / a.n, kvh = div_g(p, h), t = tok - b * a.n, g = h - kvh * G;
      const int base = cum[b], pages = pages_on_line(p, cum[b + 1] - base);
      const RowPieces q = row_pieces(p, per, b, base, pages, kvh, t, g);
      const int n = q.count();
      if (a.prefix_len == 0 && n == 1) continue;  // written by the CTA that saw all of it
      if (!waited) pdl_wait();
      waited = true;
      float x[PF][E];
      float2 v[PF];
#pragma unroll
      for (int k = 0; k < PF; ++k)
        if (w + WPR * k < n) {
          load_share(x[k], q.out(w + WPR * k) + lane * E);
          v[k] = q.stats(w + WPR * k);
        }
      const float2 st = row_stats(q);
      float o[E];
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = 0.f;
#pragma unroll
      for (int k = 0; k < PF; ++k)
        if (w + WPR * k < n) {
          const float f = piece_factor(v[k], st.x);
#pragma unroll
          for (int e = 0; e < E; ++e) o[e] += f * x[k][e];
        }
#pragma unroll 4
      for (int i = w + WPR * PF; i < n; i += WPR) {
        load_share(x[0], q.out(i) + lane * E);
        const float f = piece_factor(q.stats(i), st.x);
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] += f * x[0][e];
      }
      if constexpr (WPR > 1) {  // one row a block, and one turn of the loop
#pragma unroll
        for (int e = 0; e < E; ++e) shares[tid * E + e] = o[e];
        __syncthreads();
        if (w != 0) return;
#pragma unroll
        for (int y = 1; y < WPR; ++y)
#pragma unroll
          for (int e = 0; e < E; ++e) o[e] += shares[(tid + 32 * y) * E + e];
      }
      const float inv = st.x == -INFINITY && st.y == 0.f ? 0.f : 1.0f / st.y;
      uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<unsigned char*>(a.out) +
                                                  ((static_cast<long long>(tok) * a.Hq + h) * D + lane * E) * 2);
#pragma unroll
      for (int e = 0; e < E; e += 2) dst[e / 2] = pack_bf16x2(o[e] * inv * a.v_scale, o[e + 1] * inv * a.v_scale);
      if (a.lse != nullptr && lane == 0)
        a.lse[static_cast<long long>(h) * a.B * a.n + tok] =
            st.y == 0.f ? -INFINITY : (st.x + log2f(st.y)) * 0.69314718055994531f;
    }
    if (!waited) pdl_wait();
    return;
  }

  if constexpr (SCORES) {
    // Chunks of 1024 tokens (4 per thread) of all (sequence, kv-head) pairs, an equal share per
    // block: a pair's log-sum-exps are worked out once, then its chunks go without a barrier.
    __shared__ int chunk_cum[STEM_MAX_DECODE_SEQS + 1];
    constexpr int kSpan = kFinishThreads * 4, kChunk = kSpan / kTile;  // tokens, pages
    if (warp == 0) {
      int run = 0;
      for (int b0 = 0; b0 < a.B; b0 += 32) {
        const int b = b0 + lane;
        const int y = b < a.B ? (pages_on_line(p, cum[b + 1] - cum[b]) + kChunk - 1) / kChunk * a.Hkv : 0;
        int inc = y;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int z = __shfl_up_sync(0xffffffffu, inc, o);
          if (lane >= o) inc += z;
        }
        if (b < a.B) chunk_cum[b] = run + inc - y;
        run += __shfl_sync(0xffffffffu, inc, 31);
      }
      if (lane == 0) chunk_cum[a.B] = run;
    }
    __syncthreads();
    const int chunks = chunk_cum[a.B], nb = gridDim.x - row_blocks, share = (chunks + nb - 1) / nb;
    int c = min(chunks, static_cast<int>(blockIdx.x - row_blocks) * share);
    const int end = min(chunks, c + share);
    bool waited = false;
    while (c < end) {
      for (int b = tid; b < a.B; b += kFinishThreads)
        if (chunk_cum[b] <= c && c < chunk_cum[b + 1]) where = b;
      __syncthreads();
      const int b = where;
      const int base = cum[b], pages = pages_on_line(p, cum[b + 1] - base);
      const int off = c - chunk_cum[b], each = (pages + kChunk - 1) / kChunk, kvh = off / each;
      const int k0 = off - kvh * each, k1 = min(each, k0 + (end - c)), len = clamp_len(a, b);
      c += k1 - k0;
      const long long unit = static_cast<long long>(b) * a.Hkv + kvh;
      const float* win = a.weights_in ? a.weights_in + unit * a.weights_stride : nullptr;
      float* wout = a.weights_out + unit * a.weights_stride;
      if (!waited) pdl_wait();
      waited = true;
      for (int r0 = 0; r0 < R; r0 += 256) {
        const int nr = min(256, R - r0);
        for (int r = warp; r < nr; r += kFinishThreads / 32) {
          const int t = div_g(p, r0 + r);
          const float2 st = row_stats(row_pieces(p, per, b, base, pages, kvh, t, r0 + r - t * G));
          // a row that sees nothing adds exp2(-inf - inf) = 0
          if (lane == 0) lse2[r] = st.y == 0.f ? INFINITY : st.x + log2f(st.y);
        }
        __syncthreads();
        const float* was = r0 > 0 ? wout : win;
        for (int j = k0 * kSpan + tid * 4; j < min(len, k1 * kSpan); j += kSpan) {
          const float* sc = a.scores + (unit * R + r0) * a.score_stride + j;
          float sum[4], add[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int e = 0; e < 4; ++e) sum[e] = was && j + e < len ? was[j + e] : 0.f;
#pragma unroll 4
          for (int r = 0; r < nr; ++r) {
            const float4 x = *reinterpret_cast<const float4*>(sc + r * a.score_stride);
            const float l = lse2[r];
            add[0] += ex2_approx(x.x - l);
            add[1] += ex2_approx(x.y - l);
            add[2] += ex2_approx(x.z - l);
            add[3] += ex2_approx(x.w - l);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (j + e < len) wout[j + e] = sum[e] + add[e];
        }
        __syncthreads();
      }
    }
    if (!waited) pdl_wait();
  }
}

template <int D, bool FP8, bool SCORES>
cudaError_t run(const DecodeParams& prm, cudaStream_t st) {
  using C = Cfg<D, FP8>;
  cudaError_t e = set_smem_once<decode_kernel<D, FP8, SCORES>>(C::SMEM);
  if (e != cudaSuccess) return e;
  if (prm.pre.gangs > 0 && (e = launch_prefix(prm.a, prm.pre, FP8, st)) != cudaSuccess) return e;
  e = launch_dependent(decode_kernel<D, FP8, SCORES>, prm.gangs * prm.gang, kThreads, C::SMEM, 1, st, prm);
  if (e != cudaSuccess) return e;
  // behind it, so that its partials, the larger ones, are the last into L2
  const DecodeArgs& a = prm.a;
  const long long rows = static_cast<long long>(a.B) * a.n * a.Hq;
  const long long chunks =
      static_cast<long long>(a.B) * a.Hkv * ((a.max_kv_len + kFinishThreads * 4 - 1) / (kFinishThreads * 4));
  // As many blocks as are resident at once (three per SM), so that each plans once, ahead of
  // the wait, and then takes row after row or chunk after chunk.
  constexpr int kResident = 3 * kDecodeSms;
  // Few rows have many partials each (their tiles are spread over all CTAs): a block per row
  // then, else a warp per row.
  const bool few = rows <= 2 * kDecodeSms;
  const long long most = few ? rows : (SCORES ? kResident / 4 : kResident);
  const int row_blocks = static_cast<int>(few || (rows + 7) / 8 > most ? most : (rows + 7) / 8);
  const int left = row_blocks < kResident - 32 ? kResident - row_blocks : 32;
  const int weight_blocks = SCORES ? static_cast<int>(chunks < left ? chunks : left) : 0;
  if (few)
    return launch_dependent(decode_finish<D, SCORES, 8>, row_blocks + weight_blocks, kFinishThreads, 0, 1, st, prm,
                            row_blocks);
  return launch_dependent(decode_finish<D, SCORES, 1>, row_blocks + weight_blocks, kFinishThreads, 0, 1, st, prm,
                          row_blocks);
}

}  // namespace

cudaError_t launch_decode(const DecodeArgs& a, bool fp8, cudaStream_t st) {
  DecodeParams prm;
  memset(&prm, 0, sizeof(prm));
  const int box_d = fp8 ? 128 : 64;
  const long long kv_rows = static_cast<long long>(a.num_slots) * kTile;
  if (!make_map(&prm.tk, a.k_cache, fp8, a.d, a.Hkv, kv_rows, box_d, kTile)) return cudaErrorInvalidValue;
  if (!make_map(&prm.tv, a.v_cache, fp8, a.d, a.Hkv, kv_rows, box_d, kTile)) return cudaErrorInvalidValue;
  prm.a = a;
  const int R = a.n * a.G;
  prm.rt = (R + kDecodeRows - 1) / kDecodeRows;
  prm.pre = plan_prefix(a.B, a.n, a.Hkv, a.G, a.prefix_len);
  prm.prt = a.prefix_len > 0 && prm.pre.gangs == 0 ? (a.B * R + kDecodeRows - 1) / kDecodeRows : 0;
  prm.prefix_pages = (a.prefix_len + kTile - 1) / kTile;
  prm.g_magic = a.G > 1 ? static_cast<uint32_t>(((1ull << 32) + a.G - 1) / a.G) : 0u;
  prm.gang = gang_of(a.Hkv);
  prm.head_groups = a.Hkv / prm.gang;
  prm.prefix_span = prm.prt > 0 ? prm.head_groups * prm.prt * (prm.prefix_pages + kDecodeUnitCost) : 0;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const long long bound = static_cast<long long>(prm.head_groups) *
                          (prm.prt * prm.prefix_pages +
                           static_cast<long long>(a.B) * prm.rt * ((a.max_kv_len + kTile - 1) / kTile));
  sms = sms < kDecodeSms ? sms : kDecodeSms;
  const int per_sm = fp8 || a.d == 64 ? 3 : 2;  // Cfg::CTAS
  prm.gangs = sms * per_sm / prm.gang;
  // Behind prefix_kernel's launch the CTAs of one round on the SMs that it leaves free, where
  // that round is likely the shorter of the two (a 64-token tile here takes a quarter of a
  // 128-key tile there, at which the host's bound on the lengths is compared); otherwise as many
  // as without a prefix, the later ones starting as places become free.  64 sequences behind
  // 32768 shared tokens, one round / all: 72 / 72 us at 512 own tokens, 88 / 94 at 1024,
  // 140 / 125 at 2048, 242 / 196 at 4096.
  const int beside = (sms - prm.pre.gangs * prm.pre.gang) * per_sm / prm.gang;
  if (prm.pre.gangs > 0 && beside > 0 && bound <= 4ll * beside * prm.pre.per) prm.gangs = beside;
  if (bound < prm.gangs) prm.gangs = static_cast<int>(bound);
  const bool scores = a.scores != nullptr;
  if (fp8) return scores ? run<128, true, true>(prm, st) : run<128, true, false>(prm, st);
  if (a.d == 128) return scores ? run<128, false, true>(prm, st) : run<128, false, false>(prm, st);
  return scores ? run<64, false, true>(prm, st) : run<64, false, false>(prm, st);
}

}  // namespace stem

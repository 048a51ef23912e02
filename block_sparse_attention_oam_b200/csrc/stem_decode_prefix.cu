// The shared prefix of a decoding step on the tensor cores (tcgen05 + TMEM + TMA), sm_100a.
//
// All sequences of the batch see the same prefix, so a kv-head's rows are all of the batch's:
// B * q_len * G of them (256 for 64 sequences of Qwen3-8B's layer), over K and V that are read
// once per pair of row tiles.  Here the work is a product of that many rows, 4 d flops per row
// and key against 4 d bytes per key in BF16 (2 d in FP8): one flop a byte and row (two), so that
// the 256 rows of a pair make 256 (512), about what the tensor cores need (250).
//
// One CTA per SM, on two thirds of them; decode_kernel reads the own tokens on the others
// meanwhile (kPrefixCtas has the figures).  Work unit: one kv-head and two row tiles ("slots")
// of floor(128 / G) tokens each, G rows per token; the unit's keys, in tiles of 128 (two pages), are split
// evenly over the CTAs as in decode_kernel (a line, gangs of CTAs on neighbouring heads), and
// each CTA leaves its share's (m, l, O) for decode_finish.
//   warp 0      TMA producer: the unit's Q tiles, then K and V tiles through shared rings
//   warp 1      MMA issuer: S = Q K^T into a slot's TMEM columns, O += P V with P in TMEM;
//               the two slots take turns, one's softmax under the other's products
//   warps 2..17 softmax, eight warps per slot, two threads per row with 64 of the tile's 128
//               keys each (a quarter of the registers free, 4 % faster than one per row).  The
//               halves agree on the row's running maximum through shared memory; it is raised
//               lazily; sums of the unrounded P in float32
//   warps 18,19 (FP8) widen V's codes to f16 in shared memory: with P in f16 the product
//               carries P to 2^-11, where an e4m3 P would lose 2^-4 of every weight; S stays
//               an e4m3 product, which is exact
// A 128-key tile of 256 rows takes 2.06 us in BF16 and 1.98 in FP8 (calls of 64 sequences behind
// 32K to 128K tokens, by the difference; 4.06 thousand cycles at 1965 MHz), in which the matrix
// pipe is active 70 % and XU (exponentials, the packing of P) 72 %: with S and O of two slots
// the 512 TMEM columns are full, so a slot's S waits for its last product.  Tiles of 64 keys with a
// second S took 95 us where these took 85.
// Measured on one B200, whole calls, 32 q- and 8 kv-heads of 128: 64 sequences of up to 1K own
// tokens behind 32768 shared ones, BF16, 72 to 81 us, of which 44 are the tiles and 8 the joining
// after the last of them; 128 of up to 512 behind 16384, FP8, 71 to 73 us.
// P in f16 is taken as 2^(s - m + 7), as in decode_kernel, so that a long tail of small weights
// counts; BF16 rounds P to bf16, as V is.  V rows behind the prefix's end (the rest of its last page)
// are set to zero in shared memory, since they may hold NaN and 0 * NaN is not 0.
// Waits are bounded as in the other kernels.
#include <string.h>

#include "stem_internal.cuh"

namespace stem {
namespace {

constexpr int kBN = kPrefixTile;   // keys of a tile
constexpr int kRows = 128;         // rows of a slot
constexpr uint32_t kTmemCols = 512;

template <int D, bool FP8>
struct Cfg {
  static constexpr int ES = FP8 ? 1 : 2;
  static constexpr int CH = 128 / ES;
  static constexpr int DCH = D * ES / 128;          // 128-byte chunks of a Q, K or V row
  static constexpr int CHUNK = 128 * 128;           // 128 rows of a chunk
  static constexpr int TILE = DCH * CHUNK;
  static constexpr int VCH = D * 2 / 128;           // chunks of a V row as multiplied (16 bits)
  static constexpr int VTILE = VCH * CHUNK;
  static constexpr int NK = FP8 ? 3 : (D == 128 ? 2 : 4);
  static constexpr int NV = FP8 ? 2 : NK;
  static constexpr int NH = FP8 ? 2 : 0;            // widened V tiles
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_K = 2 * TILE;
  static constexpr int OFF_V = OFF_K + NK * TILE;
  static constexpr int OFF_H = OFF_V + NV * TILE;
  static constexpr int OFF_BAR = OFF_H + NH * VTILE;
  static constexpr int OFF_MAX = OFF_BAR + 512;     // float [2][2 slots][2 halves][128 rows]
  static constexpr int SMEM = OFF_MAX + 4096 + 1024;
  static_assert(SMEM <= 227 * 1024 && SMEM > 114 * 1024, "one CTA per SM");
  static constexpr float kLift = FP8 ? kLiftF16 : 0.f;
  static constexpr int THREADS = 32 * (FP8 ? 20 : 18);
  static constexpr int S_STEPS = D * ES / 32;
  static constexpr int PV_STEPS = kBN / 16;
  static constexpr uint32_t IDESC_S = instr_desc(FP8 ? 0u : 1u, 0, 0, kRows, kBN);
  static constexpr uint32_t IDESC_PV = instr_desc(FP8 ? 0u : 1u, 0, 1, kRows, D);  // f16 or bf16
};

struct PrefixParams {
  CUtensorMap tq;    // Q [T, Hkv, G, d]: dims (d, G, Hkv, T), box (CH, G, 1, slot_tokens)
  CUtensorMap tk, tv;
  PrefixPlan plan;
  const int32_t* table;
  int pages, len, num_slots;
  int tokens, G;     // T = B * q_len, rows per token
  float scale_log2;
  float* part_o;     // [slots, 256, d]
  float2* part_ml;   // [slots, 256]
  uint32_t* status;
};

struct Seg {
  int kvh, tok0, ns;   // head, first token, slots with tokens
  long long slot;      // where the partial goes
  int j0, j1;          // tiles
};

struct Walk {
  int t, end, gang_no, rank;
  __device__ __forceinline__ bool next(const PrefixParams& p, Seg* s) {
    const PrefixPlan& pl = p.plan;
    const int span = pl.tiles + kPrefixUnitCost;
    while (t < end) {
      const int u = t / span, at = t - u * span;
      const int stop = min(span, at + (end - t));
      t += stop - at;
      s->kvh = u / pl.pairs * pl.gang + rank;
      s->tok0 = u % pl.pairs * 2 * pl.slot_tokens;
      s->ns = s->tok0 + pl.slot_tokens < p.tokens ? 2 : 1;
      s->slot = static_cast<long long>(gang_no + u) * pl.gang + rank;
      s->j0 = max(0, at - kPrefixUnitCost);
      s->j1 = stop - kPrefixUnitCost;
      if (s->j1 > s->j0) return true;
    }
    return false;
  }
};

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0, int c1, int c2,
                                            int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}
__device__ __forceinline__ void fence_async_shared() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void st_shared16(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
// One whole 32-byte sector.
__device__ __forceinline__ void st_global32(float* at, const uint32_t* v) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(at), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]),
               "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
__device__ __forceinline__ uint4 ld_shared16(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
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

// Bounded wait by a whole warp.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag, uint32_t* status) {
  const unsigned full = 0xffffffffu;
  if (__all_sync(full, mbar_try_wait(bar, parity))) return true;
  const uint64_t t0 = global_ns();
  for (int spins = 1;; ++spins) {
    if (__all_sync(full, mbar_try_wait(bar, parity))) return true;
    if ((spins & 31) == 0) {
      if (__shfl_sync(full, *abort_flag, 0)) return false;
      if (__shfl_sync(full, (global_ns() - t0) > kWaitLimitNs ? 1 : 0, 0)) {
        if ((threadIdx.x & 31) == 0) {
          *abort_flag = 1;
          atomicOr(status, kStatusTimeout);
        }
        __syncwarp();
        return false;
      }
    }
  }
}

template <int D, bool FP8>
__global__ void __launch_bounds__(Cfg<D, FP8>::THREADS, 1) prefix_kernel(const __grid_constant__ PrefixParams p) {
  using C = Cfg<D, FP8>;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem =
      reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t sQ = sbase + C::OFF_Q, sK = sbase + C::OFF_K, sV = sbase + C::OFF_V, sH = sbase + C::OFF_H;
  const uint32_t b0 = sbase + C::OFF_BAR;
  auto q_full = [&](int s) { return b0 + 8 * s; };
  auto q_empty = [&](int s) { return b0 + 16 + 8 * s; };
  auto s_full = [&](int s) { return b0 + 32 + 8 * s; };
  auto p_full = [&](int s) { return b0 + 48 + 8 * s; };
  auto o_done = [&](int s) { return b0 + 64 + 8 * s; };
  auto k_full = [&](int t) { return b0 + 80 + 8 * t; };
  auto k_empty = [&](int t) { return b0 + 112 + 8 * t; };
  auto v_full = [&](int t) { return b0 + 144 + 8 * t; };
  auto v_empty = [&](int t) { return b0 + 176 + 8 * t; };
  auto h_full = [&](int t) { return b0 + 208 + 8 * t; };
  auto h_empty = [&](int t) { return b0 + 224 + 8 * t; };
  const uint32_t bar_drain = b0 + 240;
  auto agreed = [&](int s, int q) { return b0 + 288 + 8 * (4 * s + q); };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_BAR + 256);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_BAR + 264);

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const unsigned full = 0xffffffffu;
  if (threadIdx.x == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(q_full(s), 1);
      mbar_init(q_empty(s), 1);
      mbar_init(s_full(s), 1);
      mbar_init(p_full(s), 8);
      for (int q = 0; q < 4; ++q) mbar_init(agreed(s, q), 2);
      mbar_init(o_done(s), 1);
    }
    for (int t = 0; t < C::NK; ++t) {
      mbar_init(k_full(t), 1);
      mbar_init(k_empty(t), 1);
    }
    for (int t = 0; t < C::NV; ++t) {
      mbar_init(v_full(t), 1);
      mbar_init(v_empty(t), FP8 ? 2 : 1);
    }
    for (int t = 0; t < C::NH; ++t) {
      mbar_init(h_full(t), 2);
      mbar_init(h_empty(t), 1);
    }
    mbar_init(bar_drain, 1);
    *abort_flag = 0;
    mbar_fence_init();
    tma_prefetch_map(&p.tq);
    tma_prefetch_map(&p.tk);
    tma_prefetch_map(&p.tv);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();
  pdl_trigger();  // not earlier: decode_kernel relies on this wait
  const PrefixPlan& pl = p.plan;
  const int gang_no = static_cast<int>(blockIdx.x) / pl.gang, rank = static_cast<int>(blockIdx.x) % pl.gang;
  const int total = pl.head_groups * pl.pairs * (pl.tiles + kPrefixUnitCost);
  const int t0 = min(total, gang_no * pl.per);
  Walk walk{t0, min(total, t0 + pl.per), gang_no, rank};
  Seg sg;

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    uint32_t it = 0, tq[2] = {0, 0};
    bool alive = true;
    const int slot_rows = pl.slot_tokens * p.G;
    while (alive && walk.next(p, &sg)) {
      for (int s = 0; s < sg.ns && alive; ++s) {
        if (!warp_wait(q_empty(s), (tq[s] & 1) ^ 1, abort_flag, p.status)) {
          alive = false;
          break;
        }
        if (lane == 0) {
          mbar_arrive_expect_tx(q_full(s), C::DCH * 128 * slot_rows);
          for (int c = 0; c < C::DCH; ++c)
            tma_load_4d(sQ + s * C::TILE + c * C::CHUNK, &p.tq, q_full(s), c * C::CH, 0, sg.kvh,
                        sg.tok0 + s * pl.slot_tokens);
        }
        ++tq[s];
      }
      for (int q0 = sg.j0; q0 < sg.j1 && alive; q0 += 16) {
        // 32 pages: lanes 2 i and 2 i + 1 hold those of tile q0 + i
        int slot = 0;
        const int pg = min(2 * q0 + lane, p.pages - 1);
        if (q0 + lane / 2 < sg.j1) {
          slot = __ldg(p.table + pg);
          if (slot < 0 || slot >= p.num_slots) {
            atomicOr(p.status, kStatusBounds);
            slot = 0;
          }
        }
        const int cnt = min(16, sg.j1 - q0);
        for (int q = 0; q < cnt; ++q, ++it) {
          const int ra = __shfl_sync(full, slot, 2 * q) * STEM_PAGE_SIZE;
          const int rb = __shfl_sync(full, slot, 2 * q + 1) * STEM_PAGE_SIZE;
          const int tk = it % C::NK, tv = it % C::NV;
          if (!warp_wait(k_empty(tk), ((it / C::NK) & 1) ^ 1, abort_flag, p.status)) {
            alive = false;
            break;
          }
          if (lane == 0) {
            mbar_arrive_expect_tx(k_full(tk), C::TILE);
            for (int c = 0; c < C::DCH; ++c) {
              tma_load_3d(sK + tk * C::TILE + c * C::CHUNK, &p.tk, k_full(tk), c * C::CH, sg.kvh, ra);
              tma_load_3d(sK + tk * C::TILE + c * C::CHUNK + 64 * 128, &p.tk, k_full(tk), c * C::CH, sg.kvh, rb);
            }
          }
          if (!warp_wait(v_empty(tv), ((it / C::NV) & 1) ^ 1, abort_flag, p.status)) {
            // this tile's K is in flight and counted below
            ++it;
            alive = false;
            break;
          }
          if (lane == 0) {
            mbar_arrive_expect_tx(v_full(tv), C::TILE);
            for (int c = 0; c < C::DCH; ++c) {
              tma_load_3d(sV + tv * C::TILE + c * C::CHUNK, &p.tv, v_full(tv), c * C::CH, sg.kvh, ra);
              tma_load_3d(sV + tv * C::TILE + c * C::CHUNK + 64 * 128, &p.tv, v_full(tv), c * C::CH, sg.kvh, rb);
            }
          }
        }
      }
    }
    if (!alive) {
      // let the copies already issued land before the CTA can exit (a wait on one that was
      // never issued runs out)
      for (uint32_t q = it > C::NK ? it - C::NK : 0; q < it; ++q)
        for (int spin = 0; spin < 1000000 && !mbar_try_wait(k_full(q % C::NK), (q / C::NK) & 1); ++spin) {}
      for (uint32_t q = it > C::NV ? it - C::NV : 0; q < it; ++q)
        for (int spin = 0; spin < 1000000 && !mbar_try_wait(v_full(q % C::NV), (q / C::NV) & 1); ++spin) {}
      for (int s = 0; s < 2; ++s)
        if (tq[s] > 0)
          for (int spin = 0; spin < 1000000 && !mbar_try_wait(q_full(s), (tq[s] - 1) & 1); ++spin) {}
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      uint32_t it = 0, gb[2] = {0, 0}, tq[2] = {0, 0};
      bool alive = true;
      auto issue_s = [&](int s, uint32_t t) {
        const uint32_t d_tmem = tmem + 256 * s;
#pragma unroll
        for (int k = 0; k < C::S_STEPS; ++k) {
          const int c = k / 4, w = k % 4;
          const uint64_t ad = smem_desc_sw128(sQ + s * C::TILE + c * C::CHUNK + w * 32, 16, 1024);
          const uint64_t bd = smem_desc_sw128(sK + t * C::TILE + c * C::CHUNK + w * 32, 16, 1024);
          if (FP8)
            mma_fp8(d_tmem, ad, bd, C::IDESC_S, k > 0);
          else
            mma_bf16(d_tmem, ad, bd, C::IDESC_S, k > 0);
        }
        mma_commit(s_full(s));
      };
      while (alive && walk.next(p, &sg)) {
        const int n = sg.j1 - sg.j0;
        uint32_t tk = it % C::NK;
        if (!mbar_wait(k_full(tk), (it / C::NK) & 1, abort_flag, p.status)) break;
        for (int s = 0; s < sg.ns; ++s) {
          if (!mbar_wait(q_full(s), tq[s]++ & 1, abort_flag, p.status)) {
            alive = false;
            break;
          }
          tc_fence_after();
          issue_s(s, tk);
          if (n == 1) mma_commit(q_empty(s));
        }
        if (!alive) break;
        mma_commit(k_empty(tk));
        for (int jj = 0; jj < n && alive; ++jj, ++it) {
          const bool more = jj + 1 < n;
          // V_j and K_{j+1} land long before P_j is ready: waited for first, so that both
          // products go out back to back
          const uint32_t tv = FP8 ? it % (C::NH ? C::NH : 1) : it % C::NV;
          const uint32_t pv = FP8 ? it / (C::NH ? C::NH : 1) : it / C::NV;
          if (!mbar_wait(FP8 ? h_full(tv) : v_full(tv), pv & 1, abort_flag, p.status)) {
            alive = false;
            break;
          }
          tk = (it + 1) % C::NK;
          if (more && !mbar_wait(k_full(tk), ((it + 1) / C::NK) & 1, abort_flag, p.status)) {
            alive = false;
            break;
          }
          for (int s = 0; s < sg.ns; ++s) {
            if (!mbar_wait(p_full(s), gb[s]++ & 1, abort_flag, p.status)) {
              alive = false;
              break;
            }
            tc_fence_after();
            const uint32_t vt = FP8 ? sH + tv * C::VTILE : sV + tv * C::TILE;
#pragma unroll
            for (int k = 0; k < C::PV_STEPS; ++k)
              mma_bf16_ts(tmem + 256 * s + 128, tmem + 256 * s + k * 8,
                          smem_desc_sw128(vt + k * 16 * 128, C::CHUNK, 1024), C::IDESC_PV, jj > 0 || k > 0);
            if (more) {
              issue_s(s, tk);
              if (jj + 2 == n) mma_commit(q_empty(s));  // the unit's last S: Q may be replaced
            } else {
              mma_commit(o_done(s));
            }
          }
          if (!alive) break;
          mma_commit(FP8 ? h_empty(tv) : v_empty(tv));
          if (more) mma_commit(k_empty(tk));
        }
      }
      mma_commit(bar_drain);
      for (int spin = 0; spin < 4000000 && !mbar_try_wait(bar_drain, 0); ++spin) {}
    }
    __syncwarp();
  } else if (warp < 18) {
    // ------------------------------------------------------------ softmax
    constexpr int HN = kBN / 2;                      // keys of a half
    const int slot = (warp - 2) / 8, half = (warp - 2) / 4 % 2, quad = warp % 4;
    const int r = quad * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(quad * 32) << 16;
    const uint32_t my_S = tmem + 256 * slot + lane_off;
    const uint32_t my_O = my_S + 128 + half * (D / 2);
    volatile float* my_max = reinterpret_cast<volatile float*>(smem + C::OFF_MAX) + (slot * 2 + half) * 128 + r;
    volatile float* other_max = reinterpret_cast<volatile float*>(smem + C::OFF_MAX) + (slot * 2 + 1 - half) * 128 + r;
    const float2 sc2 = make_float2(p.scale_log2, p.scale_log2);
    uint32_t gb = 0, ga = 0, ot = 0, it = 0;
    bool alive = true;
    // Exchanges a value with the row's other thread.  Two buffers in turn: a thread writes one
    // again only after the exchange in between, to which the other came after it had read.
    auto swap = [&](float mine, float* theirs) -> bool {
      const int at = ga & 1 ? 512 : 0;
      my_max[at] = mine;
      __syncwarp();
      if (lane == 0) mbar_arrive(agreed(slot, quad));
      if (!warp_wait(agreed(slot, quad), ga++ & 1, abort_flag, p.status)) return false;
      *theirs = other_max[at];
      return true;
    };
    while (alive && walk.next(p, &sg)) {
      const int n = sg.j1 - sg.j0;
      if (slot >= sg.ns) {
        it += n;
        continue;
      }
      float m_run = -INFINITY;
      float2 l2 = make_float2(0.f, 0.f);
      for (int jj = 0; jj < n; ++jj, ++gb, ++it) {
        if (!warp_wait(s_full(slot), gb & 1, abort_flag, p.status)) {
          alive = false;
          break;
        }
        tc_fence_after();
        uint32_t sr[HN];
#pragma unroll
        for (int c = 0; c < HN / 32; ++c)
          tmem_ld32(my_S + half * HN + c * 32, *reinterpret_cast<uint32_t(*)[32]>(&sr[c * 32]));
        tmem_wait_ld();
        const int valid = p.len - (sg.j0 + jj) * kBN;
        if (valid < kBN) {
#pragma unroll
          for (int c = 0; c < HN; ++c)
            if (half * HN + c >= valid) sr[c] = __float_as_uint(-INFINITY);
          if constexpr (!FP8) {
            // V's rows behind the end
            const uint32_t tv = it % C::NV;
            if (!warp_wait(v_full(tv), (it / C::NV) & 1, abort_flag, p.status)) {
              alive = false;
              break;
            }
            if (half == 0 && r >= valid)
              for (int c = 0; c < C::DCH; ++c)
                for (int x = 0; x < 8; ++x) st_shared16(sV + tv * C::TILE + c * C::CHUNK + r * 128 + x * 16, 0, 0, 0, 0);
            fence_async_shared();
          }
        }
        float mq[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int c = 0; c < HN; c += 8)
#pragma unroll
          for (int q = 0; q < 4; ++q)
            mq[q] = max3f(mq[q], __uint_as_float(sr[c + 2 * q]), __uint_as_float(sr[c + 2 * q + 1]));
        // After the exchange both halves of S are in registers, so P may be written over them
        float mx = fmaxf(max3f(mq[0], mq[1], mq[2]), mq[3]), theirs;
        tc_fence_before();
        if (!swap(mx, &theirs)) {
          alive = false;
          break;
        }
        tc_fence_after();
        mx = fmaxf(mx, theirs);
        const float m_new = fmaxf(m_run, mx * p.scale_log2);
        const bool resc = m_new > m_run + 8.0f;
        const float m_use = resc ? m_new : m_run;
        const float alpha = resc ? ex2_approx(m_run - m_use) : 1.0f;
        const float m_sub = m_use == -INFINITY ? 0.f : m_use - C::kLift;
        const float2 bias2 = make_float2(-m_sub, -m_sub);
        float2 sq[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) sq[q] = make_float2(0.f, 0.f);
        // P packed in place over the first half of the registers
#pragma unroll
        for (int u = 0; u < HN / 2; ++u) {
          const float2 y = fma2(make_float2(__uint_as_float(sr[2 * u]), __uint_as_float(sr[2 * u + 1])), sc2, bias2);
          const float2 e = make_float2(ex2_approx(y.x), ex2_approx(y.y));
          sr[u] = FP8 ? pack_f16x2(e.x, e.y) : pack_bf16x2(e.x, e.y);
          sq[u % 4] = add2(sq[u % 4], e);
        }
        static_assert(HN / 2 == 32, "a half's P is one store");
        tmem_st32(my_S + half * 32, *reinterpret_cast<uint32_t(*)[32]>(&sr[0]));
        const float2 a2 = make_float2(alpha, alpha);
        l2 = fma2(l2, a2, add2(add2(sq[0], sq[1]), add2(sq[2], sq[3])));
        if (jj > 0 && __any_sync(full, resc)) {
          // S_j was issued after P V_{j-1} and is complete: O holds the sum up to there
#pragma unroll
          for (int c = 0; c < D / 64; ++c) {
            uint32_t o[32];
            tmem_ld32(my_O + c * 32, o);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              const float2 v = mul2(make_float2(__uint_as_float(o[e]), __uint_as_float(o[e + 1])), a2);
              o[e] = __float_as_uint(v.x);
              o[e + 1] = __float_as_uint(v.y);
            }
            tmem_st32(my_O + c * 32, o);
          }
        }
        tmem_wait_st();
        m_run = m_use;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full(slot));
      }
      if (!alive) break;
      float l = l2.x + l2.y, l_other;
      if (!swap(l, &l_other) || !warp_wait(o_done(slot), ot & 1, abort_flag, p.status)) break;
      ++ot;
      tc_fence_after();
      const int rows = min(pl.slot_tokens, p.tokens - sg.tok0 - slot * pl.slot_tokens) * p.G;
      const long long row = sg.slot * (2 * kRows) + slot * kRows + r;
      float* out = p.part_o + row * D + half * (D / 2);
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        uint32_t o[32];
        tmem_ld32(my_O + c * 32, o);
        tmem_wait_ld();
        if (r < rows) {
#pragma unroll
          for (int e = 0; e < 32; e += 8) st_global32(out + c * 32 + e, &o[e]);
        }
      }
      if (half == 0 && r < rows) p.part_ml[row] = make_float2(m_run - C::kLift, l + l_other);
      tc_fence_before();
    }
  } else {
    // ------------------------------------------------------------ V codes to f16 (FP8)
    if constexpr (FP8) {
      uint32_t it = 0;
      bool alive = true;
      while (alive && walk.next(p, &sg)) {
        for (int j = sg.j0; j < sg.j1; ++j, ++it) {
          const uint32_t tv = it % C::NV, th = it % C::NH;
          if (!warp_wait(v_full(tv), (it / C::NV) & 1, abort_flag, p.status) ||
              !warp_wait(h_empty(th), ((it / C::NH) & 1) ^ 1, abort_flag, p.status)) {
            alive = false;
            break;
          }
          const int valid = p.len - j * kBN;
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const int tok = half * 64 + (warp - 18) * 32 + lane;
            const uint32_t src = sV + tv * C::TILE + tok * 128, dst = sH + th * C::VTILE + tok * 128;
#pragma unroll
            for (int x = 0; x < 8; ++x) {   // 16 codes: 32 bytes of chunk x / 4
              uint4 v = ld_shared16(src + ((x ^ (tok & 7)) << 4));
              if (tok >= valid) v = make_uint4(0, 0, 0, 0);
              const uint32_t out = dst + (x / 4) * C::CHUNK;
              const int col = (x % 4) * 2;
              st_shared16(out + ((col ^ (tok & 7)) << 4), e4m3x2_to_h2(v.x & 0xFFFFu), e4m3x2_to_h2(v.x >> 16),
                          e4m3x2_to_h2(v.y & 0xFFFFu), e4m3x2_to_h2(v.y >> 16));
              st_shared16(out + (((col + 1) ^ (tok & 7)) << 4), e4m3x2_to_h2(v.z & 0xFFFFu), e4m3x2_to_h2(v.z >> 16),
                          e4m3x2_to_h2(v.w & 0xFFFFu), e4m3x2_to_h2(v.w >> 16));
            }
          }
          fence_async_shared();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(h_full(th));
            mbar_arrive(v_empty(tv));
          }
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, kTmemCols);
}

template <int D, bool FP8>
cudaError_t run(const PrefixParams& prm, cudaStream_t st) {
  using C = Cfg<D, FP8>;
  const cudaError_t e = set_smem_once<prefix_kernel<D, FP8>>(C::SMEM);
  if (e != cudaSuccess) return e;
  return launch_dependent(prefix_kernel<D, FP8>, prm.plan.gangs * prm.plan.gang, C::THREADS, C::SMEM, 1, st, prm);
}

}  // namespace

PrefixPlan plan_prefix(int B, int n, int Hkv, int G, int prefix_len) {
  PrefixPlan p{};
  const int tokens = B * n;
  // Up to two row tiles decode_kernel's own products are as quick and need no second launch: 8192
  // shared tokens, 32 rows there 18 us, 36 rows here 23.
  if (prefix_len < 1 || G > kRows || static_cast<long long>(tokens) * G <= kPrefixMinRows) return p;
  p.gang = gang_of(Hkv);
  p.head_groups = Hkv / p.gang;
  p.slot_tokens = kRows / G;
  p.pairs = (tokens + 2 * p.slot_tokens - 1) / (2 * p.slot_tokens);
  p.tiles = (prefix_len + kBN - 1) / kBN;
  const long long units = static_cast<long long>(p.head_groups) * p.pairs;
  p.gangs = kPrefixCtas / p.gang;
  if (units * p.tiles < p.gangs) p.gangs = static_cast<int>(units * p.tiles);
  p.per = static_cast<int>((units * (p.tiles + kPrefixUnitCost) + p.gangs - 1) / p.gangs);
  p.slots = (p.gangs + units) * p.gang;
  return p;
}

cudaError_t launch_prefix(const DecodeArgs& a, const PrefixPlan& plan, bool fp8, cudaStream_t st) {
  PrefixParams prm;
  memset(&prm, 0, sizeof(prm));
  const int box_d = fp8 ? 128 : 64;
  const long long kv_rows = static_cast<long long>(a.num_slots) * STEM_PAGE_SIZE;
  if (!make_map_rows(&prm.tq, a.q, fp8, a.d, a.G, a.Hkv, static_cast<long long>(a.B) * a.n, box_d, plan.slot_tokens))
    return cudaErrorInvalidValue;
  if (!make_map(&prm.tk, a.k_cache, fp8, a.d, a.Hkv, kv_rows, box_d, STEM_PAGE_SIZE)) return cudaErrorInvalidValue;
  if (!make_map(&prm.tv, a.v_cache, fp8, a.d, a.Hkv, kv_rows, box_d, STEM_PAGE_SIZE)) return cudaErrorInvalidValue;
  prm.plan = plan;
  prm.table = a.prefix_table;
  prm.pages = (a.prefix_len + STEM_PAGE_SIZE - 1) / STEM_PAGE_SIZE;
  prm.len = a.prefix_len;
  prm.num_slots = a.num_slots;
  prm.tokens = a.B * a.n;
  prm.G = a.G;
  prm.scale_log2 = a.scale_log2;
  prm.part_o = a.prefix_o;
  prm.part_ml = a.prefix_ml;
  prm.status = a.status;
  if (fp8) return run<128, true>(prm, st);
  return a.d == 128 ? run<128, false>(prm, st) : run<64, false>(prm, st);
}

}  // namespace stem

// Eviction from a paged K/V cache by accumulated attention weight, sm_100a.
//
// For every (sequence, kv-head): of n cached tokens the first `sink`, the last `recent` and
// the heaviest others stay, `budget` in all; the kept K/V rows go, in order, to fresh
// pages.  Two launches:
//   evict_select  the cut-off weight by radix selection (weights as ordered 32-bit keys,
//                 digits of 11, 11 and 10 bits from the top), then the kept positions in
//                 ascending order.  One cluster per (sequence, kv-head) holds all its keys in
//                 shared memory, histograms and counts joined through distributed shared memory;
//                 the weights are read once, nothing is sorted, and the order of the atomics
//                 cannot show (they count).
//   evict_move    copies the rows: the bytes are what the operator cannot do without
//                 (budget rows read and written, K and V), so each thread keeps eight
//                 16-byte loads in flight; heads are the inner index, as they are in
//                 memory, so that rows kept by several heads are read side by side.
#include <string.h>

#include <cooperative_groups.h>

#include "stem_internal.cuh"

namespace stem {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr int kMaxCluster = 8;
constexpr int kMaxKeys = 64;                  // keys a thread holds at most
static_assert(kThreads * kMaxCluster * kMaxKeys >= STEM_MAX_KV_LEN, "a cluster holds the longest sequence");
constexpr int kMoveThreads = 256;
constexpr int kMovePieces = 8;                // 16-byte pieces a thread has in flight
constexpr int kMoveRows = 512;                // (token, head) rows of a move CTA at most
static_assert(kBins == 4 * kThreads, "four bins per thread");

struct EvictParams {
  EvictArgs a;
  int kpt;             // keys of a select thread
  int move_tokens;     // tokens of a move CTA
};

// Weights in an order that unsigned comparison follows; NaN as -inf, -0 as +0.
__device__ __forceinline__ uint32_t order_key(float w) {
  if (!(w == w)) w = -INFINITY;
  const uint32_t u = w == 0.f ? 0u : __float_as_uint(w);
  return (u >> 31) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ int warp_inclusive(int x) {
  const int lane = threadIdx.x % 32;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}

struct SelectSmem {
  int hist[3][kBins];
  int sums[kWarps];
  int digit, above;         // of the pass: the cut-off's digit, candidates in higher bins
  int more[kWarps], same[kWarps];  // kept above the cut-off (forced ones too) and equal to it, by warp
  int counts[2];            // of the CTA
};

// A CTA's slice is 512 * kpt positions, their keys in shared memory: warp w takes positions
// [w, w + 1) * 32 * kpt of it, key e of lane l being number 32 e + l, so that loads are
// coalesced, no key is another lane's, and ascending order is (warp, e, lane).
__global__ void __launch_bounds__(kThreads) evict_select(const __grid_constant__ EvictParams p) {
  const EvictArgs& a = p.a;
  __shared__ SelectSmem sm;
  extern __shared__ uint32_t keys[];
  const int kpt = p.kpt;  // a multiple of 8
  cg::cluster_group cluster = cg::this_cluster();
  const int C = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
  const int unit = blockIdx.x / C, b = unit / a.Hkv, h = unit % a.Hkv;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const unsigned all = 0xffffffffu;
  pdl_trigger();
  for (int i = tid; i < 3 * kBins; i += kThreads) sm.hist[0][i] = 0;
  pdl_wait();

  const int raw = __ldg(a.kv_lens + b);
  const int n = min(max(raw, 0), a.max_kv_len), m = min(n, a.budget);
  if (rank == 0 && h == 0 && tid == 0) {
    if (raw != n) atomicOr(a.status, kStatusBounds);
    a.kv_lens_out[b] = m;
  }
  const float* w = a.weights + static_cast<long long>(unit) * a.weights_stride;
  float* wout = a.weights_out + static_cast<long long>(unit) * a.weights_out_stride;
  int32_t* keep = a.keep + static_cast<long long>(unit) * a.budget;
  for (int i = m + rank * kThreads + tid; i < a.budget; i += C * kThreads) keep[i] = -1;
  if (n <= a.budget) {  // the same for the whole cluster
    for (int i = rank * kThreads + tid; i < n; i += C * kThreads) {
      keep[i] = i;
      if (a.weights_out) wout[i] = w[i];
    }
    return;
  }

  const int lo = a.sink, hi = n - a.recent, need = a.budget - a.sink - a.recent;  // candidates: [lo, hi)
  const int first = rank * (kThreads * kpt) + warp * (32 * kpt) + lane;           // position of key 0
  uint32_t* key = keys + warp * (32 * kpt) + lane;                                // key e at [32 * e]
#pragma unroll 8
  for (int e = 0; e < kpt; ++e) key[32 * e] = first + 32 * e < n ? order_key(w[first + 32 * e]) : 0u;
  auto candidate = [&](int e) { return first + 32 * e >= lo && first + 32 * e < hi; };
  __syncthreads();

  // the cut-off key, digit by digit
  uint32_t cut = 0xFFFFFFFFu;  // no key is this large
  int ties = 0;
  if (need > 0) {
    uint32_t prefix = 0;
    int left = need;
#pragma unroll
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0), bits = pass == 2 ? 10 : 11;
      int* hist = sm.hist[pass];
#pragma unroll 8
      for (int e = 0; e < kpt; ++e) {
        const uint32_t k = key[32 * e];
        const bool in = candidate(e) && (pass == 0 || (k >> (shift + bits)) == prefix);
        const int d = in ? static_cast<int>((k >> shift) & ((1u << bits) - 1)) : -1;
        // lanes that agree with the first one add once: equal weights are common (keys that
        // nothing has looked at), and same-address atomics of a warp are done one by one
        const unsigned on = __ballot_sync(all, in);
        if (on == 0) continue;
        const int lead = __ffs(on) - 1;
        const unsigned peers = __ballot_sync(all, d == __shfl_sync(all, d, lead));
        if (lane == lead) atomicAdd(hist + d, __popc(peers));
        else if (in && !(peers >> lane & 1u)) atomicAdd(hist + d, 1);
      }
      cluster.sync();
      // bins from the top down: four per thread
      const int bin = kBins - 4 - 4 * tid;
      int4 c = make_int4(0, 0, 0, 0);
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r)
        if (r < C) {
          const int4 x = *reinterpret_cast<const int4*>(cluster.map_shared_rank(hist, r) + bin);
          c.x += x.x;
          c.y += x.y;
          c.z += x.z;
          c.w += x.w;
        }
      const int cnt[4] = {c.w, c.z, c.y, c.x};
      const int sum = c.x + c.y + c.z + c.w;
      const int inc = warp_inclusive(sum);
      if (lane == 31) sm.sums[warp] = inc;
      __syncthreads();
      int before = inc - sum;
#pragma unroll
      for (int x = 0; x < kWarps; ++x) before += x < warp ? sm.sums[x] : 0;
      if (before < left && left <= before + sum) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (before < left && left <= before + cnt[e]) {
            sm.digit = bin + 3 - e;
            sm.above = before;
          }
          before += cnt[e];
        }
      }
      __syncthreads();
      prefix = (prefix << bits) | static_cast<uint32_t>(sm.digit);
      left -= sm.above;
    }
    cut = prefix;
    ties = left;
  }
  // which keys stay, the equal ones still open; counts by warp, CTA and rank
  auto above = [&](int e) { return first + 32 * e < n && (!candidate(e) || key[32 * e] > cut); };
  auto equal = [&](int e) { return candidate(e) && key[32 * e] == cut; };
  int more = 0, same = 0;
#pragma unroll 8
  for (int e = 0; e < kpt; ++e) {
    more += __popc(__ballot_sync(all, above(e)));
    same += __popc(__ballot_sync(all, equal(e)));
  }
  if (lane == 0) {
    sm.more[warp] = more;
    sm.same[warp] = same;
  }
  __syncthreads();
  int pos = 0, eq = 0, all_more = 0, all_same = 0;
#pragma unroll
  for (int x = 0; x < kWarps; ++x) {
    pos += x < warp ? sm.more[x] : 0;
    eq += x < warp ? sm.same[x] : 0;
    all_more += sm.more[x];
    all_same += sm.same[x];
  }
  if (tid == 0) {
    sm.counts[0] = all_more;
    sm.counts[1] = all_same;
  }
  cluster.sync();
#pragma unroll
  for (int r = 0; r < kMaxCluster; ++r)
    if (r < rank) {
      const int* c = cluster.map_shared_rank(sm.counts, r);
      pos += c[0];
      eq += c[1];
    }
  cluster.sync();  // the last look into another CTA's shared memory: each may leave from here on
  // the list, in ascending order; of the equal ones the first `ties`
  const unsigned below = (1u << lane) - 1u;
  pos += min(eq, ties);
#pragma unroll 8
  for (int e = 0; e < kpt; ++e) {
    const unsigned se = __ballot_sync(all, equal(e));
    const bool take = above(e) || (equal(e) && eq + __popc(se & below) < ties);
    const unsigned te = __ballot_sync(all, take);
    if (take) {
      const int at = pos + __popc(te & below);
      keep[at] = first + 32 * e;
      if (a.weights_out) wout[at] = w[first + 32 * e];
    }
    pos += __popc(te);
    eq += __popc(se);
  }
}

__global__ void __launch_bounds__(kMoveThreads) evict_move(const __grid_constant__ EvictParams p) {
  const EvictArgs& a = p.a;
  __shared__ long long src_row[kMoveRows], dst_row[kMoveRows];  // in rows of the caches; -1: nothing to move
  const int blocks = (a.budget + p.move_tokens - 1) / p.move_tokens;
  const int b = blockIdx.x / blocks, i0 = (blockIdx.x % blocks) * p.move_tokens;
  pdl_trigger();
  pdl_wait();
  const int m = min(min(max(__ldg(a.kv_lens + b), 0), a.max_kv_len), a.budget);
  const int tokens = min(p.move_tokens, m - i0);
  if (tokens <= 0) return;
  const int rows = tokens * a.Hkv;
  for (int x = threadIdx.x; x < rows; x += kMoveThreads) {
    const int i = i0 + x / a.Hkv, h = x % a.Hkv;
    const int j = a.keep[(static_cast<long long>(b) * a.Hkv + h) * a.budget + i];
    int s = a.src_table[static_cast<long long>(b) * a.src_max_pages + j / STEM_PAGE_SIZE];
    const int d = a.dst_table[static_cast<long long>(b) * a.dst_max_pages + i / STEM_PAGE_SIZE];
    bool bad = false;
    if (s < 0 || s >= a.src_slots) {
      s = 0;
      bad = true;
    }
    const bool lost = d < 0 || d >= a.dst_slots;
    if (bad || lost) atomicOr(a.status, kStatusBounds);
    src_row[x] = (static_cast<long long>(s) * STEM_PAGE_SIZE + j % STEM_PAGE_SIZE) * a.Hkv + h;
    dst_row[x] = lost ? -1 : (static_cast<long long>(d) * STEM_PAGE_SIZE + i % STEM_PAGE_SIZE) * a.Hkv + h;
  }
  __syncthreads();
  const int shift = a.row_shift;                 // log2 of a row's 16-byte pieces
  const int half = rows << shift, pieces = 2 * half;  // K, then V
  for (int x0 = threadIdx.x; x0 < pieces; x0 += kMoveThreads * kMovePieces) {
    uint4 v[kMovePieces];
#pragma unroll
    for (int e = 0; e < kMovePieces; ++e) {
      const int x = x0 + e * kMoveThreads;
      if (x < pieces) {
        const int y = x < half ? x : x - half;
        const uint4* from = static_cast<const uint4*>(x < half ? a.src_k : a.src_v);
        v[e] = __ldg(from + (src_row[y >> shift] << shift) + (y & ((1 << shift) - 1)));
      }
    }
#pragma unroll
    for (int e = 0; e < kMovePieces; ++e) {
      const int x = x0 + e * kMoveThreads;
      if (x < pieces) {
        const int y = x < half ? x : x - half;
        const long long to = dst_row[y >> shift];
        uint4* into = static_cast<uint4*>(x < half ? a.dst_k : a.dst_v);
        if (to >= 0) into[(to << shift) + (y & ((1 << shift) - 1))] = v[e];
      }
    }
  }
}

}  // namespace

cudaError_t launch_evict(const EvictArgs& a, cudaStream_t st) {
  EvictParams p;
  p.a = a;
  // A cluster's shared memory holds a sequence: 8 keys a thread and as many CTAs as that needs
  // (short chains of atomics, and long sequences of a ragged batch spread out), then more
  // keys a thread.
  const unsigned units = static_cast<unsigned>(a.B) * a.Hkv;
  const int chunks = (a.max_kv_len + kThreads * 8 - 1) / (kThreads * 8);
  int C = 1;
  while (C < kMaxCluster && C < chunks) C *= 2;
  p.kpt = 8 * ((chunks + C - 1) / C);
  cudaError_t e = set_smem_once<evict_select>(kMaxKeys * kThreads * 4);
  if (e != cudaSuccess) return e;
  e = launch_dependent(evict_select, units * C, kThreads, static_cast<size_t>(p.kpt) * kThreads * 4, C, st, p);
  if (e != cudaSuccess) return e;
  // a move CTA's tokens: 8 pieces a thread, within its table of rows
  const int per_token = 2 * a.Hkv << a.row_shift;
  int tokens = kMoveThreads * kMovePieces / per_token;
  if (tokens * a.Hkv > kMoveRows) tokens = kMoveRows / a.Hkv;
  p.move_tokens = tokens < 1 ? 1 : tokens;
  const unsigned blocks = static_cast<unsigned>(a.B) * ((a.budget + p.move_tokens - 1) / p.move_tokens);
  return launch_dependent(evict_move, blocks, kMoveThreads, 0, 1, st, p);
}

}  // namespace stem

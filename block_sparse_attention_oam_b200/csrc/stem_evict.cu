// Eviction from a paged K/V cache by accumulated attention weight, sm_100a.
//
// For every (sequence, kv-head): of n cached tokens the first `sink`, the last `recent` and
// the heaviest others stay, `budget` in all; the kept K/V rows go, in order, to fresh
// pages.  Two launches:
//   evict_select  the cut-off weight by radix selection (weights as ordered 32-bit keys,
//                 digits of 11, 11 and 10 bits from the top), then the kept positions in
//                 ascending order.  One cluster per (sequence, kv-head), every CTA a slice
//                 of the positions, histograms and counts joined through distributed shared
//                 memory; nothing is sorted and the order of the atomics cannot show.
//   evict_move    copies the rows: the bytes are what the operator cannot do without
//                 (budget rows read and written, K and V), so each thread keeps eight
//                 16-byte loads in flight; heads are the inner index, as they are in
//                 memory, so that rows kept by several heads are read side by side.
// The weights are read four times, three of them from L2 (4 bytes a token and head,
// against 4 * d * element bytes moved per kept one).
#include <string.h>

#include <cooperative_groups.h>

#include "stem_internal.cuh"

namespace stem {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr int kPer = 8;                       // consecutive positions of a thread when lists are written
constexpr int kMoveThreads = 256;
constexpr int kMovePieces = 8;                // 16-byte pieces a thread has in flight
constexpr int kMoveRows = 512;                // (token, head) rows of a move CTA at most
static_assert(kBins == 4 * kThreads, "four bins per thread");

struct EvictParams {
  EvictArgs a;
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

// Inclusive sum over the block and its total; `sums` is used again only after the next call's
// first barrier.
__device__ __forceinline__ int block_inclusive(int x, int* sums, int* total) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  x = warp_inclusive(x);
  __syncthreads();
  if (lane == 31) sums[warp] = x;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const int s = sums[w];
    if (w < warp) before += s;
    all += s;
  }
  *total = all;
  return x + before;
}

struct SelectSmem {
  int hist[3][kBins];
  int sums[kWarps];
  int digit, above;    // of the pass: the cut-off's digit, candidates in higher bins
  int counts[2];       // of this CTA's slice: kept above the cut-off (forced ones too), equal to it
};

__global__ void __launch_bounds__(kThreads) evict_select(const __grid_constant__ EvictParams p) {
  const EvictArgs& a = p.a;
  __shared__ SelectSmem sm;
  cg::cluster_group cluster = cg::this_cluster();
  const int C = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
  const int unit = blockIdx.x / C, b = unit / a.Hkv, h = unit % a.Hkv;
  const int tid = threadIdx.x;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

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
  const int slice = (n + C - 1) / C;
  const int s0 = min(n, rank * slice), s1 = min(n, s0 + slice);
  const int c0 = max(s0, lo), c1 = min(s1, hi);
  for (int i = tid; i < 3 * kBins; i += kThreads) sm.hist[0][i] = 0;
  __syncthreads();

  // the cut-off key, digit by digit
  uint32_t cut = 0xFFFFFFFFu;  // no key is this large
  int ties = 0, mine_above = 0, mine_equal = 0;
  if (need > 0) {
    uint32_t prefix = 0;
    int left = need;
#pragma unroll
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0), bits = pass == 2 ? 10 : 11;
      int* hist = sm.hist[pass];
#pragma unroll 4
      for (int i0 = c0; i0 < c1; i0 += kThreads) {
        const int i = i0 + tid;
        const bool in = i < c1;
        const uint32_t key = in ? order_key(w[i]) : 0u;
        const int d = (key >> shift) & ((1 << bits) - 1);
        if (pass == 0) {
          // sign, exponent and two more bits: few bins hold nearly all keys, so the lanes of
          // a warp that share one add once
          const unsigned peers = __match_any_sync(0xffffffffu, in ? d : -1);
          if (in && static_cast<int>(tid % 32) == __ffs(peers) - 1) atomicAdd(hist + d, __popc(peers));
        } else if (in && (key >> (shift + bits)) == prefix) {
          atomicAdd(hist + d, 1);
        }
      }
      cluster.sync();
      // bins from the top down: four per thread
      const int top = kBins - 1 - 4 * tid;
      int cnt[4], local[4], sum = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        cnt[e] = 0;
        local[e] = hist[top - e];
        for (int r = 0; r < C; ++r) cnt[e] += cluster.map_shared_rank(hist, r)[top - e];
        sum += cnt[e];
      }
      int total;
      const int upto = block_inclusive(sum, sm.sums, &total);
      int before = upto - sum;
      if (before < left && left <= upto) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (before < left && left <= before + cnt[e]) {
            sm.digit = top - e;
            sm.above = before;
          }
          before += cnt[e];
        }
      }
      __syncthreads();
      const int digit = sm.digit;
      left -= sm.above;
      int above = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) above += top - e > digit ? local[e] : 0;
      block_inclusive(above, sm.sums, &total);
      mine_above += total;
      if (pass == 2) mine_equal = hist[digit];
      prefix = (prefix << bits) | static_cast<uint32_t>(digit);
    }
    cut = prefix;
    ties = left;
  }
  // kept tokens before this slice
  const int forced = max(0, min(s1, lo) - s0) + max(0, s1 - max(s0, hi));
  if (tid == 0) {
    sm.counts[0] = mine_above + forced;
    sm.counts[1] = mine_equal;
  }
  cluster.sync();
  int eq = 0, pos = 0;
  for (int r = 0; r < rank; ++r) {
    const int* c = cluster.map_shared_rank(sm.counts, r);
    pos += c[0];
    eq += c[1];
  }
  pos += min(eq, ties);
  // the list, in ascending order: equal weights by their index
  for (int i0 = s0; i0 < s1; i0 += kThreads * kPer) {
    const int base = i0 + tid * kPer;
    float v[kPer];
    uint32_t same = 0, more = 0;
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      const int i = base + e;
      v[e] = i < s1 ? w[i] : 0.f;
    }
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      const int i = base + e;
      if (i >= s1) continue;
      const uint32_t key = order_key(v[e]);
      if (i < lo || i >= hi || key > cut) more |= 1u << e;
      else if (key == cut) same |= 1u << e;
    }
    int total;
    int r = eq + block_inclusive(__popc(same), sm.sums, &total) - __popc(same);
    eq += total;
    uint32_t take = more;
#pragma unroll
    for (int e = 0; e < kPer; ++e)
      if (same >> e & 1u) {
        if (r < ties) take |= 1u << e;
        ++r;
      }
    int at = pos + block_inclusive(__popc(take), sm.sums, &total) - __popc(take);
    pos += total;
#pragma unroll
    for (int e = 0; e < kPer; ++e)
      if (take >> e & 1u) {
        keep[at] = base + e;
        if (a.weights_out) wout[at] = v[e];
        ++at;
      }
  }
  cluster.sync();  // no CTA leaves while another may read its shared memory
}

__global__ void __launch_bounds__(kMoveThreads) evict_move(const __grid_constant__ EvictParams p) {
  const EvictArgs& a = p.a;
  __shared__ long long src_row[kMoveRows], dst_row[kMoveRows];  // in rows of the caches; -1: nothing to move
  const int blocks = (a.budget + p.move_tokens - 1) / p.move_tokens;
  const int b = blockIdx.x / blocks, i0 = (blockIdx.x % blocks) * p.move_tokens;
  asm volatile("griddepcontrol.wait;" ::: "memory");
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
  // CTAs per (sequence, kv-head): enough that the batch's clusters cover the SMs, as long as a
  // CTA keeps 2048 positions
  const long long units = static_cast<long long>(a.B) * a.Hkv;
  int C = 1;
  while (C < 8 && units * C < 148 && a.max_kv_len / (2 * C) >= 2048) C *= 2;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(units * C));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = C;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, evict_select, p);
  if (e != cudaSuccess) return e;
  // a move CTA's tokens: 8 pieces a thread, within its table of rows
  const int per_token = 2 * a.Hkv << a.row_shift;
  int tokens = kMoveThreads * kMovePieces / per_token;
  if (tokens * a.Hkv > kMoveRows) tokens = kMoveRows / a.Hkv;
  p.move_tokens = tokens < 1 ? 1 : tokens;
  cfg.gridDim = dim3(static_cast<unsigned>(a.B) * ((a.budget + p.move_tokens - 1) / p.move_tokens));
  cfg.blockDim = dim3(kMoveThreads);
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  return cudaLaunchKernelEx(&cfg, evict_move, p);
}

}  // namespace stem

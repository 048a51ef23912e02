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
// Measured on one B200: four BF16 caches of 32K tokens and 8 heads of 128 to 8K each, 62 us
// (selection 15, move 47 of 42 at the copy rate); 32 ragged FP8 caches of up to 64K, 247 us
// (72 and 176 of 164); with softmax-like totals 62 and 249, with all weights equal 61 and 236.
// The selection is barriers, waits on other CTAs and 40 instructions a key, and the move starts
// when the last of it has ended; two tables for the first digit's counts changed nothing.  One
// kernel that selects and moves, a head's rows at a time, was slower: 285 us for a copy that this
// one does in 187.
#include <string.h>

#include <cooperative_groups.h>

#include "stem_internal.cuh"

namespace stem {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr int kMaxCluster = 8;
constexpr int kMinKeys = 16;                  // keys a thread holds, and at most
constexpr int kMaxKeys = 128;
constexpr int kBatch = 8;                     // of which read at a time
static_assert(kMinKeys % kBatch == 0, "whole batches");
static_assert(kThreads * kMaxCluster * kMaxKeys >= STEM_MAX_KV_LEN, "a cluster holds the longest sequence");
constexpr int kMoveThreads = 256;
constexpr int kMovePieces = 8;                // 16-byte pieces a thread has in flight
constexpr int kMoveRows = 512;                // (token, head) rows of a move CTA at most
constexpr int kCoarse = 64;                   // groups of bins that are looked at first
constexpr int kFine = kBins / kCoarse;
static_assert(kBins == 8 * kThreads && kThreads == 4 * kCoarse && kFine == 32 && kWarps >= kMaxCluster, "see evict_select");

struct EvictParams {
  EvictArgs a;
  int kpt;             // keys of a select thread
  int move_tokens;     // tokens of a move CTA
};

// Weights in an order that unsigned comparison follows; NaN as -inf, -0 as +0.  They run
// from that of -inf, 0x007FFFFF, to that of inf, 0xFF800000, so that two are free:
constexpr uint32_t kNone = 0u;              // behind the last token
constexpr uint32_t kForced = 0xFFFFFFFFu;   // kept whatever its weight
__device__ __forceinline__ uint32_t order_key(float w) {
  const uint32_t u = __float_as_uint(fmaxf(w + 0.f, -INFINITY));  // -0 + 0 = 0; the maximum of NaN and x is x
  return u ^ (static_cast<uint32_t>(static_cast<int>(u) >> 31) | 0x80000000u);
}

// The weight of a key; NaN where several weights have it (zeros of both signs, -inf and NaN)
// or it stands for none: those are read again.
__device__ __forceinline__ float key_weight(uint32_t k) {
  const uint32_t bits = k ^ (~static_cast<uint32_t>(static_cast<int>(k) >> 31) | 0x80000000u);
  return k == kForced || k == 0x80000000u || k == 0x007FFFFFu ? NAN : __uint_as_float(bits);
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
  int hist[2][kBins];              // passes 0 and 2, pass 1
  int coarse[3][kCoarse];          // sums of 32 bins
  int total[kCoarse];              // the same over the cluster, from the top down
  int fine[kMaxCluster][kFine];    // the bins of one group, by CTA, from the top down
  int group, digit, left;          // of the pass, found by warp 0
  int more[kWarps], same[kWarps];  // keys above the cut-off (forced ones too) and equal to it, by warp
  int counts[2];                   // of the CTA
};

// The entry that holds number `left` when the 32 lanes' counts are passed in lane order; takes
// the counts before it from `left`.
__device__ __forceinline__ int find_lane(int count, int* left) {
  const int inc = warp_inclusive(count);
  const unsigned hit = __ballot_sync(0xffffffffu, inc - count < *left && *left <= inc);
  const int at = __ffs(hit) - 1;
  *left -= __shfl_sync(0xffffffffu, inc - count, at);
  return at;
}

// A CTA's slice is 256 * kpt positions (kpt by the sequence's length, so that the cluster's CTAs
// share it evenly), their keys in shared memory: warp w takes positions [w, w + 1) * 32 * kpt
// of it, key e of lane l being number 32 e + l, so that loads are coalesced, no key is another
// lane's, and ascending order is (warp, e, lane).
// ONE: a cluster of one CTA (at most 4096 positions), whose joining is a barrier of its own
// threads and reads of its own bins (1K tokens, with the move 9.6 us a call; 10.0 as a cluster).
template <bool ONE>
__global__ void __launch_bounds__(kThreads) evict_select(const __grid_constant__ EvictParams p) {
  const EvictArgs& a = p.a;
  __shared__ SelectSmem sm;
  extern __shared__ uint32_t keys[];
  cg::cluster_group cluster = cg::this_cluster();
  const int C = ONE ? 1 : static_cast<int>(cluster.num_blocks()), rank = ONE ? 0 : static_cast<int>(cluster.block_rank());
  auto join = [&]() {
    if (ONE) __syncthreads();
    else cluster.sync();
  };
  auto of_rank = [&](int* at, int r) { return ONE ? at : cluster.map_shared_rank(at, r); };
  const int unit = blockIdx.x / C, b = unit / a.Hkv, h = unit % a.Hkv;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const unsigned all = 0xffffffffu;
  for (int i = tid; i < kBins / 2; i += kThreads) reinterpret_cast<int4*>(sm.hist[0])[i] = make_int4(0, 0, 0, 0);
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
  const int kpt = kBatch * ((n + C * kThreads * kBatch - 1) / (C * kThreads * kBatch));  // p.kpt at most
  const int first = rank * (kThreads * kpt) + warp * (32 * kpt) + lane;           // position of key 0
  uint32_t* key = keys + warp * (32 * kpt) + lane;                                // key e at [32 * e]
  __syncthreads();  // the bins are zero
  // Into shared memory, the next batch on its way, and with them the first digit's counts.
  float v[kBatch];
  auto load = [&](int e0) {
#pragma unroll
    for (int e = 0; e < kBatch; ++e) {
      const int i = first + 32 * (e0 + e);
      v[e] = i >= lo && i < hi ? w[i] : 0.f;
    }
  };
  load(0);
  for (int e0 = 0; e0 < kpt; e0 += kBatch) {
    const int at = first - lane + 32 * e0;  // of the warp's batch
    uint32_t k[kBatch];
#pragma unroll
    for (int e = 0; e < kBatch; ++e) k[e] = order_key(v[e]);
    if (e0 + kBatch < kpt) load(e0 + kBatch);
    if (at < lo || at + 32 * kBatch > hi) {  // not all of it to be ranked
#pragma unroll
      for (int e = 0; e < kBatch; ++e) {
        const int i = first + 32 * (e0 + e);
        k[e] = i >= n ? kNone : (i < lo || i >= hi ? kForced : k[e]);
      }
    }
#pragma unroll
    for (int e = 0; e < kBatch; ++e) {
      key[32 * (e0 + e)] = k[e];
      if (k[e] + 1u > 1u) atomicAdd(sm.hist[0] + (k[e] >> 21), 1);  // neither kNone nor kForced
    }
  }
  // Runs f(key) over the thread's keys, a batch read ahead: the compiler may not move a
  // shared load over f's own stores and atomics.
  auto each = [&](auto f) {
    for (int e0 = 0; e0 < kpt; e0 += kBatch) {
      uint32_t k[kBatch];
#pragma unroll
      for (int e = 0; e < kBatch; ++e) k[e] = key[32 * (e0 + e)];
#pragma unroll
      for (int e = 0; e < kBatch; ++e) f(k[e]);
    }
  };

  // the cut-off key, digit by digit
  uint32_t cut = kForced - 1;  // no weight's key is this large
  int ties = 0;
  if (need > 0) {
    uint32_t prefix = 0;
    int left = need;
#pragma unroll
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0), bits = pass == 2 ? 10 : 11;
      int* hist = sm.hist[pass & 1];
      if (pass > 0)
        each([&](uint32_t k) {
          if (k >> (shift + bits) == prefix) atomicAdd(hist + ((k >> shift) & ((1u << bits) - 1)), 1);
        });
      __syncthreads();
      // Reading all of the other CTAs' bins costs more than the rest (64 KB through distributed
      // shared memory for each CTA: 10 us); so first the groups' sums, then the bins of one group.
      const int4 x = *reinterpret_cast<const int4*>(hist + 8 * tid), y = *reinterpret_cast<const int4*>(hist + 8 * tid + 4);
      int sum = ((x.x + x.y) + (x.z + x.w)) + ((y.x + y.y) + (y.z + y.w));
      sum += __shfl_xor_sync(all, sum, 1);
      sum += __shfl_xor_sync(all, sum, 2);
      if (tid % 4 == 0) sm.coarse[pass][tid / 4] = sum;
      join();
      if (pass == 1)  // every CTA has done with pass 0's bins
        for (int i = tid; i < kBins / 4; i += kThreads) reinterpret_cast<int4*>(sm.hist[0])[i] = make_int4(0, 0, 0, 0);
      int got = 0;
#pragma unroll
      for (int r = tid % 4; r < kMaxCluster; r += 4)
        if (r < C) got += of_rank(sm.coarse[pass], r)[kCoarse - 1 - tid / 4];
      got += __shfl_xor_sync(all, got, 1);
      got += __shfl_xor_sync(all, got, 2);
      if (tid % 4 == 0) sm.total[tid / 4] = got;
      __syncthreads();
      if (warp == 0) {  // lane l holds groups 2 l and 2 l + 1
        const int c0 = sm.total[2 * lane], c1 = sm.total[2 * lane + 1];
        const int pair = find_lane(c0 + c1, &left);
        const int upper = __shfl_sync(all, c0, pair);
        if (lane == 0) {
          sm.group = kCoarse - 1 - 2 * pair - (left > upper ? 1 : 0);
          sm.left = left > upper ? left - upper : left;
        }
      }
      __syncthreads();
      const int group = sm.group;
      if (warp < C) sm.fine[warp][lane] = of_rank(hist, warp)[kFine * group + kFine - 1 - lane];
      __syncthreads();
      if (warp == 0) {
        int f = 0;
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r) f += r < C ? sm.fine[r][lane] : 0;
        left = sm.left;
        const int digit = kFine * group + kFine - 1 - find_lane(f, &left);
        if (lane == 0) {
          sm.digit = digit;
          sm.left = left;
        }
      }
      __syncthreads();
      const int digit = sm.digit;
      left = sm.left;
      prefix = (prefix << bits) | static_cast<uint32_t>(digit);
    }
    cut = prefix;
    ties = left;
  }
  // which keys stay, the equal ones still open; counts by warp, CTA and rank
  int more = 0, same = 0;
  each([&](uint32_t k) {
    more += k > cut ? 1 : 0;
    same += k == cut ? 1 : 0;
  });
  more = __reduce_add_sync(all, more);
  same = __reduce_add_sync(all, same);
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
  if (!ONE) {
    join();
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r)
      if (r < rank) {
        const int* c = of_rank(sm.counts, r);
        pos += c[0];
        eq += c[1];
      }
    join();  // the last look into another CTA's shared memory: each may leave from here on
  }
  // the list, in ascending order; of the equal ones the first `ties`
  const unsigned below = (1u << lane) - 1u;
  pos += min(eq, ties);
  for (int e0 = 0; e0 < kpt; e0 += kBatch) {
    int at[kBatch];
    float v[kBatch];
#pragma unroll
    for (int e = 0; e < kBatch; ++e) {
      const uint32_t k = key[32 * (e0 + e)];
      v[e] = key_weight(k);
      bool take = k > cut;
      if (same > 0) {  // the same for the warp
        const unsigned se = __ballot_sync(all, k == cut);
        take = take || (k == cut && eq + __popc(se & below) < ties);
        eq += __popc(se);
      }
      const unsigned te = __ballot_sync(all, take);
      at[e] = take ? pos + __popc(te & below) : -1;
      pos += __popc(te);
    }
#pragma unroll
    for (int e = 0; e < kBatch; ++e)
      if (a.weights_out && at[e] >= 0 && !(v[e] == v[e])) v[e] = w[first + 32 * (e0 + e)];
#pragma unroll
    for (int e = 0; e < kBatch; ++e)
      if (at[e] >= 0) {
        keep[at[e]] = first + 32 * (e0 + e);
        if (a.weights_out) wout[at[e]] = v[e];
      }
  }
}

__global__ void __launch_bounds__(kMoveThreads) evict_move(const __grid_constant__ EvictParams p) {
  const EvictArgs& a = p.a;
  __shared__ long long src_row[kMoveRows], dst_row[kMoveRows];  // in rows of the caches; -1: nothing to move
  const int blocks = (a.budget + p.move_tokens - 1) / p.move_tokens;
  const int b = blockIdx.x / blocks, i0 = (blockIdx.x % blocks) * p.move_tokens;
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

// Neither kernel triggers its successor early: the successor's waiting CTAs would take the
// places of its own next ones (evict_move on 32 FP8 caches: 176 us, 200 to 250 us with it).
cudaError_t launch_evict(const EvictArgs& a, cudaStream_t st) {
  EvictParams p;
  p.a = a;
  // A cluster's shared memory holds a sequence: 16 keys a thread and as many CTAs as that
  // needs (long sequences of a ragged batch are spread out), then more keys a thread.
  const unsigned units = static_cast<unsigned>(a.B) * a.Hkv;
  const int chunks = (a.max_kv_len + kThreads * kMinKeys - 1) / (kThreads * kMinKeys);
  int C = 1;
  while (C < kMaxCluster && C < chunks) C *= 2;
  p.kpt = kMinKeys * ((chunks + C - 1) / C);
  const size_t smem = static_cast<size_t>(p.kpt) * kThreads * 4;
  cudaError_t e = C > 1 ? set_smem_once<evict_select<false>>(kMaxKeys * kThreads * 4) : cudaSuccess;
  if (e == cudaSuccess)
    e = C > 1 ? launch_dependent(evict_select<false>, units * C, kThreads, smem, C, st, p)
              : launch_dependent(evict_select<true>, units, kThreads, smem, 1, st, p);
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

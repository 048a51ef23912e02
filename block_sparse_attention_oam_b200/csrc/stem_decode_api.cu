// Entry points of the decoding operators declared in include/stem.h: argument checks,
// workspace layout, and the launches.
#include <float.h>

#include <cmath>

#include "stem_internal.cuh"

namespace stem {
namespace {

bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

// [a, a + na) and [b, b + nb) share a byte
bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}

stem_status_t check_shape(int num_seqs, int Hkv, int d, stem_dtype_t dtype, int max_kv_len) {
  if (num_seqs < 1 || num_seqs > STEM_MAX_DECODE_SEQS)
    return set_last_error(STEM_ERR_INVALID, "num_seqs %d outside [1, %d]", num_seqs, STEM_MAX_DECODE_SEQS);
  if (Hkv < 1 || Hkv > 256) return set_last_error(STEM_ERR_INVALID, "num_kv_heads %d outside [1, 256]", Hkv);
  if (d != 64 && d != 128) return set_last_error(STEM_ERR_UNSUPPORTED, "head_dim %d (supported: 64, 128)", d);
  if (dtype != STEM_DT_BF16 && dtype != STEM_DT_FP8_E4M3)
    return set_last_error(STEM_ERR_INVALID, "unknown dtype %d", static_cast<int>(dtype));
  if (dtype == STEM_DT_FP8_E4M3 && d != 128) return set_last_error(STEM_ERR_UNSUPPORTED, "FP8 needs head_dim 128");
  if (max_kv_len < 1 || max_kv_len > STEM_MAX_KV_LEN)
    return set_last_error(STEM_ERR_INVALID, "max_kv_len %d outside [1, %d]", max_kv_len, STEM_MAX_KV_LEN);
  return STEM_OK;
}

stem_status_t check_cache(const stem_paged_kv_t* c, const char* what, int max_len) {
  if (c == nullptr) return set_last_error(STEM_ERR_INVALID, "%s is NULL", what);
  if (c->k_cache == nullptr || c->v_cache == nullptr || c->block_table == nullptr)
    return set_last_error(STEM_ERR_INVALID, "%s: paged cache pointers must not be NULL", what);
  if (!aligned(c->k_cache, 16) || !aligned(c->v_cache, 16))
    return set_last_error(STEM_ERR_INVALID, "%s: paged caches must be 16-byte aligned", what);
  if (c->page_size != STEM_PAGE_SIZE)
    return set_last_error(STEM_ERR_UNSUPPORTED, "%s: page_size %d (supported: %d)", what, c->page_size, STEM_PAGE_SIZE);
  if (c->num_slots < 1 || c->num_slots > (1 << 24))
    return set_last_error(STEM_ERR_INVALID, "%s: num_slots %d outside [1, 2^24]", what, c->num_slots);
  if ((max_len + STEM_PAGE_SIZE - 1) / STEM_PAGE_SIZE > c->max_pages_per_seq)
    return set_last_error(STEM_ERR_INVALID, "%s: %d tokens need more than max_pages_per_seq=%d pages", what, max_len,
                          c->max_pages_per_seq);
  return STEM_OK;
}

// sigma q_scale k_scale log2(e), what a product of codes (or BF16 values) is multiplied by
double score_scale(const stem_decode_t* de) {
  const double sigma = de->softmax_scale > 0.f ? de->softmax_scale : 1.0 / std::sqrt(static_cast<double>(de->head_dim));
  const double codes = de->dtype == STEM_DT_FP8_E4M3 ? static_cast<double>(de->q_scale) * de->k_scale : 1.0;
  return sigma * codes * 1.4426950408889634;
}

stem_status_t check_decode(const stem_decode_t* de) {
  if (de == nullptr) return set_last_error(STEM_ERR_INVALID, "decode problem is NULL");
  stem_status_t s = check_shape(de->num_seqs, de->num_kv_heads, de->head_dim, de->dtype, de->max_kv_len);
  if (s != STEM_OK) return s;
  if (de->num_q_heads < 1 || de->num_q_heads % de->num_kv_heads != 0)
    return set_last_error(STEM_ERR_INVALID, "num_q_heads %d must be a positive multiple of num_kv_heads %d",
                          de->num_q_heads, de->num_kv_heads);
  if (de->num_q_heads > 256) return set_last_error(STEM_ERR_UNSUPPORTED, "num_q_heads %d > 256", de->num_q_heads);
  if (de->q_len < 1 || de->q_len > STEM_MAX_Q_LEN)
    return set_last_error(STEM_ERR_INVALID, "q_len %d outside [1, %d]", de->q_len, STEM_MAX_Q_LEN);
  if (de->dtype == STEM_DT_FP8_E4M3)
    if (!(de->q_scale > 0.f) || !(de->k_scale > 0.f) || !(de->v_scale > 0.f) || !std::isfinite(de->q_scale) ||
        !std::isfinite(de->k_scale) || !std::isfinite(de->v_scale))
      return set_last_error(STEM_ERR_INVALID, "FP8 scales must be finite and positive");
  if (!std::isfinite(de->softmax_scale)) return set_last_error(STEM_ERR_INVALID, "softmax_scale is not finite");
  if (score_scale(de) > FLT_MAX)
    return set_last_error(STEM_ERR_INVALID, "softmax_scale x q_scale x k_scale is beyond float32");
  if (de->prefix_len < 0 || de->prefix_len > STEM_MAX_KV_LEN)
    return set_last_error(STEM_ERR_INVALID, "prefix_len %d outside [0, %d]", de->prefix_len, STEM_MAX_KV_LEN);
  if (de->collect_weights != 0 && de->collect_weights != 1)
    return set_last_error(STEM_ERR_INVALID, "collect_weights %d must be 0 or 1", de->collect_weights);
  // the line of tiles is counted in 32 bits
  const long long R = static_cast<long long>(de->q_len) * (de->num_q_heads / de->num_kv_heads);
  const long long pages = (de->max_kv_len + STEM_PAGE_SIZE - 1) / STEM_PAGE_SIZE;
  const long long ppages = (de->prefix_len + STEM_PAGE_SIZE - 1) / STEM_PAGE_SIZE;
  const long long own = de->num_kv_heads * de->num_seqs * ((R + kDecodeRows - 1) / kDecodeRows) * (pages + kDecodeUnitCost);
  const long long pre = de->num_kv_heads * ((de->num_seqs * R + kDecodeRows - 1) / kDecodeRows) * (ppages + kDecodeUnitCost);
  if (own + pre > (1ll << 30))
    return set_last_error(STEM_ERR_UNSUPPORTED, "batch x heads x pages of %lld tiles is too large", own + pre);
  return STEM_OK;
}

stem_status_t check_evict(const stem_evict_t* ev) {
  if (ev == nullptr) return set_last_error(STEM_ERR_INVALID, "evict problem is NULL");
  stem_status_t s = check_shape(ev->num_seqs, ev->num_kv_heads, ev->head_dim, ev->dtype, ev->max_kv_len);
  if (s != STEM_OK) return s;
  if (ev->budget < 1 || ev->budget > STEM_MAX_KV_LEN)
    return set_last_error(STEM_ERR_INVALID, "budget %d outside [1, %d]", ev->budget, STEM_MAX_KV_LEN);
  if (ev->sink < 0 || ev->recent < 0 || ev->sink > ev->budget || ev->recent > ev->budget - ev->sink)
    return set_last_error(STEM_ERR_INVALID, "sink %d and recent %d must be >= 0 and fit the budget %d", ev->sink,
                          ev->recent, ev->budget);
  return STEM_OK;
}

DecodeWs layout(const stem_decode_t* de) {
  DecodeWs w{};
  const size_t B = de->num_seqs, Hkv = de->num_kv_heads, d = de->head_dim;
  const size_t R = static_cast<size_t>(de->q_len) * (de->num_q_heads / de->num_kv_heads);
  const size_t rt = (R + kDecodeRows - 1) / kDecodeRows;
  const PrefixPlan pre =
      plan_prefix(de->num_seqs, de->q_len, de->num_kv_heads, de->num_q_heads / de->num_kv_heads, de->prefix_len);
  const size_t prt = de->prefix_len > 0 && pre.gangs == 0 ? (B * R + kDecodeRows - 1) / kDecodeRows : 0;
  const size_t slots = kDecodeCtas + Hkv * (prt + B * rt);
  const size_t most = prt > 0 ? B * R : R;
  w.part_rows = static_cast<int>(most < kDecodeRows ? most : kDecodeRows);
  size_t o = 256;
  w.part_ml = o;
  o = align256(o + slots * kDecodeRows * sizeof(float2));
  w.part_o = o;
  o = align256(o + slots * w.part_rows * d * 4);
  w.prefix_ml = o;
  o = align256(o + static_cast<size_t>(pre.slots) * 256 * sizeof(float2));
  w.prefix_o = o;
  o = align256(o + static_cast<size_t>(pre.slots) * 256 * d * 4);
  w.scores = o;
  w.score_stride = static_cast<long long>(de->max_kv_len + STEM_PAGE_SIZE - 1) / STEM_PAGE_SIZE * STEM_PAGE_SIZE;
  if (de->collect_weights) o = align256(o + B * Hkv * R * static_cast<size_t>(w.score_stride) * 4);
  w.total = o;
  return w;
}

stem_status_t check_ws(const void* ws, size_t ws_bytes, size_t need) {
  if (ws == nullptr) return set_last_error(STEM_ERR_WORKSPACE, "workspace is NULL");
  if (!aligned(ws, 256)) return set_last_error(STEM_ERR_WORKSPACE, "workspace must be 256-byte aligned");
  if (ws_bytes < need)
    return set_last_error(STEM_ERR_WORKSPACE, "workspace of %zu bytes is smaller than the %zu needed", ws_bytes, need);
  return STEM_OK;
}

template <typename T>
T* at(void* ws, size_t off) {
  return reinterpret_cast<T*>(static_cast<unsigned char*>(ws) + off);
}

}  // namespace
}  // namespace stem

using namespace stem;

extern "C" {

size_t stem_decode_workspace_size(const stem_decode_t* dec) {
  return check_decode(dec) == STEM_OK ? layout(dec).total : 0;
}

stem_status_t stem_decode(const stem_decode_t* dec, const void* q, const stem_paged_kv_t* cache,
                          const int32_t* kv_lens, const int32_t* prefix_table, const float* weights_in,
                          float* weights_out, int64_t weights_stride, void* out, float* lse, void* ws, size_t ws_bytes,
                          void* stream) {
  stem_status_t s = check_decode(dec);
  if (s == STEM_OK) s = check_cache(cache, "cache", dec->max_kv_len);
  if (s != STEM_OK) return s;
  if (q == nullptr || !aligned(q, 16))
    return set_last_error(STEM_ERR_INVALID, "q must be a non-NULL 16-byte aligned pointer");
  if (out == nullptr || !aligned(out, 16))
    return set_last_error(STEM_ERR_INVALID, "out must be a non-NULL 16-byte aligned pointer");
  if (kv_lens == nullptr) return set_last_error(STEM_ERR_INVALID, "kv_lens is NULL");
  if ((prefix_table != nullptr) != (dec->prefix_len > 0))
    return set_last_error(STEM_ERR_INVALID, "prefix_table and prefix_len %d must be given together", dec->prefix_len);
  if (dec->collect_weights) {
    if (weights_out == nullptr) return set_last_error(STEM_ERR_INVALID, "collect_weights without weights_out");
    if (weights_stride < dec->max_kv_len)
      return set_last_error(STEM_ERR_INVALID, "weights_stride %lld is smaller than max_kv_len %d",
                            static_cast<long long>(weights_stride), dec->max_kv_len);
    const size_t bytes = static_cast<size_t>(dec->num_seqs) * dec->num_kv_heads * weights_stride * 4;
    if (weights_in != nullptr && weights_in != weights_out && overlap(weights_in, bytes, weights_out, bytes))
      return set_last_error(STEM_ERR_INVALID, "weights_in and weights_out overlap without being the same");
  } else if (weights_in != nullptr || weights_out != nullptr) {
    return set_last_error(STEM_ERR_INVALID, "weights given without collect_weights");
  }
  const DecodeWs w = layout(dec);
  if ((s = check_ws(ws, ws_bytes, w.total)) != STEM_OK) return s;
  const bool fp8 = dec->dtype == STEM_DT_FP8_E4M3;
  DecodeArgs a{};
  a.q = q;
  a.kv_lens = kv_lens;
  a.table = cache->block_table;
  a.prefix_table = prefix_table;
  a.k_cache = cache->k_cache;
  a.v_cache = cache->v_cache;
  a.max_pages = cache->max_pages_per_seq;
  a.num_slots = cache->num_slots;
  a.B = dec->num_seqs;
  a.n = dec->q_len;
  a.Hq = dec->num_q_heads;
  a.Hkv = dec->num_kv_heads;
  a.G = a.Hq / a.Hkv;
  a.d = dec->head_dim;
  a.max_kv_len = dec->max_kv_len;
  a.prefix_len = dec->prefix_len;
  a.scale_log2 = static_cast<float>(score_scale(dec));
  a.v_scale = fp8 ? dec->v_scale : 1.0f;
  a.weights_in = weights_in;
  a.weights_out = weights_out;
  a.weights_stride = weights_stride;
  a.out = out;
  a.lse = lse;
  a.status = at<uint32_t>(ws, w.status);
  a.part_ml = at<float2>(ws, w.part_ml);
  a.part_o = at<float>(ws, w.part_o);
  a.prefix_ml = at<float2>(ws, w.prefix_ml);
  a.prefix_o = at<float>(ws, w.prefix_o);
  a.scores = dec->collect_weights ? at<float>(ws, w.scores) : nullptr;
  a.score_stride = w.score_stride;
  a.part_rows = w.part_rows;
  const cudaError_t e = launch_decode(a, fp8, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return set_last_error(STEM_ERR_CUDA, "decode: %s", cudaGetErrorString(e));
  return STEM_OK;
}

size_t stem_evict_workspace_size(const stem_evict_t* ev) { return check_evict(ev) == STEM_OK ? 256 : 0; }

stem_status_t stem_evict(const stem_evict_t* ev, const stem_paged_kv_t* src, const int32_t* kv_lens,
                         const float* weights, int64_t weights_stride, const stem_paged_kv_t* dst,
                         int32_t* kv_lens_out, float* weights_out, int64_t weights_out_stride, int32_t* keep, void* ws,
                         size_t ws_bytes, void* stream) {
  stem_status_t s = check_evict(ev);
  if (s == STEM_OK) s = check_cache(src, "src", ev->max_kv_len);
  if (s == STEM_OK) s = check_cache(dst, "dst", ev->budget < ev->max_kv_len ? ev->budget : ev->max_kv_len);
  if (s != STEM_OK) return s;
  if (kv_lens == nullptr || weights == nullptr || kv_lens_out == nullptr || keep == nullptr)
    return set_last_error(STEM_ERR_INVALID, "kv_lens, weights, kv_lens_out and keep must not be NULL");
  if (weights_stride < ev->max_kv_len)
    return set_last_error(STEM_ERR_INVALID, "weights_stride %lld is smaller than max_kv_len %d",
                          static_cast<long long>(weights_stride), ev->max_kv_len);
  const size_t units = static_cast<size_t>(ev->num_seqs) * ev->num_kv_heads;
  const size_t lens = static_cast<size_t>(ev->num_seqs) * 4;
  if (overlap(kv_lens, lens, kv_lens_out, lens))
    return set_last_error(STEM_ERR_INVALID, "kv_lens_out must not overlap kv_lens");
  if (weights_out != nullptr) {
    if (weights_out_stride < ev->budget)
      return set_last_error(STEM_ERR_INVALID, "weights_out_stride %lld is smaller than the budget %d",
                            static_cast<long long>(weights_out_stride), ev->budget);
    if (overlap(weights, units * weights_stride * 4, weights_out, units * weights_out_stride * 4))
      return set_last_error(STEM_ERR_INVALID, "weights_out must not overlap weights");
  }
  if ((s = check_ws(ws, ws_bytes, 256)) != STEM_OK) return s;
  EvictArgs a{};
  a.kv_lens = kv_lens;
  a.weights = weights;
  a.weights_stride = weights_stride;
  a.src_k = src->k_cache;
  a.src_v = src->v_cache;
  a.src_table = src->block_table;
  a.src_max_pages = src->max_pages_per_seq;
  a.src_slots = src->num_slots;
  a.dst_k = const_cast<void*>(dst->k_cache);
  a.dst_v = const_cast<void*>(dst->v_cache);
  a.dst_table = dst->block_table;
  a.dst_max_pages = dst->max_pages_per_seq;
  a.dst_slots = dst->num_slots;
  a.B = ev->num_seqs;
  a.Hkv = ev->num_kv_heads;
  const int row_bytes = ev->head_dim * (ev->dtype == STEM_DT_FP8_E4M3 ? 1 : 2);
  a.row_shift = row_bytes == 256 ? 4 : 3;  // 128 bytes otherwise: d 64 in BF16, d 128 in FP8
  a.max_kv_len = ev->max_kv_len;
  a.budget = ev->budget;
  a.sink = ev->sink;
  a.recent = ev->recent;
  a.kv_lens_out = kv_lens_out;
  a.weights_out = weights_out;
  a.weights_out_stride = weights_out_stride;
  a.keep = keep;
  a.status = at<uint32_t>(ws, 0);
  const cudaError_t e = launch_evict(a, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return set_last_error(STEM_ERR_CUDA, "evict: %s", cudaGetErrorString(e));
  return STEM_OK;
}

}  // extern "C"

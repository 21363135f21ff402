// C ABI of q3_block.h's attention sublayer and log probabilities: host-side
// validation, then the launches on the caller's stream.  Nothing here allocates
// device memory or synchronises.
#include <hip/hip_runtime.h>

#include <cmath>

#include "../../include/q3_block.h"
#include "q3_check.h"
#include "q3_internal.h"

using namespace q3::check;

namespace {

constexpr int32_t kMaxHeads = 1024;
constexpr int64_t kMaxRows = int64_t(1) << 24;   // attention and scored rows, exclusive
constexpr int64_t kMaxVocabulary = int64_t(1) << 19;
constexpr float kLog2e = 1.4426950408889634f;

bool bad_head_dim(int64_t d) { return d < 16 || d > 256 || d % 16; }
// The kernels take 1 / t, and 1 / t as a power of two.
bool bad_temperature(float t) { return !(t > 0.f) || !std::isfinite(t) || !std::isfinite(1.f / t * kLog2e); }
// The kernels take |scale| as a power of two.
bool bad_scale(float s) { return !std::isnormal(s) || !std::isfinite(s * kLog2e); }
bool bad_heads(int64_t h) { return h < 1 || h > kMaxHeads; }

q3_status check_cache(const q3_paged_cache* c) {
  if (!c) return Q3_ERR_INVALID_ARG;
  if (bad_heads(c->heads) || bad_head_dim(c->head_dim) || c->page_size < 1 || c->page_size > 1024 ||
      (c->page_size & (c->page_size - 1)) || c->pages < 1 || c->pages > kMaxM)
    return Q3_ERR_UNSUPPORTED_SHAPE;
  if (!c->k || !c->v) return Q3_ERR_INVALID_ARG;
  if (c->page_stride < int64_t(c->heads) * c->page_size * c->head_dim) return Q3_ERR_INVALID_ARG;
  if (c->page_stride % 8 || !aligned(c->k, 16) || !aligned(c->v, 16)) return Q3_ERR_MISALIGNED;
  if (c->page_stride > (int64_t(1) << 60) / c->pages) return Q3_ERR_UNSUPPORTED_SHAPE;
  return Q3_OK;
}

q3_status check_batch(const q3_paged_batch* b) {
  if (!b) return Q3_ERR_INVALID_ARG;
  if (b->sequences < 1 || b->sequences > 65535 || b->table_pages < 1) return Q3_ERR_UNSUPPORTED_SHAPE;
  if (!b->q_start || !b->kv_len || !b->page_table || b->ld_table < b->table_pages) return Q3_ERR_INVALID_ARG;
  if (!aligned(b->q_start, 4) || !aligned(b->kv_len, 4) || !aligned(b->page_table, 4)) return Q3_ERR_MISALIGNED;
  return Q3_OK;
}

q3::CacheView view_of(const q3_paged_cache* c) {
  q3::CacheView v{};
  v.k = static_cast<uint16_t*>(c->k);
  v.v = static_cast<uint16_t*>(c->v);
  v.pages = c->pages;
  v.page_stride = c->page_stride;
  while ((1 << v.shift) < c->page_size) ++v.shift;
  v.heads = c->heads;
  v.d = c->head_dim;
  return v;
}

q3::BatchView view_of(const q3_paged_batch* b) {
  q3::BatchView v{};
  v.q_start = b->q_start;
  v.kv_len = b->kv_len;
  v.table = b->page_table;
  v.ld_table = b->ld_table;
  v.table_pages = b->table_pages < kMaxM ? b->table_pages : kMaxM;   // no position is past 2^31
  v.sequences = static_cast<int32_t>(b->sequences);
  return v;
}

// The heads' layout and the fp32 rows they stand in.
q3_status check_heads(const q3_head_norms* h, const float* qkv, int64_t ld, int64_t m) {
  if (!h) return Q3_ERR_INVALID_ARG;
  if (bad_heads(h->heads_q) || bad_heads(h->heads_kv) || bad_head_dim(h->head_dim) || m < 1 || m >= kMaxM)
    return Q3_ERR_UNSUPPORTED_SHAPE;
  if (h->rotated < 0 || h->rotated > h->head_dim || h->rotated % 2) return Q3_ERR_INVALID_ARG;
  if (!qkv || !(h->eps >= 0.f) || (h->rotated && !h->inv_freq)) return Q3_ERR_INVALID_ARG;
  if (ld < int64_t(h->heads_q + 2 * h->heads_kv) * h->head_dim) return Q3_ERR_INVALID_ARG;
  if (ld % 4 || !aligned(qkv, 16) || !aligned(h->q_weight, 4) || !aligned(h->k_weight, 4) || !aligned(h->inv_freq, 4))
    return Q3_ERR_MISALIGNED;
  return Q3_OK;
}

// Rows of n elements at p, `size` bytes each, in 16-byte pieces.
q3_status check_rows(const void* p, int64_t ld, int64_t n, int size) {
  if (!p || ld < n) return Q3_ERR_INVALID_ARG;
  if (ld % (16 / size) || !aligned(p, 16)) return Q3_ERR_MISALIGNED;
  return Q3_OK;
}

// Rows and heads of one attention launch: its blocks (tiles of rows and, for
// each sequence, a part of one) have to be fewer than 2^24.
bool bad_attention(int64_t m, int64_t sequences, int64_t heads_q, int64_t heads) {
  return m < 1 || m >= kMaxRows || sequences < 1 || sequences > 65535 || bad_heads(heads_q) || bad_heads(heads) ||
         heads_q % heads || m * heads_q >= kMaxM / 2 || sequences * heads >= kMaxM / 256;
}

}  // namespace

extern "C" {

Q3_API q3_status q3_qk_norm_rope(const q3_head_norms* heads, const float* qkv, int64_t ld, const int32_t* positions,
                                 uint16_t* q, int64_t ldq, uint16_t* k, int64_t ldk, uint16_t* v, int64_t ldv,
                                 const q3_paged_cache* cache, const q3_paged_batch* batch, int64_t m, void* stream) {
  q3_status st = check_heads(heads, qkv, ld, m);
  if (st != Q3_OK) return st;
  const q3_head_norms& h = *heads;
  const int64_t nq = int64_t(h.heads_q) * h.head_dim, nk = int64_t(h.heads_kv) * h.head_dim;
  if ((st = check_rows(q, ldq, nq, 2)) != Q3_OK) return st;
  if (cache || batch) {
    if (k || v) return Q3_ERR_INVALID_ARG;
    if ((st = check_cache(cache)) != Q3_OK) return st;
    if ((st = check_batch(batch)) != Q3_OK) return st;
    if (cache->heads != h.heads_kv || cache->head_dim != h.head_dim) return Q3_ERR_UNSUPPORTED_SHAPE;
  } else {
    if ((st = check_rows(k, ldk, nk, 2)) != Q3_OK) return st;
    if ((st = check_rows(v, ldv, nk, 2)) != Q3_OK) return st;
    if (!positions && h.rotated) return Q3_ERR_INVALID_ARG;
  }
  if (!aligned(positions, 4)) return Q3_ERR_MISALIGNED;
  if ((st = check_device()) != Q3_OK) return st;
  q3::RopeArgs a{};
  a.qkv = qkv;
  a.ld = ld;
  a.hq = h.heads_q;
  a.hk = h.heads_kv;
  a.d = h.head_dim;
  a.rot = h.rotated;
  a.interleaved = h.interleaved;
  a.eps = h.eps;
  a.wq = h.q_weight;
  a.wk = h.k_weight;
  a.freq = h.inv_freq;
  a.positions = positions;
  a.q = q;
  a.ldq = ldq;
  a.k = k;
  a.ldk = ldk;
  a.v = v;
  a.ldv = ldv;
  if (cache) {
    a.cache = view_of(cache);
    a.batch = view_of(batch);
  }
  a.m = m;
  return from_hip(q3::launch_qk_norm_rope(a, static_cast<hipStream_t>(stream)));
}

Q3_API int64_t q3_qk_norm_rope_backward_workspace_bytes(int64_t m, int32_t head_dim) {
  if (m < 1 || m >= kMaxM || bad_head_dim(head_dim)) return 0;
  return align256(q3::rope_back_rows(m) * 2 * head_dim * 4);
}

Q3_API q3_status q3_qk_norm_rope_backward(const q3_head_norms* heads, const float* qkv, int64_t ld,
                                          const int32_t* positions, int64_t m, const q3_qkv_grads* grads,
                                          void* workspace, int64_t workspace_bytes, void* stream) {
  q3_status st = check_heads(heads, qkv, ld, m);
  if (st != Q3_OK) return st;
  const q3_head_norms& h = *heads;
  if (!grads) return Q3_ERR_INVALID_ARG;
  const q3_qkv_grads& g = *grads;
  if (g.d_type != Q3_F32 && g.d_type != Q3_BF16) return Q3_ERR_INVALID_ARG;
  if ((!h.q_weight && g.dq_weight) || (!h.k_weight && g.dk_weight) || (!positions && h.rotated))
    return Q3_ERR_INVALID_ARG;
  const int64_t nq = int64_t(h.heads_q) * h.head_dim, nk = int64_t(h.heads_kv) * h.head_dim;
  const int e = g.d_type == Q3_BF16 ? 2 : 4;
  if (g.dq && (st = check_rows(g.dq, g.ld_dq, nq, e)) != Q3_OK) return st;
  if (g.dk && (st = check_rows(g.dk, g.ld_dk, nk, e)) != Q3_OK) return st;
  if (g.dv && (st = check_rows(g.dv, g.ld_dv, nk, e)) != Q3_OK) return st;
  if ((st = check_rows(g.dqkv, g.ld_dqkv, nq + 2 * nk, 2)) != Q3_OK) return st;
  if (!aligned(positions, 4) || !aligned(g.dq_weight, 4) || !aligned(g.dk_weight, 4)) return Q3_ERR_MISALIGNED;
  if ((st = check_workspace(workspace, workspace_bytes, q3_qk_norm_rope_backward_workspace_bytes(m, h.head_dim))) !=
      Q3_OK)
    return st;
  if ((st = check_device()) != Q3_OK) return st;
  q3::RopeBackArgs a{};
  a.qkv = qkv;
  a.ld = ld;
  a.hq = h.heads_q;
  a.hk = h.heads_kv;
  a.d = h.head_dim;
  a.rot = h.rotated;
  a.interleaved = h.interleaved;
  a.eps = h.eps;
  a.wq = h.q_weight;
  a.wk = h.k_weight;
  a.freq = h.inv_freq;
  a.positions = positions;
  a.dq = g.dq;
  a.ld_dq = g.ld_dq;
  a.dk = g.dk;
  a.ld_dk = g.ld_dk;
  a.dv = g.dv;
  a.ld_dv = g.ld_dv;
  a.dqkv = g.dqkv;
  a.ld_out = g.ld_dqkv;
  a.dwq = g.dq_weight;
  a.dwk = g.dk_weight;
  a.part = g.dq_weight || g.dk_weight ? static_cast<float*>(workspace) : nullptr;
  a.m = m;
  return from_hip(q3::launch_qk_norm_rope_back(a, g.d_type, static_cast<hipStream_t>(stream)));
}

Q3_API int64_t q3_paged_attention_workspace_bytes(int64_t m, int64_t sequences, int32_t heads_q, int32_t heads,
                                                  int32_t head_dim) {
  if (bad_attention(m, sequences, heads_q, heads) || bad_head_dim(head_dim)) return 0;
  return align256(q3::attend_workspace_bytes(m, sequences, heads_q, heads, head_dim));
}

Q3_API q3_status q3_paged_attention(const uint16_t* q, int64_t ldq, int32_t heads_q, const q3_paged_cache* cache,
                                    const q3_paged_batch* batch, float scale, int32_t window, uint16_t* out,
                                    int64_t ldo, float* lse, int64_t m, void* workspace, int64_t workspace_bytes,
                                    void* stream) {
  q3_status st = check_cache(cache);
  if (st != Q3_OK) return st;
  if ((st = check_batch(batch)) != Q3_OK) return st;
  if (bad_attention(m, batch->sequences, heads_q, cache->heads)) return Q3_ERR_UNSUPPORTED_SHAPE;
  if (window < 0 || bad_scale(scale)) return Q3_ERR_INVALID_ARG;
  const int64_t n = int64_t(heads_q) * cache->head_dim;
  if ((st = check_rows(q, ldq, n, 2)) != Q3_OK) return st;
  if ((st = check_rows(out, ldo, n, 2)) != Q3_OK) return st;
  if (!aligned(lse, 4)) return Q3_ERR_MISALIGNED;
  const int64_t need =
      q3_paged_attention_workspace_bytes(m, batch->sequences, heads_q, cache->heads, cache->head_dim);
  if ((st = check_workspace(workspace, workspace_bytes, need)) != Q3_OK) return st;
  if ((st = check_device()) != Q3_OK) return st;
  q3::AttendArgs a{};
  a.q = q;
  a.ldq = ldq;
  a.out = out;
  a.ldo = ldo;
  a.lse = lse;
  a.hq = heads_q;
  a.scale = scale;
  a.window = window;
  a.cache = view_of(cache);
  a.batch = view_of(batch);
  a.m = m;
  return from_hip(q3::launch_attend(a, workspace, static_cast<hipStream_t>(stream)));
}

Q3_API int64_t q3_logprobs_workspace_bytes(int64_t m, int64_t n, int32_t top) {
  if (m < 1 || m >= kMaxRows || n < 1 || n > kMaxVocabulary || top < 0 || top > q3::kMaxTop) return 0;
  return align256(q3::logprobs_workspace_bytes(m, n, top));
}

Q3_API q3_status q3_logprobs(const float* logits, int64_t m, int64_t n, int64_t ld, const int32_t* targets,
                             float temperature, int32_t top, float* logprobs, float* entropy, int32_t* top_ids,
                             float* top_logprobs, float* stats, void* workspace, int64_t workspace_bytes,
                             void* stream) {
  if (!logits || !targets || !logprobs) return Q3_ERR_INVALID_ARG;
  if (m < 1 || m >= kMaxRows || n < 1 || n > kMaxVocabulary || top < 0 || top > q3::kMaxTop)
    return Q3_ERR_UNSUPPORTED_SHAPE;
  if (ld < n || bad_temperature(temperature) || (top > 0) != (top_ids != nullptr) ||
      (top > 0) != (top_logprobs != nullptr))
    return Q3_ERR_INVALID_ARG;
  if (!aligned(logits, 4) || !aligned(targets, 4) || !aligned(logprobs, 4) || !aligned(entropy, 4) ||
      !aligned(top_ids, 4) || !aligned(top_logprobs, 4) || !aligned(stats, 16))
    return Q3_ERR_MISALIGNED;
  q3_status st = check_workspace(workspace, workspace_bytes, q3_logprobs_workspace_bytes(m, n, top));
  if (st != Q3_OK) return st;
  if ((st = check_device()) != Q3_OK) return st;
  q3::LogprobArgs a{};
  a.logits = logits;
  a.ld = ld;
  a.m = m;
  a.n = static_cast<int>(n);
  a.targets = targets;
  a.inv_t = 1.f / temperature;
  a.top = top;
  a.logprobs = logprobs;
  a.entropy = entropy;
  a.top_ids = top_ids;
  a.top_logprobs = top_logprobs;
  a.stats = stats;
  return from_hip(q3::launch_logprobs(a, workspace, static_cast<hipStream_t>(stream)));
}

Q3_API q3_status q3_logprobs_backward(const float* logits, int64_t m, int64_t n, int64_t ld, const int32_t* targets,
                                      float temperature, const float* stats, const float* dlogprobs,
                                      const float* dentropy, void* dlogits, int64_t ld_d, int32_t d_type,
                                      void* stream) {
  if (!logits || !stats || !dlogits || (dlogprobs && !targets)) return Q3_ERR_INVALID_ARG;
  if (m < 1 || m >= kMaxRows || n < 1 || n > kMaxVocabulary) return Q3_ERR_UNSUPPORTED_SHAPE;
  if (d_type != Q3_F32 && d_type != Q3_BF16) return Q3_ERR_INVALID_ARG;
  if (ld < n || ld_d < n || bad_temperature(temperature)) return Q3_ERR_INVALID_ARG;
  if (dlogits == logits && (d_type != Q3_F32 || ld_d != ld)) return Q3_ERR_INVALID_ARG;
  if (!aligned(logits, 4) || !aligned(targets, 4) || !aligned(stats, 16) || !aligned(dlogprobs, 4) ||
      !aligned(dentropy, 4) || !aligned(dlogits, d_type == Q3_BF16 ? 2 : 4))
    return Q3_ERR_MISALIGNED;
  q3_status st = check_device();
  if (st != Q3_OK) return st;
  q3::LogprobBackArgs a{};
  a.logits = logits;
  a.ld = ld;
  a.m = m;
  a.n = static_cast<int>(n);
  a.targets = targets;
  a.inv_t = 1.f / temperature;
  a.stats = stats;
  a.dlogprobs = dlogprobs;
  a.dentropy = dentropy;
  a.dlogits = dlogits;
  a.ld_d = ld_d;
  return from_hip(q3::launch_logprobs_back(a, d_type, static_cast<hipStream_t>(stream)));
}

}  // extern "C"

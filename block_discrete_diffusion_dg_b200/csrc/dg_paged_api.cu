// C ABI of the paged-cache operators: argument checks and launches (include/dg.h).
#include <cmath>

#include "dg_common.cuh"
#include "dg_kernels.h"
#include "nvtx_range.h"

using namespace dg;

namespace {

inline bool aligned16(const void *p) { return ((uintptr_t)p & 15) == 0; }

// The rotation of a call: `rope`, or (null) the model's own, rotate-half over the whole head.
bool rope_spec(const dg_config *cfg, const dg_rope *rope, RopeSpec *out) {
  RopeSpec r{};
  r.theta = cfg->rope_theta;
  r.rot = cfg->head_dim;
  r.mscale = 1.0;
  r.factor = 1.0;
  if (rope) {
    r.rot = rope->rot_dim;
    r.interleaved = rope->layout == DG_ROPE_INTERLEAVED;
    r.scaling = rope->scaling;
    r.factor = rope->factor;
    r.orig_len = rope->orig_len;
    r.beta_slow = rope->beta_slow;
    r.beta_fast = rope->beta_fast;
    r.mscale = rope->mscale;
    if (rope->layout != DG_ROPE_HALF && rope->layout != DG_ROPE_INTERLEAVED) return false;
    if (r.rot < 0 || r.rot > cfg->head_dim || r.rot % 16) return false;
    if (!std::isfinite(r.mscale)) return false;
    if (r.scaling != DG_ROPE_UNSCALED && r.scaling != DG_ROPE_LINEAR &&
        r.scaling != DG_ROPE_BY_PARTS)
      return false;
    if (r.scaling != DG_ROPE_UNSCALED && !(std::isfinite(r.factor) && r.factor > 0.0)) return false;
    if (r.scaling == DG_ROPE_BY_PARTS &&
        !(std::isfinite(r.orig_len) && r.orig_len > 0.0 && std::isfinite(r.beta_slow) &&
          std::isfinite(r.beta_fast) && r.beta_slow >= 0.0 && r.beta_fast > r.beta_slow))
      return false;
  }
  *out = r;
  return true;
}

bool qkv_ok(const dg_config *cfg, const void *qkv, long long ld, long long rows) {
  const int e = cfg->act_dtype == DG_F32 ? 4 : 2;
  const long long width = (long long)(cfg->n_q_heads + 2 * cfg->n_kv_heads) * cfg->head_dim;
  return qkv && aligned16(qkv) && ld >= width && ld * e % 16 == 0 && rows <= INT32_MAX - 64 &&
         width <= INT32_MAX;
}

// Pages the calls can address: a power-of-two page, ids and rows within 32 bits.
bool pages_ok(const dg_config *cfg, const dg_paged_kv *kv) {
  if (!kv || !kv->k_pages || !kv->v_pages || !kv->page_table) return false;
  if (!aligned16(kv->k_pages) || !aligned16(kv->v_pages)) return false;
  const int ps = kv->page_size;
  if (ps < 16 || ps > 1024 || (ps & (ps - 1))) return false;
  if (kv->n_pages <= 0 || kv->max_pages <= 0) return false;
  return (long long)kv->n_pages * cfg->n_kv_heads * ps <= INT32_MAX &&
         (long long)kv->max_pages * ps <= INT32_MAX - 1024;
}

QkvCall qkv_call(const dg_config *cfg, const void *qkv, long long ld, const float *q_gain,
                 const float *k_gain, int32_t *status) {
  QkvCall c{};
  c.act = cfg->act_dtype;
  c.hd = cfg->head_dim;
  c.Hq = cfg->n_q_heads;
  c.Hkv = cfg->n_kv_heads;
  c.eps = cfg->rms_eps;
  c.qkv = qkv;
  c.ld = ld;
  c.q_gain = q_gain;
  c.k_gain = k_gain;
  c.status = status;
  return c;
}

PagedCall paged_call(const dg_config *cfg, int n_seqs, int n_tokens, int shared_len) {
  PagedCall c{};
  c.act = cfg->act_dtype;
  c.hd = cfg->head_dim;
  c.Hq = cfg->n_q_heads;
  c.Hkv = cfg->n_kv_heads;
  c.n_seqs = n_seqs;
  c.n_tokens = n_tokens;
  c.shared_len = shared_len;
  return c;
}

bool sizes_ok(const dg_config *cfg, int n_seqs, int n_tokens) {
  return cfg_ok(cfg) && n_seqs > 0 && n_seqs < (1 << 30) && n_tokens > 0 &&
         (long long)n_tokens * cfg->n_q_heads <= INT32_MAX;
}

int paged_attention(const dg_config *cfg, int n_seqs, int n_tokens, const int32_t *seq_off,
                    const int32_t *kv_len, int shared_len, const void *q, const dg_paged_kv *kv,
                    int causal, void *out, void *ws, size_t ws_bytes, int32_t *dev_status,
                    void *stream) {
  if (!sizes_ok(cfg, n_seqs, n_tokens) || !pages_ok(cfg, kv)) return DG_ERR_INVALID_ARG;
  if (!seq_off || !kv_len || !q || !out || !aligned16(q) || !aligned16(out))
    return DG_ERR_INVALID_ARG;
  if (!ws || ((uintptr_t)ws & 255)) return DG_ERR_INVALID_ARG;
  if (shared_len % kv->page_size || shared_len > kv->max_pages * kv->page_size)
    return DG_ERR_INVALID_ARG;
  if (!paged_attn_supported(cfg->act_dtype, cfg->n_q_heads, cfg->n_kv_heads, cfg->head_dim))
    return DG_ERR_UNSUPPORTED;
  PagedCall c = paged_call(cfg, n_seqs, n_tokens, shared_len);
  if (ws_bytes < paged_attn_ws_bytes(c)) return DG_ERR_WORKSPACE;
  c.seq_off = seq_off;
  c.kv_len = kv_len;
  c.q = q;
  c.out = out;
  c.k_pages = kv->k_pages;
  c.v_pages = kv->v_pages;
  c.page_table = kv->page_table;
  c.n_pages = kv->n_pages;
  c.page_size = kv->page_size;
  c.max_pages = kv->max_pages;
  c.causal = causal ? 1 : 0;
  c.status = dev_status;
  return launch_paged_attn(c, ws, (cudaStream_t)stream);
}

}  // namespace

extern "C" {

int dg_qk_norm_rope(const dg_config *cfg, int batch, int n_tokens, const void *qkv,
                    long long ld_qkv, const int32_t *cache_len, const float *q_gain,
                    const float *k_gain, const dg_rope *rope, void *q, void *k_new, void *v_new,
                    int32_t *dev_status, void *stream) {
  const NvtxRange nvtx_range("dg_qk_norm_rope");
  if (!cfg_ok(cfg) || batch <= 0 || n_tokens <= 0) return DG_ERR_INVALID_ARG;
  if (!qkv_ok(cfg, qkv, ld_qkv, (long long)batch * n_tokens) || !aligned16(q_gain) ||
      !aligned16(k_gain))
    return DG_ERR_INVALID_ARG;
  if (!cache_len || !q || !k_new || !v_new || !aligned16(q) || !aligned16(k_new) ||
      !aligned16(v_new))
    return DG_ERR_INVALID_ARG;
  QkvCall c = qkv_call(cfg, qkv, ld_qkv, q_gain, k_gain, dev_status);
  if (!rope_spec(cfg, rope, &c.rope)) return DG_ERR_INVALID_ARG;
  c.n_tokens = batch * n_tokens;
  c.n_seqs = batch;
  c.n = n_tokens;
  c.len = cache_len;
  c.q = q;
  c.k = k_new;
  c.v = v_new;
  return launch_qkv_rows(c, (cudaStream_t)stream);
}

int dg_paged_append(const dg_config *cfg, int n_seqs, int n_tokens, const int32_t *seq_off,
                    const int32_t *kv_len, const void *qkv, long long ld_qkv, const float *q_gain,
                    const float *k_gain, const dg_rope *rope, const dg_paged_kv *kv, void *q,
                    int32_t *dev_status, void *stream) {
  const NvtxRange nvtx_range("dg_paged_append");
  if (!sizes_ok(cfg, n_seqs, n_tokens) || !pages_ok(cfg, kv)) return DG_ERR_INVALID_ARG;
  if (!qkv_ok(cfg, qkv, ld_qkv, n_tokens) || !aligned16(q_gain) || !aligned16(k_gain))
    return DG_ERR_INVALID_ARG;
  if (!seq_off || !kv_len || (q && !aligned16(q))) return DG_ERR_INVALID_ARG;
  QkvCall c = qkv_call(cfg, qkv, ld_qkv, q_gain, k_gain, dev_status);
  if (!rope_spec(cfg, rope, &c.rope)) return DG_ERR_INVALID_ARG;
  c.n_tokens = n_tokens;
  c.n_seqs = n_seqs;
  c.seq_off = seq_off;
  c.len = kv_len;
  c.q = q;
  c.k_pages = kv->k_pages;
  c.v_pages = kv->v_pages;
  c.page_table = kv->page_table;
  c.n_pages = kv->n_pages;
  c.page_size = kv->page_size;
  c.max_pages = kv->max_pages;
  return launch_qkv_rows(c, (cudaStream_t)stream);
}

size_t dg_paged_workspace_size(const dg_config *cfg, int n_seqs, int n_tokens, int shared_len) {
  if (!sizes_ok(cfg, n_seqs, n_tokens) || shared_len < 0) return 0;
  if (!paged_attn_supported(cfg->act_dtype, cfg->n_q_heads, cfg->n_kv_heads, cfg->head_dim))
    return 0;
  return paged_attn_ws_bytes(paged_call(cfg, n_seqs, n_tokens, shared_len));
}

int dg_paged_attn(const dg_config *cfg, int n_seqs, int n_tokens, const int32_t *seq_off,
                  const int32_t *kv_len, const void *q, const dg_paged_kv *kv, int causal,
                  void *out, void *ws, size_t ws_bytes, int32_t *dev_status, void *stream) {
  const NvtxRange nvtx_range("dg_paged_attn");
  return paged_attention(cfg, n_seqs, n_tokens, seq_off, kv_len, 0, q, kv, causal, out, ws,
                         ws_bytes, dev_status, stream);
}

int dg_prefix_attn(const dg_config *cfg, int n_seqs, int n_tokens, const int32_t *seq_off,
                   const int32_t *kv_len, int shared_len, const void *q, const dg_paged_kv *kv,
                   int causal, void *out, void *ws, size_t ws_bytes, int32_t *dev_status,
                   void *stream) {
  const NvtxRange nvtx_range("dg_prefix_attn");
  if (shared_len <= 0) return DG_ERR_INVALID_ARG;
  return paged_attention(cfg, n_seqs, n_tokens, seq_off, kv_len, shared_len, q, kv, causal, out,
                         ws, ws_bytes, dev_status, stream);
}

}  // extern "C"

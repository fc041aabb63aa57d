// C entry points of the target-side operators: validation and launches.
#include <climits>
#include <cmath>
#include <cstring>

#include "../../include/dflash.h"
#include "kernels.h"
#include "target_ops.h"

using namespace dflash;

namespace {

int fail(int st, const char *msg) {
  set_last_error(msg);
  return st;
}

size_t elem(dflash_dtype t) { return t == DFLASH_F32 ? 4 : 2; }

bool aligned16(const void *p, int64_t stride, size_t es) {
  return (uintptr_t)p % 16 == 0 && (stride * (int64_t)es) % 16 == 0;
}

// 32-bit arrays of the device
template <typename... P> bool aligned4(const P *...p) { return (((uintptr_t)p % 4 == 0) && ...); }

int check_layer(const dflash_layer_kv *kv, int32_t batch, int32_t total_rows) {
  if (!kv) return fail(DFLASH_EINVAL, "kv is NULL");
  if (kv->dtype != DFLASH_F32 && kv->dtype != DFLASH_BF16) return fail(DFLASH_EUNSUPPORTED, "dtype");
  if (kv->head_dim != 64 && kv->head_dim != 128)
    return fail(DFLASH_EUNSUPPORTED, "head_dim must be 64 or 128");
  if (kv->n_heads <= 0 || kv->n_kv_heads <= 0 || kv->n_heads % kv->n_kv_heads)
    return fail(DFLASH_EINVAL, "n_heads must be a positive multiple of n_kv_heads");
  if (kv->n_heads / kv->n_kv_heads > 128 || kv->n_heads > 1024)
    return fail(DFLASH_EUNSUPPORTED, "at most 128 query heads per KV head and 1024 in all");
  if (!kv->k_pages || !kv->v_pages || !kv->page_table)
    return fail(DFLASH_EINVAL, "k_pages, v_pages and page_table must be non-NULL");
  if ((uintptr_t)kv->k_pages % 16 || (uintptr_t)kv->v_pages % 16)
    return fail(DFLASH_EINVAL, "pages must be 16-byte aligned");
  if (kv->n_pages <= 0 || kv->pages_per_req <= 0)
    return fail(DFLASH_EINVAL, "n_pages and pages_per_req must be positive");
  if (kv->n_pages > INT32_MAX / kPageRows || kv->pages_per_req > INT32_MAX / kPageRows / 2)
    return fail(DFLASH_EUNSUPPORTED, "n_pages or pages_per_req too large");
  if (kv->prefix_len < 0 || kv->prefix_len % kPageRows || kv->prefix_len > INT32_MAX / 2)
    return fail(DFLASH_EINVAL, "prefix_len must be a multiple of 64");
  if (kv->prefix_len > 0 && !kv->prefix_pages) return fail(DFLASH_EINVAL, "prefix_pages is NULL");
  if (!aligned4(kv->page_table, kv->prefix_pages))
    return fail(DFLASH_EINVAL, "page_table and prefix_pages must be 4-byte aligned");
  if (batch < 0 || total_rows < 0) return fail(DFLASH_EINVAL, "negative batch or total_rows");
  if (batch > 1024) return fail(DFLASH_ECAPACITY, "batch > 1024");
  if ((int64_t)total_rows * kv->n_heads > (1 << 28))
    return fail(DFLASH_ECAPACITY, "total_rows * n_heads > 2^28");
  return DFLASH_OK;
}

PagedRows paged_rows(const dflash_layer_kv *kv, int32_t batch, int32_t total_rows,
                     const int32_t *row_start, const int32_t *kv_len) {
  PagedRows r;
  r.row_start = row_start;
  r.kv_len = kv_len;
  r.page_table = kv->page_table;
  r.prefix_pages = kv->prefix_pages;
  r.B = batch;
  r.total_rows = total_rows;
  r.pages_per_req = kv->pages_per_req;
  r.n_pages = kv->n_pages;
  r.prefix_len = kv->prefix_len;
  return r;
}

int append(dflash_handle *h, const dflash_layer_kv *kv, int32_t batch, int32_t total_rows,
           const int32_t *row_start, const int32_t *kv_len, const int32_t *positions, const void *q,
           int64_t q_stride, const void *k, int64_t k_stride, const void *v,
           int64_t v_stride, const void *q_gain, const void *k_gain, float eps,
           const dflash_rope *rope, void *q_out, int64_t q_out_stride,
           dflash_stream_t stream) {
  AppendParams p;
  std::memset(&p, 0, sizeof(p));
  if (!h) return fail(DFLASH_EINVAL, "handle is NULL");
  if (int st = check_layer(kv, batch, total_rows)) return st;
  if (!rope) return fail(DFLASH_EINVAL, "rope is NULL");
  if (rope->rotary_dim < 0 || rope->rotary_dim % 2 || rope->rotary_dim > kv->head_dim)
    return fail(DFLASH_EINVAL, "rotary_dim must be even and at most head_dim");
  if (!(eps >= 0.f) || std::isinf(eps)) return fail(DFLASH_EINVAL, "eps must be >= 0 and finite");
  if ((q == nullptr) != (q_out == nullptr)) return fail(DFLASH_EINVAL, "q and q_out go together");
  if (!q && q_gain) return fail(DFLASH_EINVAL, "q_gain without q");
  const bool empty = batch == 0 || total_rows == 0;
  if (!empty && (!row_start || !kv_len || !k || !v))
    return fail(DFLASH_EINVAL, "a required pointer is NULL");
  if (!aligned4(row_start, kv_len)) return fail(DFLASH_EINVAL, "row_start and kv_len must be 4-byte aligned");
  const size_t es = elem(kv->dtype);
  const int64_t qw = (int64_t)kv->n_heads * kv->head_dim, kw = (int64_t)kv->n_kv_heads * kv->head_dim;
  if (!empty && ((q && (q_stride < qw || q_out_stride < qw)) || k_stride < kw || v_stride < kw))
    return fail(DFLASH_EINVAL, "a row stride is below the row's width");
  if ((q && (!aligned16(q, q_stride, es) || !aligned16(q_out, q_out_stride, es))) ||
      !aligned16(k, k_stride, es) || !aligned16(v, v_stride, es) || (uintptr_t)q_gain % 16 ||
      (uintptr_t)k_gain % 16)
    return fail(DFLASH_EINVAL, "pointers and row strides must be multiples of 16 bytes");
  if (q && q == q_out && q_stride != q_out_stride && total_rows > 1)
    return fail(DFLASH_EINVAL, "q_out is q with another row stride");
  if (int st = handle_ready(h, &p.err)) return st;
  if (empty) return DFLASH_OK;
  p.rows = paged_rows(kv, batch, total_rows, row_start, kv_len);
  p.q = q;
  p.k = k;
  p.v = v;
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.q_out_stride = q_out_stride;
  p.positions = positions;
  p.q_gain = q_gain;
  p.k_gain = k_gain;
  p.q_out = q_out;
  p.k_pages = kv->k_pages;
  p.v_pages = kv->v_pages;
  p.H = q ? kv->n_heads : 0;
  p.KVH = kv->n_kv_heads;
  p.eps = eps;
  p.rot = rope->rotary_dim;
  p.inter = rope->interleaved;
  p.amp = rope->amplitude;
  std::memcpy(p.turns, rope->turns, sizeof(p.turns));
  cudaStream_t s = (cudaStream_t)stream;
  const int idx = handle_timed_begin(h, "append_kv", s);
  return handle_timed_end(h, idx, "append_kv", s, launch_append_kv(kv->dtype, kv->head_dim, p, s));
}

int check_batch(int32_t batch, int32_t total_rows) {
  if (batch < 0 || total_rows < 0) return fail(DFLASH_EINVAL, "negative batch or total_rows");
  if (batch > 1024) return fail(DFLASH_ECAPACITY, "batch > 1024");
  if (total_rows > (1 << 28)) return fail(DFLASH_ECAPACITY, "total_rows > 2^28");
  return DFLASH_OK;
}

int check_mask(const uint32_t *mask, int32_t mask_words) {
  if (mask ? mask_words < 1 || mask_words > kMaxTreeRows / 32 : mask_words != 0)
    return fail(DFLASH_EINVAL, "mask_words must be 1 to 32, 0 without a mask");
  if (!aligned4(mask)) return fail(DFLASH_EINVAL, "mask must be 4-byte aligned");
  return DFLASH_OK;
}

// The two attention calls; of *p what tells them apart is filled.
int attend(dflash_handle *h, const dflash_layer_kv *kv, int32_t batch, int32_t total_rows,
           const int32_t *row_start, const int32_t *kv_len, const void *q, int64_t q_stride,
           float scale, void *out, int64_t out_stride, void *workspace, size_t bytes,
           const char *name, dflash_stream_t stream, PagedAttnParams &p) {
  if (!h) return fail(DFLASH_EINVAL, "handle is NULL");
  size_t need = 0;
  if (int st = dflash_paged_attention_workspace_size(kv, batch, total_rows, &need)) return st;
  if (p.causal != 0 && p.causal != 1) return fail(DFLASH_EINVAL, "causal must be 0 or 1");
  if (std::isnan(scale) || std::isinf(scale)) return fail(DFLASH_EINVAL, "scale must be finite");
  if (batch == 0 || total_rows == 0) return handle_ready(h, &p.err);
  if (!row_start || !kv_len || !q || !out) return fail(DFLASH_EINVAL, "a required pointer is NULL");
  if (q == out) return fail(DFLASH_EINVAL, "out must not be q");
  if (!aligned4(row_start, kv_len)) return fail(DFLASH_EINVAL, "row_start and kv_len must be 4-byte aligned");
  const size_t es = elem(kv->dtype);
  const int64_t qw = (int64_t)kv->n_heads * kv->head_dim;
  if (q_stride < qw || out_stride < qw) return fail(DFLASH_EINVAL, "a row stride is below the row's width");
  if (!aligned16(q, q_stride, es) || !aligned16(out, out_stride, es))
    return fail(DFLASH_EINVAL, "pointers and row strides must be multiples of 16 bytes");
  if (!workspace || (uintptr_t)workspace % 256)
    return fail(DFLASH_EINVAL, "workspace must be non-NULL and 256-byte aligned");
  if (bytes < need) return fail(DFLASH_ECAPACITY, "workspace too small");
  if (int st = handle_ready(h, &p.err)) return st;
  p.rows = paged_rows(kv, batch, total_rows, row_start, kv_len);
  p.q = q;
  p.k_pages = kv->k_pages;
  p.v_pages = kv->v_pages;
  p.out = out;
  p.q_stride = q_stride;
  p.out_stride = out_stride;
  p.H = kv->n_heads;
  p.KVH = kv->n_kv_heads;
  p.D = kv->head_dim;
  p.scale = scale;
  cudaStream_t s = (cudaStream_t)stream;
  const int idx = handle_timed_begin(h, name, s);
  return handle_timed_end(h, idx, name, s,
                          kv->dtype == DFLASH_BF16 ? launch_paged_attention_tc(p, workspace, s)
                                                   : launch_paged_attention_simt(p, s));
}

// Checks shared by the two sampling calls; *p is filled but for the outputs.
int sampling_params(dflash_handle *h, int32_t rows, int32_t vocab, const void *logits,
                    dflash_dtype dtype, int64_t row_stride, const dflash_sampling *sp,
                    SampleParams *p) {
  if (!h) return fail(DFLASH_EINVAL, "handle is NULL");
  if (rows < 0 || vocab <= 0) return fail(DFLASH_EINVAL, "negative rows or vocab <= 0");
  if (dtype != DFLASH_F32 && dtype != DFLASH_BF16) return fail(DFLASH_EUNSUPPORTED, "dtype");
  if (vocab > sampling_max_vocab(dtype))
    return fail(DFLASH_EUNSUPPORTED, "vocab > 524288 (bf16) or 262144 (fp32)");
  if (rows > (1 << 24)) return fail(DFLASH_ECAPACITY, "rows > 2^24");
  if (!sp) return fail(DFLASH_EINVAL, "params is NULL");
  if (sp->rows_per_entry <= 0 || rows % sp->rows_per_entry)
    return fail(DFLASH_EINVAL, "rows_per_entry must be positive and divide rows");
  if (rows > 0 && !logits) return fail(DFLASH_EINVAL, "logits is NULL");
  if (row_stride < vocab) return fail(DFLASH_EINVAL, "row_stride < vocab");
  if ((uintptr_t)logits % elem(dtype)) return fail(DFLASH_EINVAL, "logits misaligned");
  if (!aligned4(sp->temperature, sp->top_k, sp->top_p, sp->min_p))
    return fail(DFLASH_EINVAL, "sampling parameters must be 4-byte aligned");
  std::memset(p, 0, sizeof(*p));
  p->logits = logits;
  p->ld = row_stride;
  p->rows = rows;
  p->vocab = vocab;
  p->temperature = sp->temperature;
  p->top_k = sp->top_k;
  p->top_p = sp->top_p;
  p->min_p = sp->min_p;
  p->rows_per_entry = sp->rows_per_entry;
  return DFLASH_OK;
}

}  // namespace

extern "C" {

int dflash_rope_init(int32_t rotary_dim, int32_t interleaved, double theta,
                     dflash_rope_scaling scaling, double factor, double original_positions,
                     double low, double high, dflash_rope *out) {
  if (!out) return fail(DFLASH_EINVAL, "out is NULL");
  if (rotary_dim < 0 || rotary_dim > 128 || rotary_dim % 2)
    return fail(DFLASH_EUNSUPPORTED, "rotary_dim must be even and in [0, 128]");
  if (interleaved != 0 && interleaved != 1) return fail(DFLASH_EINVAL, "interleaved must be 0 or 1");
  if (!(theta > 1.0) || std::isinf(theta)) return fail(DFLASH_EINVAL, "theta must be finite and > 1");
  const int sc = (int)scaling;
  if (sc < DFLASH_ROPE_NONE || sc > DFLASH_ROPE_YARN) return fail(DFLASH_EUNSUPPORTED, "scaling");
  if (sc != DFLASH_ROPE_NONE && (!(factor >= 1.0) || std::isinf(factor)))
    return fail(DFLASH_EINVAL, "factor must be finite and >= 1");
  if (sc >= DFLASH_ROPE_BANDS) {
    if (!(original_positions > 0.0) || std::isinf(original_positions))
      return fail(DFLASH_EINVAL, "original_positions must be positive and finite");
    if (low == 0.0) low = 1.0;
    if (high == 0.0) high = sc == DFLASH_ROPE_BANDS ? 4.0 : 32.0;
    if (!(low > 0.0) || !(high > low) || std::isinf(high))
      return fail(DFLASH_EINVAL, "0 < low < high required");
  }
  std::memset(out, 0, sizeof(*out));
  out->rotary_dim = rotary_dim;
  out->interleaved = interleaved;
  out->amplitude = sc == DFLASH_ROPE_YARN ? (float)(0.1 * std::log(factor) + 1.0) : 1.0f;
  const double two_pi = 6.283185307179586476925;
  double lo = 0, hi = 0;
  if (sc == DFLASH_ROPE_YARN && rotary_dim > 0) {
    auto at = [&](double turns) {
      return rotary_dim * std::log(original_positions / (turns * two_pi)) / (2.0 * std::log(theta));
    };
    lo = std::fmax(std::floor(at(high)), 0.0);
    hi = std::fmin(std::ceil(at(low)), rotary_dim - 1.0);
  }
  for (int i = 0; i < rotary_dim / 2; ++i) {
    double f = std::pow(theta, -2.0 * i / rotary_dim);
    if (sc == DFLASH_ROPE_LINEAR) {
      f /= factor;
    } else if (sc == DFLASH_ROPE_BANDS) {
      const double turns = original_positions * f / two_pi;
      const double s = std::fmin(1.0, std::fmax(0.0, (turns - low) / (high - low)));
      f *= (1.0 - s) / factor + s;
    } else if (sc == DFLASH_ROPE_YARN) {
      const double a = std::fmin(1.0, std::fmax(0.0, (i - lo) / std::fmax(hi - lo, 0.001)));
      f *= a / factor + 1.0 - a;
    }
    // turns per position (below 0.16) as a fraction of 2^64
    out->turns[i] = (uint64_t)std::ldexp(f / two_pi, 64);
  }
  return DFLASH_OK;
}

int dflash_append_kv(dflash_handle *h, const dflash_layer_kv *kv, int32_t batch, int32_t total_rows,
                     const int32_t *row_start, const int32_t *kv_len, const void *q,
                     int64_t q_stride, const void *k, int64_t k_stride, const void *v,
                     int64_t v_stride, const void *q_gain, const void *k_gain, float eps,
                     const dflash_rope *rope, void *q_out, int64_t q_out_stride,
                     dflash_stream_t stream) {
  return append(h, kv, batch, total_rows, row_start, kv_len, nullptr, q, q_stride, k, k_stride, v, v_stride,
                q_gain, k_gain, eps, rope, q_out, q_out_stride, stream);
}

int dflash_append_kv_at(dflash_handle *h, const dflash_layer_kv *kv, int32_t batch,
                        int32_t total_rows, const int32_t *row_start, const int32_t *kv_len,
                        const int32_t *positions, const void *q, int64_t q_stride, const void *k,
                        int64_t k_stride, const void *v, int64_t v_stride, const void *q_gain,
                        const void *k_gain, float eps, const dflash_rope *rope, void *q_out,
                        int64_t q_out_stride, dflash_stream_t stream) {
  if (batch > 0 && total_rows > 0 && !positions) return fail(DFLASH_EINVAL, "positions is NULL");
  if (!aligned4(positions)) return fail(DFLASH_EINVAL, "positions must be 4-byte aligned");
  return append(h, kv, batch, total_rows, row_start, kv_len, positions, q, q_stride, k, k_stride, v, v_stride,
                q_gain, k_gain, eps, rope, q_out, q_out_stride, stream);
}

int dflash_paged_attention_workspace_size(const dflash_layer_kv *kv, int32_t batch,
                                          int32_t total_rows, size_t *bytes) {
  if (!bytes) return fail(DFLASH_EINVAL, "bytes is NULL");
  if (int st = check_layer(kv, batch, total_rows)) return st;
  *bytes = kv->dtype == DFLASH_BF16
               ? paged_attention_tc_workspace(batch, total_rows, kv->n_heads, kv->n_kv_heads,
                                              kv->head_dim, kv->prefix_len)
               : 256;
  return DFLASH_OK;
}

int dflash_paged_attention(dflash_handle *h, const dflash_layer_kv *kv, int32_t batch,
                           int32_t total_rows, const int32_t *row_start, const int32_t *kv_len,
                           const void *q, int64_t q_stride, float scale, int32_t causal, void *out,
                           int64_t out_stride, void *workspace, size_t bytes,
                           dflash_stream_t stream) {
  PagedAttnParams p;
  std::memset(&p, 0, sizeof(p));
  p.causal = causal;
  return attend(h, kv, batch, total_rows, row_start, kv_len, q, q_stride, scale, out, out_stride, workspace, bytes,
                "paged_attention", stream, p);
}

int dflash_tree_attention(dflash_handle *h, const dflash_layer_kv *kv, int32_t batch,
                          int32_t total_rows, const int32_t *row_start, const int32_t *kv_len,
                          const uint32_t *mask, int32_t mask_words, const void *q, int64_t q_stride,
                          float scale, void *out, int64_t out_stride, float *lse, void *workspace,
                          size_t bytes, dflash_stream_t stream) {
  if (int st = check_mask(mask, mask_words)) return st;
  if (!aligned4(lse)) return fail(DFLASH_EINVAL, "lse must be 4-byte aligned");
  PagedAttnParams p;
  std::memset(&p, 0, sizeof(p));
  p.causal = mask == nullptr;
  p.mask = mask;
  p.mask_words = mask_words;
  p.lse = lse;
  p.tree = 1;
  return attend(h, kv, batch, total_rows, row_start, kv_len, q, q_stride, scale, out, out_stride, workspace, bytes,
                "tree_attention", stream, p);
}

int dflash_tree_plan(dflash_handle *h, int32_t batch, int32_t total_rows, const int32_t *row_start,
                     const int32_t *parent, const int32_t *root_pos, int32_t mask_words,
                     uint32_t *mask, int32_t *positions, dflash_stream_t stream) {
  TreePlanParams p;
  if (!h) return fail(DFLASH_EINVAL, "handle is NULL");
  if (int st = check_batch(batch, total_rows)) return st;
  if (mask_words < 1 || mask_words > kMaxTreeRows / 32) return fail(DFLASH_EUNSUPPORTED, "mask_words must be 1 to 32");
  const bool empty = batch == 0 || total_rows == 0;
  if (!empty && (!row_start || !parent || !root_pos || !mask))
    return fail(DFLASH_EINVAL, "a required pointer is NULL");
  if (!aligned4(row_start, parent, root_pos, mask, positions))
    return fail(DFLASH_EINVAL, "arrays must be 4-byte aligned");
  if (int st = handle_ready(h, &p.err)) return st;
  if (empty) return DFLASH_OK;
  p.row_start = row_start;
  p.parent = parent;
  p.root_pos = root_pos;
  p.mask = mask;
  p.positions = positions;
  p.B = batch;
  p.total_rows = total_rows;
  p.mask_words = mask_words;
  cudaStream_t s = (cudaStream_t)stream;
  const int idx = handle_timed_begin(h, "tree_plan", s);
  return handle_timed_end(h, idx, "tree_plan", s, launch_tree_plan(p, s));
}

int dflash_accept_commit_tree(dflash_handle *h, int32_t batch, int32_t total_rows,
                              const int32_t *row_start, const int32_t *parent,
                              const int32_t *tokens, const int32_t *posterior, int32_t max_path,
                              int32_t *seq_len, int32_t *accept_len, int32_t *commit_len,
                              int32_t *bonus, int32_t *out_tokens, int32_t *path,
                              float *row_weight, int32_t *output_ids, int32_t out_stride,
                              dflash_stream_t stream) {
  AcceptTreeParams p;
  if (!h) return fail(DFLASH_EINVAL, "handle is NULL");
  if (int st = check_batch(batch, total_rows)) return st;
  if (max_path < 1 || max_path > kMaxTreeRows) return fail(DFLASH_EUNSUPPORTED, "max_path must be 1 to 1024");
  const bool empty = batch == 0 || total_rows == 0;
  if (!empty && (!row_start || !parent || !tokens || !posterior || !seq_len || !accept_len || !commit_len || !bonus ||
                 !out_tokens || !path))
    return fail(DFLASH_EINVAL, "a required pointer is NULL");
  if (output_ids && out_stride <= 0) return fail(DFLASH_EINVAL, "out_stride must be positive");
  if (!aligned4(row_start, parent, tokens, posterior, seq_len, accept_len, commit_len, bonus, out_tokens, path,
                row_weight, output_ids))
    return fail(DFLASH_EINVAL, "arrays must be 4-byte aligned");
  if (int st = handle_ready(h, &p.err)) return st;
  if (empty) return DFLASH_OK;
  p.row_start = row_start;
  p.parent = parent;
  p.tokens = tokens;
  p.posterior = posterior;
  p.seq_len = seq_len;
  p.accept_len = accept_len;
  p.commit_len = commit_len;
  p.bonus = bonus;
  p.out_tokens = out_tokens;
  p.path = path;
  p.row_weight = row_weight;
  p.output_ids = output_ids;
  p.B = batch;
  p.total_rows = total_rows;
  p.max_path = max_path;
  p.out_stride = out_stride;
  const void *lm_head;
  int hidden, dtype;
  if (int st = handle_lm_head(h, &lm_head, &hidden, &p.vocab, &dtype)) return st;
  cudaStream_t s = (cudaStream_t)stream;
  const int idx = handle_timed_begin(h, "accept_tree", s);
  return handle_timed_end(h, idx, "accept_tree", s, launch_accept_tree(p, s));
}

int dflash_key_weights(dflash_handle *h, const dflash_layer_kv *kv, int32_t batch,
                       int32_t total_rows, const int32_t *row_start, const int32_t *kv_len,
                       const uint32_t *mask, int32_t mask_words, const void *q, int64_t q_stride,
                       float scale, const float *lse, const float *row_weight, float decay,
                       float *weights, int32_t width, dflash_stream_t stream) {
  KeyWeightParams p;
  std::memset(&p, 0, sizeof(p));
  if (!h) return fail(DFLASH_EINVAL, "handle is NULL");
  if (int st = check_layer(kv, batch, total_rows)) return st;
  if (int st = check_mask(mask, mask_words)) return st;
  if (std::isnan(scale) || std::isinf(scale)) return fail(DFLASH_EINVAL, "scale must be finite");
  if (scale != 0.f && (std::fabs(scale) < 0x1p-100f || std::fabs(scale) > 0x1p100f))
    return fail(DFLASH_EUNSUPPORTED, "scale must be 0 or of magnitude 2^-100 to 2^100");
  if (!(decay >= 0.f && decay <= 1.f)) return fail(DFLASH_EINVAL, "decay must be 0 to 1");
  if (width <= 0) return fail(DFLASH_EINVAL, "width must be positive");
  const bool empty = batch == 0 || total_rows == 0;
  if (!empty && (!row_start || !kv_len || !q || !lse || !weights))
    return fail(DFLASH_EINVAL, "a required pointer is NULL");
  if (!aligned4(row_start, kv_len, lse, row_weight, weights))
    return fail(DFLASH_EINVAL, "arrays must be 4-byte aligned");
  if (q_stride < (int64_t)kv->n_heads * kv->head_dim) return fail(DFLASH_EINVAL, "a row stride is below the row's width");
  if (!aligned16(q, q_stride, elem(kv->dtype)))
    return fail(DFLASH_EINVAL, "pointers and row strides must be multiples of 16 bytes");
  if (int st = handle_ready(h, &p.err)) return st;
  if (empty) return DFLASH_OK;
  p.rows = paged_rows(kv, batch, total_rows, row_start, kv_len);
  p.mask = mask;
  p.mask_words = mask_words;
  p.q = q;
  p.k_pages = kv->k_pages;
  p.q_stride = q_stride;
  p.H = kv->n_heads;
  p.KVH = kv->n_kv_heads;
  p.D = kv->head_dim;
  p.scale = scale;
  p.lse = lse;
  p.row_weight = row_weight;
  p.decay = decay;
  p.weights = weights;
  p.width = width;
  cudaStream_t s = (cudaStream_t)stream;
  const int idx = handle_timed_begin(h, "key_weights", s);
  return handle_timed_end(h, idx, "key_weights", s,
                          kv->dtype == DFLASH_BF16 ? launch_key_weights_tc(p, s) : launch_key_weights_simt(p, s));
}

int dflash_choose_rows(dflash_handle *h, const dflash_layer_kv *kv, int32_t batch,
                       const int32_t *kv_len, const float *weights, int32_t width,
                       const int32_t *keep, int32_t first, int32_t last, int32_t max_keep,
                       int32_t *rows, int32_t *count, dflash_stream_t stream) {
  ChooseParams p;
  std::memset(&p, 0, sizeof(p));
  if (!h) return fail(DFLASH_EINVAL, "handle is NULL");
  if (int st = check_layer(kv, batch, 0)) return st;
  if (width <= 0 || max_keep <= 0) return fail(DFLASH_EINVAL, "width and max_keep must be positive");
  if (first < 0 || last < 0) return fail(DFLASH_EINVAL, "negative first or last");
  if (batch > 0 && (!kv_len || !weights || !keep || !rows || !count))
    return fail(DFLASH_EINVAL, "a required pointer is NULL");
  if (!aligned4(kv_len, weights, keep, rows, count)) return fail(DFLASH_EINVAL, "arrays must be 4-byte aligned");
  if (int st = handle_ready(h, &p.err)) return st;
  if (batch == 0) return DFLASH_OK;
  p.kv_len = kv_len;
  p.keep = keep;
  p.weights = weights;
  p.rows = rows;
  p.count = count;
  p.B = batch;
  p.KVH = kv->n_kv_heads;
  p.width = width;
  p.prefix_len = kv->prefix_len;
  p.first = first;
  p.last = last;
  p.max_keep = max_keep;
  cudaStream_t s = (cudaStream_t)stream;
  const int idx = handle_timed_begin(h, "choose_rows", s);
  return handle_timed_end(h, idx, "choose_rows", s, launch_choose_rows(p, s));
}

int dflash_keep_rows(dflash_handle *h, const dflash_layer_kv *kv, int32_t batch,
                     const int32_t *first, int32_t lists, int32_t max_rows, const int32_t *rows,
                     const int32_t *count, float *weights, int32_t width, dflash_stream_t stream) {
  KeepParams p;
  std::memset(&p, 0, sizeof(p));
  if (!h) return fail(DFLASH_EINVAL, "handle is NULL");
  if (int st = check_layer(kv, batch, 0)) return st;
  if (lists != 1 && lists != kv->n_kv_heads) return fail(DFLASH_EINVAL, "lists must be 1 or n_kv_heads");
  if (max_rows <= 0) return fail(DFLASH_EINVAL, "max_rows must be positive");
  if (weights && width <= 0) return fail(DFLASH_EINVAL, "width must be positive");
  if (batch > 0 && (!rows || !count)) return fail(DFLASH_EINVAL, "a required pointer is NULL");
  if (!aligned4(first, rows, count, weights)) return fail(DFLASH_EINVAL, "arrays must be 4-byte aligned");
  if (int st = handle_ready(h, &p.err)) return st;
  if (batch == 0) return DFLASH_OK;
  p.first = first;
  p.rows = rows;
  p.count = count;
  p.page_table = kv->page_table;
  p.k_pages = kv->k_pages;
  p.v_pages = kv->v_pages;
  p.weights = weights;
  p.B = batch;
  p.KVH = kv->n_kv_heads;
  p.lists = lists;
  p.max_rows = max_rows;
  p.width = width;
  p.prefix_len = kv->prefix_len;
  p.pages_per_req = kv->pages_per_req;
  p.n_pages = kv->n_pages;
  p.row_bytes = kv->head_dim * (int)elem(kv->dtype);
  cudaStream_t s = (cudaStream_t)stream;
  const int idx = handle_timed_begin(h, "keep_rows", s);
  return handle_timed_end(h, idx, "keep_rows", s, launch_keep_rows(p, s));
}

int dflash_target_probs(dflash_handle *h, int32_t rows, int32_t vocab, const void *logits,
                        dflash_dtype dtype, int64_t row_stride, const dflash_sampling *params,
                        float *probs, dflash_stream_t stream) {
  SampleParams p;
  if (int st = sampling_params(h, rows, vocab, logits, dtype, row_stride, params, &p)) return st;
  if (rows == 0) return handle_ready(h, &p.err);
  if (!probs || (uintptr_t)probs % 4) return fail(DFLASH_EINVAL, "probs is NULL or misaligned");
  const char *a = (const char *)logits, *b = (const char *)probs;
  const char *a_end = a + ((int64_t)(rows - 1) * row_stride + vocab) * (int64_t)elem(dtype);
  const char *b_end = b + (int64_t)rows * vocab * 4;
  if (a < b_end && b < a_end) return fail(DFLASH_EINVAL, "probs overlaps logits");
  if (int st = handle_ready(h, &p.err)) return st;
  p.probs = probs;
  cudaStream_t s = (cudaStream_t)stream;
  const int idx = handle_timed_begin(h, "target_probs", s);
  return handle_timed_end(h, idx, "target_probs", s, launch_sampling(dtype, p, s));
}

int dflash_sample_tokens(dflash_handle *h, int32_t rows, int32_t vocab, const void *logits,
                         dflash_dtype dtype, int64_t row_stride, const dflash_sampling *params,
                         const float *exp_noise, int32_t *ids, float *prob,
                         dflash_stream_t stream) {
  SampleParams p;
  if (int st = sampling_params(h, rows, vocab, logits, dtype, row_stride, params, &p)) return st;
  if (rows == 0) return handle_ready(h, &p.err);
  if (!exp_noise || !ids) return fail(DFLASH_EINVAL, "exp_noise or ids is NULL");
  if (!aligned4(exp_noise, ids, prob)) return fail(DFLASH_EINVAL, "exp_noise, ids and prob must be 4-byte aligned");
  if (int st = handle_ready(h, &p.err)) return st;
  p.noise = exp_noise;
  p.ids = ids;
  p.prob = prob;
  cudaStream_t s = (cudaStream_t)stream;
  const int idx = handle_timed_begin(h, "sample_tokens", s);
  return handle_timed_end(h, idx, "sample_tokens", s, launch_sampling(dtype, p, s));
}

}  // extern "C"

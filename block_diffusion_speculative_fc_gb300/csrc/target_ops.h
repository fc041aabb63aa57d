// Internal launch interface of the target-side operators (append, paged
// attention, sampling) and their access to the handle.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/dflash.h"

namespace dflash {

// ---- the handle (dflash_api.cu) ----
// Status of a call that needs a bound workspace on the current device; *err =
// the device error word.
int handle_ready(const dflash_handle *h, unsigned int **err);
// Event bracket of one timed launch (a no-op unless profiling is on).
int handle_timed_begin(dflash_handle *h, const char *name, cudaStream_t s);
int handle_timed_end(dflash_handle *h, int idx, const char *name, cudaStream_t s, cudaError_t e);

// ---- ragged rows over a paged cache ----
struct PagedRows {
  const int *row_start;      // [B + 1]
  const int *kv_len;         // [B]
  const int *page_table;     // [B, pages_per_req]
  const int *prefix_pages;   // [prefix_len / 64]
  int B, total_rows, pages_per_req, n_pages, prefix_len;
};
constexpr int kPageRows = 64;

struct AppendParams {
  PagedRows rows;
  const void *q, *k, *v;
  int64_t q_stride, k_stride, v_stride, q_out_stride;   // elements
  const void *q_gain, *k_gain;
  void *q_out, *k_pages, *v_pages;
  int H, KVH;                // H = 0: no queries
  float eps;
  int rot, inter;
  float amp;
  uint64_t turns[64];
  unsigned int *err;
};
cudaError_t launch_append_kv(int dtype, int head_dim, const AppendParams &p, cudaStream_t s);

struct PagedAttnParams {
  PagedRows rows;
  const void *q, *k_pages, *v_pages;
  void *out;
  int64_t q_stride, out_stride;
  int H, KVH, D;
  float scale;
  int causal;
  unsigned int *err;
};
cudaError_t launch_paged_attention_simt(const PagedAttnParams &p, cudaStream_t s);   // fp32
cudaError_t prepare_paged_attention_simt();
// bf16 on the tensor cores; device scratch of the size below.
size_t paged_attention_tc_workspace(int B, int total_rows, int H, int KVH, int D, int prefix);
cudaError_t launch_paged_attention_tc(const PagedAttnParams &p, void *workspace, cudaStream_t s);
cudaError_t prepare_paged_attention_tc();

struct SampleParams {
  const void *logits;
  int64_t ld;
  int rows, vocab;
  const float *temperature;
  const int *top_k;
  const float *top_p, *min_p;
  int rows_per_entry;
  float *probs;              // distribution, or
  const float *noise;        // tokens
  int *ids;
  float *prob;
  unsigned int *err;
};
// Largest vocabulary whose row fits the shared memory of one cluster.
int sampling_max_vocab(int dtype);
cudaError_t launch_sampling(int dtype, const SampleParams &p, cudaStream_t s);
cudaError_t prepare_sampling();

}  // namespace dflash

// CUDA-core attention of new rows over a paged fp32 cache (the tensor cores
// have no exact-fp32 kind).  One CTA per (row, KV head) holds the group's query
// heads and streams the row's keys in tiles of 32 with an online softmax: a
// lane per key for the scores, a lane per dim for the weighted sum.
#include <math.h>

#include "common.cuh"
#include "paged_rows.cuh"
#include "target_ops.h"

namespace dflash {
namespace {

constexpr int KT = 32, THREADS = 128, MAX_SMEM = 200 * 1024;

template <typename T, int D>
__global__ void __launch_bounds__(THREADS) paged_simt_kernel(const __grid_constant__ PagedAttnParams p) {
  pdl_wait();
  const int t = blockIdx.x, g = blockIdx.y, tid = threadIdx.x;
  const int warp = tid >> 5, lane = tid & 31;
  const int G = p.H / p.KVH;
  const PagedRows &r = p.rows;
  extern __shared__ float sm[];
  float *Ks = sm;                    // [KT][D + 1]
  float *Vs = Ks + KT * (D + 1);     // [KT][D]
  float *Qs = Vs + KT * D;           // [G][D]
  float *Os = Qs + G * D;            // [G][D]
  float *ms = Os + G * D, *ls = ms + G;
  __shared__ RowOwner s_owner;
  if (!owner_of_row(r, t, p.err, &s_owner)) return;
  const int b = s_owner.b, kv = s_owner.kv, a = s_owner.start, n = r.row_start[b + 1] - a;
  if (kv < r.prefix_len ||
      (int64_t)kv + n - r.prefix_len > (int64_t)r.pages_per_req * kPageRows) {
    if (tid == 0) raise_error(p.err, DFLASH_DERR_KV_CAPACITY);
    return;
  }
  const int keys = p.causal ? kv + (t - a) + 1 : kv + n;
  const T *q = (const T *)p.q + (int64_t)t * p.q_stride + (int64_t)g * G * D;
  for (int i = tid; i < G * D; i += THREADS) {
    Qs[i] = to_f32(q[i]) * p.scale;
    Os[i] = 0.f;
  }
  for (int j = tid; j < G; j += THREADS) {
    ms[j] = -INFINITY;
    ls[j] = 0.f;
  }
  for (int k0 = 0; k0 < keys; k0 += KT) {
    __syncthreads();
    for (int i = tid; i < KT * D; i += THREADS) {
      const int k = i / D, d = i % D, pos = k0 + k;
      float kk = 0.f, vv = 0.f;
      if (pos < keys) {
        int page = pos < r.prefix_len
                       ? r.prefix_pages[pos / kPageRows]
                       : r.page_table[(int64_t)b * r.pages_per_req + (pos - r.prefix_len) / kPageRows];
        if (page < 0 || page >= r.n_pages) {
          if (d == 0) raise_error(p.err, DFLASH_DERR_PAGE_RANGE);
          page = 0;
        }
        const int64_t at = (((int64_t)page * kPageRows + pos % kPageRows) * p.KVH + g) * D + d;
        kk = to_f32(((const T *)p.k_pages)[at]);
        vv = to_f32(((const T *)p.v_pages)[at]);
      }
      Ks[k * (D + 1) + d] = kk;
      Vs[i] = vv;
    }
    __syncthreads();
    const int live = min(KT, keys - k0);
    for (int j = warp; j < G; j += THREADS / 32) {
      float s = 0.f;
#pragma unroll 8
      for (int d = 0; d < D; ++d) s = fmaf(Qs[j * D + d], Ks[lane * (D + 1) + d], s);
      if (lane >= live) s = -INFINITY;
      const float m_old = ms[j], m = fmaxf(m_old, warp_max(s));
      // where every score so far is -infinity there is nothing to rescale
      const float base = m == -INFINITY ? 0.f : m;
      const float w = expf(s - base), alpha = expf(m_old - base);
      const float l = ls[j] * alpha + warp_sum(w);
      float o[D / 32];
#pragma unroll
      for (int c = 0; c < D / 32; ++c) o[c] = Os[j * D + c * 32 + lane] * alpha;
      for (int k = 0; k < live; ++k) {
        const float wk = __shfl_sync(0xffffffffu, w, k);
#pragma unroll
        for (int c = 0; c < D / 32; ++c) o[c] = fmaf(wk, Vs[k * D + c * 32 + lane], o[c]);
      }
#pragma unroll
      for (int c = 0; c < D / 32; ++c) Os[j * D + c * 32 + lane] = o[c];
      __syncwarp();   // every lane has read m and l of this row
      if (lane == 0) {
        ms[j] = m;
        ls[j] = l;
      }
      __syncwarp();
    }
  }
  __syncthreads();
  T *out = (T *)p.out + (int64_t)t * p.out_stride + (int64_t)g * G * D;
  for (int i = tid; i < G * D; i += THREADS) out[i] = from_f32<T>(Os[i] / ls[i / D]);
}

template <typename T, int D> cudaError_t launch(const PagedAttnParams &p, cudaStream_t s) {
  const int G = p.H / p.KVH;
  const size_t smem = sizeof(float) * (KT * (D + 1) + KT * D + 2 * (size_t)G * D + 2 * G);
  return launch_pdl(paged_simt_kernel<T, D>, dim3(p.rows.total_rows, p.KVH), dim3(THREADS), smem, s, p);
}
template <typename T, int D> cudaError_t prepare() {
  return cudaFuncSetAttribute(paged_simt_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              MAX_SMEM);
}

}  // namespace

cudaError_t launch_paged_attention_simt(const PagedAttnParams &p, cudaStream_t s) {
  return p.D == 64 ? launch<float, 64>(p, s) : launch<float, 128>(p, s);
}

cudaError_t prepare_paged_attention_simt() {
  const cudaError_t e = prepare<float, 64>();
  return e == cudaSuccess ? prepare<float, 128>() : e;
}

}  // namespace dflash

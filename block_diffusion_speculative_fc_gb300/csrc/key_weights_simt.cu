// Attention weight that falls on every row of a paged fp32 cache, on the CUDA cores:
// w[p] = decay w[p] + sum_r row_weight exp(scale q_r . K_p - lse_r) over the query rows
// r = (token, head of the group) that see key p.
//
// A CTA holds 64 keys of a (request, KV head) and takes its query rows 64 at a time,
// a thread 4 keys by 4 rows of a block's scores: fp32 arithmetic and the shared-memory
// reads that feed it bound it.  A key's sum stays in the CTA: fixed order, no atomics.
#include "common.cuh"
#include "target_ops.h"

namespace dflash {
namespace {

constexpr int KT = 64, RT = 64, THREADS = 256;

template <int D>
__global__ void __launch_bounds__(THREADS) key_weights_simt_kernel(const __grid_constant__ KeyWeightParams p) {
  constexpr int LD = D + 4, C4 = D / 4;
  extern __shared__ __align__(16) float sm[];
  float *s_k = sm, *s_q = s_k + KT * LD, *s_lse = s_q + RT * LD, *s_w = s_lse + RT;   // [KT][LD], [RT][LD], [RT], [RT]
  const int b = blockIdx.z, g = blockIdx.y, k0 = blockIdx.x * KT, tid = threadIdx.x;
  const int tx = tid & 15, ty = tid >> 4, G = p.H / p.KVH;
  const PagedRows &r = p.rows;
  const bool first = blockIdx.x == 0 && g == 0 && tid == 0;
  pdl_wait();
  const int start = r.row_start[b], end = r.row_start[b + 1], kv = r.kv_len[b];
  if (start < 0 || start > end || end > r.total_rows) {
    if (first) raise_error(p.err, DFLASH_DERR_ROW_RANGE);
    return;
  }
  const int n = end - start;
  if (n == 0) return;
  const int64_t own = (int64_t)kv + n - r.prefix_len;
  if (kv < r.prefix_len || own > (int64_t)r.pages_per_req * kPageRows || own > p.width) {
    if (first) raise_error(p.err, DFLASH_DERR_KV_CAPACITY);
    return;
  }
  if (p.mask && n > 32 * p.mask_words) {
    if (first) raise_error(p.err, DFLASH_DERR_TREE);
    return;
  }
  const int ctx = kv - r.prefix_len, keys = (int)own;
  if (k0 >= keys) return;
  int page = r.page_table[(int64_t)b * r.pages_per_req + k0 / kPageRows];   // a tile is a page
  if (page < 0 || page >= r.n_pages) {
    if (tid == 0) raise_error(p.err, DFLASH_DERR_PAGE_RANGE);
    page = 0;
  }
  for (int i = tid; i < KT * C4; i += THREADS) {
    const int k = i / C4, c = i % C4;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (k0 + k < keys)
      x = reinterpret_cast<const float4 *>(p.k_pages)[(((int64_t)page * kPageRows + k) * p.KVH + g) * C4 + c];
    *reinterpret_cast<float4 *>(s_k + k * LD + 4 * c) = x;
  }
  float sum[4] = {0.f, 0.f, 0.f, 0.f};
  // rows that see none of these keys are passed over
  const int rows = n * G, skip = p.mask || k0 < ctx ? 0 : (k0 - ctx) * G / RT * RT;
  for (int r0 = skip; r0 < rows; r0 += RT) {
    __syncthreads();
    for (int i = tid; i < RT * C4; i += THREADS) {
      const int q = i / C4, c = i % C4, row = r0 + q;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      if (row < rows)
        x = *(reinterpret_cast<const float4 *>((const float *)p.q + (int64_t)(start + row / G) * p.q_stride +
                                               (int64_t)(g * G + row % G) * D) + c);
      *reinterpret_cast<float4 *>(s_q + q * LD + 4 * c) = x;
    }
    if (tid < RT) {
      const int row = r0 + tid, tok = start + row / G;
      float l = 0.f, w = 0.f;
      if (row < rows) {
        l = p.lse[(int64_t)tok * p.H + g * G + row % G];
        w = p.row_weight ? p.row_weight[tok] : 1.f;
        if (!isfinite(l) || !(w > 0.f) || !isfinite(w)) w = 0.f;
      }
      s_lse[tid] = l;
      s_w[tid] = w;
    }
    __syncthreads();
    float s[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
#pragma unroll 4
    for (int c = 0; c < C4; ++c) {
      float4 k[4], q[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        k[i] = *reinterpret_cast<const float4 *>(s_k + (ty + 16 * i) * LD + 4 * c);
        q[i] = *reinterpret_cast<const float4 *>(s_q + (tx + 16 * i) * LD + 4 * c);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          s[i][j] = fmaf(k[i].w, q[j].w, fmaf(k[i].z, q[j].z, fmaf(k[i].y, q[j].y, fmaf(k[i].x, q[j].x, s[i][j]))));
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int row = tx + 16 * j, tok = (r0 + row) / G;
      const float l = s_lse[row], w = s_w[row];
      if (w == 0.f) continue;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int num = k0 + ty + 16 * i - ctx;        // among the new rows
        bool sees = num < 0 || (!p.mask && num <= tok);
        if (p.mask && num >= 0 && num < n)
          sees = p.mask[(int64_t)(start + tok) * p.mask_words + (num >> 5)] >> (num & 31) & 1u;
        if (sees) sum[i] = fmaf(w, expf(fmaf(s[i][j], p.scale, -l)), sum[i]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], o);
    const int key = k0 + ty + 16 * i;
    if (tx == 0 && key < keys) {
      float *out = p.weights + ((int64_t)b * p.KVH + g) * p.width + key;
      const float old = key < ctx && p.decay != 0.f ? *out : 0.f;
      *out = old * p.decay + sum[i];
    }
  }
}

template <int D> size_t smem() { return sizeof(float) * ((KT + RT) * (D + 4) + 2 * RT); }

template <int D> cudaError_t launch(const KeyWeightParams &p, cudaStream_t s) {
  const int64_t most = std::min<int64_t>(p.width, (int64_t)p.rows.pages_per_req * kPageRows);
  const dim3 grid((unsigned)((most + KT - 1) / KT), p.KVH, p.rows.B);
  return launch_pdl(key_weights_simt_kernel<D>, grid, dim3(THREADS), smem<D>(), s, p);
}

}  // namespace

cudaError_t launch_key_weights_simt(const KeyWeightParams &p, cudaStream_t s) {
  return p.D == 64 ? launch<64>(p, s) : launch<128>(p, s);
}

cudaError_t prepare_key_weights_simt() {
  const cudaError_t e = cudaFuncSetAttribute(key_weights_simt_kernel<64>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem<64>());
  return e == cudaSuccess ? cudaFuncSetAttribute(key_weights_simt_kernel<128>,
                                                 cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem<128>())
                          : e;
}

}  // namespace dflash

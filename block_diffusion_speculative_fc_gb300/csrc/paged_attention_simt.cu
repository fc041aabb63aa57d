// Attention of new rows over a paged fp32 cache, on the CUDA cores (the tensor
// cores have no exact-fp32 kind), with a running softmax over tiles of 32 keys.
//
// A CTA holds up to 64 query rows of one KV head: `tokens` consecutive tokens
// times up to 64 heads of the group, each warp RPW of them.  Scores: a lane a
// key, the query rows broadcast; weighted sum: a lane D/32 dims, the weights
// broadcast; both sides of either product come from shared memory as 16-byte
// reads that RPW rows share, so fp32 arithmetic and those reads bound it.  K/V
// rows are staged once for all of a CTA's rows.  Where that makes few CTAs, a
// cluster of them splits the keys and joins its (max, sum, weighted sum)
// through distributed shared memory in rank order.
//
// Measured (inputs beyond L2): 8 requests x 16 rows of 32 heads over 2064 keys
// of 8 heads 235 us (18 TFLOP/s); one token over 1001 keys 24 us; 64 tokens over
// 2001 keys each 350 us.
//
// Tokens of one CTA that belong to different requests are taken in turn, so a
// CTA has no more tokens than requests have on average.
#include <cooperative_groups.h>
#include <math.h>

#include <algorithm>

#include "common.cuh"
#include "target_ops.h"

namespace dflash {
namespace {

namespace cg = cooperative_groups;

constexpr int KT = 32, WARPS = 8, THREADS = 32 * WARPS, MAX_TOKENS = 16, MAX_ROWS = 64, MAXC = 8;

struct Split {
  int tokens, heads, blocks;   // of a CTA; blocks of heads in a group
};

template <int D, int RPW>
__global__ void __launch_bounds__(THREADS) paged_simt_kernel(const __grid_constant__ PagedAttnParams p,
                                                             const Split split) {
  constexpr int QR = WARPS * RPW, KS = D + 4, PS = KT + 4, C4 = D / 4, V = D / 32;
  extern __shared__ __align__(16) float sm[];
  float *Ks = sm;                    // [KT][KS]
  float *Vs = Ks + KT * KS;          // [KT][D]
  float *Qs = Vs + KT * D;           // [QR][D]: queries, then the weighted sums to be joined
  float *Ps = Qs + QR * D;           // [QR][PS]
  __shared__ int s_owner[MAX_TOKENS], s_owners[MAX_TOKENS];
  __shared__ float s_m[QR], s_l[QR];
  unsigned &s_claimed = *reinterpret_cast<unsigned *>(Ps);   // rows of all ranges, until the first weights
  cg::cluster_group cl = cg::this_cluster();
  const int C = (int)cl.num_blocks(), rank = (int)cl.block_rank();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int t0 = (int)(blockIdx.x / C) * split.tokens, g = blockIdx.y / split.blocks;
  const int G = p.H / p.KVH, h0 = blockIdx.y % split.blocks * split.heads, hn = min(split.heads, G - h0);
  const PagedRows &r = p.rows;
  pdl_wait();
  if (tid < MAX_TOKENS) s_owners[tid] = 0;
  if (tid == 0) s_claimed = 0;
  __syncthreads();
  unsigned claimed = 0;              // up to one more than there are (at most 2^28)
  const unsigned over = (unsigned)r.total_rows + 1;
  for (int i = tid; i < r.B; i += THREADS) {
    const int a = r.row_start[i], e = r.row_start[i + 1];
    if (a < 0 || a > e || e > r.total_rows) {
      if (t0 == 0) raise_error(p.err, DFLASH_DERR_ROW_RANGE);
      continue;
    }
    claimed = min(claimed + (unsigned)(e - a), over);
    for (int t = max(a, t0); t < min(e, t0 + split.tokens); ++t) {
      s_owner[t - t0] = i;
      atomicAdd(&s_owners[t - t0], 1);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) claimed = min(claimed + __shfl_xor_sync(0xffffffffu, claimed, o), over);
  if (lane == 0 && claimed) atomicAdd(&s_claimed, claimed);
  __syncthreads();
  if (tid < split.tokens && s_owners[tid] > 1) raise_error(p.err, DFLASH_DERR_ROW_RANGE);
  if (s_claimed >= over) {           // every CTA finds the same, and none writes
    if (tid == 0) raise_error(p.err, DFLASH_DERR_ROW_RANGE);
    return;
  }

  for (int first = 0, next; first < split.tokens; first = next) {
    next = first + 1;
    if (s_owners[first] != 1) continue;
    const int b = s_owner[first];
    while (next < split.tokens && s_owners[next] == 1 && s_owner[next] == b) ++next;
    const int a = r.row_start[b], n = r.row_start[b + 1] - a, kv = r.kv_len[b];
    if (kv < r.prefix_len || (int64_t)kv + n - r.prefix_len > (int64_t)r.pages_per_req * kPageRows) {
      if (tid == 0) raise_error(p.err, DFLASH_DERR_KV_CAPACITY);
      continue;
    }
    const int rows = (next - first) * hn, tok = t0 + first;   // query row i: token tok + i / hn
    const int low = p.causal ? kv + (tok - a) + 1 : kv + n;   // keys that the first token sees
    const int keys = p.causal ? low + (next - first) - 1 : low;
    for (int i = tid; i < rows * C4; i += THREADS) {
      const int q = i / C4;
      const float4 x = *(reinterpret_cast<const float4 *>((const float *)p.q + (int64_t)(tok + q / hn) * p.q_stride +
                                                          (int64_t)(g * G + h0 + q % hn) * D) + i % C4);
      reinterpret_cast<float4 *>(Qs)[i] = make_float4(x.x * p.scale, x.y * p.scale, x.z * p.scale, x.w * p.scale);
    }
    float m[RPW], l[RPW], o[RPW][V];
    int lim[RPW];                    // keys that the row sees
#pragma unroll
    for (int i = 0; i < RPW; ++i) {
      m[i] = -INFINITY;
      l[i] = 0.f;
      lim[i] = p.causal ? low + (warp + WARPS * i) / hn : low;
#pragma unroll
      for (int c = 0; c < V; ++c) o[i][c] = 0.f;
    }
    for (int k0 = KT * rank; k0 < keys; k0 += KT * C) {
      __syncthreads();
#pragma unroll
      for (int i = tid; i < KT * C4; i += THREADS) {
        const int k = i / C4, c = i % C4, pos = k0 + k;
        float4 kk = make_float4(0.f, 0.f, 0.f, 0.f), vv = kk;
        if (pos < keys) {
          int page = pos < r.prefix_len
                         ? r.prefix_pages[pos / kPageRows]
                         : r.page_table[(int64_t)b * r.pages_per_req + (pos - r.prefix_len) / kPageRows];
          if (page < 0 || page >= r.n_pages) {
            if (c == 0) raise_error(p.err, DFLASH_DERR_PAGE_RANGE);
            page = 0;
          }
          const int64_t at = (((int64_t)page * kPageRows + pos % kPageRows) * p.KVH + g) * C4 + c;
          kk = reinterpret_cast<const float4 *>(p.k_pages)[at];
          vv = reinterpret_cast<const float4 *>(p.v_pages)[at];
        }
        *reinterpret_cast<float4 *>(Ks + k * KS + 4 * c) = kk;
        reinterpret_cast<float4 *>(Vs)[i] = vv;
      }
      __syncthreads();
      if (warp >= rows) continue;
      float s[RPW];
#pragma unroll
      for (int i = 0; i < RPW; ++i) s[i] = 0.f;
#pragma unroll 4
      for (int c = 0; c < C4; ++c) {
        const float4 kk = *reinterpret_cast<const float4 *>(Ks + lane * KS + 4 * c);
#pragma unroll
        for (int i = 0; i < RPW; ++i) {
          const float4 q = reinterpret_cast<const float4 *>(Qs + (warp + WARPS * i) * D)[c];
          s[i] = fmaf(q.x, kk.x, s[i]);
          s[i] = fmaf(q.y, kk.y, s[i]);
          s[i] = fmaf(q.z, kk.z, s[i]);
          s[i] = fmaf(q.w, kk.w, s[i]);
        }
      }
#pragma unroll
      for (int i = 0; i < RPW; ++i) {
        const float x = k0 + lane < lim[i] ? s[i] : -INFINITY;
        const float mx = fmaxf(m[i], warp_max(x));
        // where every score so far is -infinity there is nothing to rescale
        const float base = mx == -INFINITY ? 0.f : mx;
        const float w = expf(x - base), alpha = expf(m[i] - base);
        l[i] = l[i] * alpha + warp_sum(w);
        m[i] = mx;
#pragma unroll
        for (int c = 0; c < V; ++c) o[i][c] *= alpha;
        Ps[(warp + WARPS * i) * PS + lane] = w;
      }
      __syncwarp();
      auto value = [&](int k, float *v) {
        if (V == 4) *reinterpret_cast<float4 *>(v) = *reinterpret_cast<const float4 *>(Vs + k * D + 4 * lane);
        else *reinterpret_cast<float2 *>(v) = *reinterpret_cast<const float2 *>(Vs + k * D + 2 * lane);
      };
      if (k0 + KT <= low) {
#pragma unroll 2
        for (int k = 0; k < KT; k += 4) {
          __align__(16) float v[4][V];
#pragma unroll
          for (int j = 0; j < 4; ++j) value(k + j, v[j]);
#pragma unroll
          for (int i = 0; i < RPW; ++i) {
            const float4 w = *reinterpret_cast<const float4 *>(Ps + (warp + WARPS * i) * PS + k);
#pragma unroll
            for (int c = 0; c < V; ++c)
              o[i][c] = fmaf(w.w, v[3][c], fmaf(w.z, v[2][c], fmaf(w.y, v[1][c], fmaf(w.x, v[0][c], o[i][c]))));
          }
        }
      } else {                       // a key that a row does not see may hold anything
#pragma unroll
        for (int i = 0; i < RPW; ++i)
          for (int k = 0; k < min(KT, lim[i] - k0); ++k) {
            __align__(16) float v[V];
            value(k, v);
            const float w = Ps[(warp + WARPS * i) * PS + k];
#pragma unroll
            for (int c = 0; c < V; ++c) o[i][c] = fmaf(w, v[c], o[i][c]);
          }
      }
    }
    auto store = [&](int q, const float *x) {
      float *out = (float *)p.out + (int64_t)(tok + q / hn) * p.out_stride + (int64_t)(g * G + h0 + q % hn) * D;
      if (V == 4) reinterpret_cast<float4 *>(out)[lane] = *reinterpret_cast<const float4 *>(x);
      else reinterpret_cast<float2 *>(out)[lane] = *reinterpret_cast<const float2 *>(x);
    };
    __syncthreads();                 // the queries have been read
    if (C == 1) {
#pragma unroll
      for (int i = 0; i < RPW; ++i) {
        __align__(16) float x[V];
#pragma unroll
        for (int c = 0; c < V; ++c) x[c] = o[i][c] / l[i];
        if (warp + WARPS * i < rows) store(warp + WARPS * i, x);
      }
      continue;
    }
#pragma unroll
    for (int i = 0; i < RPW; ++i) {
      const int q = warp + WARPS * i;
#pragma unroll
      for (int c = 0; c < V; ++c) Qs[q * D + V * lane + c] = o[i][c];
      if (lane == 0) {
        s_m[q] = m[i];
        s_l[q] = l[i];
      }
    }
    cl.sync();
    for (int q = rank + C * warp; q < rows; q += C * WARPS) {
      float mx = -INFINITY, sum = 0.f;
      __align__(16) float x[V];
#pragma unroll
      for (int c = 0; c < V; ++c) x[c] = 0.f;
      for (int k = 0; k < C; ++k) mx = fmaxf(mx, *cl.map_shared_rank(&s_m[q], k));
      const float base = mx == -INFINITY ? 0.f : mx;
      for (int k = 0; k < C; ++k) {
        const float f = expf(*cl.map_shared_rank(&s_m[q], k) - base);
        const float lk = *cl.map_shared_rank(&s_l[q], k);
        const float *ok = cl.map_shared_rank(Qs + q * D + V * lane, k);
        if (lk == 0.f) continue;     // a rank whose keys the row does not see
        sum = fmaf(f, lk, sum);
#pragma unroll
        for (int c = 0; c < V; ++c) x[c] = fmaf(f, ok[c], x[c]);
      }
#pragma unroll
      for (int c = 0; c < V; ++c) x[c] /= sum;
      store(q, x);
    }
    cl.sync();                       // read by every rank before the next tokens' queries come
  }
}

template <int D, int RPW> size_t smem() {
  return sizeof(float) * (KT * (D + 4) + KT * D + WARPS * RPW * (D + KT + 4));
}

template <int D, int RPW>
cudaError_t launch(const PagedAttnParams &p, const Split &split, int sms, cudaStream_t s) {
  const int64_t tiles = (p.rows.total_rows + split.tokens - 1) / split.tokens;
  const int64_t ctas = tiles * p.KVH * split.blocks;
  // Keys split while the CTAs are fewer than two an SM: one token over 1001 keys 24 us against 134
  // unsplit, 8 x 16 rows over 2064 keys 235 against 508.  (Up to four an SM: 32 x 16 rows 1212 us
  // against 1377, but 64 single tokens 380 against 351.)
  int C = 1;
  while (C < MAXC && ctas * C < 2 * sms) C *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = smem<D, RPW>();
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = C;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  cfg.gridDim = dim3((unsigned)(tiles * C), (unsigned)(p.KVH * split.blocks));
  return cudaLaunchKernelEx(&cfg, paged_simt_kernel<D, RPW>, p, split);
}

template <int D> cudaError_t launch(const PagedAttnParams &p, cudaStream_t s) {
  int dev = 0, sms = 0;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  const int G = p.H / p.KVH;
  Split split;
  split.heads = std::min(G, MAX_ROWS);
  split.blocks = (G + split.heads - 1) / split.heads;
  // (a token a CTA stages every key once a token: 8 x 16 rows 623 us against 235, 2000 rows of one
  // prompt 3546 against 1442)
  split.tokens = 1;
  while (split.tokens < MAX_TOKENS && 2 * split.tokens * split.heads <= MAX_ROWS &&
         2LL * split.tokens * p.rows.B <= p.rows.total_rows)
    split.tokens *= 2;
  const int rows = split.tokens * split.heads;
  if (rows <= WARPS) return launch<D, 1>(p, split, sms, s);
  if (rows <= 2 * WARPS) return launch<D, 2>(p, split, sms, s);
  if (rows <= 4 * WARPS) return launch<D, 4>(p, split, sms, s);
  return launch<D, 8>(p, split, sms, s);
}
template <int D, int RPW> cudaError_t prepare() {
  return cudaFuncSetAttribute(paged_simt_kernel<D, RPW>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              (int)smem<D, RPW>());
}
template <int D> cudaError_t prepare() {
  cudaError_t e = prepare<D, 1>();
  if (e == cudaSuccess) e = prepare<D, 2>();
  if (e == cudaSuccess) e = prepare<D, 4>();
  return e == cudaSuccess ? prepare<D, 8>() : e;
}

}  // namespace

cudaError_t launch_paged_attention_simt(const PagedAttnParams &p, cudaStream_t s) {
  return p.D == 64 ? launch<64>(p, s) : launch<128>(p, s);
}

cudaError_t prepare_paged_attention_simt() {
  const cudaError_t e = prepare<64>();
  return e == cudaSuccess ? prepare<128>() : e;
}

}  // namespace dflash

// Head norms, rotary positions and the append of new K/V rows to a paged
// cache, in one pass over the projected rows.
//
// Per token and head: y = R(p f) (x / sqrt(mean x^2 + eps) * g) for queries
// and keys, R the rotation of the pairs (i, i + rd/2) or (2i, 2i + 1) by the
// angle of position p; values are copied.  Each element is read once and
// written once and costs about ten operations, so HBM bounds it.
//
// Angles.  A frequency is held as its turns per position times 2^64; position
// times that, in 64-bit arithmetic, wraps modulo one turn, so its high word is
// the reduced angle for any position (2^-32 turn) without a table or a
// floating-point reduction.  sin and cos are formed once per token and pair
// (rd/2 calls of sincospif) and shared by its heads through shared memory.
//
// One CTA per token; 16 bytes per thread and chunk, the 16-byte chunks of a
// head in consecutive lanes: the mean square is a shuffle reduction over those
// lanes, and the rotation partner rd/2 dims away sits in the same slot of
// another lane (through shared memory where rd/2 is not a multiple of the
// chunk).  A thread's first kU chunks are in flight before the CTA looks up
// its request, position and page (three dependent loads).
#include "common.cuh"
#include "paged_rows.cuh"
#include "target_ops.h"

namespace dflash {
namespace {

constexpr int kU = 4;

template <typename T> struct Chunk;
template <> struct Chunk<bf16> {
  static constexpr int E = 8;
  static __device__ __forceinline__ void unpack(const uint4 &u, float *x) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ uint4 pack(const float *x) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<uint32_t *>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <> struct Chunk<float> {
  static constexpr int E = 4;
  static __device__ __forceinline__ void unpack(const uint4 &u, float *x) {
    x[0] = __uint_as_float(u.x);
    x[1] = __uint_as_float(u.y);
    x[2] = __uint_as_float(u.z);
    x[3] = __uint_as_float(u.w);
  }
  static __device__ __forceinline__ uint4 pack(const float *x) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                      __float_as_uint(x[3]));
  }
};

// LPR lanes per head row; D = LPR * E.
template <typename T, int LPR>
__global__ void __launch_bounds__(256) append_kv_kernel(const __grid_constant__ AppendParams p) {
  constexpr int E = Chunk<T>::E, D = LPR * E;
  __shared__ float2 s_cs[64];
  __shared__ int s_b;
  extern __shared__ float s_x[];   // [threads][E], rotations across chunk borders only
  pdl_wait();
  const int t = blockIdx.x, tid = threadIdx.x, nt = blockDim.x;
  const int lane = tid & (LPR - 1);
  const int chunks = (p.H + 2 * p.KVH) * LPR;
  // chunk c: head c / LPR of [q heads | k heads | v heads]
  auto source = [&](int c) -> const uint4 * {
    const int head = c / LPR;
    const T *row;
    if (head < p.H) row = (const T *)p.q + (int64_t)t * p.q_stride + head * D;
    else if (head < p.H + p.KVH) row = (const T *)p.k + (int64_t)t * p.k_stride + (head - p.H) * D;
    else row = (const T *)p.v + (int64_t)t * p.v_stride + (head - p.H - p.KVH) * D;
    return reinterpret_cast<const uint4 *>(row) + lane;
  };
  uint4 raw[kU];
#pragma unroll
  for (int u = 0; u < kU; ++u)
    if (tid + u * nt < chunks) raw[u] = *source(tid + u * nt);

  const PagedRows &r = p.rows;
  const int b = owner_of_row(r, t, p.err, &s_b);
  if (b < 0) return;
  const int kv = r.kv_len[b];
  const int64_t pos64 = (int64_t)kv + (t - r.row_start[b]);
  if (kv < r.prefix_len || pos64 - r.prefix_len >= (int64_t)r.pages_per_req * kPageRows) {
    if (tid == 0) raise_error(p.err, DFLASH_DERR_KV_CAPACITY);
    return;
  }
  const int pos = (int)pos64, own = pos - r.prefix_len;
  const int page = r.page_table[(int64_t)b * r.pages_per_req + own / kPageRows];
  if (page < 0 || page >= r.n_pages) {
    if (tid == 0) raise_error(p.err, DFLASH_DERR_PAGE_RANGE);
    return;
  }
  const int half = p.rot >> 1;
  for (int i = tid; i < half; i += nt) {
    const unsigned long long turn = (unsigned long long)pos * p.turns[i];
    float sn, cs;   // of pi * x, x in [-1, 1): half turns
    sincospif((float)(int)(turn >> 32) * 0x1p-31f, &sn, &cs);
    s_cs[i] = make_float2(cs * p.amp, sn * p.amp);
  }
  __syncthreads();

  const int64_t slot = (int64_t)page * kPageRows + own % kPageRows;
  const bool shuffled = !p.inter && half % E == 0;
  for (int c0 = 0; c0 < chunks; c0 += kU * nt) {
    if (c0 > 0) {
#pragma unroll
      for (int u = 0; u < kU; ++u)
        if (c0 + tid + u * nt < chunks) raw[u] = *source(c0 + tid + u * nt);
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int c = c0 + tid + u * nt;
      if (c0 + u * nt >= chunks) break;          // the whole CTA is past the end
      const int head = c / LPR;
      const bool live = c < chunks;
      const bool is_q = head < p.H, is_v = head >= p.H + p.KVH;
      uint4 res = raw[u];
      // heads differ within a warp: every lane takes part in the exchanges
      float x[E];
      Chunk<T>::unpack(live ? raw[u] : make_uint4(0, 0, 0, 0), x);
      const T *gain = (const T *)(is_q ? p.q_gain : p.k_gain);
      if (p.q_gain || p.k_gain) {
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o, LPR);
        if (gain && !is_v) {
          const float rs = rsqrtf(ss * (1.0f / D) + p.eps);
          float g[E];
          Chunk<T>::unpack(__ldg(reinterpret_cast<const uint4 *>(gain) + lane), g);
#pragma unroll
          for (int e = 0; e < E; ++e) x[e] = x[e] * rs * g[e];
        }
      }
      if (p.inter) {
#pragma unroll
        for (int e = 0; e < E; e += 2) {
          const int i = (lane * E + e) >> 1;
          if (i < half) {
            const float2 cs = s_cs[i];
            const float a = x[e], bb = x[e + 1];
            x[e] = a * cs.x - bb * cs.y;
            x[e + 1] = bb * cs.x + a * cs.y;
          }
        }
      } else if (shuffled) {
        const int hl = half / E;                 // lanes of half the rotated dims
        const bool lo = lane < hl, rotated = lane < 2 * hl;
        const int from = rotated ? (lo ? lane + hl : lane - hl) : lane;
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const float y = __shfl_sync(0xffffffffu, x[e], from, LPR);
          if (rotated) {
            const float2 cs = s_cs[(lo ? lane : lane - hl) * E + e];
            x[e] = lo ? x[e] * cs.x - y * cs.y : x[e] * cs.x + y * cs.y;
          }
        }
      } else {
        float *row = s_x + (tid - lane) * E;     // this head's D values
#pragma unroll
        for (int e = 0; e < E; ++e) row[lane * E + e] = x[e];
        __syncwarp();
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const int d = lane * E + e;
          if (d < p.rot) {
            const bool lo = d < half;
            const float y = row[lo ? d + half : d - half];
            const float2 cs = s_cs[lo ? d : d - half];
            x[e] = lo ? x[e] * cs.x - y * cs.y : x[e] * cs.x + y * cs.y;
          }
        }
        __syncwarp();
      }
      if (!live) continue;
      if (!is_v) res = Chunk<T>::pack(x);
      T *dst;
      if (is_q) dst = (T *)p.q_out + (int64_t)t * p.q_out_stride + head * D;
      else if (!is_v) dst = (T *)p.k_pages + (slot * p.KVH + (head - p.H)) * D;
      else dst = (T *)p.v_pages + (slot * p.KVH + (head - p.H - p.KVH)) * D;
      *(reinterpret_cast<uint4 *>(dst) + lane) = res;
    }
  }
}

template <typename T, int LPR>
cudaError_t launch(const AppendParams &p, cudaStream_t s) {
  const int chunks = (p.H + 2 * p.KVH) * LPR;
  // kU chunks a thread and pass, in as few passes as 256 threads allow
  const int passes = (chunks + 256 * kU - 1) / (256 * kU);
  int nt = (chunks + passes * kU - 1) / (passes * kU);
  nt = (nt + 31) / 32 * 32;
  const bool across = !p.inter && (p.rot / 2) % Chunk<T>::E != 0;
  const size_t smem = across ? sizeof(float) * Chunk<T>::E * nt : 0;
  return launch_pdl(append_kv_kernel<T, LPR>, dim3(p.rows.total_rows), dim3(nt), smem, s, p);
}

}  // namespace

cudaError_t launch_append_kv(int dtype, int head_dim, const AppendParams &p, cudaStream_t s) {
  if (dtype == DFLASH_BF16)
    return head_dim == 64 ? launch<bf16, 8>(p, s) : launch<bf16, 16>(p, s);
  return head_dim == 64 ? launch<float, 16>(p, s) : launch<float, 32>(p, s);
}

}  // namespace dflash

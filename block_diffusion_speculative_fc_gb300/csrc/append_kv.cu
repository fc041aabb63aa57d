// Head norms, rotary positions and the append of new K/V rows to a paged
// cache, in one pass over the projected rows.
//
// Measured: 16153 rows of 64 + 8 + 8 heads of 128 in bf16 109 us, 6.0 TB/s; 2048
// rows of 32 + 8 + 8 heads 16.6 us, 3.0 TB/s (three waves of CTAs, each a chain
// of loads); one row 3.3 us.
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
// One CTA per token.  A thread holds two 16-byte chunks of a head D/2 dims
// apart, the chunks of a head's half in consecutive lanes: the mean square is a
// shuffle reduction over those lanes, and where the rotation covers the whole
// head both sides of a pair are in one thread (in another lane where it covers
// at most half of the head; other halves go through shared memory).  A thread's sines and cosines serve all its heads and
// stay in registers.  With a chunk a thread and the pair's other side in another
// lane, shared-memory accesses and shuffles bound it instead of HBM: 2048 tokens
// of 32 + 8 + 8 heads of 128 took 24.0 us.  A thread's first kU units (pairs of
// chunks) are in flight before the CTA looks up its request, position and page
// (two dependent loads).
#include "common.cuh"
#include "paged_rows.cuh"
#include "target_ops.h"

namespace dflash {
namespace {

constexpr int kU = 2;   // units of a thread and pass

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

// pairs (2i, 2i+1); halves of the whole head; halves within a head's first half, of whole chunks;
// any other halves
enum Rotation { kInterleaved, kWholeHalves, kLowHalves, kPartHalves };

// L lanes per head; D = 2 L E.  AT: rotary positions are given.  (A branch instead of the parameter costs the call
// without them a twentieth: 2048 rows 16.5 -> 17.4 us.)
template <typename T, int L, int ROT, bool AT>
__global__ void __launch_bounds__(256) append_kv_kernel(const __grid_constant__ AppendParams p) {
  constexpr int E = Chunk<T>::E, D = 2 * L * E;
  __shared__ float2 s_cs[64];
  __shared__ RowOwner s_owner;
  __shared__ uint4 s_gain[2][2 * L];   // of queries, of keys
  extern __shared__ float s_x[];       // [2 E][threads]: kPartHalves only
  pdl_wait();
  const int t = blockIdx.x, tid = threadIdx.x, nt = blockDim.x;
  const int lane = tid & (L - 1);
  const int units = (p.H + 2 * p.KVH) * L;
  // unit c: chunks `lane` and L + `lane` of head c / L of [q heads | k heads | v heads]
  auto source = [&](int c) -> const uint4 * {
    const int head = c / L;
    const T *row;
    if (head < p.H) row = (const T *)p.q + (int64_t)t * p.q_stride + head * D;
    else if (head < p.H + p.KVH) row = (const T *)p.k + (int64_t)t * p.k_stride + (head - p.H) * D;
    else row = (const T *)p.v + (int64_t)t * p.v_stride + (head - p.H - p.KVH) * D;
    return reinterpret_cast<const uint4 *>(row) + lane;
  };
  uint4 raw[kU][2];
#pragma unroll
  for (int u = 0; u < kU; ++u)
    if (tid + u * nt < units) {
      const uint4 *src = source(tid + u * nt);
      raw[u][0] = src[0];
      raw[u][1] = src[L];
    }

  const PagedRows &r = p.rows;
  for (int i = tid; i < 4 * L; i += nt) {
    const uint4 *gain = (const uint4 *)(i < 2 * L ? p.q_gain : p.k_gain);
    if (gain) s_gain[i / (2 * L)][i % (2 * L)] = gain[i % (2 * L)];
  }
  if (!owner_of_row(r, t, p.err, &s_owner)) return;
  const int b = s_owner.b, kv = s_owner.kv;
  const int64_t pos64 = (int64_t)kv + (t - s_owner.start);
  if (kv < r.prefix_len || pos64 - r.prefix_len >= (int64_t)r.pages_per_req * kPageRows) {
    if (tid == 0) raise_error(p.err, DFLASH_DERR_KV_CAPACITY);
    return;
  }
  const int pos = (int)pos64, own = pos - r.prefix_len;
  const int page = r.page_table[(int64_t)b * r.pages_per_req + own / kPageRows];
  const int half = p.rot >> 1, at = AT ? p.positions[t] : pos;
  for (int i = tid; i < half; i += nt) {
    const unsigned long long turn = (unsigned long long)at * p.turns[i];
    float sn, cs;   // of pi * x, x in [-1, 1): half turns
    sincospif((float)(int)(turn >> 32) * 0x1p-31f, &sn, &cs);
    s_cs[i] = make_float2(cs * p.amp, sn * p.amp);
  }
  if (page < 0 || page >= r.n_pages) {
    if (tid == 0) raise_error(p.err, DFLASH_DERR_PAGE_RANGE);
    return;
  }
  __syncthreads();

  // the pairs of this thread's values
  const int hl = half / E;             // lanes of half the rotated dims (kLowHalves)
  const bool lo = lane < hl, rotated = lane < 2 * hl;
  float2 cs[E];
  if (ROT != kPartHalves) {
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int i = ROT == kWholeHalves ? lane * E + e
                    : ROT == kLowHalves ? (lo ? lane : lane - hl) * E + e
                                        : (e / (E / 2)) * (D / 4) + lane * (E / 2) + e % (E / 2);
      cs[e] = s_cs[i < half ? i : 0];
    }
  }
  const int64_t slot = (int64_t)page * kPageRows + own % kPageRows;
  for (int c0 = 0; c0 < units; c0 += kU * nt) {
    if (c0 > 0) {
#pragma unroll
      for (int u = 0; u < kU; ++u)
        if (c0 + tid + u * nt < units) {
          const uint4 *src = source(c0 + tid + u * nt);
          raw[u][0] = src[0];
          raw[u][1] = src[L];
        }
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int c = c0 + tid + u * nt;
      if (c0 + u * nt >= units) break;           // the whole CTA is past the end
      const int head = c / L;
      const bool live = c < units;
      const bool is_q = head < p.H, is_v = head >= p.H + p.KVH;
      // heads differ within a warp: every lane takes part in the exchanges
      const uint4 zero = make_uint4(0, 0, 0, 0);
      float x[2 * E];
      Chunk<T>::unpack(live ? raw[u][0] : zero, x);
      Chunk<T>::unpack(live ? raw[u][1] : zero, x + E);
      if (p.q_gain || p.k_gain) {
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < 2 * E; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o, L);
        if ((is_q ? p.q_gain : p.k_gain) && !is_v) {
          const float rs = rsqrtf(ss * (1.0f / D) + p.eps);
          float g[2 * E];
          Chunk<T>::unpack(s_gain[is_q ? 0 : 1][lane], g);
          Chunk<T>::unpack(s_gain[is_q ? 0 : 1][L + lane], g + E);
#pragma unroll
          for (int e = 0; e < 2 * E; ++e) x[e] = x[e] * rs * g[e];
        }
      }
      if (ROT == kInterleaved) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const int k = (e / (E / 2)) * E + 2 * (e % (E / 2));   // first side, in x
          const int i = (e / (E / 2)) * (D / 4) + lane * (E / 2) + e % (E / 2);
          if (i < half) {
            const float a = x[k], bb = x[k + 1];
            x[k] = a * cs[e].x - bb * cs[e].y;
            x[k + 1] = bb * cs[e].x + a * cs[e].y;
          }
        }
      } else if (ROT == kWholeHalves) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const float a = x[e], bb = x[E + e];
          x[e] = a * cs[e].x - bb * cs[e].y;
          x[E + e] = bb * cs[e].x + a * cs[e].y;
        }
      } else if (ROT == kLowHalves) {
        const int from = rotated ? (lo ? lane + hl : lane - hl) : lane;
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const float y = __shfl_sync(0xffffffffu, x[e], from, L);
          if (rotated) x[e] = lo ? x[e] * cs[e].x - y * cs[e].y : x[e] * cs[e].x + y * cs[e].y;
        }
      } else {
        // dim d of this head: side d / (D / 2), lane d / E % L, value d % E
        float *at = s_x + (tid - lane);
#pragma unroll
        for (int e = 0; e < 2 * E; ++e) at[e * nt + lane] = x[e];
        __syncwarp();
#pragma unroll
        for (int e = 0; e < 2 * E; ++e) {
          const int d = (e / E) * (D / 2) + lane * E + e % E;
          if (d < p.rot) {
            const bool lo = d < half;
            const int o = lo ? d + half : d - half;
            const float y = at[((o / (D / 2)) * E + o % E) * nt + o / E % L];
            const float2 w = s_cs[lo ? d : d - half];
            x[e] = lo ? x[e] * w.x - y * w.y : x[e] * w.x + y * w.y;
          }
        }
        __syncwarp();
      }
      if (!live) continue;
      T *dst;
      if (is_q) dst = (T *)p.q_out + (int64_t)t * p.q_out_stride + head * D;
      else if (!is_v) dst = (T *)p.k_pages + (slot * p.KVH + (head - p.H)) * D;
      else dst = (T *)p.v_pages + (slot * p.KVH + (head - p.H - p.KVH)) * D;
      uint4 *to = reinterpret_cast<uint4 *>(dst) + lane;
      to[0] = is_v ? raw[u][0] : Chunk<T>::pack(x);
      to[L] = is_v ? raw[u][1] : Chunk<T>::pack(x + E);
    }
  }
}

template <typename T, int L, bool AT>
cudaError_t launch(const AppendParams &p, cudaStream_t s) {
  constexpr int E = Chunk<T>::E, D = 2 * L * E;
  const int units = (p.H + 2 * p.KVH) * L;
  // kU units a thread and pass, in as few passes as 256 threads allow
  const int passes = (units + 256 * kU - 1) / (256 * kU);
  int nt = (units + passes * kU - 1) / (passes * kU);
  nt = (nt + 31) / 32 * 32;
  const dim3 grid(p.rows.total_rows), block(nt);
  if (p.inter || p.rot == 0) return launch_pdl(append_kv_kernel<T, L, kInterleaved, AT>, grid, block, 0, s, p);
  if (p.rot == D) return launch_pdl(append_kv_kernel<T, L, kWholeHalves, AT>, grid, block, 0, s, p);
  if (p.rot <= D / 2 && p.rot / 2 % E == 0)
    return launch_pdl(append_kv_kernel<T, L, kLowHalves, AT>, grid, block, 0, s, p);
  return launch_pdl(append_kv_kernel<T, L, kPartHalves, AT>, grid, block, sizeof(float) * 2 * E * nt, s, p);
}
template <typename T, int L> cudaError_t launch(const AppendParams &p, cudaStream_t s) {
  return p.positions ? launch<T, L, true>(p, s) : launch<T, L, false>(p, s);
}

}  // namespace

cudaError_t launch_append_kv(int dtype, int head_dim, const AppendParams &p, cudaStream_t s) {
  if (dtype == DFLASH_BF16)
    return head_dim == 64 ? launch<bf16, 4>(p, s) : launch<bf16, 8>(p, s);
  return head_dim == 64 ? launch<float, 8>(p, s) : launch<float, 16>(p, s);
}

}  // namespace dflash

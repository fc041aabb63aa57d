// Attention weight that falls on every row of a paged bf16 cache, on the tensor
// cores (tcgen05 + TMEM).
//
// w[p] = decay w[p] + sum_r 2^(c s[p, r] + z[r]), s = K Q^T, c = scale log2 e, over
// the query rows r = (token, head of the group) of a request that see key p; z[r]
// = log2(row_weight) - lse log2 e is known before, so keys need no second look.  A
// key tile (128 keys, two pages) is the product's A operand and up to 128 query
// rows its B operand: a TMEM lane is a key, and the sum over its columns stays
// in one thread, without exchange or atomics; every key has one CTA and one
// thread, so sums are in a fixed order.
//
// Few rows (decoding): HBM bounds it, K is read once and V not at all.  Many rows:
// an exponential per key and row bounds it (MUFU); the product of a 128 x 128 tile
// takes half of its exponentials' time.  Rows beyond 256 of a request and KV head
// are further passes over the CTA's keys.
//
// Every CTA lays out the same plan from the requests' lengths: the tiles of all
// (request, KV head)s in a row, a tile's cost its blocks of 128 query rows, and takes
// an equal share.  Within a (request, KV head) early and late tiles alternate: new
// keys are seen by few rows, so that shares of equal cost take equal time.
//
// Warps 0-3, 4-7: sums of the even and odd tiles; 8: TMA producer (a ring of key
// tiles); 9: issues the MMAs.
#include <cuda.h>

#include <cstring>
#include <type_traits>

#include "common.cuh"
#include "target_ops.h"
#include "tcgen.cuh"

namespace dflash {
namespace {

constexpr int KT = 128;                   // keys of a tile
constexpr int CH = 128;                   // query rows of a product (of its columns)
constexpr int NBUF = 4;                   // products' results in TMEM, two a sum group
constexpr int SUM_THREADS = 256, THREADS = SUM_THREADS + 64;
constexpr int MAX_B = 1024;

// QB: query rows held at a time
template <int D, int QB> struct Cfg {
  static constexpr int TILE = KT * D * 2;
  static constexpr int NSLOT = (QB == 128 ? 5 : 4) * (D == 128 ? 1 : 2);
  static constexpr int Q_TILE = CH * D * 2;
  static constexpr int OFF_RING = (QB / CH) * Q_TILE;
  static constexpr int OFF_Z = OFF_RING + NSLOT * TILE;       // [QB] float
  static constexpr int OFF_COUNTS = OFF_Z + QB * 4;           // [QB / 32]
  static constexpr int OFF_PLAN = OFF_COUNTS + QB / 8;        // [MAX_B + 1] int64
  static constexpr int OFF_BARS = OFF_PLAN + (MAX_B + 1) * 8;
  static constexpr int N_BARS = 2 * NSLOT + 2 * NBUF + 2;
  static constexpr int SMEM = 1024 + OFF_BARS + N_BARS * 8 + 16;
  static_assert(SMEM <= 227 * 1024, "one CTA per SM");
};

struct Params {
  CUtensorMap tmK;                        // dims {D, KVH, n_pages * 64}, box {64, 1, 64}
  KeyWeightParams a;
  float c;                                // scale log2 e
};

// A request's new rows and own keys before them.
struct Request {
  int start, n, ctx;
};
// false: without rows, or not to be served (flagged by `flag`)
__device__ __forceinline__ bool read_request(const KeyWeightParams &a, int b, bool flag, Request &q) {
  const PagedRows &r = a.rows;
  const int s = r.row_start[b], e = r.row_start[b + 1], kv = r.kv_len[b];
  if (s < 0 || s > e || e > r.total_rows) {
    if (flag) raise_error(a.err, DFLASH_DERR_ROW_RANGE);
    return false;
  }
  if (e == s) return false;
  const int64_t own = (int64_t)kv + (e - s) - r.prefix_len;
  if (kv < r.prefix_len || own > (int64_t)r.pages_per_req * kPageRows || own > a.width) {
    if (flag) raise_error(a.err, DFLASH_DERR_KV_CAPACITY);
    return false;
  }
  if (a.mask && e - s > 32 * a.mask_words) {
    if (flag) raise_error(a.err, DFLASH_DERR_TREE);
    return false;
  }
  q.start = s;
  q.n = e - s;
  q.ctx = kv - r.prefix_len;
  return true;
}

// A run of tiles j0 .. j1-1 of one (request, KV head).
struct Run {
  Request q;
  int b, g, tiles, j0, j1, rows, blocks;  // tiles of the request; query rows, blocks of QB of them
};
__device__ __forceinline__ int tile_of(const Run &u, int j) { return j & 1 ? u.tiles - 1 - (j >> 1) : j >> 1; }
// Whether any of the query rows up to row `last` sees a key of the tile that begins at key k0.
__device__ __forceinline__ bool reaches(const Run &u, bool masked, int G, int k0, int last) {
  return masked || k0 - u.q.ctx <= min(last, u.rows - 1) / G;
}

template <int D, int QB>
__global__ void __launch_bounds__(THREADS, 1) key_weights_kernel(const __grid_constant__ Params p) {
  using C = Cfg<D, QB>;
  constexpr int NS = C::NSLOT, NB = D / 64;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint8_t *ring = smem + C::OFF_RING;
  float *s_z = (float *)(smem + C::OFF_Z);                    // what a row's exponents begin with
  uint32_t *s_counts = (uint32_t *)(smem + C::OFF_COUNTS);    // rows that count
  long long *s_base = (long long *)(smem + C::OFF_PLAN);      // cost of the requests before
  uint64_t *full = (uint64_t *)(smem + C::OFF_BARS), *empty = full + NS;
  uint64_t *s_full = empty + NS, *s_free = s_full + NBUF, *q_full = s_free + NBUF, *done = q_full + 1;
  uint32_t *s_tmem = (uint32_t *)(done + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const KeyWeightParams &a = p.a;
  const PagedRows &r = a.rows;
  const int G = a.H / a.KVH, KVH = a.KVH;
  const bool masked = a.mask != nullptr;

  if (threadIdx.x == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < NBUF; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_free[i], 128);
    }
    mbar_init(q_full, SUM_THREADS);
    mbar_init(done, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 9) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(su32(s_tmem))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (warp == 8 && lane == 0) asm volatile("prefetch.tensormap [%0];" ::"l"((uint64_t)&p.tmK) : "memory");
  pdl_wait();
  // ---- plan: cost of the requests before each, by one warp's scan
  for (int b = threadIdx.x; b < r.B; b += THREADS) {
    Request q;
    long long cost = 0;
    if (read_request(a, b, blockIdx.x == 0, q))
      cost = (long long)KVH * ((q.ctx + q.n + KT - 1) / KT) * (((int64_t)q.n * G + CH - 1) / CH);
    s_base[b + 1] = cost;
  }
  if (threadIdx.x == 0) s_base[0] = 0;
  __syncthreads();
  if (warp == 0) {
    long long sum = 0;
    for (int b0 = 0; b0 < r.B; b0 += 32) {
      const int b = b0 + lane;
      long long v = b < r.B ? s_base[b + 1] : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += x;
      }
      if (b < r.B) s_base[b + 1] = sum + v;
      sum += __shfl_sync(0xffffffffu, v, 31);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;
  const long long total = s_base[r.B];
  const long long lo = total * blockIdx.x / gridDim.x, hi = total * (blockIdx.x + 1) / gridDim.x;

  // the next run of this CTA's share at or behind cost `at`: tiles whose cost begins in [at, hi)
  auto next_run = [&](long long &at, Run &u) {
    while (at < hi) {
      int s0 = 0, s1 = r.B - 1;            // last request whose base is <= at
      while (s0 < s1) {
        const int mid = (s0 + s1 + 1) >> 1;
        if (s_base[mid] <= at) s0 = mid;
        else s1 = mid - 1;
      }
      u.b = s0;
      read_request(a, s0, false, u.q);     // (it has a cost: it is served)
      u.rows = u.q.n * G;
      u.tiles = (u.q.ctx + u.q.n + KT - 1) / KT;
      u.blocks = (u.rows + QB - 1) / QB;
      const int per = (u.rows + CH - 1) / CH;
      const long long in = at - s_base[s0], span = (long long)u.tiles * per;
      u.g = (int)(in / span);
      const long long head = s_base[s0] + u.g * span;
      u.j0 = (int)((at - head + per - 1) / per);
      u.j1 = (int)min((long long)u.tiles, (hi - head + per - 1) / per);
      at = head + span;
      if (u.j0 < u.j1) return true;
    }
    return false;
  };
  bool ok = true;
  long long at = lo;
  Run u;

  if (warp == 8) {
    // -------------------------------------------------------------- producer
    uint32_t n_tile = 0;
    while (ok && next_run(at, u)) {
      const int *list = r.page_table + (int64_t)u.b * r.pages_per_req;
      const int keys = u.q.ctx + u.q.n, npages = (keys + kPageRows - 1) / kPageRows;
      for (int rb = 0; rb < u.blocks && ok; ++rb) {
        auto pages_of = [&](int j) {       // of 16 tiles, one a lane
          const int jj = j + (lane >> 1), pn = jj < u.j1 ? 2 * tile_of(u, jj) + (lane & 1) : npages;
          return pn < npages ? __ldg(list + pn) : 0;
        };
        int ahead = pages_of(u.j0), batch = 0;
        for (int j = u.j0; j < u.j1 && ok; ++j) {
          if ((j - u.j0) % 16 == 0) {
            batch = ahead;
            ahead = pages_of(j + 16);
            if (batch < 0 || batch >= r.n_pages) {
              raise_error(a.err, DFLASH_DERR_PAGE_RANGE);
              batch = 0;
            }
          }
          const int t = tile_of(u, j), i = (j - u.j0) % 16;
          const int pg0 = __shfl_sync(0xffffffffu, batch, 2 * i), pg1 = __shfl_sync(0xffffffffu, batch, 2 * i + 1);
          if (!reaches(u, masked, G, t * KT, rb * QB + QB - 1)) continue;
          bool good = true;
          if (lane == 0) {
            const uint32_t slot = n_tile % NS;
            good = mbar_wait(&empty[slot], ((n_tile / NS) & 1) ^ 1);
            if (good) {
              const bool two = 2 * t + 1 < npages;
              asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(su32(&full[slot])),
                           "r"(two ? C::TILE : C::TILE / 2)
                           : "memory");
              uint8_t *dst = ring + slot * C::TILE;
#pragma unroll
              for (int c = 0; c < NB; ++c) {
                tma3(dst + c * (KT * 128), &p.tmK, &full[slot], 64 * c, u.g, pg0 * kPageRows);
                if (two) tma3(dst + c * (KT * 128) + 8192, &p.tmK, &full[slot], 64 * c, u.g, pg1 * kPageRows);
              }
            }
          }
          ok = __shfl_sync(0xffffffffu, good, 0) != 0;
          if (ok) ++n_tile;
        }
      }
    }
    if (lane == 0) {
      if (!ok) raise_error(a.err, DFLASH_DERR_TIMEOUT);
      // every copy has landed before the CTA exits
      for (uint32_t v = n_tile > (uint32_t)NS ? n_tile - NS : 0; v < n_tile; ++v)
        mbar_wait(&full[v % NS], (v / NS) & 1);
    }
  } else if (warp == 9) {
    // -------------------------------------------------------------- MMA issuer
    if (lane == 0) {
      const uint64_t k_desc = desc_k(su32(ring)), q_desc = desc_k(su32(smem));
      uint32_t n_tile = 0, n_q = 0, prod0 = 0, prod1 = 0;   // tiles, query blocks, products of either group
      while (ok && next_run(at, u)) {
        for (int rb = 0; rb < u.blocks && ok; ++rb) {
          ok = mbar_wait(q_full, n_q++ & 1);
          for (int j = u.j0; j < u.j1 && ok; ++j) {
            const int t = tile_of(u, j), x = j & 1;
            if (!reaches(u, masked, G, t * KT, rb * QB + QB - 1)) continue;
            const uint32_t slot = n_tile % NS;
            ok = mbar_wait(&full[slot], (n_tile / NS) & 1);
            ++n_tile;
            for (int ch = 0; ch < QB / CH && ok; ++ch) {
              const int row0 = rb * QB + ch * CH;
              if (row0 >= u.rows || !reaches(u, masked, G, t * KT, row0 + CH - 1)) continue;
              const int rows = min(CH, u.rows - row0);
              const uint32_t n_prod = x ? prod1++ : prod0++, buf = 2 * x + (n_prod & 1);
              ok = mbar_wait(&s_free[buf], ((n_prod >> 1) & 1) ^ 1);
              if (!ok) break;
              tc_fence_after();
              const uint32_t id = idesc(128, rows <= 16 ? 16 : (rows + 31) / 32 * 32, false);
              const uint64_t kd = k_desc + slot * (C::TILE >> 4), qd = q_desc + ch * (C::Q_TILE >> 4);
#pragma unroll
              for (int i = 0; i < D / 16; ++i)
                umma_ss(tmem + buf * CH, kd + (i >> 2) * ((KT * 128) >> 4) + 2 * (i & 3),
                        qd + (i >> 2) * ((CH * 128) >> 4) + 2 * (i & 3), id, i ? 1u : 0u);
              umma_commit(&s_full[buf]);
            }
            umma_commit(&empty[slot]);
          }
        }
      }
      umma_commit(done);
      if (!mbar_wait(done, 0)) ok = false;   // every MMA has ended before TMEM is freed
      if (!ok) raise_error(a.err, DFLASH_DERR_TIMEOUT);
    }
  } else {
    // -------------------------------------------------------------- sums, a key a thread
    const int x = warp >> 2, tid = threadIdx.x, key_lane = tid & 127;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    auto wait = [&](uint64_t *b, uint32_t parity) {
      if (ok && !mbar_wait(b, parity)) ok = false;
      ok = __all_sync(0xffffffffu, ok);
    };
    uint32_t n_prod = 0;
    // (after a wait that gave up the loops go on, without work, to the barriers that both groups share)
    while (next_run(at, u)) {
      float *out = a.weights + ((int64_t)u.b * KVH + u.g) * a.width;
      for (int rb = 0; rb < u.blocks; ++rb) {
        // the block's queries and what their exponents begin with; every product with the block
        // before has been read
        asm volatile("bar.sync 1, 256;" ::: "memory");
        if (tid < QB) {
          const int row = rb * QB + tid, tok = u.q.start + row / G, h = u.g * G + row % G;
          float z = -INFINITY;
          if (row < u.rows) {
            const float l = a.lse[(int64_t)tok * a.H + h], w = a.row_weight ? a.row_weight[tok] : 1.f;
            if (isfinite(l) && w > 0.f && isfinite(w)) z = log2f(w) - l * 1.4426950408889634f;
          }
          s_z[tid] = z;
          const uint32_t counts = __ballot_sync(0xffffffffu, z != -INFINITY);
          if (lane == 0) s_counts[warp] = counts;
        }
        asm volatile("bar.sync 1, 256;" ::: "memory");
        const int held = min(QB, (u.rows - rb * QB + 31) / 32 * 32);
#pragma unroll 8
        for (int i = tid; i < held * (D / 8); i += SUM_THREADS) {
          const int row = i / (D / 8), c = i % (D / 8), at_row = rb * QB + row;
          uint4 v = make_uint4(0, 0, 0, 0);    // rows that count for nothing
          if (s_counts[row >> 5] >> (row & 31) & 1u)
            v = *(reinterpret_cast<const uint4 *>((const bf16 *)a.q + (int64_t)(u.q.start + at_row / G) * a.q_stride +
                                                  (int64_t)(u.g * G + at_row % G) * D) + c);
          const int in = row & (CH - 1);
          *reinterpret_cast<uint4 *>(smem + (row / CH) * C::Q_TILE + (c >> 3) * (CH * 128) + in * 128 +
                                     (((c & 7) ^ (in & 7)) << 4)) = v;
        }
        fence_async_smem();
        mbar_arrive(q_full);
        const int keys = u.q.ctx + u.q.n;
        auto begins = [&](int k0) { return rb == 0 || !reaches(u, masked, G, k0, rb * QB - 1); };
        // what the sum of tile j's key is added to (loaded a tile ahead)
        auto read_old = [&](int j) {
          float old = 0.f;
          if (j < u.j1) {
            const int k0 = tile_of(u, j) * KT, key = k0 + key_lane;
            if (reaches(u, masked, G, k0, rb * QB + QB - 1) && key < keys &&
                (begins(k0) ? key < u.q.ctx && a.decay != 0.f : true))
              old = out[key];
          }
          return old;
        };
        const int first = u.j0 + ((u.j0 ^ x) & 1);
        float next_old = read_old(first);
        for (int j = first; j < u.j1; j += 2) {
          const float old = next_old;
          next_old = read_old(j + 2);
          const int k0 = tile_of(u, j) * KT, key = k0 + key_lane;
          if (!ok || !reaches(u, masked, G, k0, rb * QB + QB - 1)) continue;
          const bool live = key < keys;
          const int num = key - u.q.ctx;       // among the new rows
          float sum = 0.f;
          for (int ch = 0; ch < QB / CH; ++ch) {
            const int row0 = rb * QB + ch * CH;
            if (row0 >= u.rows || !reaches(u, masked, G, k0, row0 + CH - 1)) continue;
            const int rows = min(CH, u.rows - row0);
            const uint32_t buf = 2 * x + (n_prod & 1);
            wait(&s_full[buf], (n_prod >> 1) & 1);
            ++n_prod;
            if (!ok) break;
            tc_fence_after();
            const uint32_t t_s = tmem + lanes + buf * CH;
            const float *z = s_z + ch * CH;
            const uint32_t *counts = s_counts + ch * (CH / 32);
            // columns c .. c+31 whose row sees this key
            auto sees = [&](int c) {
              const int r0 = row0 + c;
              if (num < 0 || !live) return 0xffffffffu;
              if (!masked) {
                const int64_t from = (int64_t)num * G - r0;
                return from <= 0 ? 0xffffffffu : from >= 32 ? 0u : 0xffffffffu << from;
              }
              uint32_t cols = 0;
              int tok = r0 / G;
              for (int at = tok * G - r0; at < 32 && tok < u.q.n; at += G, ++tok)
                if (__ldg(a.mask + (int64_t)(u.q.start + tok) * a.mask_words + (num >> 5)) >> (num & 31) & 1u) {
                  const uint32_t upto = at + G >= 32 ? 0xffffffffu : (1u << (at + G)) - 1u;
                  cols |= upto & (at > 0 ? 0xffffffffu << at : 0xffffffffu);
                }
              return cols;
            };
            const float2 c2 = make_float2(p.c, p.c);
            float2 s0, s1;
            // a piece's terms; with SELECT those of `cols` alone
            auto add = [&](const uint32_t *v, const float *zz, uint32_t cols, auto select) {
              constexpr bool SELECT = decltype(select)::value;
#pragma unroll
              for (int i = 0; i < 32; i += 4) {
                const float4 z4 = *reinterpret_cast<const float4 *>(zz + i);
                const float2 e0 = fma2(make_float2(__uint_as_float(v[i]), __uint_as_float(v[i + 1])), c2,
                                       make_float2(z4.x, z4.y));
                const float2 e1 = fma2(make_float2(__uint_as_float(v[i + 2]), __uint_as_float(v[i + 3])), c2,
                                       make_float2(z4.z, z4.w));
                float2 w0 = make_float2(ex2(e0.x), ex2(e0.y)), w1 = make_float2(ex2(e1.x), ex2(e1.y));
                if (SELECT) {
                  w0.x = cols >> i & 1u ? w0.x : 0.f;
                  w0.y = cols >> (i + 1) & 1u ? w0.y : 0.f;
                  w1.x = cols >> (i + 2) & 1u ? w1.x : 0.f;
                  w1.y = cols >> (i + 3) & 1u ? w1.y : 0.f;
                }
                s0 = add2(s0, w0);
                s1 = add2(s1, w1);
              }
            };
            // every row of the product sees every key of the tile
            const bool whole = k0 + KT <= u.q.ctx || (!masked && k0 + KT - 1 - u.q.ctx <= row0 / G);
            // Terms one by one where rows see some of the keys, or where a row that counts for nothing has
            // met a key that is not finite.
            auto pass = [&](auto select) {
              s0 = s1 = make_float2(0.f, 0.f);
              uint32_t v0[32], v1[32];
              auto cols = [&](int c) { return decltype(select)::value ? counts[c >> 5] & (whole ? 0xffffffffu : sees(c)) : 0u; };
              if (rows <= 16) {
                tmem_ld16(t_s, v0);
#pragma unroll
                for (int i = 16; i < 32; ++i) v0[i] = 0;         // (beyond the rows: weigh 0)
                tmem_ld_wait32(v0);
                add(v0, z, cols(0), select);
              } else {
                tmem_ld32(t_s, v0);
                for (int i = 0; i < rows; i += 64) {             // the next piece is on its way
                  tmem_ld_wait32(v0);
                  if (i + 32 < rows) tmem_ld32(t_s + i + 32, v1);
                  add(v0, z + i, cols(i), select);
                  if (i + 32 < rows) {
                    tmem_ld_wait32(v1);
                    if (i + 64 < rows) tmem_ld32(t_s + i + 64, v0);
                    add(v1, z + i + 32, cols(i + 32), select);
                  }
                }
              }
              return (s0.x + s0.y) + (s1.x + s1.y);
            };
            float part = 0.f;
            if (whole) part = pass(std::false_type());
            if (!whole || __any_sync(0xffffffffu, live && isnan(part))) part = pass(std::true_type());
            sum += part;
            tc_fence_before();
            mbar_arrive(&s_free[buf]);
          }
          if (live && ok) out[key] = (begins(k0) ? old * a.decay : old) + sum;
        }
      }
    }
    if (!ok && lane == 0) raise_error(a.err, DFLASH_DERR_TIMEOUT);
  }
  tc_fence_before();
  __syncthreads();
  pdl_trigger();
  if (warp == 9) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }
}

template <int D, int QB> cudaError_t launch(const KeyWeightParams &a, cudaStream_t s) {
  Params p;
  memset(&p, 0, sizeof(p));
  if (!encode_pages(&p.tmK, a.k_pages, a.rows.n_pages, a.KVH, D)) return cudaErrorInvalidValue;
  int dev = 0, sms = 0;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  p.a = a;
  p.c = a.scale * 1.4426950408889634f;
  return launch_pdl(key_weights_kernel<D, QB>, dim3(sms), dim3(THREADS), Cfg<D, QB>::SMEM, s, p);
}
template <int D, int QB> cudaError_t prepare() {
  return cudaFuncSetAttribute(key_weights_kernel<D, QB>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              Cfg<D, QB>::SMEM);
}
template <int D> cudaError_t launch(const KeyWeightParams &a, cudaStream_t s) {
  const bool few = (int64_t)a.rows.total_rows * (a.H / a.KVH) <= 128LL * a.rows.B;
  return few ? launch<D, 128>(a, s) : launch<D, 256>(a, s);
}

}  // namespace

cudaError_t launch_key_weights_tc(const KeyWeightParams &p, cudaStream_t s) {
  return p.D == 64 ? launch<64>(p, s) : launch<128>(p, s);
}

cudaError_t prepare_key_weights_tc() {
  cudaError_t e = prepare<64, 128>();
  if (e == cudaSuccess) e = prepare<64, 256>();
  if (e == cudaSuccess) e = prepare<128, 128>();
  return e == cudaSuccess ? prepare<128, 256>() : e;
}

}  // namespace dflash

// Attention weight that falls on every row of a paged bf16 cache, on the tensor
// cores (tcgen05 + TMEM).
//
// w[p] = decay w[p] + sum_r 2^(c (s[p, r] + z[r] / c)), s = K Q^T, c = scale log2 e,
// over the query rows r = (token, head of the group) of a request that see key p;
// z[r] = log2(row_weight) - lse log2 e is known before, so keys need no second look.
// A key tile (128 keys, two pages) is the product's A operand and up to 256 query
// rows its B operand: a TMEM lane is a key, and the sum over the columns stays in
// one thread (two where a product has more than 32 columns, joined through shared
// memory), without atomics; every key has one CTA, so sums are in a fixed order.
// z / c is a row of the product too: 16 more columns along K, 1 1 1 0 ... of every
// key against z / c as the sum of three bf16 values (24 bits).  Read from shared
// memory by the summing threads instead, it took as much of its bandwidth as the
// products' operands (windows 77 us against 60).
//
// Few rows (decoding): HBM bounds it, K is read once and V not at all.  Many rows:
// an exponential per key and row (1024 clocks of the MUFU for 128 keys by 256 rows)
// and the product (1150 clocks) bound it.  Rows of a request and KV head
// beyond a block (128, 256 or 512) are further passes over the CTA's keys.
//
// Every CTA lays out the same plan from the requests' lengths: the tiles of all
// (request, KV head)s in a row, a tile's cost its blocks of 128 query rows, and takes
// an equal share.  Within a (request, KV head) early and late tiles alternate: new
// keys are seen by few rows, so that shares of equal cost take equal time.
//
// Measured (calls in a row; 8 KV heads of 128, inputs beyond L2): 32 requests, a token
// each, over 500 to 16000 rows (558 MB) 90 us, 6.2 TB/s; the last 64 rows of two
// prompts, 64 heads, over 8000 and 30000 rows 53 us (156 million exponentials and 40
// GFLOP: 17 and 20 us at the units' rates; per 128 keys and 512 rows about 4600
// clocks, of which the sums take 3100 and a product that nothing hides 1000).  Tried
// for it and no faster: products of 128 columns with two places a group, so that one
// runs while another is summed (8% more: more waits a column), an issuer a group,
// both products of a tile one after the other (5% more), key tiles fetched to the L2
// ahead, an arrival a warp instead of a thread, waits that poll.
//
// Warps: the groups that sum (of even and odd tiles; 128 or 256 threads each), the TMA
// producer (a ring of key tiles), the MMA issuer.
#include <cuda.h>

#include <climits>
#include <cstring>
#include <type_traits>

#include "common.cuh"
#include "target_ops.h"
#include "tcgen.cuh"

namespace dflash {
namespace {

constexpr int KT = 128;                   // keys of a tile
constexpr int NG = 2;                     // groups that sum, each with a product's result in TMEM
constexpr int MAX_B = 1024;

// QB: query rows held at a time; PC of them are the columns of a product, whose halves of 128 are summed by
// 128 threads each
template <int D, int QB> struct Cfg {
  static constexpr int TILE = KT * D * 2;
  static constexpr int PC = QB < 256 ? QB : 256, HALVES = PC / 128;
  static constexpr int PER_SM = QB == 128 ? 2 : 1;            // CTAs
  static constexpr int NSLOT = (QB == 256 ? 4 : 2) * (D == 128 ? 1 : 2);
  static constexpr int GROUP = 128 * HALVES, SUM_THREADS = NG * GROUP, THREADS = SUM_THREADS + 64;
  static constexpr int OFF_RING = QB * D * 2;
  static constexpr int OFF_ONES = OFF_RING + NSLOT * TILE;    // [KT][16] bf16
  static constexpr int OFF_Z = OFF_ONES + KT * 32;            // [QB][16] bf16
  static constexpr int OFF_COUNTS = OFF_Z + QB * 32;          // [QB / 32]
  static constexpr int OFF_PARTS = OFF_COUNTS + QB / 8;       // [NG][2][128] float, with two halves
  static constexpr int OFF_PLAN = OFF_PARTS + (HALVES - 1) * NG * 2 * 128 * 4;   // [MAX_B + 2] uint32
  static constexpr int OFF_BARS = OFF_PLAN + (MAX_B + 2) * 4;
  static constexpr int N_BARS = 2 * NSLOT + 4 * NG + 2;
  static constexpr int SMEM = 1024 + OFF_BARS + N_BARS * 8 + 16;
  static_assert(OFF_BARS % 8 == 0 && PER_SM * (SMEM + 1024) <= 228 * 1024, "shared memory of an SM");
};

struct Params {
  CUtensorMap tmK;                        // dims {D, KVH, n_pages * 64}, box {64, 1, 64}
  KeyWeightParams a;
  float c, inv_c;                         // scale log2 e, and 1 / c
  int no_scores;                          // scale 0: every score is 0 (c is 1)
};

// Element (row, k) of an operand of 16 columns along K without swizzle, in bf16 elements.
__device__ __forceinline__ int plain_at(int row, int k) {
  return (row >> 3) * 128 + (k >> 3) * 64 + (row & 7) * 8 + (k & 7);
}

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
  int b, g, tiles, j0, j1, rows;          // tiles of the request; query rows
  int block0, blocks;                     // blocks of QB of them: the first that sees a key of the run, and behind the last
};
__device__ __forceinline__ int tile_of(const Run &u, int j) { return j & 1 ? u.tiles - 1 - (j >> 1) : j >> 1; }
// The last key that the rows of a block, and of the block before, may see; up to which key all rows
// of a block see all of them.
struct Limits {
  int before, block, whole;
  __device__ __forceinline__ Limits(const Run &u, bool masked, int G, int row0, int rows) {
    before = row0 == 0 ? -1 : masked ? INT_MAX : u.q.ctx + (row0 - 1) / G;
    block = masked ? INT_MAX : u.q.ctx + min(row0 + rows - 1, u.rows - 1) / G;
    whole = masked ? u.q.ctx : u.q.ctx + row0 / G + 1;
  }
};

template <int D, int QB>
__global__ void __launch_bounds__(Cfg<D, QB>::THREADS, Cfg<D, QB>::PER_SM)
key_weights_kernel(const __grid_constant__ Params p) {
  using C = Cfg<D, QB>;
  constexpr int NS = C::NSLOT, NB = D / 64, PC = C::PC, TMEM_COLS = NG * PC;
  constexpr int PRODUCER = C::SUM_THREADS / 32, ISSUER = PRODUCER + 1;   // first warps of their kind
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint8_t *ring = smem + C::OFF_RING;
  bf16 *s_ones = (bf16 *)(smem + C::OFF_ONES), *s_z = (bf16 *)(smem + C::OFF_Z);
  uint32_t *s_counts = (uint32_t *)(smem + C::OFF_COUNTS);    // rows that count
  uint32_t *s_base = (uint32_t *)(smem + C::OFF_PLAN);        // cost of the requests before, in units of 2^shift
  uint64_t *full = (uint64_t *)(smem + C::OFF_BARS), *empty = full + NS;
  uint64_t *s_full = empty + NS, *s_free = s_full + NG, *parts = s_free + NG, *q_full = parts + 2 * NG, *done = q_full + 1;
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
    for (int i = 0; i < NG; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_free[i], C::GROUP);
      mbar_init(&parts[2 * i], 128);
      mbar_init(&parts[2 * i + 1], 128);
    }
    mbar_init(q_full, C::SUM_THREADS);
    mbar_init(done, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == ISSUER) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(su32(s_tmem)), "n"(TMEM_COLS)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  // the columns that add a row's term z / c (in three parts) to its scores: 1, 1, 1, 0, ... of a key
  for (int i = threadIdx.x; i < KT * 2; i += C::THREADS)     // (groups of 8 rows: k 0..7, then 8..15)
    reinterpret_cast<uint4 *>(s_ones)[i] = i & 8 ? make_uint4(0, 0, 0, 0) : make_uint4(0x3f803f80u, 0x3f80u, 0, 0);
  for (int i = threadIdx.x; i < QB * 2; i += C::THREADS) reinterpret_cast<uint4 *>(s_z)[i] = make_uint4(0, 0, 0, 0);
  fence_async_smem();
  if (warp == PRODUCER && lane == 0) asm volatile("prefetch.tensormap [%0];" ::"l"((uint64_t)&p.tmK) : "memory");
  pdl_wait();
  // ---- plan, by one warp: the requests' costs added up, then scanned in units that 32 bits hold
  auto cost_of = [&](int b, bool flag) {
    Request q;
    if (b >= r.B || !read_request(a, b, flag, q)) return 0LL;
    return (long long)KVH * ((q.ctx + q.n + KT - 1) / KT) * (((int64_t)q.n * G + 127) / 128);
  };
  if (warp == 0) {
    const long long first = cost_of(lane, blockIdx.x == 0);
    long long sum = first;
    for (int b = 32 + lane; b < r.B; b += 32) sum += cost_of(b, blockIdx.x == 0);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const int shift = max(0, 34 - __clzll(sum));   // (rounding up adds less than one a request)
    uint32_t before = 0;
    for (int b0 = 0; b0 < r.B; b0 += 32) {
      uint32_t v = (uint32_t)(((b0 == 0 ? first : cost_of(b0 + lane, false)) + (1LL << shift) - 1) >> shift);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t x = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += x;
      }
      if (b0 + lane < r.B) s_base[b0 + lane + 1] = before + v;
      before += __shfl_sync(0xffffffffu, v, 31);
    }
    if (lane == 0) {
      s_base[0] = 0;
      s_base[MAX_B + 1] = (uint32_t)shift;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *s_tmem, total = s_base[r.B];
  const int shift = (int)s_base[MAX_B + 1];
  const uint32_t lo = (uint32_t)((uint64_t)total * blockIdx.x / gridDim.x);
  const uint32_t hi = (uint32_t)((uint64_t)total * (blockIdx.x + 1) / gridDim.x);

  // The next run of this CTA's share: of the first request at or behind `b`, from its KV head `g` on;
  // tiles whose cost begins in [lo, hi).
  auto next_run = [&](int &b, int &g, Run &u) {
    while (lo < hi && b < r.B && s_base[b] < hi) {
      if (s_base[b + 1] <= lo || s_base[b + 1] == s_base[b]) {
        ++b, g = 0;
        continue;
      }
      read_request(a, b, false, u.q);      // (it has a cost: it is served)
      u.b = b;
      u.rows = u.q.n * G;
      u.tiles = (u.q.ctx + u.q.n + KT - 1) / KT;
      u.blocks = (u.rows + QB - 1) / QB;
      const long long per = (u.rows + 127) / 128, span = u.tiles * per;
      const long long from = lo > s_base[b] ? (long long)(lo - s_base[b]) << shift : 0;
      const long long upto = min(span * KVH, (long long)(hi - s_base[b]) << shift);
      g = max(g, (int)(from / span));
      if (g >= KVH || g * span >= upto) {
        ++b, g = 0;
        continue;
      }
      u.g = g++;
      u.j0 = from > u.g * span ? (int)((from - u.g * span + per - 1) / per) : 0;
      u.j1 = (int)min((long long)u.tiles, (upto - u.g * span + per - 1) / per);
      // Blocks before block0 see nothing of the run and are not loaded: every block that is has a product,
      // which the sums wait for, so that a block is loaded when the one before has been taken.  (The first
      // tile of a run is its first early one, if it has one.)
      const int t0 = u.j0 + (u.j0 & 1) < u.j1 ? (u.j0 + 1) >> 1 : tile_of(u, u.j0);
      u.block0 = masked || t0 * KT <= u.q.ctx ? 0 : (t0 * KT - u.q.ctx) * G / QB;
      if (u.j0 < u.j1) return true;
    }
    return false;
  };
  int at_b = 0, at_g = 0;
  {
    int s1 = r.B - 1;                      // last request that begins at or before lo
    while (at_b < s1) {
      const int mid = (at_b + s1 + 1) >> 1;
      if (s_base[mid] <= lo) at_b = mid;
      else s1 = mid - 1;
    }
  }
  bool ok = true;

  if (warp == PRODUCER) {
    // -------------------------------------------------------------- producer
    uint32_t n_tile = 0;
    Run u, next;
    auto pages_of = [&](const Run &u, int j) {     // of 16 tiles, one a lane
      const int jj = j + (lane >> 1), pn = jj < u.j1 ? 2 * tile_of(u, jj) + (lane & 1) : INT_MAX;
      return pn < (u.q.ctx + u.q.n + kPageRows - 1) / kPageRows
                 ? __ldg(r.page_table + (int64_t)u.b * r.pages_per_req + pn)
                 : 0;
    };
    bool more = next_run(at_b, at_g, next);
    int first = more ? pages_of(next, next.j0) : 0;
    while (ok && more) {
      u = next;
      int head = first;
      // the run after this one and its first pages, before they are wanted
      more = next_run(at_b, at_g, next);
      if (more) first = pages_of(next, next.j0);
      const int npages = (u.q.ctx + u.q.n + kPageRows - 1) / kPageRows;
      for (int rb = u.block0; rb < u.blocks && ok; ++rb) {
        const Limits lim(u, masked, G, rb * QB, QB);
        int ahead = head, batch = 0;
        for (int j = u.j0; j < u.j1 && ok; ++j) {
          if ((j - u.j0) % 16 == 0) {
            batch = ahead;
            ahead = pages_of(u, j + 16);
            if (batch < 0 || batch >= r.n_pages) {
              raise_error(a.err, DFLASH_DERR_PAGE_RANGE);
              batch = 0;
            }
          }
          const int t = tile_of(u, j), i = (j - u.j0) % 16;
          const int pg0 = __shfl_sync(0xffffffffu, batch, 2 * i), pg1 = __shfl_sync(0xffffffffu, batch, 2 * i + 1);
          if (t * KT > lim.block) continue;
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
  } else if (warp >= ISSUER) {
    // -------------------------------------------------------------- MMA issuer
    // Two tiles at a time, a group's each: their first products, then their second ones.  So the groups
    // stay out of phase, one's sums run while the other's product does.  (With an issuer a group they
    // fell into step and waited for each other's products: windows 60 us.)
    if (lane == 0) {
      const uint64_t k_desc = desc_k(su32(ring)), q_desc = desc_k(su32(smem));
      const uint64_t ones_desc = desc_plain(su32(s_ones), 128, 256), z_desc = desc_plain(su32(s_z), 128, 256);
      uint32_t n_tile = 0, n_q = 0, parity = 0;   // tiles and query blocks before; bit x: of group x's products
      Run u;
      while (ok && next_run(at_b, at_g, u)) {
        for (int rb = u.block0; rb < u.blocks && ok; ++rb) {
          const Limits lim(u, masked, G, rb * QB, QB);
          const int rows = min(QB, u.rows - rb * QB), products = (rows + PC - 1) / PC;
          ok = mbar_wait(q_full, n_q++ & 1);
          for (int j0 = u.j0 & ~1; j0 < u.j1 && ok; j0 += 2) {
            const bool has0 = j0 >= u.j0 && tile_of(u, j0) * KT <= lim.block;
            const bool has1 = j0 + 1 < u.j1 && tile_of(u, j0 + 1) * KT <= lim.block;
            for (int pr = 0; pr < products; ++pr) {
              const int cols = min(PC, rows - pr * PC);
              const uint32_t id = idesc(128, cols <= 16 ? 16 : (cols + 31) / 32 * 32, false);
              const uint64_t qd = q_desc + pr * ((PC * D * 2) >> 4), zd = z_desc + pr * ((PC * 32) >> 4);
#pragma unroll
              for (int x = 0; x < NG; ++x) {
                if (!(x ? has1 : has0) || !ok) continue;
                const uint32_t tile = n_tile + (x && has0 ? 1 : 0), slot = tile % NS;
                const uint64_t kd = k_desc + slot * (C::TILE >> 4);
                ok = mbar_wait(&full[slot], (tile / NS) & 1) && mbar_wait(&s_free[x], (parity >> x & 1) ^ 1);
                parity ^= 1u << x;
                if (!ok) continue;
                tc_fence_after();
#pragma unroll
                for (int i = 0; i < D / 16; ++i)
                  umma_ss(tmem + x * PC, kd + (i >> 2) * ((KT * 128) >> 4) + 2 * (i & 3),
                          qd + (i >> 2) * ((PC * 128) >> 4) + 2 * (i & 3), id, i ? 1u : 0u);
                umma_ss(tmem + x * PC, ones_desc, zd, id, 1u);
                umma_commit(&s_full[x]);
                if (pr == products - 1) umma_commit(&empty[slot]);
              }
            }
            n_tile += has0 + has1;
          }
        }
      }
      umma_commit(done);
      if (!mbar_wait(done, 0)) ok = false;   // every MMA has ended before TMEM is freed
      if (!ok) raise_error(a.err, DFLASH_DERR_TIMEOUT);
    }
  } else {
    // -------------------------------------------------------------- sums, a key a thread
    const int tid = threadIdx.x, x = tid / C::GROUP, half = tid / 128 % C::HALVES, key_lane = tid & 127;
    const uint32_t t_s = tmem + ((uint32_t)((warp & 3) * 32) << 16) + x * PC;
    float *s_parts = (float *)(smem + C::OFF_PARTS) + x * 256 + key_lane;   // of the second half, for even and odd products
    auto sync = [] { asm volatile("bar.sync 1, %0;" ::"n"(C::SUM_THREADS) : "memory"); };
    auto wait = [&](uint64_t *b, uint32_t parity) {
      if (ok && !mbar_wait(b, parity)) ok = false;
      ok = __all_sync(0xffffffffu, ok);
    };
    uint32_t n = 0, n_join = 0;            // products of the group before; of those with two halves
    Run u;
    // (after a wait that gave up the loops go on, without work, to the barriers that all groups share)
    while (next_run(at_b, at_g, u)) {
      float *out = a.weights + ((int64_t)u.b * KVH + u.g) * a.width;
      for (int rb = u.block0; rb < u.blocks; ++rb) {
        // The block's queries, and every row's z / c = (log2(row_weight) - lse log2 e) / c as the sum of three
        // bf16 values; every product with the block before has been read.  (A row that counts for nothing
        // gets a term that no score outweighs.)
        constexpr int R = C::SUM_THREADS / (D / 8), UNITS = QB / R < 8 ? QB / R : 8;   // rows at a time; chunks of a thread
        const int chunk = tid % (D / 8), row0 = rb * QB, rows = min(QB, u.rows - row0);
        auto load_q = [&](int r0, uint4 *q) {
#pragma unroll
          for (int k = 0; k < UNITS; ++k) {
            const int i = r0 + tid / (D / 8) + k * R, row = row0 + i;
            q[k] = make_uint4(0, 0, 0, 0);
            if (i < rows && !p.no_scores)
              q[k] = *(reinterpret_cast<const uint4 *>((const bf16 *)a.q + (int64_t)(u.q.start + row / G) * a.q_stride +
                                                       (int64_t)(u.g * G + row % G) * D) + chunk);
          }
        };
        auto store_q = [&](int r0, const uint4 *q) {
#pragma unroll
          for (int k = 0; k < UNITS; ++k) {
            const int i = r0 + tid / (D / 8) + k * R, in = i % PC;
            *reinterpret_cast<uint4 *>(smem + i / PC * (PC * D * 2) + (chunk >> 3) * (PC * 128) + in * 128 +
                                       (((chunk & 7) ^ (in & 7)) << 4)) = q[k];
          }
        };
        uint4 q[UNITS];
        load_q(0, q);
        bool counts = false;
        float z = copysignf(3e38f, -p.c);
        if (tid < rows) {
          const int row = row0 + tid, tok = u.q.start + row / G;
          const float l = a.lse[(int64_t)tok * a.H + u.g * G + row % G], w = a.row_weight ? a.row_weight[tok] : 1.f;
          counts = isfinite(l) && w > 0.f && isfinite(w);
          if (counts) z = fminf(fmaxf((log2f(w) - l * 1.4426950408889634f) * p.inv_c, -3e38f), 3e38f);
        }
        const uint32_t these = __ballot_sync(0xffffffffu, counts);
        sync();
        if (tid < QB) {
          bf16 part[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            part[k] = __float2bfloat16_rn(k < 3 ? z : 0.f);
            z -= __bfloat162float(part[k]);
          }
          *reinterpret_cast<uint4 *>(s_z + plain_at(tid, 0)) = *reinterpret_cast<const uint4 *>(part);
          if (lane == 0) s_counts[warp] = these;
        }
        store_q(0, q);
        for (int r0 = R * UNITS; r0 < rows; r0 += R * UNITS) {
          load_q(r0, q);
          store_q(r0, q);
        }
        fence_async_smem();
        mbar_arrive(q_full);
        const Limits lim(u, masked, G, row0, QB);
        const int keys = u.q.ctx + u.q.n;
        const int products = (rows + PC - 1) / PC;
        const bool joined = C::HALVES > 1 && rows > 32;
        // what the sum of tile j's key is added to (loaded a tile ahead)
        auto read_old = [&](int j) {
          float old = 0.f;
          if (j < u.j1 && half == 0) {
            const int k0 = tile_of(u, j) * KT, key = k0 + key_lane;
            // (the first block that sees a key takes the weight from before the call)
            if (k0 <= lim.block && key < keys && (k0 <= lim.before || (key < u.q.ctx && a.decay != 0.f)))
              old = out[key];
          }
          return old;
        };
        const int first = u.j0 + ((x - u.j0) & (NG - 1));
        float next_old = read_old(first);
        for (int j = first; j < u.j1; j += NG) {
          const float old = next_old;
          next_old = read_old(j + NG);
          const int k0 = tile_of(u, j) * KT, key = k0 + key_lane;
          if (!ok || k0 > lim.block) continue;
          const bool live = key < keys;
          const int num = key - u.q.ctx;       // among the new rows
          // every row of the block sees every key of the tile
          const bool whole = k0 + KT <= lim.whole;
          // columns c .. c+31 whose row sees this key
          auto sees = [&](int c) {
            const int r0 = row0 + c;
            if (num < 0 || !live) return 0xffffffffu;
            if (!masked) {
              const int64_t first_row = (int64_t)num * G - r0;
              return first_row <= 0 ? 0xffffffffu : first_row >= 32 ? 0u : 0xffffffffu << first_row;
            }
            uint32_t cols = 0;
            int tok = r0 / G;
            for (int at = tok * G - r0; at < 32 && tok < u.q.n; at += G, ++tok)
              if (__ldg(a.mask + (int64_t)(u.q.start + tok) * a.mask_words + (num >> 5)) >> (num & 31) & 1u) {
                const uint32_t ends = at + G >= 32 ? 0xffffffffu : (1u << (at + G)) - 1u;
                cols |= ends & (at > 0 ? 0xffffffffu << at : 0xffffffffu);
              }
            return cols;
          };
          // the sum of a piece's terms, of columns c .. c+W-1
          auto piece = [&](const uint32_t *v, int c, auto width) {
            constexpr int W = decltype(width)::value;
            const float2 c2 = make_float2(p.c, p.c);
            auto terms = [&](uint32_t cols, auto select) {   // with SELECT those of `cols` alone
              constexpr bool SELECT = decltype(select)::value;
              float2 s0 = make_float2(0.f, 0.f), s1 = s0;
#pragma unroll
              for (int i = 0; i < W; i += 4) {
                const float2 e0 = mul2(make_float2(__uint_as_float(v[i]), __uint_as_float(v[i + 1])), c2);
                const float2 e1 = mul2(make_float2(__uint_as_float(v[i + 2]), __uint_as_float(v[i + 3])), c2);
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
              return (s0.x + s0.y) + (s1.x + s1.y);
            };
            // Terms one by one where rows see some of the keys, or where what is not finite may be a row's
            // that counts for nothing.
            float part = 0.f;
            if (whole) part = terms(0u, std::false_type());
            if (!whole || __any_sync(0xffffffffu, live && !(part < INFINITY)))
              part = terms(s_counts[c >> 5] & (whole ? 0xffffffffu : sees(c)), std::true_type());
            return part;
          };
          float sum = 0.f;
#pragma unroll 1
          for (int pr = 0; pr < products; ++pr) {
            wait(&s_full[x], n & 1);
            ++n;
            if (!ok) break;
            tc_fence_after();
            auto release = [&] {               // the product is in registers
              tc_fence_before();
              mbar_arrive(&s_free[x]);
            };
            // this half's columns: whole pieces of 32
            const int cols = min(PC, rows - pr * PC), split = C::HALVES == 1 ? cols : (cols + 63) / 64 * 32;
            const int from = half == 0 ? 0 : split, upto = half == 0 ? min(split, cols) : cols;
            if (cols <= 16 && half == 0) {
              uint32_t v[16];
              tmem_ld16(t_s, v);
              tmem_ld_wait<16>(v);
              release();
              sum += piece(v, pr * PC, std::integral_constant<int, 16>());
            } else {
#pragma unroll 1
              for (int c = from; c < upto; c += 32) {
                uint32_t v[32];
                tmem_ld32(t_s + c, v);
                tmem_ld_wait<32>(v);
                if (c + 32 >= upto) release();
                sum += piece(v, pr * PC + c, std::integral_constant<int, 32>());
              }
              if (from >= upto) release();
            }
          }
          if (!ok) continue;
          if (joined) {
            const uint32_t e = n_join & 1;
            if (half == 1) {
              s_parts[e * 128] = sum;          // (read before the product after the next is there)
              mbar_arrive(&parts[2 * x + e]);
            } else {
              wait(&parts[2 * x + e], n_join >> 1 & 1);
              if (ok) sum += s_parts[e * 128];
            }
            ++n_join;
          }
          if (half == 0 && live && ok) out[key] = (k0 <= lim.before ? old : old * a.decay) + sum;
        }
      }
    }
    if (!ok && lane == 0) raise_error(a.err, DFLASH_DERR_TIMEOUT);
  }
  tc_fence_before();
  __syncthreads();
  pdl_trigger();
  if (warp == ISSUER) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(TMEM_COLS) : "memory");
  }
}

template <int D, int QB> cudaError_t launch(const KeyWeightParams &a, cudaStream_t s) {
  using C = Cfg<D, QB>;
  Params p;
  memset(&p, 0, sizeof(p));
  if (!encode_pages(&p.tmK, a.k_pages, a.rows.n_pages, a.KVH, D)) return cudaErrorInvalidValue;
  int dev = 0, sms = 0;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  p.a = a;
  p.no_scores = a.scale == 0.f;
  p.c = p.no_scores ? 1.f : a.scale * 1.4426950408889634f;
  p.inv_c = 1.f / p.c;
  return launch_pdl(key_weights_kernel<D, QB>, dim3(sms * C::PER_SM), dim3(C::THREADS), C::SMEM, s, p);
}
template <int D, int QB> cudaError_t prepare() {
  return cudaFuncSetAttribute(key_weights_kernel<D, QB>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              Cfg<D, QB>::SMEM);
}
template <int D> cudaError_t launch(const KeyWeightParams &a, cudaStream_t s) {
  // Blocks of 128 query rows and two CTAs an SM, or of 512 and one: 32 requests over 3000 to 6000 rows with
  // 4 query rows each (a token) 57 us against 72, with 128 65 against 85; with 192 112 against 97, with 256 121
  // against 111; 2 requests with 512 over 8000 and 30000 168 against 58.  Blocks of 256, with twice the key
  // tiles on their way, against those of 512: with 192 77 against 90, with 256 93 against 97, with 384 148 both
  // ways, with 400 37 against 35 (4 requests).
  const int64_t rows = (int64_t)a.rows.total_rows * (a.H / a.KVH);
  if (rows <= 128LL * a.rows.B) return launch<D, 128>(a, s);
  return rows <= 256LL * a.rows.B ? launch<D, 256>(a, s) : launch<D, 512>(a, s);
}

}  // namespace

cudaError_t launch_key_weights_tc(const KeyWeightParams &p, cudaStream_t s) {
  return p.D == 64 ? launch<64>(p, s) : launch<128>(p, s);
}

cudaError_t prepare_key_weights_tc() {
  cudaError_t e = prepare<64, 128>();
  if (e == cudaSuccess) e = prepare<64, 256>();
  if (e == cudaSuccess) e = prepare<64, 512>();
  if (e == cudaSuccess) e = prepare<128, 128>();
  if (e == cudaSuccess) e = prepare<128, 256>();
  return e == cudaSuccess ? prepare<128, 512>() : e;
}

}  // namespace dflash

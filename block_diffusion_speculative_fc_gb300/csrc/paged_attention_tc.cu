// bf16 attention of new rows over a paged cache with a shared prefix, on the
// tensor cores (tcgen05 + TMEM).
//
// Per KV head g, query row r = (token, head of g's group) attends to a list of
// keys; the rows of a batch fall into segments that share their keys: the
// shared prefix (the rows of all requests) and each request's own rows (its
// rows).  A work item is up to 256 rows of a segment times a range of 128-key
// tiles (two cache pages).  Partial results (o / l, log2 of the weight) of a
// row that several items hold are joined by a last launch.
//
// The softmax is the running one: tile by tile S = Q K^T, w = 2^(S c - m), O +=
// w V, l += sum w, with c = scale log2 e; m is a running reference that follows
// the row maximum only when that exceeds it by more than 2^8 (the result o / l
// does not depend on m; w <= 2^8 keeps fp32 sums far from overflow), so that
// O in TMEM is rarely rescaled.
//
// Two streams of 128 threads (a thread per row: TMEM lane = row, no exchange
// between threads) share the tensor cores: while one takes the softmax of its
// tile, the other's products run.  A stream's row tile is 128 / group
// whole tokens.  With more rows than that the streams
// hold a row tile each and share every K/V tile (32 bytes of K/V per SM clock at
// full tensor rate; one row tile would need the 64 that L2 can just deliver).  With
// fewer, both hold the same rows and take even and odd tiles, which halves the
// serial chain of a tile: those items are bound by the K/V bytes.  S and the
// rounded weights w share their TMEM columns (w is the second product's A
// operand, read from TMEM; V is read as staged, keys by dims).  The rounding of
// w to bf16 is what the product's A operand holds beside bf16 values: 2^-8 of
// sum_p softmax_p |V_p| at most, while l sums the unrounded weights.
//
// Measured (32 query heads on 8 KV heads of 128, graph replays): two prompts of
// 2500 and 4096 tokens 216 us, 875 TFLOP/s of visible products; 32 requests x 16
// rows over a shared prefix of 8192 and 256..4096 rows of their own 149 us
// (kernel 130, plan and join 19); 64 single tokens of 64 heads over a prefix of
// 16384 118 us; 128 requests x 16 rows over 64..14755 rows of their own and no
// prefix 625 us (3.9 GB of keys and values at 6.3 TB/s: HBM bounds it), with one
// row each 610 us; one token over 1001 keys 19 us.  Where HBM does not bound it a
// 128-key step takes a stream about 5000 clocks: 2350 in the softmax (TMEM reads,
// the maximum, exponentials and the rounding of 128 scores a thread), 1400 in its
// two products, the rest waiting for its turn at the tensor pipe and for
// barriers; the tensor pipe is 40% busy.
//
// Warps 0-3, 4-7: the streams; 8: TMA producer (a ring of K and V tiles, one
// copy per page and 64 dims); 9, 10: issue the MMAs of a stream each; 11
// completes the register split of the last warpgroup.
#include <cuda.h>

#include <algorithm>
#include <cstring>

#include "common.cuh"
#include "paged_rows.cuh"
#include "target_ops.h"

namespace dflash {
namespace {

constexpr int KT = 128;                   // keys of a tile
constexpr int THREADS = 384;
// registers a thread: 168 at launch (384 threads), then 208 for the streams and 80 for the rest
// (256 * 208 + 128 * 80 <= 384 * 168)
constexpr int REGS_STREAM = 208, REGS_REST = 80;
constexpr int PLAN_THREADS = 1024;
constexpr int NQ = 4;                     // items known ahead in a CTA
constexpr int EXTRA = 1024;               // items beyond one per (segment, head, row tile pair)
constexpr int MAX_SMS = EXTRA * 3 / 4;    // CTAs at most
constexpr int BUCKETS = 128;              // sizes that the item list is ordered by
// The weights of a tile go to the upper half of its S columns, so that the lower half can be read
// a second time.
constexpr int P_COL = KT / 2;
constexpr float TAU = 8.f;
constexpr uint32_t WAIT_NS = 20000;       // longest sleep of one try
constexpr uint32_t WAIT_LIMIT = 1u << 16; // tries (about a second)

template <int D> struct Cfg {
  static constexpr int TILE = KT * D * 2;             // K (or V) tile
  static constexpr int NSLOT = D == 128 ? 5 : 10;
  static constexpr int Q_TILE = 128 * D * 2;
  static constexpr int OFF_RING = 2 * Q_TILE;
  static constexpr int OFF_ML = OFF_RING + NSLOT * TILE;      // [128] float2
  static constexpr int OFF_BARS = OFF_ML + 128 * 8;
  // full[NSLOT], empty[NSLOT], s_full[2], turn[2], p_full[2], o_full[2], o_read[2], item_full[NQ],
  // item_empty[NQ], q_full, q_free, ml_full, ml_free, done; then the queue entries and a word
  static constexpr int N_BARS = 2 * NSLOT + 10 + 2 * NQ + 5;
  static constexpr int SMEM = 1024 + OFF_BARS + N_BARS * 8 + NQ * 48 + 32;
  static_assert(SMEM <= 227 * 1024, "one CTA per SM");
};

struct Item {
  int g, tok0, ntok, req;                 // KV head, first token, tokens, request (-1: prefix)
  int page0, ntiles, keys_left, part;     // first page, tiles, keys from the first to the segment's end, partial rows (-1: final)
  int lim_base, lim_slope, pad0, pad1;    // keys that row's token sees: lim_base + lim_slope * token
};
struct Request {
  int start, n, ctx, splits;              // first row, rows (0: skipped), own rows before them
  int tiles, part, pad0, pad1;            // key tiles of a split, first partial row (-1: none)
};
struct Head {
  int items, merge, prefix_splits, prefix_tiles;
  int first_row, rows, taken, redo;       // rows that meet the prefix; items handed out past one a CTA; rows to do again
};

// A row of an item to do again.
struct Redo {
  int at, req, page0, lim;                // token * H + head, request, first page, keys that the row sees
  int part, next, pad0, pad1;             // partial row (-1: final), next of the CTA's list (-1: none)
};

struct Params {
  CUtensorMap tmK, tmV;                   // dims {D, KVH, n_pages * 64}, box {64, 1, 64}
  CUtensorMap tmQ;                        // dims {D, H, total_rows}, box {64, G, 128 / G}
  PagedAttnParams a;
  Head *head;
  Item *items;
  Request *req;
  int *row_req;                           // [total_rows]
  Redo *redo;                             // [total_rows * H]
  float *part_o, *part_lse;               // [partial rows][D], [partial rows]
  int sms;
  float scale_log2;                       // |scale| log2 e
  int negative;                           // scale < 0: S changes its sign
};

// ------------------------------------------------------------------ PTX
__device__ __forceinline__ uint32_t su32(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void mbar_init(uint64_t *b, uint32_t n) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(su32(b)), "r"(n));
}
__device__ __forceinline__ void mbar_arrive(uint64_t *b) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(su32(b)) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t *b, uint32_t count) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(su32(b)), "r"(count) : "memory");
}
__device__ __forceinline__ bool mbar_try(uint32_t b, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(b), "r"(parity), "r"(WAIT_NS)
      : "memory");
  return ok != 0;
}
// Bounded wait for the phase of parity `parity`; false = gave up.  The thread
// sleeps in the barrier: eight warps that polled took a quarter of the shared
// memory bandwidth that the products need.
__device__ __forceinline__ bool mbar_wait(uint32_t b, uint32_t parity) {
  for (uint32_t i = 0; i < WAIT_LIMIT; ++i)
    if (mbar_try(b, parity)) return true;
  return false;
}
__device__ __forceinline__ bool mbar_wait(uint64_t *b, uint32_t parity) { return mbar_wait(su32(b), parity); }
__device__ __forceinline__ void tma3(void *dst, const CUtensorMap *tm, uint64_t *bar, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(su32(dst)),
      "l"((uint64_t)tm), "r"(su32(bar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}
__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void fence_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
// D += A B^T: both operands in shared memory, or A in TMEM
__device__ __forceinline__ void umma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void umma_commit(uint64_t *bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(su32(bar))
               : "memory");
}
// 32 columns of the warp's TMEM lanes, without the wait
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t *r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, "
      "%28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t *v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, "
      "%28, %29, %30, %31, %32};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
      "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]),
      "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]), "r"(v[21]),
      "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]),
      "r"(v[29]), "r"(v[30]), "r"(v[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(*reinterpret_cast<uint64_t *>(&d))
      : "l"(*reinterpret_cast<uint64_t *>(&a)), "l"(*reinterpret_cast<uint64_t *>(&b)),
        "l"(*reinterpret_cast<uint64_t *>(&c)));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(*reinterpret_cast<uint64_t *>(&d))
      : "l"(*reinterpret_cast<uint64_t *>(&a)), "l"(*reinterpret_cast<uint64_t *>(&b)));
  return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ void store32(void *p, const uint32_t *v) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
               "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Shared-memory operand descriptors, 128-byte swizzle: K-major (rows of 128
// bytes along K, 8-row groups 1 KB apart); MN-major (a row per K index, 64
// elements along N; `lbo` bytes between 64-element blocks).
__device__ __forceinline__ uint64_t desc_base(uint32_t saddr) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) |
         ((uint64_t)2 << 61);
}
__device__ __forceinline__ uint64_t desc_k(uint32_t saddr) { return desc_base(saddr) | ((uint64_t)1 << 16); }
__device__ __forceinline__ uint64_t desc_mn(uint32_t saddr, uint32_t lbo) {
  return desc_base(saddr) | ((uint64_t)((lbo >> 4) & 0x3FFFu) << 16);
}
// kind::f16: bf16 A and B, fp32 D; b_mn: B is MN-major
constexpr uint32_t idesc(int M, int N, bool b_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (b_mn ? (1u << 16) : 0u) | ((uint32_t)(N >> 3) << 17) |
         ((uint32_t)(M >> 4) << 24);
}

// Places of V(t) and K(t) in an item's load order: the first `ahead` K tiles,
// then V(0), K(ahead), V(1), K(ahead + 1), ...
__device__ __forceinline__ int order_v(int t, int n, int ahead) {
  return min(ahead, n) + t + min(t, max(0, n - ahead));
}

__device__ __forceinline__ int order_k(int t, int n, int ahead) {
  return t < ahead ? t : order_v(t - ahead, n, ahead) + 1;
}

__device__ __forceinline__ Item read_item(const int *p) {
  const int4 *s = reinterpret_cast<const int4 *>(p);
  const int4 a = s[0], b = s[1], c = s[2];
  Item it;
  it.g = a.x, it.tok0 = a.y, it.ntok = a.z, it.req = a.w;
  it.page0 = b.x, it.ntiles = b.y, it.keys_left = b.z, it.part = b.w;
  it.lim_base = c.x, it.lim_slope = c.y;
  return it;
}

// ------------------------------------------------------------------ plan
// One CTA: checks every request, chooses the key split of every segment (items
// of about U units, U an SM's share of them all; a unit is a 128-row tile by
// 128 keys), lays out partial rows and lists the items,
// large ones first (the CTAs take them from the list one by one).
__device__ __forceinline__ long long block_sum(long long v, long long *s) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
  __syncthreads();
  v = (threadIdx.x & 31) < (blockDim.x >> 5) ? s[threadIdx.x & 31] : 0;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
// exclusive scan; total in `total`
__device__ __forceinline__ int block_scan(int v, int *s, int &total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += x;
  }
  __syncthreads();
  if (lane == 31) s[warp] = inc;
  __syncthreads();
  int w = lane < (blockDim.x >> 5) ? s[lane] : 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += x;
  }
  total = __shfl_sync(0xffffffffu, w, 31);
  const int before = __shfl_sync(0xffffffffu, w, warp > 0 ? warp - 1 : 0);
  return (warp > 0 ? before : 0) + inc - v;
}
struct Split {
  int tiles, splits;
};
__device__ __forceinline__ Split split_keys(int nkt, int n, int tpt, long long U) {
  const int unit = n > tpt ? 2 : 1;       // row tiles of an item
  long long per = (U + unit - 1) / unit;
  per = per < 1 ? 1 : per;
  const int ns = nkt > 0 ? (int)((nkt + per - 1) / per) : 0;
  Split s;
  s.tiles = ns > 0 ? (nkt + ns - 1) / ns : 1;
  s.splits = (nkt + s.tiles - 1) / s.tiles;
  return s;
}
__device__ __forceinline__ int ceil_div(int a, int b) { return (a + b - 1) / b; }

__global__ void __launch_bounds__(PLAN_THREADS) paged_plan_kernel(const __grid_constant__ Params p) {
  pdl_wait();
  pdl_trigger();   // the attention CTAs set up their barriers and TMEM meanwhile, then wait for the plan
  __shared__ long long s_sum[32];
  __shared__ int s_scan[32];
  __shared__ int s_first[PLAN_THREADS + 2];     // first item of every segment (prefix, requests)
  __shared__ int s_start[PLAN_THREADS], s_n[PLAN_THREADS], s_ctx[PLAN_THREADS], s_tiles[PLAN_THREADS];
  __shared__ int s_part[PLAN_THREADS], s_splits[PLAN_THREADS];
  __shared__ int s_lo, s_hi;
  __shared__ int s_bucket[BUCKETS];             // items of a size, then the next place for one
  const PagedRows &r = p.a.rows;
  const int b = threadIdx.x, nt = blockDim.x, G = p.a.H / p.a.KVH, KVH = p.a.KVH, prefix = r.prefix_len;
  const int tpt = 128 / G;                      // tokens of a row tile
  if (b == 0) {
    s_lo = r.total_rows;
    s_hi = 0;
  }
  __syncthreads();
  int start = 0, n = 0, ctx = 0, claimed = 0;
  if (b < r.B) {
    const int a = r.row_start[b], e = r.row_start[b + 1], kv = r.kv_len[b];
    if (a < 0 || a > e || e > r.total_rows) {
      raise_error(p.a.err, DFLASH_DERR_ROW_RANGE);
    } else if (e > a) {
      claimed = e - a;
      if (kv < prefix || (int64_t)kv + (e - a) - prefix > (int64_t)r.pages_per_req * kPageRows) {
        raise_error(p.a.err, DFLASH_DERR_KV_CAPACITY);
      } else {
        start = a;
        n = e - a;
        ctx = kv - prefix;
        atomicMin(&s_lo, a);
        atomicMax(&s_hi, e);
      }
    }
  }
  __syncthreads();
  // more rows than there are: ranges overlap (a decreasing pair among them is flagged already), and
  // the workspace has no room for them; rows of requests that are skipped count too
  const bool fits = block_sum(claimed, s_sum) <= r.total_rows;
  if (!fits) {
    n = 0;
    if (b == 0) raise_error(p.a.err, DFLASH_DERR_ROW_RANGE);
  }
  const int lo = s_lo, rows = fits ? max(0, s_hi - s_lo) : 0;
  const int R = n * G, keys = ctx + n, nkt = n > 0 ? (keys + KT - 1) / KT : 0;
  const int Rp = prefix > 0 ? rows * G : 0, nktp = Rp > 0 ? prefix / KT + (prefix % KT != 0) : 0;
  const long long W = block_sum((long long)KVH * nkt * ceil_div(n, tpt), s_sum) +
                      (long long)KVH * nktp * ceil_div(rows, tpt);
  // At half an SM's share the SMs end more evenly, but there are twice the partial rows to write
  // and join: shared-prefix verification 160 us against 149, shared-prefix tokens 124 against 118,
  // prompts (whose requests' items are smaller than either) 216 both ways.
  long long U = (W + p.sms - 1) / p.sms;
  U = U < 2 ? 2 : U;
  // Items beyond one per (segment, KV head, pair of row tiles) are fewer than 4/3 W / U <= 4/3 SMs <=
  // EXTRA (a pair costs two units of its U in split_keys; segments of c row tiles have (c + 1) / 2
  // pairs and count c in W), each with the rows of at most 2 tpt tokens and of no more than there
  // are: the workspace has room for them.
  const Split sp = split_keys(nkt, n, tpt, U), spp = split_keys(nktp, rows, tpt, U);
  const bool joined = n > 0 && (prefix > 0 || sp.splits > 1);
  const int nrt = ceil_div(n, 2 * tpt), nrtp = Rp > 0 ? ceil_div(rows, 2 * tpt) : 0;
  const int prefix_rows = spp.splits * KVH * Rp, prefix_items = KVH * nrtp * spp.splits;
  int total_rows = 0, total_items = 0;
  const int part = block_scan(joined ? sp.splits * KVH * R : 0, s_scan, total_rows) + prefix_rows;
  const int items = block_scan(KVH * nrt * sp.splits, s_scan, total_items) + prefix_items;
  total_rows += prefix_rows;
  total_items += prefix_items;
  s_first[b + 1] = items;
  if (b == 0) {
    s_first[0] = 0;
    Head h;
    h.items = 0;                                // set below
    h.prefix_splits = spp.splits;
    h.prefix_tiles = spp.tiles;
    h.first_row = lo;
    h.rows = rows;
    h.merge = total_rows > 0;
    h.taken = h.redo = 0;
    *p.head = h;
  }
  s_start[b] = start;
  s_n[b] = n;
  s_ctx[b] = ctx;
  s_tiles[b] = sp.tiles;
  s_splits[b] = sp.splits;
  s_part[b] = joined ? part : -1;
  if (b < r.B) {
    Request q;
    q.start = start, q.n = n, q.ctx = ctx, q.splits = sp.splits;
    q.tiles = sp.tiles, q.part = joined ? part : -1, q.pad0 = q.pad1 = 0;
    p.req[b] = q;
  }
  __syncthreads();
  auto item_at = [&](int i) {
    // last segment whose first item is <= i (empty segments share a first item)
    int s0 = 0, s1 = r.B;
    while (s0 < s1) {
      const int mid = (s0 + s1 + 1) >> 1;
      if (s_first[mid] <= i) s0 = mid;
      else s1 = mid - 1;
    }
    Item it;
    const int j = i - s_first[s0];
    if (s0 == 0) {
      const int per = KVH * spp.splits, rt = j / per, g = j % per / spp.splits, s = j % spp.splits;
      it.g = g;
      it.tok0 = lo + rt * 2 * tpt;
      it.ntok = min(2 * tpt, rows - rt * 2 * tpt);
      it.req = -1;
      it.page0 = s * spp.tiles * 2;
      it.ntiles = min(spp.tiles, nktp - s * spp.tiles);
      it.keys_left = prefix - s * spp.tiles * KT;
      it.part = (g * spp.splits + s) * Rp + rt * 2 * tpt * G;
      it.lim_base = it.keys_left;
      it.lim_slope = 0;
    } else {
      const int q = s0 - 1, ns = s_splits[q], tiles = s_tiles[q], nq = s_n[q], c = s_ctx[q], st = s_start[q];
      const int Rq = nq * G, per = KVH * ns;
      const int rt = j / per, g = j % per / ns, s = j % ns;
      const int last = min(nq, (rt + 1) * 2 * tpt) - 1;        // last token of the row tiles
      const int seen = p.a.causal ? c + last + 1 : c + nq;
      it.g = g;
      it.tok0 = st + rt * 2 * tpt;
      it.ntok = min(2 * tpt, nq - rt * 2 * tpt);
      it.req = q;
      it.page0 = s * tiles * 2;
      it.ntiles = max(0, min(tiles, (seen + KT - 1) / KT - s * tiles));
      it.keys_left = c + nq - s * tiles * KT;
      it.part = s_part[q] >= 0 ? s_part[q] + (g * ns + s) * Rq + rt * 2 * tpt * G : -1;
      it.lim_slope = p.a.causal;
      it.lim_base = (p.a.causal ? c + 1 - st : c + nq) - s * tiles * KT;
    }
    it.pad0 = it.pad1 = 0;
    return it;
  };
  // larger items first (in units of half a row tile, so that a lone row tile counts three: its
  // products have half the rows but its K/V tiles are its own)
  auto bucket_of = [&](const Item &it) {
    const int size = it.ntiles * (it.ntok > tpt ? 4 : 3);
    return BUCKETS - 1 - min(BUCKETS - 1, size <= 64 ? size : 64 + (size - 64) / 16);
  };
  for (int i = b; i < BUCKETS; i += nt) s_bucket[i] = 0;
  __syncthreads();
  for (int i = b; i < total_items; i += nt) {
    const Item it = item_at(i);
    if (it.ntiles > 0) atomicAdd(&s_bucket[bucket_of(it)], 1);
  }
  __syncthreads();
  int listed = 0;
  {
    const int v = b < BUCKETS ? s_bucket[b] : 0;
    const int at = block_scan(v, s_scan, listed);
    __syncthreads();
    if (b < BUCKETS) s_bucket[b] = at;
  }
  __syncthreads();
  if (b == 0) p.head->items = listed;
  for (int i = b; i < total_items; i += nt) {
    const Item it = item_at(i);
    if (it.ntiles > 0) p.items[atomicAdd(&s_bucket[bucket_of(it)], 1)] = it;
  }
  if (total_rows > 0) {   // the owner of every row, for the join
    for (int t = b; t < r.total_rows; t += nt) p.row_req[t] = -1;
    __syncthreads();
    for (int q = b >> 5; q < r.B; q += nt / 32)
      for (int t = b & 31; t < s_n[q]; t += 32) p.row_req[s_start[q] + t] = q;
  }
}

// ------------------------------------------------------------------ attention
// The matrix product multiplies the values of keys that a row does not see by 0, which is not 0 for
// a value that is not finite.  Such keys are in the tiles that hold a row tile's own tokens, where
// the result gives them away (`odd`); the warp then looks for the last of them here (fewer than 2 * 128 +
// 128 keys lie between `lim`, the keys that a row sees, and `end`) and lists the rows before it, which
// the CTA does again once it has no more items: nothing waits for it then, however many keys they see.
template <int D>
__device__ __noinline__ void list_spoiled(const Params &p, int *s_redo, int req, int g, int page0, int at, int part,
                                          int lim, int end, bool odd) {
  const int from = __reduce_min_sync(0xffffffffu, odd ? lim : end);
  const int *list = p.a.rows.page_table + (int64_t)req * p.a.rows.pages_per_req + page0;
  constexpr int C = D / 8;                 // 16-byte chunks of a key's values
  int last = -1;
  for (int i = (int)(threadIdx.x & 31); i < (end - from) * C; i += 32) {
    const int key = from + i / C, pg = list[key / kPageRows];
    const int64_t slot = (int64_t)(pg >= 0 && pg < p.a.rows.n_pages ? pg : 0) * kPageRows + key % kPageRows;
    const uint4 v = *(reinterpret_cast<const uint4 *>((const bf16 *)p.a.v_pages + (slot * p.a.KVH + g) * D) + i % C);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e)            // exponents of all ones
      if ((w[e] & 0x7f80u) == 0x7f80u || (w[e] & 0x7f800000u) == 0x7f800000u) last = key;
  }
  last = __reduce_max_sync(0xffffffffu, last);
  if (odd && lim <= last) {                // (a row has such keys in one split at most)
    const int i = atomicAdd(&p.head->redo, 1);
    Redo e;
    e.at = at, e.req = req, e.page0 = page0, e.lim = lim;
    e.part = part, e.next = atomicExch(s_redo, i), e.pad0 = e.pad1 = 0;
    p.redo[i] = e;
  }
}

// The rows of the CTA's list over their visible keys alone, by its first 256 threads.  A warp takes 32
// keys at a time, a key a lane for the scores, D / 32 dims a lane for the values; the row's weight (lse)
// stands already, as no score of a hidden key enters it.  24 ns a key and row (12 with 64 dims): 16 rows
// over 200000 keys 78 ms.
template <int D> __device__ __noinline__ void redo_rows(const Params &p, int first, float *sm) {
  constexpr int W = 8, V = D / 32;
  float *s_q = sm, *s_m = s_q + D, *s_l = s_m + W, *s_o = s_l + W;      // [D], [W], [W], [W][D]
  const int H = p.a.H, KVH = p.a.KVH, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const PagedRows &r = p.a.rows;
  const float scale = p.negative ? -p.scale_log2 : p.scale_log2;
  auto sync = [] { asm volatile("bar.sync 1, 256;" ::: "memory"); };
  for (int next; first >= 0; first = next) {
    const Redo e = p.redo[first];
    next = e.next;
    const int t = e.at / H, h = e.at % H, g = h / (H / KVH);
    const int *list = r.page_table + (int64_t)e.req * r.pages_per_req + e.page0;
    sync();                                // the row before has been read
    for (int d = threadIdx.x; d < D; d += 256)
      s_q[d] = to_f32(((const bf16 *)p.a.q)[(int64_t)t * p.a.q_stride + (int64_t)h * D + d]);
    sync();
    float m = -INFINITY, l = 0.f, o[V];
#pragma unroll
    for (int c = 0; c < V; ++c) o[c] = 0.f;
    for (int k0 = 32 * warp; k0 < e.lim; k0 += 32 * W) {
      const int key = k0 + lane, n = min(32, e.lim - k0);
      int64_t slot = 0;
      float x = -INFINITY;
      if (lane < n) {
        const int pg = list[key / kPageRows];
        slot = (((int64_t)(pg >= 0 && pg < r.n_pages ? pg : 0) * kPageRows + key % kPageRows) * KVH + g) * D;
        const uint4 *k = reinterpret_cast<const uint4 *>((const bf16 *)p.a.k_pages + slot);
        float dot = 0.f;
#pragma unroll 8
        for (int c = 0; c < D / 8; ++c) {
          const uint4 u = k[c];
          const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            dot = fmaf(s_q[8 * c + 2 * i], __uint_as_float(w[i] << 16), dot);
            dot = fmaf(s_q[8 * c + 2 * i + 1], __uint_as_float(w[i] & 0xffff0000u), dot);
          }
        }
        x = dot * scale;
      }
      const float mx = fmaxf(m, warp_max(x)), base = mx == -INFINITY ? 0.f : mx;
      const float w = ex2(x - base), alpha = ex2(m - base);
      m = mx;
      l = l * alpha + warp_sum(w);
#pragma unroll
      for (int c = 0; c < V; ++c) o[c] *= alpha;
      for (int j0 = 0; j0 < n; j0 += 8) {  // eight keys' values in flight
        uint32_t u[8][V / 2];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const bf16 *v = (const bf16 *)p.a.v_pages + __shfl_sync(0xffffffffu, slot, j0 + j) + lane * V;
#pragma unroll
          for (int c = 0; c < V / 2; ++c)
            u[j][c] = j0 + j < n ? reinterpret_cast<const uint32_t *>(v)[c] : 0u;   // (a key that is none weighs 0)
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float wj = __shfl_sync(0xffffffffu, w, j0 + j);
#pragma unroll
          for (int c = 0; c < V / 2; ++c) {
            o[2 * c] = fmaf(wj, __uint_as_float(u[j][c] << 16), o[2 * c]);
            o[2 * c + 1] = fmaf(wj, __uint_as_float(u[j][c] & 0xffff0000u), o[2 * c + 1]);
          }
        }
      }
    }
#pragma unroll
    for (int c = 0; c < V; ++c) s_o[warp * D + lane * V + c] = o[c];
    if (lane == 0) {
      s_m[warp] = m;
      s_l[warp] = l;
    }
    sync();
    for (int d = threadIdx.x; d < D; d += 256) {
      float mx = -INFINITY, den = 0.f, num = 0.f;
      for (int w = 0; w < W; ++w) mx = fmaxf(mx, s_m[w]);
      const float base = mx == -INFINITY ? 0.f : mx;
      for (int w = 0; w < W; ++w) {
        if (s_l[w] == 0.f) continue;       // a warp without keys
        const float f = ex2(s_m[w] - base);
        den = fmaf(f, s_l[w], den);
        num = fmaf(f, s_o[w * D + d], num);
      }
      const float x = num / den;
      if (e.part >= 0) p.part_o[(int64_t)e.part * D + d] = x;
      else ((bf16 *)p.a.out)[(int64_t)t * p.a.out_stride + (int64_t)h * D + d] = __float2bfloat16_rn(x);
    }
  }
}

template <int D>
__global__ void __launch_bounds__(THREADS, 1) paged_attention_kernel(const __grid_constant__ Params p) {
  using C = Cfg<D>;
  constexpr int NS = C::NSLOT, NB = D / 64;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint8_t *ring = smem + C::OFF_RING;
  float2 *s_ml = (float2 *)(smem + C::OFF_ML);
  uint64_t *full = (uint64_t *)(smem + C::OFF_BARS), *empty = full + NS;
  uint64_t *s_full = empty + NS, *turn = s_full + 2, *p_full = turn + 2, *o_full = p_full + 2;
  uint64_t *o_read = o_full + 2, *item_full = o_read + 2, *item_empty = item_full + NQ;
  uint64_t *q_full = item_empty + NQ, *q_free = q_full + 1, *ml_full = q_free + 1, *ml_free = ml_full + 1;
  uint64_t *done = ml_free + 1;
  int *s_items = (int *)(((uintptr_t)(done + 1) + 15) & ~(uintptr_t)15);   // [NQ][12]
  uint32_t *s_tmem = (uint32_t *)(s_items + NQ * 12);
  int *s_redo = s_items + NQ * 12 + 1;   // last of the CTA's rows to do again (-1: none)
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = p.a.H / p.a.KVH, tpt = 128 / G, rt_rows = tpt * G;   // tokens and rows of a row tile

  if (threadIdx.x == 0) {
    *s_redo = -1;
    for (int i = 0; i < NS; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 2);            // released by both streams, or twice by the one that used it
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&turn[i], 1);
      mbar_init(&p_full[i], 128);
      mbar_init(&o_full[i], 1);
      mbar_init(&o_read[i], 128);
    }
    for (int i = 0; i < NQ; ++i) {
      mbar_init(&item_full[i], 1);
      mbar_init(&item_empty[i], 10);      // a lane of each MMA and stream warp
    }
    mbar_init(q_full, 1);
    mbar_init(q_free, 2);
    mbar_init(ml_full, 128);
    mbar_init(ml_free, 128);
    mbar_init(done, 2);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 9) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(su32(s_tmem))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (warp == 8 && lane == 0) {
    asm volatile("prefetch.tensormap [%0];" ::"l"((uint64_t)&p.tmK) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"((uint64_t)&p.tmV) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"((uint64_t)&p.tmQ) : "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;
  pdl_wait();
  const int n_items = __ldcg(&p.head->items);
  bool ok = true;
  // consumers: the CTA's i-th item (a warp's wait); false at the end or after a timeout
  uint32_t n_item = 0;
  auto next_item = [&](Item &it) {
    const int e = n_item % NQ;
    if (ok && !mbar_wait(&item_full[e], (n_item / NQ) & 1)) ok = false;
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) return false;
    it = read_item(s_items + e * 12);
    __syncwarp();
    if (lane == 0) mbar_arrive(&item_empty[e]);
    ++n_item;
    return it.ntiles > 0;
  };

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_REST));
    if (warp == 8) {
      // ------------------------------------------------------------ producer (one warp)
      uint32_t u = 0, k = 0;                // tiles issued, items begun
      int slot = 0, phase = 1;              // place in the ring; parity of its empty barrier
      Item it;
      int prev0 = 0, prev1 = 0, cur0 = 0, cur1 = 0;   // pages of the last two K tiles
      // the next item of the list, to the other warps as well (0 tiles: no more)
      auto take_item = [&] {
        const int e = n_item % NQ;
        int idx = 0;
        if (lane == 0) {
          if (!mbar_wait(&item_empty[e], ((n_item / NQ) & 1) ^ 1)) idx = -1;
          else idx = n_item == 0 ? blockIdx.x : gridDim.x + atomicAdd(&p.head->taken, 1);
        }
        idx = __shfl_sync(0xffffffffu, idx, 0);
        if (idx < 0) {
          ok = false;
          return false;
        }
        if (lane < 12) s_items[e * 12 + lane] = idx < n_items ? __ldcg((const int *)(p.items + idx) + lane) : 0;
        __syncwarp();
        it = read_item(s_items + e * 12);
        if (lane == 0) mbar_arrive(&item_full[e]);
        ++n_item;
        return it.ntiles > 0;
      };
      while (ok && take_item()) {
        const int n = it.ntiles, ahead = it.ntok > tpt ? 1 : 2;
        const int npages = (min(it.keys_left, n * KT) + kPageRows - 1) / kPageRows;
        const int *list = (it.req < 0 ? p.a.rows.prefix_pages
                                      : p.a.rows.page_table + (int64_t)it.req * p.a.rows.pages_per_req) + it.page0;
        int batch = 0;
        auto issue = [&](const CUtensorMap *tm, int t, int pg0, int pg1) {
          bool good = true;
          if (lane == 0) {
            good = mbar_wait(&empty[slot], phase);
            if (good) {
              const bool two = 2 * t + 1 < npages;
              asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(su32(&full[slot])),
                           "r"(two ? C::TILE : C::TILE / 2)
                           : "memory");
              uint8_t *dst = ring + slot * C::TILE;
#pragma unroll
              for (int c = 0; c < NB; ++c) {
                tma3(dst + c * (KT * 128), tm, &full[slot], 64 * c, it.g, pg0 * kPageRows);
                if (two) tma3(dst + c * (KT * 128) + 8192, tm, &full[slot], 64 * c, it.g, pg1 * kPageRows);
              }
            }
          }
          ok = __shfl_sync(0xffffffffu, good, 0) != 0;
          if (!ok) return;
          ++u;
          if (++slot == NS) {
            slot = 0;
            phase ^= 1;
          }
        };
        auto issue_k = [&](int t) {
          const int j = 2 * t;
          if (j % 32 == 0) {                // the next 32 pages, one a lane
            int pg = 0;
            if (j + lane < npages) {
              pg = __ldg(list + j + lane);
              if (pg < 0 || pg >= p.a.rows.n_pages) {
                raise_error(p.a.err, DFLASH_DERR_PAGE_RANGE);
                pg = 0;
              }
            }
            batch = pg;
          }
          prev0 = cur0, prev1 = cur1;
          cur0 = __shfl_sync(0xffffffffu, batch, j % 32);
          cur1 = __shfl_sync(0xffffffffu, batch, j % 32 + 1);
          issue(&p.tmK, t, cur0, cur1);
        };
        // the query rows, once the last S of the item before has read its own
        auto issue_q = [&] {
          bool good = true;
          if (lane == 0) {
            if (k > 0) good = mbar_wait(q_free, (k - 1) & 1);
            if (good) {
              const int tiles = it.ntok > tpt ? 2 : 1;
              asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(su32(q_full)),
                           "r"(tiles * rt_rows * D * 2)
                           : "memory");
              for (int x = 0; x < tiles; ++x)
#pragma unroll
                for (int c = 0; c < NB; ++c)
                  tma3(smem + x * C::Q_TILE + c * (128 * 128), &p.tmQ, q_full, 64 * c, it.g * G, it.tok0 + x * tpt);
            }
          }
          ok = __shfl_sync(0xffffffffu, good, 0) != 0;
          if (ok) ++k;
        };
        // the K tiles that go ahead find free slots before Q is free
        for (int t = 0; t < min(ahead, n) && ok; ++t) issue_k(t);
        if (ok) issue_q();
        for (int t = 0; t < n && ok; ++t) {
          // K(t) is the last K tile issued, or the one before it
          const bool older = ahead == 2 && t + 1 < n;
          issue(&p.tmV, t, older ? prev0 : cur0, older ? prev1 : cur1);
          if (ok && t + ahead < n) issue_k(t + ahead);
        }
      }
      if (lane == 0) {
        if (!ok) raise_error(p.a.err, DFLASH_DERR_TIMEOUT);
        // every copy has landed before the CTA exits
        for (uint32_t v = u > (uint32_t)NS ? u - NS : 0; v < u; ++v) mbar_wait(&full[v % NS], (v / NS) & 1);
        if (k > 0) mbar_wait(q_full, (k - 1) & 1);
      }
    } else if (warp <= 10) {
      // ------------------------------------------------------------ MMA issuers: a lane a stream
      // Groups of MMAs alternate between the streams (a token goes back and forth), which keeps
      // them out of phase: one's softmax runs while the other's products do.  Without the token
      // the two fall into step, both S ready at once, then both in the softmax and the tensor
      // cores idle; one issuer for both needs 2300 clocks a step, half of them for waits and
      // addresses.  Commits cost the tensor pipe 40 to 80 clocks each, so a step has one: S of the
      // stream's next tile, after which the tiles that the step has read are released by the
      // stream that waits for that S.
      const uint32_t x = warp - 9;
      if (lane == 0) {
        constexpr uint32_t ID_S = idesc(128, KT, false), ID_O = idesc(128, D, true);
        const uint64_t k_desc = desc_k(su32(ring)), v_desc = desc_mn(su32(ring), KT * 128);
        const uint32_t full_at = su32(full), p_at = su32(&p_full[x]);
        const uint32_t t_s = tmem + x * KT, t_o = tmem + 256 + x * 128;
        uint32_t k = 0, u = 0, c = 0;     // items, ring tiles, tiles of this stream before
        uint32_t n_o = 0, n_turn = 0;     // items of this stream, tokens received before
        int owner = 0;                    // stream of the group before
        auto wait = [&](uint32_t bar, uint32_t parity) {
          if (mbar_try(bar, parity)) return;
          if (ok && !mbar_wait(bar, parity)) ok = false;
        };
        auto take_turn = [&] { wait(su32(&turn[x]), n_turn++ & 1); };
        Item it;
        while (ok) {
          const int e = k % NQ;
          wait(su32(&item_full[e]), (k / NQ) & 1);
          if (!ok) break;
          it = read_item(s_items + e * 12);
          mbar_arrive(&item_empty[e]);
          if (it.ntiles == 0) break;
          // The stream's tiles t0, t0 + dt, ...: all of a pair's, every other one of a single row
          // tile's.  Groups: S of stream 0's first tile, of stream 1's, then step by step O += w V(t)
          // and S of the stream's next tile; streams 0, 1, 0, ... in both kinds.
          const int n = it.ntiles, pair = it.ntok > tpt ? 1 : 0, dt = 2 - pair, t0 = pair ? 0 : (int)x;
          const bool two = (n << pair) > 1;                    // stream 1 has tiles
          const int last_owner = ((n << pair) - 1) & 1;
          const uint64_t q_desc = desc_k(su32(smem) + (pair & x) * C::Q_TILE);
          auto wait_tile = [&](int order) { wait(full_at + 8 * ((u + order) % NS), ((u + order) / NS) & 1); };
          auto issue_s = [&](int order) {
            const uint64_t kd = k_desc + ((u + order) % NS) * (C::TILE >> 4);
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
              umma_ss(t_s, q_desc + (i >> 2) * ((128 * 128) >> 4) + 2 * (i & 3),
                      kd + (i >> 2) * ((KT * 128) >> 4) + 2 * (i & 3), ID_S, i ? 1u : 0u);
            umma_commit(&s_full[x]);
          };
          wait(su32(q_full), k & 1);
          ++k;
          if (t0 < n) {
            const int order = order_k(t0, n, dt);
            wait_tile(order);
            if (x == 1 || owner == 1) take_turn();
            if (!ok) break;
            tc_fence_after();
            issue_s(order);
            if (two) mbar_arrive(&turn[x ^ 1]);
          }
#pragma unroll 1
          for (int t = t0; t < n; t += dt) {
            const int order = order_v(t, n, dt);
            const uint64_t vd = v_desc + ((u + order) % NS) * (C::TILE >> 4);
            const bool more = t + dt < n;
            if (t == t0) {                // the item before has read this stream's O
              if (n_o > 0) wait(su32(&o_read[x]), (n_o - 1) & 1);
              ++n_o;
            }
            wait_tile(order);
            if (more) wait_tile(order + 1);
            wait(p_at, c & 1);
            ++c;
            if (two) take_turn();
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < KT / 16; ++kk)
              umma_ts(t_o, t_s + P_COL + kk * 8, vd + kk * (2048 >> 4), ID_O, (t == t0 && kk == 0) ? 0u : 1u);
            if (more) issue_s(order + 1);
            else umma_commit(&o_full[x]);
            // the other stream's step, or after the item's last the next item's first group, stream 0's
            if (two && (x == 1 || more || !(last_owner == 0))) mbar_arrive(&turn[x ^ 1]);
          }
          if (!ok) break;
          owner = last_owner;
          u += 2 * n;
        }
        umma_commit(done);
        if (!mbar_wait(su32(done), 0)) ok = false;   // every MMA has ended before TMEM is freed
        if (!ok) raise_error(p.a.err, DFLASH_DERR_TIMEOUT);
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS_STREAM));
    // ------------------------------------------------------------ softmax, a row a thread
    const int x = warp >> 2, row = threadIdx.x & 127;          // stream, row of its tile
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t t_s = tmem + lanes + x * KT;
    const float sl = p.scale_log2;
    const bool wide = (((uintptr_t)p.a.out | (uint64_t)(p.a.out_stride * 2)) & 31) == 0;   // 32-byte rows
    // every wait is one for the warp, so that its lanes stay together
    auto wait = [&](uint64_t *b, uint32_t parity) {
      if (ok && !mbar_wait(b, parity)) ok = false;
      ok = __all_sync(0xffffffffu, ok);
    };
    uint32_t c = 0, u = 0, o_par = 0, n_ml = 0;   // o_par bit x: parity of o_full[x]
    const int row_tok = row / G, row_head = row % G;
    Item it;
    while (ok && next_item(it)) {
      const int n = it.ntiles;
      const bool pair = it.ntok > tpt;
      const int ahead = pair ? 1 : 2;
      const int mine = (pair ? x * tpt : 0) + row_tok;         // this thread's token of the item
      const bool own = row < rt_rows && mine < it.ntok;
      const bool live = ((pair ? x * tpt : 0) + ((warp & 3) * 32) / G) < it.ntok && (warp & 3) * 32 < rt_rows;
      const int tok = it.tok0 + mine, h = it.g * G + row_head;
      // (rows that nobody owns see every key: the mask costs a warp its fast path)
      const int lim = own ? it.lim_base + it.lim_slope * tok : 1 << 30;
      float m = -INFINITY, l = 0.f;
      const uint32_t uses = pair ? 1 : 2;   // of a tile by this stream, of the two that free it
      auto release = [&](int order) { mbar_arrive(&empty[(u + order) % NS], uses); };
      // V rows past the segment's last key may hold anything: 0 times it has to be 0
      auto clear_v = [&](int t) {
        if (t != n - 1 || it.keys_left >= n * KT) return;
        const int ov = u + order_v(t, n, ahead);
        wait(&full[ov % NS], (ov / NS) & 1);
        if (!ok) return;
        uint8_t *vt = ring + (ov % NS) * C::TILE;
        for (int i = (it.keys_left - t * KT) * 8 + row; i < KT * 8; i += 128)
#pragma unroll
          for (int b = 0; b < NB; ++b)
            *reinterpret_cast<uint4 *>(vt + b * (KT * 128) + i * 16) = make_uint4(0, 0, 0, 0);
        fence_async_smem();
      };
      for (int t = pair ? 0 : x; t < n && ok; t += pair ? 1 : 2) {
        wait(&s_full[x], c & 1);
        if (!ok) break;
        ++c;
        tc_fence_after();
        if (row == 96) {                   // S has read K(t), and the product before it its V
          release(order_k(t, n, ahead));
          if (t >= ahead) release(order_v(t - ahead, n, ahead));
          if (t + ahead >= n) mbar_arrive(q_free, !pair && n == 1 ? 2 : 1);   // its last S
        }
        if (live) {
          // keys 0..63 for their maximum, then keys 64..127 and their weights, then keys 0..63 again: reading TMEM twice is cheaper than 128 live registers
          uint32_t sv[KT / 2];
          auto load = [&](int half) {
            tmem_ld32(t_s + half * 64, sv);
            tmem_ld32(t_s + half * 64 + 32, sv + 32);
            tmem_ld_wait();
            if (p.negative) {
#pragma unroll
              for (int i = 0; i < 64; ++i) sv[i] ^= 0x80000000u;
            }
          };
          const int vis = lim - t * KT;                        // visible keys of this tile
          const bool whole = __all_sync(0xffffffffu, vis >= KT);
          auto maximum = [&](int half, float a0) {
            if (whole) {
              float a1 = __uint_as_float(sv[0]), a2 = __uint_as_float(sv[1]), a3 = __uint_as_float(sv[2]);
              a0 = fmaxf(a0, __uint_as_float(sv[3]));
#pragma unroll
              for (int i = 4; i < 60; i += 8) {
                a0 = max3(a0, __uint_as_float(sv[i]), __uint_as_float(sv[i + 1]));
                a1 = max3(a1, __uint_as_float(sv[i + 2]), __uint_as_float(sv[i + 3]));
                a2 = max3(a2, __uint_as_float(sv[i + 4]), __uint_as_float(sv[i + 5]));
                a3 = max3(a3, __uint_as_float(sv[i + 6]), __uint_as_float(sv[i + 7]));
              }
              a0 = max3(a0, __uint_as_float(sv[60]), __uint_as_float(sv[61]));
              a1 = max3(a1, __uint_as_float(sv[62]), __uint_as_float(sv[63]));
              return max3(fmaxf(a0, a1), a2, a3);
            }
#pragma unroll
            for (int i = 0; i < 64; ++i) a0 = half * 64 + i < vis ? fmaxf(a0, __uint_as_float(sv[i])) : a0;
            return a0;
          };
          load(0);
          float mx = maximum(0, -INFINITY);
          load(1);
          mx = maximum(1, mx);
          mx = vis > 0 ? mx * sl : -INFINITY;
          float alpha = 1.f;
          if (mx > m + TAU || m == -INFINITY) {
            if (m != -INFINITY) alpha = ex2(m - mx);
            m = mx;
          }
          const float mm = m == -INFINITY ? 0.f : m;
          const float2 sl2 = make_float2(sl, sl), mm2 = make_float2(-mm, -mm);
          float2 sum = make_float2(0.f, 0.f);
          auto weights = [&](int half) {
            uint32_t w[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const int e = half * 64 + 2 * i;
              const float2 a = fma2(make_float2(__uint_as_float(sv[2 * i]), __uint_as_float(sv[2 * i + 1])), sl2, mm2);
              float2 q = make_float2(ex2(a.x), ex2(a.y));
              if (!whole) {
                q.x = e < vis ? q.x : 0.f;
                q.y = e + 1 < vis ? q.y : 0.f;
              }
              sum = add2(sum, q);
              __nv_bfloat162 h2 = __floats2bfloat162_rn(q.x, q.y);
              w[i] = *reinterpret_cast<uint32_t *>(&h2);
            }
            tmem_st32(t_s + P_COL + half * 32, w);
          };
          weights(1);
          if (__any_sync(0xffffffffu, alpha != 1.f)) {
            // S of this tile was issued after the last O product of the stream: O is at rest
#pragma unroll
            for (int i = 0; i < D; i += 32) {
              uint32_t o[32];
              tmem_ld32(tmem + lanes + 256 + x * 128 + i, o);
              tmem_ld_wait();
#pragma unroll
              for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * alpha);
              tmem_st32(tmem + lanes + 256 + x * 128 + i, o);
            }
          }
          load(0);
          weights(0);
          l = fmaf(l, alpha, sum.x + sum.y);
          tmem_st_wait();
        }
        clear_v(t);
        tc_fence_before();
        mbar_arrive(&p_full[x]);
      }
      if (!ok) break;
      // ---- the item's rows: o / l and log2 of their weight, or the result
      const bool both = !pair && n > 1;    // the other stream holds the odd tiles' share
      if (both && x == 1) {
        if (n_ml > 0) wait(ml_free, (n_ml - 1) & 1);
        if (!ok) break;
        s_ml[row] = make_float2(m, l);
        mbar_arrive(ml_full);
      }
      if (pair || x == 0) {
        wait(&o_full[x], (o_par >> x) & 1);
        float a0 = 1.f, a1 = 0.f;
        if (both) {
          wait(&o_full[1], (o_par >> 1) & 1);
          wait(ml_full, n_ml & 1);
          if (!ok) break;
          const float2 ml = s_ml[row];
          const float ms = fmaxf(m, ml.x), base = ms == -INFINITY ? 0.f : ms;
          a0 = ex2(m - base);
          a1 = ex2(ml.x - base);
          l = l * a0 + ml.y * a1;
          m = ms;
          mbar_arrive(ml_free);
        }
        if (!ok) break;
        tc_fence_after();
        if (row == 0) {                    // the last V tiles
          release(order_v(n - 1, n, ahead));
          if (both) release(order_v(n - 2, n, ahead));
        }
        if (live) {
          // a split may hold no key that the row sees; a whole row of -infinities has no result (NaN)
          const float inv = l == 0.f && it.part >= 0 ? 0.f : 1.f / l;
          // keys of these tiles that the row does not see
          const int end = min(n * KT, it.keys_left);
          const bool hides = own && lim < end && l != 0.f;
          bool odd = false;
          a0 *= inv;
          a1 *= inv;
          bf16 *out = (bf16 *)p.a.out + (int64_t)tok * p.a.out_stride + (int64_t)h * D;
          const int at = it.part + mine * G + row_head;        // partial row
          float *po = p.part_o + (int64_t)at * D;
          if (own && it.part >= 0) p.part_lse[at] = l == 0.f ? -INFINITY : m + log2f(l);
#pragma unroll
          for (int i = 0; i < D; i += 32) {
            uint32_t o[32];
            tmem_ld32(tmem + lanes + 256 + x * 128 + i, o);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(a0 != 0.f ? __uint_as_float(o[j]) * a0 : 0.f);
            if (both) {
              uint32_t q[32];
              tmem_ld32(tmem + lanes + 256 + 128 + i, q);
              tmem_ld_wait();
#pragma unroll
              for (int j = 0; j < 32; ++j)
                o[j] = __float_as_uint(__uint_as_float(o[j]) + (a1 != 0.f ? __uint_as_float(q[j]) * a1 : 0.f));
            }
            if (hides) {
#pragma unroll
              for (int j = 0; j < 32; ++j) odd = odd || !isfinite(__uint_as_float(o[j]));
            }
            // 32 bytes a store: whole sectors, as a lane's rows are far apart
            if (own && it.part >= 0) {
#pragma unroll
              for (int j = 0; j < 32; j += 8) store32(po + i + j, o + j);
            } else if (own) {
#pragma unroll
              for (int j = 0; j < 32; j += 16) {
                uint32_t w[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                  __nv_bfloat162 h2 = __floats2bfloat162_rn(__uint_as_float(o[j + 2 * e]),
                                                            __uint_as_float(o[j + 2 * e + 1]));
                  w[e] = *reinterpret_cast<uint32_t *>(&h2);
                }
                if (wide) {
                  store32(out + i + j, w);
                } else {
                  *reinterpret_cast<uint4 *>(out + i + j) = make_uint4(w[0], w[1], w[2], w[3]);
                  *reinterpret_cast<uint4 *>(out + i + j + 8) = make_uint4(w[4], w[5], w[6], w[7]);
                }
              }
            }
          }
          if (__builtin_expect(__any_sync(0xffffffffu, odd), 0))
            list_spoiled<D>(p, s_redo, it.req, it.g, it.page0, tok * p.a.H + h, it.part >= 0 ? at : -1, lim, end, odd);
        }
        tc_fence_before();
        mbar_arrive(&o_read[x]);
        if (both) mbar_arrive(&o_read[1]);
      }
      // streams that took part in this item
      o_par ^= pair || n > 1 ? 3u : 1u;
      if (both) ++n_ml;
      u += 2 * n;
    }
    if (!ok && lane == 0) raise_error(p.a.err, DFLASH_DERR_TIMEOUT);
  }
  tc_fence_before();
  __syncthreads();
  // (every copy has landed and every product ended: the ring is free)
  if (__builtin_expect(*s_redo >= 0, 0)) {
    if (threadIdx.x < 256) redo_rows<D>(p, *s_redo, reinterpret_cast<float *>(ring));
    __syncthreads();
  }
  pdl_trigger();   // every global write of this CTA is done
  if (warp == 9) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }
}

// ------------------------------------------------------------------ join
// A warp a (row, head): out = sum_i 2^(lse_i - max) o_i / sum_i 2^(lse_i - max)
// over the prefix splits and the own splits whose first key the row sees.
// Eight lanes read one partial row, so that a warp has four in flight.
template <int D>
__global__ void __launch_bounds__(256) paged_join_kernel(const __grid_constant__ Params p) {
  pdl_wait();
  const Head *head = p.head;
  const int4 h0 = __ldcg(reinterpret_cast<const int4 *>(head)), h1 = __ldcg(reinterpret_cast<const int4 *>(head) + 1);
  if (!h0.y) return;
  constexpr int C = D / 32;                // 16-byte chunks a lane
  const int lane = threadIdx.x & 31, sub = lane & 7, quarter = lane >> 3;
  const int H = p.a.H, KVH = p.a.KVH, G = H / KVH;
  const int nsp = h0.z, first = h1.x, Rp = p.a.rows.prefix_len > 0 ? h1.y * G : 0;
  const int total = p.a.rows.total_rows * H, step = gridDim.x * (blockDim.x >> 5);
  for (int idx = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); idx < total; idx += step) {
    const int t = idx / H, h = idx % H, g = h / G;
    const int b = __ldcg(p.row_req + t);
    if (b < 0) continue;
    const int4 r0 = __ldcg(reinterpret_cast<const int4 *>(p.req + b));
    const int4 r1 = __ldcg(reinterpret_cast<const int4 *>(p.req + b) + 1);
    if (r1.y < 0) continue;                // written by its one item
    const int R = r0.y * G, seen = p.a.causal ? r0.z + (t - r0.x) + 1 : r0.z + r0.y;
    const int span = r1.x * KT, own = min(r0.w, (seen + span - 1) / span);
    const int64_t at_p = (int64_t)g * nsp * Rp + (int64_t)(t - first) * G + h % G;
    const int64_t at_o = r1.y + (int64_t)g * r0.w * R + (int64_t)(t - r0.x) * G + h % G;
    const int parts = (Rp > 0 ? nsp : 0) + own, np = parts - own;
    auto place = [&](int i) { return i < np ? at_p + (int64_t)i * Rp : at_o + (int64_t)(i - np) * R; };
    float mx = -INFINITY, den = 0.f;
    float4 acc[C];
#pragma unroll
    for (int c = 0; c < C; ++c) acc[c] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = 0; i0 < parts; i0 += 32) {
      float w = i0 + lane < parts ? __ldcg(p.part_lse + place(i0 + lane)) : -INFINITY;
      const float m = fmaxf(mx, warp_max(w)), base = m == -INFINITY ? 0.f : m, old = ex2(mx - base);
      mx = m;
      w = ex2(w - base);
      den = den * old + w;
      const int n = min(32, parts - i0);
#pragma unroll
      for (int c = 0; c < C; ++c) {
        acc[c].x *= old;
        acc[c].y *= old;
        acc[c].z *= old;
        acc[c].w *= old;
      }
#pragma unroll 2
      for (int i = 0; i < n; i += 4) {
        const float wi = __shfl_sync(0xffffffffu, w, i + quarter);
        if (i + quarter < n) {
          const float4 *o = reinterpret_cast<const float4 *>(p.part_o + place(i0 + i + quarter) * D) + sub;
#pragma unroll
          for (int c = 0; c < C; ++c) {
            const float4 x = __ldcg(o + 8 * c);
            acc[c].x = fmaf(wi, x.x, acc[c].x);
            acc[c].y = fmaf(wi, x.y, acc[c].y);
            acc[c].z = fmaf(wi, x.z, acc[c].z);
            acc[c].w = fmaf(wi, x.w, acc[c].w);
          }
        }
      }
    }
    const float inv = 1.f / warp_sum(den);
#pragma unroll
    for (int c = 0; c < C; ++c) {
#pragma unroll
      for (int o = 8; o < 32; o <<= 1) {
        acc[c].x += __shfl_xor_sync(0xffffffffu, acc[c].x, o);
        acc[c].y += __shfl_xor_sync(0xffffffffu, acc[c].y, o);
        acc[c].z += __shfl_xor_sync(0xffffffffu, acc[c].z, o);
        acc[c].w += __shfl_xor_sync(0xffffffffu, acc[c].w, o);
      }
    }
    // quarter q writes chunk q
    bf16 *out = (bf16 *)p.a.out + (int64_t)t * p.a.out_stride + (int64_t)h * D;
#pragma unroll
    for (int c = 0; c < C; ++c)
      if (c == quarter) {
        __nv_bfloat162 w2[2] = {__floats2bfloat162_rn(acc[c].x * inv, acc[c].y * inv),
                                __floats2bfloat162_rn(acc[c].z * inv, acc[c].w * inv)};
        *reinterpret_cast<uint2 *>(out + (8 * c + sub) * 4) = *reinterpret_cast<uint2 *>(w2);
      }
  }
}

// ------------------------------------------------------------------ host
typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                  const cuuint64_t *, const cuuint32_t *, const cuuint32_t *,
                                  CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                                  CUtensorMapFloatOOBfill);
EncodeTiledFn encoder() {
  static EncodeTiledFn fn = [] {
    void *ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) !=
            cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      ptr = nullptr;
    return (EncodeTiledFn)ptr;
  }();
  return fn;
}
bool encode_pages(CUtensorMap *tm, const void *base, int n_pages, int kvh, int D) {
  EncodeTiledFn fn = encoder();
  if (!fn) return false;
  cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)kvh, (cuuint64_t)n_pages * kPageRows};
  cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)kvh * D * 2};
  cuuint32_t box[3] = {64, 1, 64};
  cuuint32_t estr[3] = {1, 1, 1};
  return fn(tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool encode_rows(CUtensorMap *tm, const void *q, int total_rows, int H, int D, int64_t stride, int G) {
  EncodeTiledFn fn = encoder();
  if (!fn) return false;
  cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)H, (cuuint64_t)total_rows};
  cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)stride * 2};
  cuuint32_t box[3] = {64, (cuuint32_t)G, (cuuint32_t)(128 / G)};
  cuuint32_t estr[3] = {1, 1, 1};
  return fn(tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(q), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct Layout {
  size_t head, items, req, row_req, redo, part_o, part_lse, total;
};
// Partial rows: at most one per row and segment plus those of every item beyond
// one per (segment, head, row tile pair), which has no more tokens than the call.
Layout layout(int B, int total_rows, int H, int KVH, int D, int prefix) {
  Layout L;
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o += (bytes + 255) / 256 * 256;
    return at;
  };
  const int tpt = 128 / (H / KVH);
  const int64_t rows = (int64_t)total_rows * H, tiles = (int64_t)total_rows / (2 * tpt) + 1;
  const int64_t max_items = KVH * (B + tiles) + (prefix > 0 ? KVH * tiles : 0) + EXTRA;
  const int64_t cap = rows * (prefix > 0 ? 2 : 1) +
                      (int64_t)EXTRA * std::min(2 * tpt, total_rows) * (H / KVH);
  L.head = take(sizeof(Head));
  L.items = take(sizeof(Item) * max_items);
  L.req = take(sizeof(Request) * B);
  L.row_req = take(4 * (size_t)total_rows);
  L.redo = take(sizeof(Redo) * (size_t)rows);
  L.part_lse = take(4 * cap);
  L.part_o = take(4 * cap * D);
  L.total = o;
  return L;
}

template <int D> cudaError_t launch(const PagedAttnParams &a, void *workspace, cudaStream_t s) {
  const Layout L = layout(a.rows.B, a.rows.total_rows, a.H, a.KVH, D, a.rows.prefix_len);
  char *ws = (char *)workspace;
  Params p;
  memset(&p, 0, sizeof(p));
  if (!encode_pages(&p.tmK, a.k_pages, a.rows.n_pages, a.KVH, D) ||
      !encode_pages(&p.tmV, a.v_pages, a.rows.n_pages, a.KVH, D) ||
      !encode_rows(&p.tmQ, a.q, a.rows.total_rows, a.H, D, a.q_stride, a.H / a.KVH))
    return cudaErrorInvalidValue;
  int dev = 0, sms = 0;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  p.a = a;
  p.head = (Head *)(ws + L.head);
  p.items = (Item *)(ws + L.items);
  p.req = (Request *)(ws + L.req);
  p.row_req = (int *)(ws + L.row_req);
  p.redo = (Redo *)(ws + L.redo);
  p.part_o = (float *)(ws + L.part_o);
  p.part_lse = (float *)(ws + L.part_lse);
  p.sms = std::max(1, std::min(sms, MAX_SMS));
  p.scale_log2 = fabsf(a.scale) * 1.4426950408889634f;
  p.negative = a.scale < 0.f;
  // a thread a request; barriers of 256 threads are cheaper than those of 1024
  cudaError_t e = launch_pdl(paged_plan_kernel, dim3(1), dim3(a.rows.B <= 256 ? 256 : PLAN_THREADS), 0, s, p);
  if (e != cudaSuccess) return e;
  e = launch_pdl(paged_attention_kernel<D>, dim3(p.sms), dim3(THREADS), Cfg<D>::SMEM, s, p);
  if (e != cudaSuccess) return e;
  const int64_t warps = (int64_t)a.rows.total_rows * a.H;
  const int grid = (int)std::min<int64_t>((warps + 7) / 8, 16LL * p.sms);
  return launch_pdl(paged_join_kernel<D>, dim3(grid), dim3(256), 0, s, p);
}
template <int D> cudaError_t prepare() {
  return cudaFuncSetAttribute(paged_attention_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              Cfg<D>::SMEM);
}

}  // namespace

size_t paged_attention_tc_workspace(int B, int total_rows, int H, int KVH, int D, int prefix) {
  return layout(B, total_rows, H, KVH, D, prefix).total;
}

cudaError_t launch_paged_attention_tc(const PagedAttnParams &p, void *workspace, cudaStream_t s) {
  return p.D == 64 ? launch<64>(p, workspace, s) : launch<128>(p, workspace, s);
}

cudaError_t prepare_paged_attention_tc() {
  const cudaError_t e = prepare<64>();
  return e == cudaSuccess ? prepare<128>() : e;
}

}  // namespace dflash

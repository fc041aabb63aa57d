// Eviction from a paged cache: which rows a budget keeps, and moving listed rows
// together.
//
// Choosing: per (request, KV head) the m-th largest of up to 10^5 weights.  A CTA (a
// cluster of them where lists are few) turns its weights to order-preserving images,
// holds them in shared memory where they fit (else it reads them again in each pass),
// and takes a histogram of their high 11 bits.  Rows that share the cut's bin, a few
// per cent, go to a list, whose two further histograms (11 and 10 bits) give the cut
// exactly; bins with more rows than the list holds are first split by further
// histograms of all rows.  Counts are whole numbers, so nothing depends on their order.
// A row's place is the number of kept rows before it: counts by warp, then a pass that
// writes.  Waits bound it: of 256 lists the SMs issue 30% of the time, most stalls are at
// barriers and for loads; 93 KB of shared memory leave two CTAs an SM, so that 512 CTAs of
// uneven lists take 1.7 waves.  (Its instructions, some 80 for 32 rows over all passes,
// would take about 10 us.)
// Measured: 32 requests x 8 heads, 2000 to 32000 rows, 4096 kept: 29 us (52 us with
// three histograms of all rows and ballots for every count); one request x 8 heads, 2048
// of 4096: 9 us, of which half are barriers of the cluster and the list's histograms.
//
// Moving: rows ascend, so row i's source is never before its destination, and a CTA
// that goes through its list in order, each step's loads before its stores, never
// reads what it has overwritten.  CTAs share nothing: one takes a slice of the bytes
// of a (request, KV head, keys or values).  Measured: 8 requests x 8 heads, 4096 rows
// kept of 5000 to 16000, 134 MB read and written, 54 us (a plain copy of as much takes
// 45).  More bytes on their way (through shared memory) and wider slices did not help.
#include <cooperative_groups.h>

#include "common.cuh"
#include "target_ops.h"

namespace dflash {
namespace {

namespace cg = cooperative_groups;

// ------------------------------------------------------------------ choose
constexpr int CHOOSE_THREADS = 512, CHOOSE_WARPS = CHOOSE_THREADS / 32, BINS = 2048;
constexpr int MAXC = 8;
constexpr int MOST_HELD = 16384;          // weights that a CTA holds in shared memory
constexpr int LIST = 2048;                // rows near the cut that are told apart in a list
constexpr int PER = LIST / CHOOSE_THREADS;

// larger image: larger weight; NaN as -infinity, -0 as 0
__device__ __forceinline__ uint32_t order_image(float v) {
  const uint32_t u = __float_as_uint(v + 0.f), x = u ^ ((uint32_t)((int)u >> 31) | 0x80000000u);
  return x > 0xff800000u ? 0x007fffffu : max(x, 0x007fffffu);
}

// HELD: the images of a CTA's rows stay in shared memory; else the weights are read again in each pass.
template <bool HELD>
__global__ void __launch_bounds__(CHOOSE_THREADS, 3) choose_rows_kernel(const __grid_constant__ ChooseParams p) {
  extern __shared__ uint32_t s_image[];                         // [rows of the CTA], a warp's after another's
  __shared__ __align__(16) uint32_t s_hist[2][BINS];
  __shared__ uint32_t s_list[LIST];
  __shared__ uint8_t s_from[LIST];                              // warp of the cluster that listed a row
  __shared__ int s_warp[2][CHOOSE_WARPS], s_of[2][MAXC * CHOOSE_WARPS], s_total[2];
  __shared__ int s_bin, s_above, s_count, s_listed, s_need;
  __shared__ uint32_t s_cut;
  cg::cluster_group cl = cg::this_cluster();
  const int C = (int)cl.num_blocks(), rank = (int)cl.block_rank();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int list = blockIdx.x / C, b = list / p.KVH;
  pdl_wait();
  const int kv = p.kv_len[b], keep = p.keep[b];
  const bool bad_len = kv < p.prefix_len || kv - p.prefix_len > p.width, bad_keep = keep < 0 || keep > p.max_keep;
  if (bad_len || bad_keep) {                                    // (the whole cluster)
    if (tid == 0 && bad_len) raise_error(p.err, DFLASH_DERR_KV_CAPACITY);
    if (tid == 0 && bad_keep) raise_error(p.err, DFLASH_DERR_ROW_LIST);
    return;
  }
  const int n = kv - p.prefix_len;
  int *rows = p.rows + (int64_t)list * p.max_keep;
  if (rank == 0 && tid == 0) p.count[list] = min(n, keep);
  if (n <= keep) {
    for (int i = rank * CHOOSE_THREADS + tid; i < n; i += C * CHOOSE_THREADS) rows[i] = i;
    return;
  }
  const float *w = p.weights + (int64_t)list * p.width;
  const int a = min(p.first, keep), z = min(p.last, keep - a), m = keep - a - z;
  for (int i = rank * CHOOSE_THREADS + tid; i < a + z; i += C * CHOOSE_THREADS)
    rows[i < a ? i : m + i] = i < a ? i : n - z + (i - a);
  if (m == 0) return;
  // a warp's rows: a run of those between, whole steps of 32
  const int M = n - a - z, id = rank * CHOOSE_WARPS + warp;
  const int run = (int)(((int64_t)M + C * CHOOSE_WARPS * 32 - 1) / (C * CHOOSE_WARPS * 32)) * 32;
  const int w0 = a + (int)min((int64_t)M, (int64_t)id * run), w1 = min(n - z - w0, run) + w0;
  uint32_t *held = s_image + warp * run;
  // f(row, its image, whether there is one) for all of the warp's rows, in order
  auto each = [&](auto read, auto f) {
    constexpr int U = 8;
    int i0 = w0;
    for (; i0 + 32 * U <= w1; i0 += 32 * U) {
      uint32_t x[U];
#pragma unroll
      for (int e = 0; e < U; ++e) x[e] = read(i0 + 32 * e + lane);
#pragma unroll
      for (int e = 0; e < U; ++e) f(i0 + 32 * e + lane, x[e], true);
    }
    for (; i0 < w1; i0 += 32) {
      const int i = i0 + lane;
      f(i, i < w1 ? read(i) : 0u, i < w1);
    }
  };
  auto from_weights = [&](int i) { return order_image(w[i]); };
  auto image = [&](int i) { return HELD ? held[i - w0] : order_image(w[i]); };
  // the bin from the top where the counts reach `need`: it, those above it, those in it (all threads)
  auto find_bin = [&](uint32_t *hist, int ranks, int need) {
    uint4 c = make_uint4(0, 0, 0, 0);      // four bins a thread
    for (int k = 0; k < ranks; ++k) {
      const uint4 h = reinterpret_cast<const uint4 *>(cl.map_shared_rank(hist, ranks > 1 ? k : rank))[BINS / 4 - 1 - tid];
      c.x += h.w, c.y += h.z, c.z += h.y, c.w += h.x;
    }
    const int own = (int)(c.x + c.y + c.z + c.w);
    int inc = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += x;
    }
    if (lane == 31) s_warp[0][warp] = inc;
    __syncthreads();
    int above = __reduce_add_sync(0xffffffffu, lane < warp ? s_warp[0][lane] : 0) + inc - own;
    if (above < need && need <= above + own) {
      const int cs[4] = {(int)c.x, (int)c.y, (int)c.z, (int)c.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (above < need && need <= above + cs[k]) {
          s_bin = BINS - 1 - 4 * tid - k;
          s_above = above;
          s_count = cs[k];
        }
        above += cs[k];
      }
    }
    __syncthreads();
  };
  // ---- the cut, the m-th largest image: as many of its high bits as it takes to leave few rows
  uint32_t cut = 0;                       // those bits
  int need = m, count = M, shift = 32;    // of the rows that agree with them, how many are taken; the bits below
  if (tid == 0) s_listed = 0;
  for (int i = tid; i < 2 * MAXC * CHOOSE_WARPS; i += CHOOSE_THREADS) (&s_of[0][0])[i] = 0;
  for (int pass = 0; pass < 3 && need < count && (pass == 0 || count > LIST); ++pass) {
    const int upper = shift, bits = pass == 2 ? 10 : 11;
    uint32_t *hist = s_hist[pass & 1];
    reinterpret_cast<uint4 *>(hist)[tid] = make_uint4(0, 0, 0, 0);
    __syncthreads();
    shift -= bits;
    const uint32_t mask = (1u << bits) - 1;
    if (pass == 0)
      each(from_weights, [&](int i, uint32_t x, bool live) {
        if (HELD && live) held[i - w0] = x;
        if (live) atomicAdd(&hist[x >> 21], 1u);
      });
    else
      each(image, [&](int, uint32_t x, bool live) {
        if (live && x >> upper == cut) atomicAdd(&hist[x >> shift & mask], 1u);
      });
    cl.sync();
    find_bin(hist, C, need);
    cut = cut << bits | (uint32_t)s_bin;
    need -= s_above;
    count = s_count;
  }
  // ---- rows above the cut's bits, by warp; those that agree with them are all taken, or all alike, or
  // go to a list
  const bool listed = need < count && shift > 0;
  int above = 0, equal = 0;
  each(image, [&](int, uint32_t x, bool live) {
    const uint32_t high = x >> shift;
    above += live && high > cut;
    if (live && high == cut) {
      ++equal;
      if (listed) {
        const int at = atomicAdd(&s_listed, 1);
        s_list[at] = x;
        s_from[at] = (uint8_t)id;
      }
    }
  });
  above = __reduce_add_sync(0xffffffffu, above);
  equal = __reduce_add_sync(0xffffffffu, equal);
  if (listed) {
    cl.sync();
    if (rank == 0) {
      // the cluster's lists, PER rows a thread, and the rest of the cut's bits
      uint32_t x[PER];
      int from[PER], total = 0;
      for (int k = 0; k < C; ++k) total += *cl.map_shared_rank(&s_listed, k);
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        int at = j * CHOOSE_THREADS + tid, k = 0;
        from[j] = -1;
        x[j] = 0;
        if (at < total) {
          for (int c = *cl.map_shared_rank(&s_listed, 0); at >= c; c = *cl.map_shared_rank(&s_listed, k)) {
            at -= c;
            ++k;
          }
          x[j] = cl.map_shared_rank(s_list, k)[at];
          from[j] = cl.map_shared_rank(s_from, k)[at];
        }
      }
      for (int low = shift; low > 0;) {
        const int upper = low, bits = min(low, 11);
        low -= bits;
        __syncthreads();
        reinterpret_cast<uint4 *>(s_hist[0])[tid] = make_uint4(0, 0, 0, 0);
        __syncthreads();
#pragma unroll
        for (int j = 0; j < PER; ++j)
          if (from[j] >= 0 && x[j] >> upper == cut) atomicAdd(&s_hist[0][x[j] >> low & ((1u << bits) - 1)], 1u);
        __syncthreads();
        find_bin(s_hist[0], 1, need);
        cut = cut << bits | (uint32_t)s_bin;
        need -= s_above;
      }
#pragma unroll
      for (int j = 0; j < PER; ++j)
        if (from[j] >= 0 && x[j] >= cut) atomicAdd(&s_of[x[j] > cut ? 0 : 1][from[j]], 1);
      if (tid == 0) {
        s_cut = cut;
        s_need = need;
      }
    }
    cl.sync();
    cut = *cl.map_shared_rank(&s_cut, 0);
    need = *cl.map_shared_rank(&s_need, 0);
    above += *cl.map_shared_rank(&s_of[0][id], 0);
    equal = *cl.map_shared_rank(&s_of[1][id], 0);
    shift = 0;
  }
  // ---- places
  __syncthreads();
  if (lane == 0) {
    s_warp[0][warp] = above;
    s_warp[1][warp] = equal;
  }
  __syncthreads();
  above = __reduce_add_sync(0xffffffffu, lane < warp ? s_warp[0][lane] : 0);
  equal = __reduce_add_sync(0xffffffffu, lane < warp ? s_warp[1][lane] : 0);
  if (warp == CHOOSE_WARPS - 1 && lane == 0) {
    s_total[0] = above + s_warp[0][warp];
    s_total[1] = equal + s_warp[1][warp];
  }
  cl.sync();
  above += a;
  for (int k = 0; k < rank; ++k) {
    above += *cl.map_shared_rank(&s_total[0], k);
    equal += *cl.map_shared_rank(&s_total[1], k);
  }
  // a row's place: kept rows before it
  const uint32_t before = (1u << lane) - 1;
  int at = above + min(equal, need), left = need - min(equal, need);   // alike rows that are still taken
  each(image, [&](int i, uint32_t x, bool live) {
    const uint32_t high = x >> shift;
    bool kept = live && high > cut;
    const bool alike = live && high == cut;
    if (left > 0 && __any_sync(0xffffffffu, alike)) {
      const uint32_t be = __ballot_sync(0xffffffffu, alike);
      kept = kept || (alike && __popc(be & before) < left);
      left -= min(left, __popc(be));
    }
    const uint32_t bk = __ballot_sync(0xffffffffu, kept);
    if (kept) rows[at + __popc(bk & before)] = i;
    at += __popc(bk);
  });
  cl.sync();                              // no CTA leaves while another reads its totals
}

// ------------------------------------------------------------------ keep
constexpr int KEEP_THREADS = 256, UNITS = 4;

// A slice of 16 LANES bytes of the listed rows, UNITS rows a thread and step.  List, page and row are three
// loads that wait for one another, so they are three steps, two and one ahead of the store (sources of
// later steps lie behind the places of this one).
template <int LANES>
__device__ __forceinline__ void move_rows(uint4 *pages, const int *table, const int *list, int count, int own,
                                          int64_t row_step, int lane16) {
  // pages: head g of cache row 0; row_step: 16-byte chunks from one cache row to the next
  constexpr int RP = KEEP_THREADS / LANES, ROWS = RP * UNITS;
  const int r = threadIdx.x / LANES, c = threadIdx.x % LANES + lane16;
  struct Step {
    int from[UNITS], to[UNITS];            // slots; -1: stays where it is
    uint4 v[UNITS];
  };
  int src[UNITS];
  auto look_up = [&](int i0) {
#pragma unroll
    for (int u = 0; u < UNITS; ++u) {
      const int i = i0 + u * RP + r;
      src[u] = i < count ? __ldg(list + i) : i;
    }
  };
  auto find = [&](int i0, Step &s) {
#pragma unroll
    for (int u = 0; u < UNITS; ++u) {
      const int i = i0 + u * RP + r, f = own + src[u], t = own + i;
      s.from[u] = s.to[u] = -1;
      if (src[u] != i) {
        s.from[u] = __ldg(table + f / kPageRows) * kPageRows + f % kPageRows;
        s.to[u] = __ldg(table + t / kPageRows) * kPageRows + t % kPageRows;
      }
    }
  };
  auto load = [&](Step &s) {
#pragma unroll
    for (int u = 0; u < UNITS; ++u)
      if (s.from[u] >= 0) s.v[u] = pages[s.from[u] * row_step + c];
  };
  auto store = [&](const Step &s) {
#pragma unroll
    for (int u = 0; u < UNITS; ++u)
      if (s.to[u] >= 0) pages[s.to[u] * row_step + c] = s.v[u];
  };
  Step a, b;
  auto advance = [&](int i0, Step &now, Step &next) {
    find(i0 + ROWS, next);
    look_up(i0 + 2 * ROWS);
    __syncthreads();                       // the rows of this step are loaded
    load(next);
    store(now);
  };
  look_up(0);
  find(0, a);
  look_up(ROWS);
  load(a);
  for (int i0 = 0; i0 < count; i0 += 2 * ROWS) {
    advance(i0, a, b);
    if (i0 + ROWS >= count) break;
    advance(i0 + ROWS, b, a);
  }
}

template <int LANES>
__global__ void __launch_bounds__(KEEP_THREADS, 4) keep_rows_kernel(const __grid_constant__ KeepParams p) {
  const int b = blockIdx.z, g = blockIdx.y, tid = threadIdx.x, part = blockIdx.x;
  const int chunks = p.row_bytes / 16, slices = chunks / LANES;
  const bool reports = part == 0 && tid == 0;
  pdl_wait();
  const int l = b * p.lists + (p.lists > 1 ? g : 0), count = p.count[l];
  const int first = p.first ? p.first[b] : p.prefix_len;
  const int *list = p.rows + (int64_t)l * p.max_rows;
  const int *table = p.page_table + (int64_t)b * p.pages_per_req;
  if (count < 0 || count > p.max_rows) {
    if (reports) raise_error(p.err, DFLASH_DERR_ROW_LIST);
    return;
  }
  if (count == 0) return;
  const int own = first - p.prefix_len;
  // ---- the list as a whole: ascending, its last row and its pages there
  bool falls = false;
#pragma unroll 4
  for (int i = tid; i < count; i += KEEP_THREADS) falls = falls || list[i] <= (i > 0 ? list[i - 1] : -1);
  if (__syncthreads_or(falls)) {
    if (reports) raise_error(p.err, DFLASH_DERR_ROW_LIST);
    return;
  }
  const int64_t last = (int64_t)own + list[count - 1];
  if (first < p.prefix_len || last >= (int64_t)p.pages_per_req * kPageRows || (p.weights && last >= p.width)) {
    if (reports) raise_error(p.err, DFLASH_DERR_KV_CAPACITY);
    return;
  }
  bool bad = false;
  for (int i = own / kPageRows + tid; i <= (int)last / kPageRows; i += KEEP_THREADS)
    bad = bad || table[i] < 0 || table[i] >= p.n_pages;
  if (__syncthreads_or(bad)) {
    if (reports) raise_error(p.err, DFLASH_DERR_PAGE_RANGE);
    return;
  }
  if (part == 2 * slices) {                // the weights
    float *w = p.weights + ((int64_t)b * p.KVH + g) * p.width + own;
    for (int i0 = 0; i0 < count; i0 += KEEP_THREADS * UNITS) {
      float v[UNITS];
#pragma unroll
      for (int u = 0; u < UNITS; ++u) {
        const int i = i0 + u * KEEP_THREADS + tid;
        if (i < count) v[u] = w[list[i]];
      }
      __syncthreads();
#pragma unroll
      for (int u = 0; u < UNITS; ++u) {
        const int i = i0 + u * KEEP_THREADS + tid;
        if (i < count) w[i] = v[u];
      }
    }
    return;
  }
  uint4 *pages = (uint4 *)(part < slices ? p.k_pages : p.v_pages);
  move_rows<LANES>(pages + (int64_t)g * chunks, table, list, count, own, (int64_t)p.KVH * chunks,
                   part % slices * LANES);
}

template <int LANES> cudaError_t launch_keep(const KeepParams &p, cudaStream_t s) {
  const int slices = p.row_bytes / 16 / LANES;
  return launch_pdl(keep_rows_kernel<LANES>, dim3(2 * slices + (p.weights ? 1 : 0), p.KVH, p.B), dim3(KEEP_THREADS),
                    0, s, p);
}

}  // namespace

cudaError_t launch_choose_rows(const ChooseParams &p, cudaStream_t s) {
  int dev = 0, sms = 0;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  const int64_t lists = (int64_t)p.B * p.KVH;
  int C = 1;
  // CTAs for two an SM, of 4096 rows at least: 256 lists of up to 32000 rows 33 us with 2 CTAs a list,
  // 42 with 4
  while (C < MAXC && C * 4096LL < p.width && lists * C < 2 * sms) C *= 2;
  // (a run of a warp is whole steps of 32 rows)
  const int64_t held = ((int64_t)p.width + C * CHOOSE_THREADS - 1) / (C * CHOOSE_THREADS) * CHOOSE_THREADS;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(lists * C));
  cfg.blockDim = dim3(CHOOSE_THREADS);
  cfg.dynamicSmemBytes = held <= MOST_HELD ? held * 4 : 0;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = C;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return held <= MOST_HELD ? cudaLaunchKernelEx(&cfg, choose_rows_kernel<true>, p)
                           : cudaLaunchKernelEx(&cfg, choose_rows_kernel<false>, p);
}

cudaError_t prepare_choose_rows() {
  return cudaFuncSetAttribute(choose_rows_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, MOST_HELD * 4);
}

cudaError_t launch_keep_rows(const KeepParams &p, cudaStream_t s) {
  int dev = 0, sms = 0;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  // slices of a row, down to a sector, while the CTAs are few: 64 (request, head)s of 256-byte rows in
  // slices of 256, 128, 64 and 32 bytes 97, 74, 58 and 74 us
  const int64_t heads = 2LL * p.B * p.KVH;
  int lanes = p.row_bytes / 16;
  while (lanes > 2 && heads * (p.row_bytes / 16 / lanes) < 2 * sms) lanes /= 2;
  switch (lanes) {
    case 32: return launch_keep<32>(p, s);
    case 16: return launch_keep<16>(p, s);
    case 8: return launch_keep<8>(p, s);
    case 4: return launch_keep<4>(p, s);
    default: return launch_keep<2>(p, s);
  }
}

}  // namespace dflash

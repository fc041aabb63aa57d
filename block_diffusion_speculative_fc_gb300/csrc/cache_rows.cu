// Eviction from a paged cache: which rows a budget keeps, and moving listed rows
// together.
//
// Choosing: per (request, KV head) the m-th largest of up to 10^5 weights.  A cluster
// of CTAs holds a list's weights in shared memory (what does not fit is read again)
// and finds the cut by three histograms of 11, 11 and 10 bits of the order-preserving
// image of the weights, most significant first; counts are whole numbers, so nothing
// depends on their order.  Row i then goes to place (rows before it above the cut) +
// min(rows before it at the cut, how many of those are taken): a scan of two counts.
//
// Moving: rows ascend, so row i's source is never before its destination, and a CTA
// that goes through its list in order, each step's loads before its stores, never
// reads what it has overwritten.  CTAs share nothing: one takes a slice of the bytes
// of a (request, KV head, keys or values).  HBM bounds it, in large batches.
#include <cooperative_groups.h>

#include "common.cuh"
#include "target_ops.h"

namespace dflash {
namespace {

namespace cg = cooperative_groups;

// ------------------------------------------------------------------ choose
constexpr int CHOOSE_THREADS = 1024, CHOOSE_WARPS = CHOOSE_THREADS / 32, BINS = 2048;
constexpr int HELD = 48 * 1024;           // weights that a CTA holds
constexpr size_t CHOOSE_SMEM = HELD * 4 + 2 * BINS * 4;

// larger image: larger weight; NaN as -infinity, -0 as 0
__device__ __forceinline__ uint32_t order_image(float v) {
  if (isnan(v)) v = -INFINITY;
  const uint32_t u = __float_as_uint(v + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__global__ void __launch_bounds__(CHOOSE_THREADS) choose_rows_kernel(const __grid_constant__ ChooseParams p) {
  extern __shared__ uint32_t s_dyn[];
  uint32_t *s_val = s_dyn, *s_hist = s_dyn + HELD;             // [HELD], [2][BINS]
  __shared__ int s_warp[2][CHOOSE_WARPS], s_bin, s_above, s_total[2];
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
  // this CTA's rows
  const int seg = (n + C - 1) / C, lo = min(n, rank * seg), hi = min(n, lo + seg);
  auto image = [&](int i) { return i - lo < HELD ? s_val[i - lo] : order_image(w[i]); };
  for (int i = lo + tid; i < min(hi, lo + HELD); i += CHOOSE_THREADS) s_val[i - lo] = order_image(w[i]);
  // ---- the cut: the m-th largest image of rows a .. n-z-1
  uint32_t cut = 0;                       // its bits found so far
  int need = m;                           // how many of those that agree with them are taken
  const int from = max(lo, a), to = min(hi, n - z);
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
    uint32_t *hist = s_hist + (pass & 1) * BINS;
    for (int i = tid; i < BINS; i += CHOOSE_THREADS) hist[i] = 0;
    __syncthreads();
    for (int i = from + tid; i < to; i += CHOOSE_THREADS) {
      const uint32_t u = image(i);
      if (pass == 0 || (u ^ cut) >> (shift + bits) == 0) atomicAdd(&hist[u >> shift & ((1u << bits) - 1)], 1u);
    }
    cl.sync();
    // bins from the top, two a thread: counts of all CTAs, those above, and the bin that holds the cut
    const int hi_bin = BINS - 1 - 2 * tid;
    uint32_t c0 = 0, c1 = 0;
    for (int k = 0; k < C; ++k) {
      const uint32_t *h = cl.map_shared_rank(hist, k);
      c0 += h[hi_bin];
      c1 += h[hi_bin - 1];
    }
    int inc = (int)(c0 + c1);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += x;
    }
    if (lane == 31) s_warp[0][warp] = inc;
    __syncthreads();
    int before = lane < warp ? s_warp[0][lane] : 0;             // (as many warps as lanes)
    before = __reduce_add_sync(0xffffffffu, before);
    const int above = before + inc - (int)(c0 + c1);
    if (above < need && need <= above + (int)c0) {
      s_bin = hi_bin;
      s_above = above;
    } else if (above + (int)c0 < need && need <= above + (int)(c0 + c1)) {
      s_bin = hi_bin - 1;
      s_above = above + (int)c0;
    }
    __syncthreads();
    if (need > 0) {
      cut |= (uint32_t)s_bin << shift;
      need -= s_above;
    }
  }
  // m == 0: nothing of the middle is taken
  const bool none = m == 0;
  auto above_cut = [&](int i, uint32_t u) { return i < a || i >= n - z || (!none && u > cut); };
  auto at_cut = [&](int i, uint32_t u) { return i >= a && i < n - z && !none && u == cut; };
  // ---- places: a warp a run of consecutive rows
  const int run = ((hi - lo + CHOOSE_WARPS - 1) / CHOOSE_WARPS + 31) / 32 * 32;
  const int w0 = min(hi, lo + warp * run), w1 = min(hi, w0 + run);
  int above = 0, equal = 0;
  for (int i0 = w0; i0 < w1; i0 += 32) {
    const int i = i0 + lane;
    const uint32_t u = i < w1 ? image(i) : 0;
    above += __popc(__ballot_sync(0xffffffffu, i < w1 && above_cut(i, u)));
    equal += __popc(__ballot_sync(0xffffffffu, i < w1 && at_cut(i, u)));
  }
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
  for (int k = 0; k < rank; ++k) {
    above += *cl.map_shared_rank(&s_total[0], k);
    equal += *cl.map_shared_rank(&s_total[1], k);
  }
  for (int i0 = w0; i0 < w1; i0 += 32) {
    const int i = i0 + lane;
    const uint32_t u = i < w1 ? image(i) : 0, before = (1u << lane) - 1;
    const bool is_above = i < w1 && above_cut(i, u), is_equal = i < w1 && at_cut(i, u);
    const uint32_t ba = __ballot_sync(0xffffffffu, is_above), be = __ballot_sync(0xffffffffu, is_equal);
    const int eq = equal + __popc(be & before);
    if (is_above || (is_equal && eq < need)) rows[above + __popc(ba & before) + min(eq, need)] = i;
    above += __popc(ba);
    equal += __popc(be);
  }
  cl.sync();                              // no CTA leaves while another reads its totals
}

// ------------------------------------------------------------------ keep
constexpr int KEEP_THREADS = 256, UNITS = 8;

// `bytes` of a row in this CTA's slice: 16 a lane.
template <int LANES>
__device__ __forceinline__ void move_rows(uint4 *pages, const int *table, const int *list, int count, int own,
                                          int64_t row_step, int lane16) {
  // pages: the slice of head g in cache row 0; row_step: 16-byte chunks from one cache row to the next
  constexpr int RP = KEEP_THREADS / LANES;
  const int r = threadIdx.x / LANES, c = threadIdx.x % LANES + lane16;
  auto slot = [&](int row) { return ((int64_t)table[row / kPageRows] * kPageRows + row % kPageRows) * row_step + c; };
  for (int i0 = 0; i0 < count; i0 += RP * UNITS) {
    uint4 v[UNITS];
    int64_t to[UNITS];
#pragma unroll
    for (int u = 0; u < UNITS; ++u) {
      const int i = i0 + u * RP + r;
      to[u] = -1;
      if (i < count) {
        const int src = list[i];
        if (src != i) {
          v[u] = pages[slot(own + src)];
          to[u] = slot(own + i);
        }
      }
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < UNITS; ++u)
      if (to[u] >= 0) pages[to[u]] = v[u];
  }
}

template <int LANES>
__global__ void __launch_bounds__(KEEP_THREADS) keep_rows_kernel(const __grid_constant__ KeepParams p) {
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
  while (C < 8 && lists * C * 2 <= sms && p.width / C >= 2048) C *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(lists * C));
  cfg.blockDim = dim3(CHOOSE_THREADS);
  cfg.dynamicSmemBytes = CHOOSE_SMEM;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = C;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, choose_rows_kernel, p);
}

cudaError_t prepare_choose_rows() {
  return cudaFuncSetAttribute(choose_rows_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)CHOOSE_SMEM);
}

cudaError_t launch_keep_rows(const KeepParams &p, cudaStream_t s) {
  int dev = 0, sms = 0;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  // slices of a row, down to a sector, while the CTAs are few
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

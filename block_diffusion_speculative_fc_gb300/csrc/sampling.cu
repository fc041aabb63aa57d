// Sampling distribution of a row of logits (temperature, top-k, top-p, min-p)
// and the draw of a token from it.
//
// With m the row's maximum and c = log2(e) / T, token v weighs w = 2^-a, a =
// (m - x) c.  The order is by logit, lower ids first among equal ones, so the
// 64-bit key (order-preserving image of x, ~id) has no ties and every filter
// is a cut of that order: the k-th key, the last key whose predecessors weigh
// less than p of the total, the smallest x with w >= min_p.  The kept set is
// "key >= the largest of the cuts"; probabilities are w over its sum.
//
// A row belongs to one thread-block cluster, whose CTAs hold its slices in
// shared memory: the logits are read from HBM once and the result written
// once (6 or 8 bytes an element, the operator's floor); every pass in between
// runs on shared memory.  Batches of many rows take a CTA a row, which reads it
// again from L2 (or HBM) instead.
//
// Measured: 16 rows of 151936 bf16 logits with top-k and top-p 13.5 us (clusters
// of 8, latency: loads, five cluster barriers, the list's sort); 2048 rows of
// mixed kinds 520 us, 3.6 TB/s of the floor's bytes (two CTAs of 16 warps an SM
// take turns loading, scanning and storing; 417 us with top-k and top-p in every
// row, 650 us with top-p alone, where 8% of the rows need the histogram); one
// draw 8.8 us, 128 draws of 163840 logits 54 to 68 us by their logits (the rows
// with the histogram take about 50 us each, the others 10).
//
// Most rows keep few tokens, and those are found without a histogram or a
// sort of the row.  Every CTA takes the j-th largest of its threads' maxima
// (j C >= k, so at least k tokens of the row reach the smallest of the C
// values, L); one pass gathers the tokens >= L in the cluster's first CTA --
// a few times k -- and adds up the weight of the rest where top-p needs it.
// That CTA sorts and walks the list while the others write zeros; then every
// CTA writes its kept tokens over them.
//
// Rows whose list overflows, or whose nucleus is larger than it, take a
// histogram over a (32 bins per unit, so a bin's weights are alike) of counts
// and weights; the tokens of the bin that holds the cut are gathered, sorted
// and walked, and a bin with more tokens than the list holds is split by key
// until it fits (equal logits split by id).
//
// Sums that decide a border are whole numbers: a weight is rounded once to
// about 2^-26 relative and sums are exact multiples of 2^-44, so they do not
// go by the order of atomics (the weight of the tokens outside a list, which
// lie beyond the border, comes from the hardware's exponential, good to
// 2^-20).  A border falls where 64-bit arithmetic puts it except within about
// 1e-9 of the total (single roundings of 2^-27 average out) plus 2^-20 of the
// weight outside the list.  min-p compares logits with m + T ln
// min_p formed in 64 bits (by one thread: fp64 runs at 2 lanes a clock here,
// so everything else stays out of it).
#include <cooperative_groups.h>
#include <float.h>
#include <math.h>

#include <algorithm>

#include "common.cuh"
#include "target_ops.h"

namespace dflash {
namespace {

namespace cg = cooperative_groups;

constexpr int NT = 512;          // threads of a CTA
constexpr int NB = 1024;         // histogram bins: a = 0 .. 31.95 and one for the rest
constexpr float TAIL = 31.95f;   // a of the last bin's first token (inside the bin before it)
constexpr int PB = NB / NT;      // bins of a thread in a scan
constexpr int CAP = 1024;        // gathered tokens (two a thread)
// Top-k of the short way at most.  k = 512 by the list and by the histogram: 16 rows of 151936 50 us and
// 65, 128 fp32 rows of 50257 69 and 112; k = 700 73 and 67, 103 and 114.  (512 rows of 151936, a CTA each:
// k = 400 185 and 788; at 500 the list overflows, 846 and 787.)
constexpr int MAX_K = 512;
// Tokens that its list holds at least for top-p alone: 64, 128, 256 take 33, 34, 41 us for 96 fp32 rows
// of 50257, 649, 656, 666 for 2048 rows of 151936, 31.8, 30.9, 32.0 for 16.
constexpr int TOP_P_LIST = 128;
constexpr int MAXC = 8;          // CTAs of a cluster
constexpr int GROUPS = NT / 4;
// A bound of up to this place comes from the maxima of groups of threads, a later one from a search
// over the threads' own.  512 rows of 151936: k = 100 and 120 by the search 118 and 120 us, by groups
// 122 and 134 (a lower bound, a longer list), k = 128 120 and 393 (it overflows).
constexpr int GROUP_PLACES = GROUPS * 3 / 4;
constexpr int STREAM_VOCAB = 1 << 18;   // tokens of a CTA at most (sums of the histogram)
constexpr int MAX_SMEM = 220 * 1024;
// Up to here two logits whose difference passes the largest float differ by a weight of 0; above it
// they need not, and an infinite difference says nothing of the place of the lower one.
constexpr float MAX_T = 0x1p100f;

struct Tables {
  uint32_t u[32];                // round(2^26 2^(-i/32))
  float f[32];                   // 2^26 2^(-i/32)
};

typedef unsigned long long u64;

struct Fixed {
  u64 list[CAP];
  union {
    struct {
      uint32_t cnt[NB], lo[NB], hi[NB];   // tokens (top-k only), sums of u % 2^13 and u / 2^13
    };
    u64 sorted[CAP];
  };
  u64 warp_m[NT / 32];
  int warp_c[NT / 32];
  float group[GROUPS];           // maxima of groups of four threads
  int own_n, own_at;             // tokens that this CTA lists, their place in the leader's list
  u64 own_rest;                  // weight outside the histogram
  u64 w_rest[NT / 32], w_listed[NT / 32];
  float fred[NT / 32];
  u64 kred[NT / 32];
  double t_log;                  // min-p: T ln min_p
  float x_min;                   // and the smallest logit kept
  // exchanged between the CTAs of the cluster, one slot per rank
  float x_max[MAXC], x_low[MAXC], x_sum[MAXC];
  int x_n[MAXC];
  u64 x_rest[MAXC], x_listed[MAXC], x_race[MAXC];
  int n_list;
  // the leader's command to every CTA
  int cmd, bin, sh;
  u64 range_lo, range_hi, cut;
  // leader: the bin that holds a cut
  int sel_bin, sel_n, sel_above;
  u64 sel_above_m, target;
};

enum { CMD_GATHER = 0, CMD_SPLIT = 1, CMD_DONE = 2 };

__device__ __forceinline__ uint32_t order_image(float x) {
  const uint32_t u = __float_as_uint(x);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float order_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}
__device__ __forceinline__ unsigned long long key_of(float x, int idx) {
  return ((unsigned long long)order_image(x) << 32) | (uint32_t)~(uint32_t)idx;
}
// The image of -0 is one below that of +0, but equal logits go by id: one image for both.  (Applied where
// keys are few, not in order_image: there its registers take 128 unfiltered draws from 48 to 50 us.)
__device__ __forceinline__ uint32_t one_zero(uint32_t image) { return image + (image == 0x7fffffffu); }
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Bin and weight of a token.  The weight is u 2^-(26 + octave(bin)).  a is
// carried as a pair of floats; 2^-r on |r| <= 1/64 is a Taylor polynomial in r
// ln 2 (next term below 2e-12).  Explicit roundings: every pass gets the same
// bin for a token.
struct Weigher {
  float m, c_hi, c_lo;
  __device__ __forceinline__ void distance(float x, float &a, float &al) const {
    const float d = __fsub_rn(m, x);
    const float bb = __fsub_rn(d, m);   // d + err = m - x exactly
    const float err = __fsub_rn(__fsub_rn(m, __fsub_rn(d, bb)), __fadd_rn(x, bb));
    a = __fmul_rn(d, c_hi);
    al = __fmaf_rn(err, c_hi, __fmaf_rn(d, c_lo, __fmaf_rn(d, c_hi, -a)));
  }
  __device__ __forceinline__ void operator()(float x, const Tables &t, int &bin, uint32_t &u) const {
    float a, al;
    distance(x, a, al);
    if (!(a < TAIL)) {                  // far tail (a may be infinite, al then NaN)
      bin = NB - 1;
      u = (uint32_t)(ex2(31.f - a) * 0x1p26f);
      return;
    }
    const float big = __fmaf_rn(a, 32.f, 12582912.f);   // 1.5 2^23: rounds 32 a to a whole number
    bin = (int)(__float_as_uint(big) & 0x3fffffu);
    const float r = __fadd_rn(__fmaf_rn(__fsub_rn(big, 12582912.f), -0.03125f, a), al);
    const float y = __fmul_rn(r, -0.69314718f);
    float q = __fmaf_rn(y, 1.f / 24.f, 1.f / 6.f);
    q = __fmaf_rn(y, q, 0.5f);
    q = __fmaf_rn(__fmul_rn(y, y), q, y);               // 2^-r - 1
    u = t.u[bin & 31] + __float2int_rn(__fmul_rn(t.f[bin & 31], q));
  }
};
// A sum of weights of one octave in units of 2^-44.
__device__ __forceinline__ u64 units(u64 sum, int bin) {
  const int octave = bin >> 5;
  return octave <= 18 ? sum << (18 - octave) : sum >> (octave - 18);
}
// p of a sum, rounded up: "below" it as whole numbers is below p of it.
__device__ __forceinline__ u64 share_of(u64 total, float p) {
  if (!(p > 0.f)) return 1;
  const double t = ceil((double)p * (double)total);
  return t < 1.0 ? 1 : (u64)t;
}

__device__ __forceinline__ void cluster_arrive_relaxed() {
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}

template <typename T> struct Elem;
template <> struct Elem<bf16> {
  static constexpr int E = 8;
  typedef uint2 Quad;
  static __device__ __forceinline__ void unpack4(const Quad &t, float *x) {
    x[0] = __uint_as_float(t.x << 16);
    x[1] = __uint_as_float(t.x & 0xffff0000u);
    x[2] = __uint_as_float(t.y << 16);
    x[3] = __uint_as_float(t.y & 0xffff0000u);
  }
  static __device__ __forceinline__ void unpack(const uint4 &v, float *x) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ float largest() { return __uint_as_float(0x7f7f0000u); }
  // the largest of a vector, NaN if any is
  static __device__ __forceinline__ float max_of(const uint4 &v) {
    const __nv_bfloat162 *h = reinterpret_cast<const __nv_bfloat162 *>(&v);
    const __nv_bfloat162 t = __hmax2_nan(__hmax2_nan(h[0], h[1]), __hmax2_nan(h[2], h[3]));
    return __bfloat162float(__hmax_nan(__low2bfloat16(t), __high2bfloat16(t)));
  }
};
template <> struct Elem<float> {
  static constexpr int E = 4;
  typedef float4 Quad;
  static __device__ __forceinline__ void unpack4(const Quad &t, float *x) {
    x[0] = t.x, x[1] = t.y, x[2] = t.z, x[3] = t.w;
  }
  static __device__ __forceinline__ void unpack(const uint4 &v, float *x) {
    x[0] = __uint_as_float(v.x);
    x[1] = __uint_as_float(v.y);
    x[2] = __uint_as_float(v.z);
    x[3] = __uint_as_float(v.w);
  }
  static __device__ __forceinline__ float largest() { return FLT_MAX; }
  static __device__ __forceinline__ float max_of(const uint4 &v) {
    float t;
    asm("{\n\t.reg .f32 a, b;\n\tmax.NaN.f32 a, %1, %2;\n\tmax.NaN.f32 b, %3, %4;\n\tmax.NaN.f32 %0, a, b;\n\t}"
        : "=f"(t)
        : "f"(__uint_as_float(v.x)), "f"(__uint_as_float(v.y)), "f"(__uint_as_float(v.z)),
          "f"(__uint_as_float(v.w)));
    return t;
  }
};

__device__ __forceinline__ u64 warp_max_key(u64 k) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const unsigned long long other = __shfl_xor_sync(0xffffffffu, k, o);
    k = other > k ? other : k;
  }
  return k;
}

// Exclusive scan over the CTA of a thread's (count, weight); returns the totals.
__device__ void block_scan(Fixed &f, int &c, u64 &m, int &total_c, u64 &total_m) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c0 = c;
  const u64 m0 = m;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int oc = __shfl_up_sync(0xffffffffu, c, o);
    const u64 om = __shfl_up_sync(0xffffffffu, m, o);
    if (lane >= o) {
      c += oc;
      m += om;
    }
  }
  __syncthreads();
  if (lane == 31) {
    f.warp_c[warp] = c;
    f.warp_m[warp] = m;
  }
  __syncthreads();
  int wc = lane < NT / 32 ? f.warp_c[lane] : 0;
  u64 wm = lane < NT / 32 ? f.warp_m[lane] : 0;
  const int own_c = wc;
  const u64 own_m = wm;
#pragma unroll
  for (int o = 1; o < NT / 32; o <<= 1) {
    const int oc = __shfl_up_sync(0xffffffffu, wc, o);
    const u64 om = __shfl_up_sync(0xffffffffu, wm, o);
    if (lane >= o) {
      wc += oc;
      wm += om;
    }
  }
  total_c = __shfl_sync(0xffffffffu, wc, NT / 32 - 1);
  total_m = __shfl_sync(0xffffffffu, wm, NT / 32 - 1);
  c = __shfl_sync(0xffffffffu, wc - own_c, warp) + c - c0;
  m = __shfl_sync(0xffffffffu, wm - own_m, warp) + m - m0;
}

// f.list[0 .. n) in descending order to f.sorted: a key's place is the number
// of larger ones (n is mostly a few hundred; keys are distinct).
__device__ void sort_list(Fixed &f, int n) {
  if (threadIdx.x == 0 && (n & 1)) f.list[n] = 0;   // n < CAP when odd
  __syncthreads();
  const ulonglong2 *l2 = reinterpret_cast<const ulonglong2 *>(f.list);
  for (int i = threadIdx.x; i < n; i += NT) {
    const u64 k = f.list[i];
    int place = 0;
#pragma unroll 4
    for (int j = 0; j < (n + 1) / 2; ++j) {
      const ulonglong2 o = l2[j];
      place += (o.x > k ? 1 : 0) + (o.y > k ? 1 : 0);
    }
    f.sorted[place] = k;
  }
  __syncthreads();
}

struct KernelParams {
  SampleParams p;
  Tables t;
  int per;                       // tokens of a slice
};

// A CTA's tokens of a row.  RESIDENT: in shared memory, cleaned (NaN to -inf,
// +inf to the largest finite value, -inf around the ends); otherwise read from
// the logits (L2) in every pass and cleaned where an element needs it.
template <typename T, bool RESIDENT> struct Slice {
  static constexpr int E = Elem<T>::E;
  const T *src;                  // the slice's first token
  T *held;                       // its place in shared memory, -mis elements (16-byte aligned)
  int start, n, mis, nv;         // first id, tokens, elements before it in its first vector, vectors
  bool dirty;
  __device__ __forceinline__ const uint4 *vectors() const {
    return RESIDENT ? reinterpret_cast<const uint4 *>(held) : reinterpret_cast<const uint4 *>(src - mis);
  }
  __device__ __forceinline__ bool whole(int v) const { return v * E >= mis && (v + 1) * E <= mis + n; }
  static __device__ __forceinline__ float clean(float x) {
    return isnan(x) ? -INFINITY : fminf(x, Elem<T>::largest());
  }
  __device__ __forceinline__ float slow(int v, int e) const {   // an element at an end or in need of cleaning
    const int i = v * E + e - mis;
    return i >= 0 && i < n ? clean(to_f32(src[i])) : -INFINITY;
  }
  // fn(first id, E values) of every vector, U of them in flight
  template <int U, typename F> __device__ __forceinline__ void each_vector(F fn) const {
    each_vector<U>([](int, int, const float *) {}, [&](int, int id, const float *x) { fn(id, x); });
  }
  // ahead(u, first id, values) of U vectors, then fn(u, first id, values) of them
  template <int U, typename A, typename F> __device__ __forceinline__ void each_vector(A ahead, F fn) const {
    const uint4 *at = vectors();
    for (int v0 = threadIdx.x; v0 < nv; v0 += U * NT) {
      uint4 t[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int v = v0 + u * NT;
        t[u] = make_uint4(0, 0, 0, 0);
        if (RESIDENT ? v < nv : v < nv && whole(v)) t[u] = at[v];
      }
      auto values = [&](int u, int v, float *x) {
        Elem<T>::unpack(t[u], x);
        if (!RESIDENT && (dirty || !whole(v))) {
#pragma unroll
          for (int e = 0; e < E; ++e) x[e] = slow(v, e);
        }
      };
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int v = v0 + u * NT;
        float x[E];
        if (v < nv) {
          values(u, v, x);
          ahead(u, start + v * E - mis, x);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int v = v0 + u * NT;
        float x[E];
        if (v < nv) {
          values(u, v, x);
          fn(u, start + v * E - mis, x);
        }
      }
    }
  }
  template <typename F> __device__ __forceinline__ void each(F fn) const {   // fn(x, id)
    each_vector<2>([&](int id, const float *x) {
#pragma unroll
      for (int e = 0; e < E; ++e) fn(x[e], id + e);
    });
  }
  __device__ __forceinline__ float at(int i) const {
    return RESIDENT ? to_f32(held[mis + i]) : clean(to_f32(src[i]));
  }
};

// The general cut (the histogram way); every CTA of the cluster calls it.
template <typename Row>
__device__ __noinline__ u64 general_cut(Fixed &f, const Tables &tab, const Weigher weigh, float temp, int top_k,
                                        float top_p, int vocab, u64 cut, unsigned int *err, const Row tokens) {
  cg::cluster_group cl = cg::this_cluster();
  const int C = (int)cl.num_blocks(), rank = (int)cl.block_rank(), tid = threadIdx.x;
  const float m = weigh.m;
  Fixed &lead = *cl.map_shared_rank(&f, 0);
  auto clear = [&] {
    for (int i = tid; i < NB; i += NT) f.cnt[i] = f.lo[i] = f.hi[i] = 0;
    __syncthreads();
  };
  // u < 2^26.1 and at most 2^18 tokens a CTA: both sums fit 32 bits, and nothing is read back
  auto add = [&](int b, uint32_t u) {
    if (top_k > 0) atomicAdd(&f.cnt[b], 1u);
    atomicAdd(&f.lo[b], u & 0x1fffu);
    atomicAdd(&f.hi[b], u >> 13);
  };
  // With top-p alone, tokens beyond this exponent are outside the nucleus
  // whatever the rest is (vocab of them weigh half of 1 - p at most, the
  // maximum alone weighs 1): their sum is all that counts.
  const float far = top_k > 0 ? INFINITY : log2f((float)vocab) - log2f(fmaxf(1.f - top_p, 1e-9f)) + 1.f;
  auto is_far = [&](float x) { return __fmul_rn(__fsub_rn(m, x), weigh.c_hi) > far; };
  __syncthreads();
  clear();
  float part = 0.f;
  tokens.each([&](float x, int) {
    if (is_far(x)) {
      part += ex2((x - m) * weigh.c_hi);
    } else if (x > -INFINITY) {
      int b;
      uint32_t u;
      weigh(x, tab, b, u);
      add(b, u);
    }
  });
  {
    u64 rest = (u64)(part * 0x1p44f);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) rest += __shfl_xor_sync(0xffffffffu, rest, o);
    if ((tid & 31) == 0) f.w_rest[tid >> 5] = rest;
    __syncthreads();
    if (tid == 0) {
      u64 r = 0;
      for (int w = 0; w < NT / 32; ++w) r += f.w_rest[w];
      f.own_rest = r;
    }
  }
  cl.sync();

  // The leader keeps its bins' (tokens, weight) above them; the others follow its commands.
  int n0[PB], above0[PB];
  u64 above_m0[PB];
  int stage = 0;               // leader: 0 top-k, 1 top-p
  int bin = 0, above = 0;      // leader: the current range and what lies above it
  u64 above_m = 0, target = 0; // leader: the weight that the cut's predecessors stay below
  u64 lo = 0, hi = 0;
  // bins tid * PB ..: sums over the cluster (of: the bin whose octave they have, -1: their own)
  auto totals = [&](int *nn, u64 *mm, int of) {
    for (int i = 0; i < PB; ++i) {
      const int b = tid * PB + i;
      nn[i] = 0;
      u64 s = 0;
      for (int r = 0; r < C; ++r) {
        const Fixed &o = *cl.map_shared_rank(&f, r);
        nn[i] += (int)o.cnt[b];
        s += ((u64)o.hi[b] << 13) + o.lo[b];
      }
      mm[i] = units(s, of < 0 ? b : of);
      if (top_k <= 0) nn[i] = s > 0;   // not counted: a list that overflows tells
    }
  };
  auto scan = [&](const int *nn, const u64 *mm, int *ab, u64 *abm, int &tc, u64 &tm) {
    int c = 0;
    u64 w = 0;
    for (int i = 0; i < PB; ++i) {
      c += nn[i];
      w += mm[i];
    }
    block_scan(f, c, w, tc, tm);
    for (int i = 0; i < PB; ++i) {
      ab[i] = c;
      abm[i] = w;
      c += nn[i];
      w += mm[i];
    }
  };
  // the bin that holds the cut, given what lies above every bin
  auto select = [&](const int *nn, const int *ab, const u64 *abm, int base, u64 base_m) {
    if (tid == 0) f.sel_bin = -1;
    __syncthreads();
    int mine = -1;
    for (int i = 0; i < PB; ++i)
      if (nn[i] > 0 && (stage == 0 ? base + ab[i] < top_k : base_m + abm[i] < target)) mine = tid * PB + i;
    if (mine >= 0) atomicMax(&f.sel_bin, mine);
    __syncthreads();
    const int s = max(f.sel_bin, 0);
    if (s / PB == tid) {
      const int i = s % PB;
      f.sel_n = nn[i];
      f.sel_above = base + ab[i];
      f.sel_above_m = base_m + abm[i];
    }
    __syncthreads();
    above = f.sel_above;
    above_m = f.sel_above_m;
    return s;
  };
  // thread r of the leader: command to CTA r
  auto tell = [&](int cmd, int sh) {
    if (tid < C) {
      Fixed &o = *cl.map_shared_rank(&f, tid);
      o.cmd = cmd;
      o.bin = bin;
      o.sh = sh;
      o.range_lo = lo;
      o.range_hi = hi;
      o.cut = cut;
    }
  };
  auto tell_range = [&](int count) {
    int sh = 0;
    while (((hi - lo - 1) >> sh) >= NB) ++sh;
    if (tid == 0) f.n_list = 0;
    tell(count <= CAP ? CMD_GATHER : CMD_SPLIT, sh);
  };
  // start of a stage: the first histogram's bin, and its range of keys, wider than it: a bin begins half
  // a bin before its number, the last one at TAIL, which is 0.6 before
  auto begin = [&] {
    bin = select(n0, above0, above_m0, 0, 0);
    float x_hi = FLT_MAX, x_lo = -FLT_MAX;
    if (tid < C) {
      const double inv = (double)temp * 0.6931471805599453 / 32.0;
      static_assert(32.0 * TAIL > NB - 1 - 0.61, "the last bin's tokens are in its range");
      x_hi = __double2float_ru(fmax((double)m - fmax(0.0, (bin - 0.62) * inv), -(double)FLT_MAX));
      if (bin < NB - 1) x_lo = __double2float_rd(fmax((double)m - (bin + 0.51) * inv, -(double)FLT_MAX));
    }
    x_hi = __shfl_sync(0xffffffffu, x_hi, 0);
    x_lo = __shfl_sync(0xffffffffu, x_lo, 0);
    if (tid == 0) {
      f.range_lo = (u64)order_image(x_lo) << 32;
      f.range_hi = ((u64)one_zero(order_image(x_hi)) + 1) << 32;
    }
    __syncthreads();
    lo = f.range_lo;
    hi = f.range_hi;
    __syncthreads();
    tell_range(f.sel_n);
  };
  auto set_target = [&](u64 total) {
    if (tid == 0) f.target = share_of(total, top_p);
    __syncthreads();
    target = f.target;
  };
  for (int guard = 0;; ++guard) {
    if (rank == 0) {
      if (guard == 0) {
        u64 mm[PB], total_m;
        int total;
        totals(n0, mm, -1);
        scan(n0, mm, above0, above_m0, total, total_m);
        for (int r = 0; r < C; ++r) total_m += cl.map_shared_rank(&f, r)->own_rest;
        stage = top_k > 0 && top_k < total ? 0 : 1;
        set_target(total_m);
        if (stage == 1 && !(top_p < 1.f)) tell(CMD_DONE, 0);
        else begin();
      } else if (f.cmd == CMD_SPLIT) {
        int nn[PB], ab[PB], tc;
        u64 mm[PB], abm[PB], tm;
        totals(nn, mm, bin);
        scan(nn, mm, ab, abm, tc, tm);
        const int s = select(nn, ab, abm, above, above_m);
        const int sh = f.sh;
        const u64 v = (u64)(NB - 1 - s);
        const u64 l = lo + (v << sh), h = l + (1ull << sh);
        lo = l;
        hi = h < hi ? h : hi;
        __syncthreads();   // sh has been read
        tell_range(f.sel_n);
      } else if (f.n_list > CAP || f.n_list == 0) {
        // (no token at all: bins and key ranges would disagree; the rounds run out, which is flagged)
        const int over = f.n_list;
        __syncthreads();
        tell_range(over);
      } else {
        // the gathered tokens: sort, then walk to the cut
        const int cnt = f.n_list;
        sort_list(f, cnt);
        int nn[2], ab[2], tc;
        u64 mm[2], abm[2], tm;
        static_assert(CAP == 2 * NT && PB == 2, "two tokens and two bins a thread");
        for (int i = 0; i < 2; ++i) {
          const int at = 2 * tid + i;
          nn[i] = at < cnt ? 1 : 0;
          mm[i] = 0;
          if (at < cnt) {
            int b;
            uint32_t u;
            weigh(order_value((uint32_t)(f.sorted[at] >> 32)), tab, b, u);
            mm[i] = units(u, bin);
          }
        }
        scan(nn, mm, ab, abm, tc, tm);
        const int s = select(nn, ab, abm, above, above_m);   // the cut's place in the list
        cut = f.sorted[s];
        if (stage == 0 && top_p < 1.f) {
          if (s / 2 == tid) f.range_lo = above_m + mm[s % 2];   // weight through the cut
          __syncthreads();
          const u64 through = f.range_lo;
          __syncthreads();
          stage = 1;
          set_target(through);
          begin();
        } else {
          tell(CMD_DONE, 0);
        }
      }
    }
    cl.sync();
    const int cmd = f.cmd;
    if (cmd == CMD_DONE) break;
    const int want = f.bin, sh = f.sh;
    const u64 r_lo = f.range_lo, r_hi = f.range_hi;
    if (guard > 24) {   // 64-bit keys end long before
      if (rank == 0 && tid == 0) raise_error(err, DFLASH_DERR_TIMEOUT);
      break;
    }
    if (cmd == CMD_SPLIT) clear();
    const float x_lo = order_value((uint32_t)(r_lo >> 32)), x_hi = order_value((uint32_t)((r_hi - 1) >> 32));
    tokens.each([&](float x, int id) {
      if (x < x_lo || x > x_hi || is_far(x)) return;
      const u64 k = ((u64)one_zero(order_image(x)) << 32) | (uint32_t)~(uint32_t)id;
      if (k < r_lo || k >= r_hi) return;
      int b;
      uint32_t u;
      weigh(x, tab, b, u);
      if (b != want) return;
      if (cmd == CMD_GATHER) {
        const int at = atomicAdd(&lead.n_list, 1);
        if (at < CAP) lead.list[at] = k;
      } else {
        add(NB - 1 - (int)((k - r_lo) >> sh), u);
      }
    });
    cl.sync();
  }
  return f.cut;
}

// RESIDENT: the row's slices stay in the cluster's shared memory.  Otherwise a
// CTA a row, which reads it again from L2 in every pass.
template <typename T, bool DRAW, bool RESIDENT>
__global__ void __launch_bounds__(NT, 2) sampling_kernel(const __grid_constant__ KernelParams kp) {
  constexpr int E = Elem<T>::E;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ Tables tab;
  Fixed &f = *reinterpret_cast<Fixed *>(smem);
  T *slice = reinterpret_cast<T *>(smem + ((sizeof(Fixed) + 15) / 16) * 16);
  cg::cluster_group cl = cg::this_cluster();
  const int C = (int)cl.num_blocks(), rank = (int)cl.block_rank(), tid = threadIdx.x;
  const int lane = tid & 31, warp = tid >> 5;
  const SampleParams &p = kp.p;
  const int row = blockIdx.x / C, V = p.vocab;
  pdl_wait();
  if (tid < 32) {
    tab.u[tid] = kp.t.u[tid];
    tab.f[tid] = kp.t.f[tid];
  }

  const int entry = row / p.rows_per_entry;
  float temp = p.temperature ? p.temperature[entry] : 1.f;
  int top_k = p.top_k ? p.top_k[entry] : 0;
  float top_p = p.top_p ? p.top_p[entry] : 1.f;
  float min_p = p.min_p ? p.min_p[entry] : 0.f;

  // ---- the slice and its maximum
  Slice<T, RESIDENT> tokens;
  tokens.start = min(rank * kp.per, V);
  tokens.n = min(kp.per, V - tokens.start);
  tokens.src = (const T *)p.logits + (int64_t)row * p.ld + tokens.start;
  tokens.held = slice;
  tokens.mis = (int)(((uintptr_t)tokens.src & 15) / sizeof(T));
  tokens.nv = tokens.n > 0 ? (tokens.mis + tokens.n + E - 1) / E : 0;
  tokens.dirty = false;
  const int start = tokens.start, n = tokens.n, mis = tokens.mis, nv = tokens.nv;
  if (temp < FLT_MIN) {  // the largest logit alone: one token, whatever the weights
    if (temp >= 0.f && !isnan(top_p) && min_p <= 1.f) {
      temp = 1.f;
      top_k = 1;
      top_p = 1.f;
      min_p = 0.f;
    }
  }
  if (top_p < 0.f) top_p = 0.f;   // the first token alone, as 0 (NaN stays for the check below)
  if (top_k <= 0 || top_k >= V) top_k = 0;
  const bool filtered = top_k > 0 || top_p < 1.f;
  // nothing is dropped: the sum of the weights goes along with the first pass, relative to the
  // thread's running maximum
  const bool plain = !DRAW && !filtered && !(min_p > 0.f);
  const float c0 = __fdiv_rn(1.44269502f, temp);
  if (min_p > 0.f && tid == NT - 1) f.t_log = (double)temp * log((double)min_p);
  float mx = -INFINITY, sum_x = 0.f;
  {
    const uint4 *gv = reinterpret_cast<const uint4 *>(tokens.src - mis);
    uint4 *sv = reinterpret_cast<uint4 *>(slice);
    bool dirty = false;
    constexpr int U = 8;
    for (int v0 = tid; v0 < nv; v0 += U * NT) {
      uint4 t[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int v = v0 + u * NT;
        t[u] = make_uint4(~0u, ~0u, ~0u, ~0u);        // NaN: the ends come element by element
        if (v < nv && tokens.whole(v)) t[u] = RESIDENT ? __ldcs(gv + v) : gv[v];
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int v = v0 + u * NT;
        if (v < nv) {
          const float vm = Elem<T>::max_of(t[u]);
          if (vm <= Elem<T>::largest()) {
            if (RESIDENT) sv[v] = t[u];
            if (plain && vm > mx) {
              if (mx > -INFINITY) sum_x *= ex2((mx - vm) * c0);
              mx = vm;
            }
            if (plain && mx > -INFINITY) {
              float x[E], s0 = 0.f;
              Elem<T>::unpack(t[u], x);
#pragma unroll
              for (int e = 0; e < E; ++e) s0 += ex2((x[e] - mx) * c0);
              sum_x += s0;
            }
            mx = fmaxf(mx, vm);
          } else {                                    // an end, a NaN or an infinity
            if (tokens.whole(v)) dirty = true;
            for (int e = 0; e < E; ++e) {
              const float x = tokens.slow(v, e);
              if (plain && x > -INFINITY)
                sum_x = x > mx ? (mx > -INFINITY ? sum_x * ex2((mx - x) * c0) : 0.f) + 1.f
                               : sum_x + ex2((x - mx) * c0);
              mx = fmaxf(mx, x);
              if (RESIDENT) slice[v * E + e] = from_f32<T>(x);
            }
          }
        }
      }
    }
    if (!RESIDENT) tokens.dirty = __syncthreads_or(dirty) != 0;
  }
  if (!(temp >= 0.f && temp <= MAX_T) || isnan(top_p) || !(min_p <= 1.f)) {
    if (rank == 0 && tid == 0) raise_error(p.err, DFLASH_DERR_SAMPLING);
    return;   // the whole cluster, before any of its barriers
  }
  cl.barrier_arrive();   // every CTA of the cluster runs before the first remote access
  const float own_mx = mx;   // what sum_x is relative to
  const bool by_min_p = !filtered && min_p > 0.f;   // min-p alone: its border is known once the maximum is
  const bool brief = (filtered && top_k <= MAX_K) || by_min_p;
  const int j = brief && !by_min_p ? ((top_k > 0 ? top_k : TOP_P_LIST) + C - 1) / C : 0;
  float low = -INFINITY;
  if (j > GROUP_PLACES) {
    const uint32_t own = order_image(mx);
    uint32_t found = 0;
#pragma unroll 1
    for (int bit = 31; bit >= 12; --bit) {
      const uint32_t want = found | (1u << bit);
      if (__syncthreads_count(own >= want) >= j) found = want;
    }
    low = found >= order_image(-FLT_MAX) ? order_value(found) : -INFINITY;
  }
  mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
  mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
  if ((tid & 3) == 0) f.group[tid >> 2] = mx;
  if (tid == 0) {
    f.n_list = 0;
    f.own_n = 0;
  }
  __syncthreads();
  if (j > 1 && j <= GROUP_PLACES) {
    // the j-th largest is the smallest with fewer than j larger ones
    if (tid < GROUPS) {
      const float own = f.group[tid];
      int place = 0;
#pragma unroll 8
      for (int i = 0; i < GROUPS / 4; ++i) {
        const float4 o = reinterpret_cast<const float4 *>(f.group)[i];
        place += (o.x > own) + (o.y > own) + (o.z > own) + (o.w > own);
      }
      const float l = -warp_max(place < j ? -own : -INFINITY);
      if (lane == 0) f.fred[warp] = l;
    }
    __syncthreads();
    low = f.fred[0];
    for (int w = 1; w < GROUPS / 32; ++w) low = fminf(low, f.fred[w]);
  }
  {
    const float4 g = reinterpret_cast<const float4 *>(f.group)[lane];
    mx = warp_max(fmaxf(fmaxf(g.x, g.y), fmaxf(g.z, g.w)));
  }
  if (j == 1) low = mx;
  cl.barrier_wait();
  if (tid < C) {
    Fixed &o = *cl.map_shared_rank(&f, tid);
    o.x_max[rank] = mx;
    o.x_low[rank] = low;
  }
  cl.sync();
  float m = f.x_max[0];
  low = f.x_low[0];
  for (int r = 1; r < C; ++r) {
    m = fmaxf(m, f.x_max[r]);
    low = fminf(low, f.x_low[r]);
  }
  if (top_k == 1) low = m;

  float *out = DRAW ? nullptr : p.probs + (int64_t)row * V + start;
  const int head = DRAW ? 0 : min(n, (int)((16 - ((uintptr_t)out & 15)) & 15) / 4);
  const int quads = DRAW ? 0 : (n - head) / 4, done = head + 4 * quads;
  auto write_zeros = [&] {
    if (tid < head) out[tid] = 0.f;
    for (int q = tid; q < quads; q += NT)
      __stcs(reinterpret_cast<float4 *>(out + head + 4 * q), make_float4(0.f, 0.f, 0.f, 0.f));
    if (tid < n - done) out[done + tid] = 0.f;
  };
  if (m == -INFINITY) {
    if (!DRAW) write_zeros();
    if (rank == 0 && tid == 0) {
      if (DRAW) {
        p.ids[row] = -1;
        if (p.prob) p.prob[row] = 0.f;
      }
      raise_error(p.err, DFLASH_DERR_EMPTY_ROW);
    }
    return;   // the whole cluster, nothing remote in flight
  }

  Weigher weigh;
  weigh.m = m;
  {
    // log2(e) / T as a pair: quotient, and its remainder over T
    const float l2e = 1.44269502f, l2e_lo = 1.92596299e-8f;
    weigh.c_hi = __fdiv_rn(l2e, temp);
    weigh.c_lo = __fdiv_rn(__fadd_rn(__fmaf_rn(-weigh.c_hi, temp, l2e), l2e_lo), temp);
  }
  const float c = weigh.c_hi;
  // min-p: w >= min_p is x >= m + T ln min_p
  if (tid == 0) f.x_min = min_p > 0.f ? __double2float_ru(fmax((double)m + f.t_log, -(double)FLT_MAX)) : -FLT_MAX;
  if (by_min_p) {
    __syncthreads();
    low = f.x_min;
  }
  const float *noise = DRAW ? p.noise + (int64_t)row * V : nullptr;

  u64 cut = (u64)order_image(-FLT_MAX) << 32;   // every finite logit
  if (brief) {
    // ---- the short way: tokens >= low to the leader's list, the weight of the others
    Fixed &lead = *cl.map_shared_rank(&f, 0);
    const bool weights = top_k == 0 && !by_min_p;
    u64 listed = 0, rest = 0;
    float part0 = 0.f, part1 = 0.f;
    // to this CTA's list first (weighed and sent together below): what a token costs here, all lanes
    // of its warp wait for
    auto list_token = [&](float x, int id) {
      const int at = atomicAdd(&f.own_n, 1);
      if (at < CAP) f.sorted[at] = key_of(x, id);
    };
    // most vectors hold no token of the list
    auto list_some = [&](int id, const float *x) {
      float vm = x[0];
#pragma unroll
      for (int e = 1; e < E; ++e) vm = fmaxf(vm, x[e]);
      if (vm >= low && vm > -INFINITY) {
#pragma unroll
        for (int e = 0; e < E; ++e)
          if (x[e] >= low && x[e] > -INFINITY) list_token(x[e], id + e);
      }
    };
    if (weights) {
      tokens.template each_vector<2>([&](int id, const float *x) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const float w = ex2((x[e] - m) * c);
          if (e & 1) part1 += x[e] >= low ? 0.f : w;
          else part0 += x[e] >= low ? 0.f : w;
        }
        list_some(id, x);
      });
    } else {
      tokens.template each_vector<4>(list_some);
    }
    __syncthreads();
    const int own_n = min(f.own_n, CAP);
    if (tid == 0) f.own_at = own_n > 0 ? atomicAdd(&lead.n_list, own_n) : 0;
    if (weights) {
      for (int i = tid; i < own_n; i += NT) {
        int b;
        uint32_t u;
        weigh(order_value((uint32_t)(f.sorted[i] >> 32)), tab, b, u);
        listed += units(u, b);
      }
      rest = (u64)((part0 + part1) * 0x1p44f);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        rest += __shfl_xor_sync(0xffffffffu, rest, o);
        listed += __shfl_xor_sync(0xffffffffu, listed, o);
      }
      if (lane == 0) {
        f.w_rest[warp] = rest;
        f.w_listed[warp] = listed;
      }
    }
    __syncthreads();
    for (int i = tid; i < own_n; i += NT)
      if (f.own_at + i < CAP)
        lead.list[f.own_at + i] = ((u64)one_zero((uint32_t)(f.sorted[i] >> 32)) << 32) | (uint32_t)f.sorted[i];
    if (tid < C) {
      Fixed &o = *cl.map_shared_rank(&f, tid);
      u64 r = 0, l = 0;
      if (weights) {
#pragma unroll
        for (int w = 0; w < NT / 32; ++w) {
          r += f.w_rest[w];
          l += f.w_listed[w];
        }
      }
      o.x_n[rank] = f.own_n;
      o.x_rest[rank] = r;
      o.x_listed[rank] = l;
    }
    cl.sync();   // the list is complete
    int all = 0;
    u64 all_rest = 0, all_listed = 0;
    for (int r = 0; r < C; ++r) {
      all += f.x_n[r];
      all_rest += f.x_rest[r];
      all_listed += f.x_listed[r];
    }
    // with top-k the list holds the k largest (or every finite logit); for top-p alone the
    // nucleus is inside when the list's weight reaches p of the total
    bool inside = all <= CAP;
    if (inside && weights) {
      if (tid == 0) f.target = share_of(all_rest + all_listed, top_p);
      __syncthreads();
      inside = all_listed >= f.target || all_rest == 0;
    }
    if (inside) {
      if (rank != 0) {
        if (DRAW) return;
        // zeros meanwhile; this arrival passes nothing on, so it does not wait for them
        cluster_arrive_relaxed();
        write_zeros();
      } else {
        sort_list(f, all);
        const int kk = top_k > 0 ? min(top_k, all) : all;
        u64 w[2], sum2 = 0, total;
        float x[2];
        for (int i = 0; i < 2; ++i) {
          const int at = 2 * tid + i;
          w[i] = 0;
          x[i] = -INFINITY;
          if (at < kk) {
            x[i] = order_value((uint32_t)(f.sorted[at] >> 32));
            int b;
            uint32_t u;
            weigh(x[i], tab, b, u);
            w[i] = units(u, b);
          }
          sum2 += w[i];
        }
        u64 target = ~0ull, before = 0;
        if (top_p < 1.f) {
          int zero = 0, none;
          before = sum2;
          block_scan(f, zero, before, none, total);
          if (tid == 0) f.target = share_of(total + (weights ? all_rest : 0), top_p);
          __syncthreads();
          target = f.target;
        }
        const float x_min = f.x_min;
        bool keep[2];
        float e[2], sum_f = 0.f;
        int ids[2];
        u64 best = 0;
        for (int i = 0; i < 2; ++i) {
          const int at = 2 * tid + i;
          keep[i] = at < kk && (before < target || at == 0) && x[i] >= x_min;
          before += w[i];
          e[i] = keep[i] ? ex2((x[i] - m) * c) : 0.f;
          sum_f += e[i];
          ids[i] = keep[i] ? (int)~(uint32_t)f.sorted[at] : 0;
          if (DRAW && keep[i]) {
            const float score = e[i] / noise[ids[i]];
            const u64 k = score > 0.f ? argmax_key(score, ids[i]) : 0;
            best = k > best ? k : best;
          }
        }
        sum_f = warp_sum(sum_f);
        if (DRAW) best = warp_max_key(best);
        if (lane == 0) {
          f.fred[warp] = sum_f;
          f.kred[warp] = best;
        }
        const int n_kept = __syncthreads_count(keep[0]) + __syncthreads_count(keep[1]);
        const float inv = 1.f / warp_sum(lane < NT / 32 ? f.fred[lane] : 0.f);
        if (DRAW) {
          if (warp == 0) {
            best = warp_max_key(f.kred[lane & (NT / 32 - 1)]);
            if (lane == 0) {
              const int id = best ? argmax_key_index(best) : -1;
              p.ids[row] = id;
              if (id < 0) raise_error(p.err, DFLASH_DERR_SAMPLING);
              if (p.prob && id < 0) p.prob[row] = 0.f;
              else if (p.prob) {
                const float xd = to_f32(((const T *)p.logits)[(int64_t)row * p.ld + id]);
                p.prob[row] = ex2((fminf(xd, Elem<T>::largest()) - m) * c) * inv;
              }
            }
          }
          return;
        }
        // the kept tokens are a prefix of the sorted list: (probability, id) to every CTA
        for (int r = 0; r < C; ++r) {
          Fixed &o = *cl.map_shared_rank(&f, r);
          for (int i = 0; i < 2; ++i)
            if (keep[i]) o.list[2 * tid + i] = ((u64)__float_as_uint(e[i] * inv) << 32) | (uint32_t)ids[i];
          if (tid == 0) o.n_list = n_kept;
        }
        cl.barrier_arrive();
        write_zeros();
      }
      cl.barrier_wait();
      __syncthreads();   // this CTA's zeros come before its tokens
      for (int i = tid; i < f.n_list; i += NT) {
        const u64 t = f.list[i];
        const int id = (int)(uint32_t)t - start;
        if (id >= 0 && id < n) out[id] = __uint_as_float((uint32_t)(t >> 32));
      }
      return;
    }
  }
  if (filtered) {
    cl.sync();   // the list and the exchange slots of the short way have been read
    cut = general_cut(f, tab, weigh, temp, top_k, top_p, V, cut, p.err, tokens);
  }
  __syncthreads();   // x_min
  {
    const u64 k = (u64)order_image(f.x_min) << 32;
    cut = k > cut ? k : cut;
  }

  // ---- the kept tokens' sum (and the race)
  const float xc = order_value((uint32_t)(cut >> 32));
  const uint32_t idc = ~(uint32_t)cut;
  const bool ties = idc != 0xffffffffu;   // some tokens equal to the cut are dropped
  auto kept = [&](float x, int id) { return x >= xc && !(ties && x == xc && (uint32_t)id > idc); };
  float s0 = 0.f, s1 = 0.f;
  u64 best = 0;
  if (plain) {
    s0 = own_mx > -INFINITY ? sum_x * ex2((own_mx - m) * c) : 0.f;
  } else if (!DRAW) {
    tokens.each([&](float x, int id) {
      const float w = kept(x, id) ? ex2((x - m) * c) : 0.f;
      if (id & 1) s1 += w;
      else s0 += w;
    });
  } else {
    // the exact quotient only where an approximate one (2^-21) reaches the best so far; a thread's
    // ids ascend, so the first of equal scores has the lowest
    float top = 0.f;
    int top_id = 0;
    float e[2][E];                       // the noise of two vectors is in flight
    bool any[2];
    auto fetch = [&](int u, int id, const float *x) {
      any[u] = false;
#pragma unroll
      for (int i = 0; i < E; ++i) any[u] = any[u] || kept(x[i], id + i);
      if (!any[u]) return;
      if (((uintptr_t)(noise + id) & 15) == 0 && id >= start && id + E <= start + n) {
#pragma unroll
        for (int i = 0; i < E; i += 4) {
          const float4 t = __ldcs(reinterpret_cast<const float4 *>(noise + id + i));
          e[u][i] = t.x, e[u][i + 1] = t.y, e[u][i + 2] = t.z, e[u][i + 3] = t.w;
        }
      } else {
#pragma unroll
        for (int i = 0; i < E; ++i) e[u][i] = kept(x[i], id + i) ? noise[id + i] : 1.f;
      }
    };
    tokens.template each_vector<2>(fetch, [&](int u, int id, const float *x) {
      if (!any[u]) return;
#pragma unroll
      for (int i = 0; i < E; ++i) {
        const bool k = kept(x[i], id + i);
        const float w = k ? ex2((x[i] - m) * c) : 0.f;
        if (i & 1) s1 += w;
        else s0 += w;
        if (k && __fdividef(w, e[u][i]) * 1.000001f >= top) {
          const float score = __fdiv_rn(w, e[u][i]);
          if (score > top) {
            top = score;
            top_id = id + i;
          }
        }
      }
    });
    if (top > 0.f) best = argmax_key(top, top_id);
  }
  const float sum = warp_sum(s0 + s1);
  if (DRAW) best = warp_max_key(best);
  __syncthreads();
  if (lane == 0) {
    f.fred[warp] = sum;
    if (DRAW) f.kred[warp] = best;
  }
  __syncthreads();
  if (tid < 32) {
    const float s = warp_sum(lane < NT / 32 ? f.fred[lane] : 0.f);
    if (DRAW) best = warp_max_key(f.kred[lane & (NT / 32 - 1)]);
    if (tid < C) {
      Fixed &o = *cl.map_shared_rank(&f, tid);
      o.x_sum[rank] = s;
      if (DRAW) o.x_race[rank] = best;
    }
  }
  cl.sync();   // the last exchange: nothing remote after it
  float total = 0;
  for (int r = 0; r < C; ++r) total += f.x_sum[r];
  const float inv = 1.f / total;
  if (DRAW) {
    if (rank == 0 && tid == 0) {
      best = 0;
      for (int r = 0; r < C; ++r) best = f.x_race[r] > best ? f.x_race[r] : best;
      // no score above 0: every kept token's variate is negative, infinite or NaN
      const int id = best ? argmax_key_index(best) : -1;
      p.ids[row] = id;
      if (id < 0) raise_error(p.err, DFLASH_DERR_SAMPLING);
      if (p.prob && id < 0) p.prob[row] = 0.f;
      else if (p.prob) {
        float x = to_f32(((const T *)p.logits)[(int64_t)row * p.ld + id]);
        x = fminf(x, Elem<T>::largest());
        p.prob[row] = ex2((x - m) * c) * inv;
      }
    }
    return;
  }
  // ---- probabilities: 16-byte stores from the row's first aligned element
  auto prob_of = [&](float x, int id) { return kept(x, id) ? ex2((x - m) * c) * inv : 0.f; };
  auto prob_at = [&](int i) { return prob_of(tokens.at(i), start + i); };
  if (tid < head) out[tid] = prob_at(tid);
  if ((mis + head) % 4 == 0) {
    constexpr int U = 4;                   // four elements a load, U of them in flight
    typedef typename Elem<T>::Quad Quad;
    const T *from = RESIDENT ? slice + mis + head : tokens.src + head;
    for (int q0 = tid; q0 < quads; q0 += U * NT) {
      Quad t[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (q0 + u * NT < quads) t[u] = *reinterpret_cast<const Quad *>(from + 4 * (q0 + u * NT));
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = head + 4 * (q0 + u * NT), id = start + i;
        if (q0 + u * NT < quads) {
          float x[4];
          Elem<T>::unpack4(t[u], x);
          if (!RESIDENT && tokens.dirty) {
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = tokens.clean(x[e]);
          }
          __stcs(reinterpret_cast<float4 *>(out + i), make_float4(prob_of(x[0], id), prob_of(x[1], id + 1),
                                                                  prob_of(x[2], id + 2), prob_of(x[3], id + 3)));
        }
      }
    }
  } else {
    for (int q = tid; q < quads; q += NT) {
      const int i = head + 4 * q;
      *reinterpret_cast<float4 *>(out + i) =
          make_float4(prob_at(i), prob_at(i + 1), prob_at(i + 2), prob_at(i + 3));
    }
  }
  if (tid < n - done) out[done + tid] = prob_at(done + tid);
}

size_t smem_bytes(int per, int es) {
  return (sizeof(Fixed) + 15) / 16 * 16 + (size_t)per * es + 32;
}
int slice_of(int vocab, int C) { return ((vocab + C - 1) / C + 15) / 16 * 16; }

template <typename T, bool DRAW, bool RESIDENT>
cudaError_t launch(const SampleParams &p, int C, cudaStream_t s) {
  KernelParams kp;
  kp.p = p;
  kp.per = slice_of(p.vocab, C);
  for (int i = 0; i < 32; ++i) {
    const double w = std::exp2(26.0 - i / 32.0);
    kp.t.u[i] = (uint32_t)std::llround(w);
    kp.t.f[i] = (float)w;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.rows * C));
  cfg.blockDim = dim3(NT);
  cfg.dynamicSmemBytes = smem_bytes(RESIDENT ? kp.per : 0, sizeof(T));
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = C;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, sampling_kernel<T, DRAW, RESIDENT>, kp);
}

template <typename T, bool DRAW> cudaError_t launch(const SampleParams &p, cudaStream_t s) {
  const int es = sizeof(T);
  int dev = 0, sms = 0;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  // A CTA a row once that fills the GPU: no cluster barriers, at the price of reading the row again
  // (304 rows of 151936: 66 us against 84 with top-k and top-p, 67 against 74 unfiltered; 128 rows 35
  // against 40 and 40 against 34).
  if (p.rows >= 2 * sms && p.vocab <= STREAM_VOCAB) return launch<T, DRAW, false>(p, 1, s);
  // The fewest CTAs whose slices leave room for two of them on an SM (128 rows of 151936: 40 us with
  // clusters of 4, 52 with 8); more while rows are too few to fill the GPU and a slice stays worth a CTA
  // (down to half of 4096: unfiltered rows of 4000 to 16000 0.1 to 0.4 us less, 16 filtered ones of
  // 16000 9.5 us against 8.2; no smaller than 16384: 0.3 to 1.5 us more for 1 to 8 rows)
  int C = 1;
  while (C < MAXC && smem_bytes(slice_of(p.vocab, C), es) > 108 * 1024) C *= 2;
  while (C < MAXC && (int64_t)p.rows * C * 2 <= sms && slice_of(p.vocab, C) > 4096) C *= 2;
  return launch<T, DRAW, true>(p, C, s);
}

template <typename T, bool DRAW> cudaError_t prepare() {
  return cudaFuncSetAttribute(sampling_kernel<T, DRAW, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              MAX_SMEM);
}

}  // namespace

int sampling_max_vocab(int dtype) { return dtype == DFLASH_BF16 ? 524288 : 262144; }

cudaError_t launch_sampling(int dtype, const SampleParams &p, cudaStream_t s) {
  if (dtype == DFLASH_BF16) return p.probs ? launch<bf16, false>(p, s) : launch<bf16, true>(p, s);
  return p.probs ? launch<float, false>(p, s) : launch<float, true>(p, s);
}

cudaError_t prepare_sampling() {
  cudaError_t e;
  if ((e = prepare<bf16, false>()) != cudaSuccess || (e = prepare<bf16, true>()) != cudaSuccess ||
      (e = prepare<float, false>()) != cudaSuccess)
    return e;
  return prepare<float, true>();
}

}  // namespace dflash

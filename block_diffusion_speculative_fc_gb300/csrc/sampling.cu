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
// once, which bounds the operator (6 or 8 bytes an element); every pass in
// between runs on shared memory.  Cuts are found without sorting the row: a
// histogram over a (32 bins per unit, so a bin's weights are alike) gives
// counts and weights above every bin; the few tokens of the bin that holds
// the cut are gathered in the cluster's first CTA, sorted, and walked.  A bin
// with more tokens than that list holds is split by key until it fits (equal
// logits split by id).
//
// Sums that decide a border are whole numbers: a weight is rounded once to a
// multiple of 2^-28 of its bin's octave (about 2^-28 relative), so they do not
// go by the order of atomics, and a border falls where 64-bit arithmetic puts
// it except within about 1e-9 of a tie.  min-p compares logits with m + T ln
// min_p formed in 64 bits.
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
constexpr int NB = 1024;         // histogram bins: a = 0 .. 31.97 and one for the rest
constexpr int PB = NB / NT;      // bins of a thread in a scan
constexpr int CAP = 1024;        // gathered tokens (two a thread)
constexpr int MAXC = 8;          // CTAs of a cluster
constexpr int MAX_SMEM = 220 * 1024;

struct Tables {
  uint32_t u[32];                // round(2^28 2^(-i/32))
  float f[32];                   // 2^28 2^(-i/32)
};

struct Fixed {
  unsigned long long list[CAP];
  uint32_t cnt[NB], lo[NB], hi[NB];   // tokens, and weight as a 64-bit sum
  double warp_m[NT / 32];
  int warp_c[NT / 32];
  float fred[NT / 32];
  unsigned long long kred[NT / 32];
  // exchanged between the CTAs of the cluster, one slot per rank
  float x_max[MAXC];
  unsigned long long x_arg[MAXC], x_race[MAXC];
  double x_sum[MAXC];
  float pruned;                  // weight this CTA left out of the histogram
  // the leader's command to every CTA
  int cmd, bin, sh;
  unsigned long long range_lo, range_hi, cut;
  int n_list;
  // leader: the bin that holds a cut
  int sel_bin, sel_n, sel_above;
  double sel_above_m, sel_through;
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
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Bin and weight of a token.  The weight is u 2^-(28 + octave(bin)).  a is
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
    if (!(a < 31.95f)) {                // far tail (a may be infinite, al then NaN)
      bin = NB - 1;
      u = (uint32_t)(ex2(31.f - a) * 0x1p28f);
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
__device__ __forceinline__ double octave_scale(int bin) {   // 2^-(28 + octave)
  return __longlong_as_double((long long)(1023 - 28 - (bin >> 5)) << 52);
}

template <typename T> struct Elem;
template <> struct Elem<bf16> {
  static constexpr int E = 8;
  static __device__ __forceinline__ void unpack(const uint4 &v, float *x) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ float largest() { return __uint_as_float(0x7f7f0000u); }
};
template <> struct Elem<float> {
  static constexpr int E = 4;
  static __device__ __forceinline__ void unpack(const uint4 &v, float *x) {
    x[0] = __uint_as_float(v.x);
    x[1] = __uint_as_float(v.y);
    x[2] = __uint_as_float(v.z);
    x[3] = __uint_as_float(v.w);
  }
  static __device__ __forceinline__ float largest() { return FLT_MAX; }
};

__device__ __forceinline__ unsigned long long warp_max_key(unsigned long long k) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const unsigned long long other = __shfl_xor_sync(0xffffffffu, k, o);
    k = other > k ? other : k;
  }
  return k;
}

// Exclusive scan over the CTA of a thread's (count, mass); returns the totals.
__device__ void block_scan(Fixed &f, int &c, double &m, int &total_c, double &total_m) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c0 = c;
  const double m0 = m;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int oc = __shfl_up_sync(0xffffffffu, c, o);
    const double om = __shfl_up_sync(0xffffffffu, m, o);
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
  int bc = 0;
  double bm = 0;
  total_c = 0;
  total_m = 0;
  for (int w = 0; w < NT / 32; ++w) {
    if (w == warp) {
      bc = total_c;
      bm = total_m;
    }
    total_c += f.warp_c[w];
    total_m += f.warp_m[w];
  }
  c = bc + c - c0;
  m = bm + (m - m0);
}

struct KernelParams {
  SampleParams p;
  Tables t;
  int per;                       // tokens of a slice
};

template <typename T, bool DRAW>
__global__ void __launch_bounds__(NT) sampling_kernel(const __grid_constant__ KernelParams kp) {
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
  const float temp = p.temperature ? p.temperature[entry] : 1.f;
  const int top_k = p.top_k ? p.top_k[entry] : 0;
  const float top_p = p.top_p ? p.top_p[entry] : 1.f;
  const float min_p = p.min_p ? p.min_p[entry] : 0.f;
  if (!(temp >= 0.f) || isinf(temp) || isnan(top_p) || !(min_p <= 1.f)) {
    if (rank == 0 && tid == 0) raise_error(p.err, DFLASH_DERR_SAMPLING);
    return;   // the whole cluster
  }
  const bool greedy = temp < FLT_MIN;
  cl.barrier_arrive();   // every CTA of the cluster runs before the first remote access

  // ---- the slice, cleaned (NaN to -inf, +inf to the largest finite value), and its maximum
  const int start = min(rank * kp.per, V), n = min(kp.per, V - start);
  const T *src = (const T *)p.logits + (int64_t)row * p.ld + start;
  const int mis = (int)(((uintptr_t)src & 15) / sizeof(T));
  const int nv = n > 0 ? (mis + n + E - 1) / E : 0;
  uint4 *sv = reinterpret_cast<uint4 *>(slice);
  float mx = -INFINITY;
  {
    const uint4 *gv = reinterpret_cast<const uint4 *>(src - mis);
    constexpr int U = 4;
    for (int v0 = tid; v0 < nv; v0 += U * NT) {
      uint4 t[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int v = v0 + u * NT;
        // whole vectors only; the ends come element by element
        if (v < nv && v * E >= mis && (v + 1) * E <= mis + n) t[u] = __ldcs(gv + v);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int v = v0 + u * NT;
        if (v >= nv) break;
        float x[E];
        bool dirty = false;
        if (v * E >= mis && (v + 1) * E <= mis + n) {
          Elem<T>::unpack(t[u], x);
          sv[v] = t[u];
        } else {
#pragma unroll
          for (int e = 0; e < E; ++e) {
            const int i = v * E + e - mis;
            x[e] = i >= 0 && i < n ? to_f32(src[i]) : -INFINITY;
          }
          dirty = true;
        }
#pragma unroll
        for (int e = 0; e < E; ++e) {
          if (!(x[e] <= Elem<T>::largest())) {
            x[e] = isnan(x[e]) ? -INFINITY : Elem<T>::largest();
            dirty = true;
          }
          mx = fmaxf(mx, x[e]);
        }
        if (dirty) {
#pragma unroll
          for (int e = 0; e < E; ++e) slice[v * E + e] = from_f32<T>(x[e]);
        }
      }
    }
  }
  mx = warp_max(mx);
  if (lane == 0) f.fred[warp] = mx;
  __syncthreads();
  mx = f.fred[0];
  for (int w = 1; w < NT / 32; ++w) mx = fmaxf(mx, f.fred[w]);
  cl.barrier_wait();
  if (tid < C) cl.map_shared_rank(&f, tid)->x_max[rank] = mx;
  cl.sync();
  float m = f.x_max[0];
  for (int r = 1; r < C; ++r) m = fmaxf(m, f.x_max[r]);

  float *out = DRAW ? nullptr : p.probs + (int64_t)row * V + start;
  if (m == -INFINITY) {
    if (DRAW) {
      if (rank == 0 && tid == 0) {
        p.ids[row] = -1;
        if (p.prob) p.prob[row] = 0.f;
      }
    } else {
      for (int i = tid; i < n; i += NT) out[i] = 0.f;
    }
    if (rank == 0 && tid == 0) raise_error(p.err, DFLASH_DERR_EMPTY_ROW);
    return;   // the whole cluster, nothing remote in flight
  }

  Weigher weigh;
  weigh.m = m;
  {
    const double c = greedy ? 1.0 : 1.4426950408889634 / (double)temp;
    weigh.c_hi = (float)c;
    weigh.c_lo = (float)(c - (double)weigh.c_hi);
  }
  // every token of the slice: fn(x, id); ids before and past the slice hold -inf
  auto each = [&](auto fn) {
    for (int v = tid; v < nv; v += NT) {
      float x[E];
      Elem<T>::unpack(sv[v], x);
#pragma unroll
      for (int e = 0; e < E; ++e) fn(x[e], start + v * E + e - mis);
    }
  };

  unsigned long long cut = (unsigned long long)order_image(-FLT_MAX) << 32;   // every finite logit
  if (greedy) {
    unsigned long long best = 0;
    each([&](float x, int id) {
      if (x == m) {
        const unsigned long long k = key_of(x, id);
        best = k > best ? k : best;
      }
    });
    best = warp_max_key(best);
    if (lane == 0) f.kred[warp] = best;
    __syncthreads();
    if (tid < C) {
      for (int w = 0; w < NT / 32; ++w) best = f.kred[w] > best ? f.kred[w] : best;
      cl.map_shared_rank(&f, tid)->x_arg[rank] = best;
    }
    cl.sync();
    for (int r = 0; r < C; ++r) cut = f.x_arg[r] > cut ? f.x_arg[r] : cut;
  } else if ((top_k > 0 && top_k < V) || top_p < 1.f) {
    Fixed &lead = *cl.map_shared_rank(&f, 0);
    // Tokens that cannot be in the nucleus whatever the rest is (V of them
    // weigh less than half of 1 - p, and the maximum alone weighs 1) add
    // to the total without the histogram.
    float far = 3.0e38f;
    if (!(top_k > 0 && top_k < V))
      far = log2f((float)V) - log2f(fmaxf(1.f - top_p, 1e-9f)) + 1.f;
    auto is_far = [&](float x) { return __fmul_rn(__fsub_rn(m, x), weigh.c_hi) > far; };
    auto clear = [&] {
      for (int i = tid; i < NB; i += NT) f.cnt[i] = f.lo[i] = f.hi[i] = 0;
      if (tid == 0) f.n_list = 0;
      __syncthreads();
    };
    auto add = [&](int b, uint32_t u) {
      atomicAdd(&f.cnt[b], 1u);
      const uint32_t old = atomicAdd(&f.lo[b], u);
      if (old + u < old) atomicAdd(&f.hi[b], 1u);
    };
    clear();
    float pruned = 0.f;
    each([&](float x, int) {
      if (x == -INFINITY) return;
      if (is_far(x)) {
        pruned += ex2((x - m) * weigh.c_hi);
        return;
      }
      int b;
      uint32_t u;
      weigh(x, tab, b, u);
      add(b, u);
    });
    pruned = warp_sum(pruned);
    if (lane == 0) f.fred[warp] = pruned;
    __syncthreads();
    if (tid == 0) {
      float s = 0.f;
      for (int w = 0; w < NT / 32; ++w) s += f.fred[w];
      f.pruned = s;
    }
    cl.sync();

    // The leader keeps its bins' (tokens, weight) above them; the others follow its commands.
    int n0[PB], above0[PB];
    double above_m0[PB], total_m = 0;
    int stage = 0;               // leader: 0 top-k, 1 top-p
    bool started = false;
    double target = 0;           // leader: weight that the cut's predecessors stay below
    int kth = 0;                 // leader: or the cut's place
    int bin = 0, above = 0;      // leader: the current range and what lies above it
    double above_m = 0;
    unsigned long long lo = 0, hi = 0;
    // bins tid * PB ..: sums over the cluster (scale: of a split bin, else the bin's own)
    auto totals = [&](int *nn, double *mm, double scale) {
      for (int i = 0; i < PB; ++i) {
        const int b = tid * PB + i;
        nn[i] = 0;
        unsigned long long s = 0;
        for (int r = 0; r < C; ++r) {
          const Fixed &o = *cl.map_shared_rank(&f, r);
          nn[i] += (int)o.cnt[b];
          s += ((unsigned long long)o.hi[b] << 32) + o.lo[b];
        }
        mm[i] = (double)s * (scale > 0 ? scale : octave_scale(b));
      }
    };
    auto scan = [&](const int *nn, const double *mm, int *ab, double *abm, int &tc, double &tm) {
      int c = 0;
      double w = 0;
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
    auto select = [&](const int *nn, const int *ab, const double *abm, int base, double base_m) {
      if (tid == 0) f.sel_bin = -1;
      __syncthreads();
      int mine = -1;
      for (int i = 0; i < PB; ++i)
        if (nn[i] > 0 && (stage == 0 ? base + ab[i] < kth : base_m + abm[i] < target)) mine = tid * PB + i;
      if (mine >= 0) atomicMax(&f.sel_bin, mine);
      __syncthreads();
      const int s = f.sel_bin;
      if (s >= 0 && s / PB == tid) {
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
      tell(count <= CAP ? CMD_GATHER : CMD_SPLIT, sh);
    };
    // start of a stage: the first histogram's bin, and its range of keys
    auto begin = [&] {
      const int s = select(n0, above0, above_m0, 0, 0);
      bin = s;
      const double inv = (double)temp * 0.6931471805599453 / 32.0;
      const double x_hi = (double)m - fmax(0.0, (bin - 0.51) * inv);
      const double x_lo = bin == NB - 1 ? -(double)FLT_MAX : (double)m - (bin + 0.51) * inv;
      lo = (unsigned long long)order_image(__double2float_rd(fmax(x_lo, -(double)FLT_MAX))) << 32;
      hi = ((unsigned long long)order_image(__double2float_ru(fmax(x_hi, -(double)FLT_MAX))) + 1) << 32;
      tell_range(f.sel_n);
    };
    for (int guard = 0;; ++guard) {
      if (rank == 0) {
        if (!started) {
          started = true;
          double mm[PB];
          int total;
          totals(n0, mm, 0);
          scan(n0, mm, above0, above_m0, total, total_m);
          for (int r = 0; r < C; ++r) total_m += (double)cl.map_shared_rank(&f, r)->pruned;
          stage = top_k > 0 && top_k < total ? 0 : 1;
          kth = top_k;
          target = fmax((double)top_p * total_m, 1e-300);
          if (stage == 1 && !(top_p < 1.f)) tell(CMD_DONE, 0);
          else begin();
        } else if (f.cmd == CMD_SPLIT) {
          int nn[PB], ab[PB], tc;
          double mm[PB], abm[PB], tm;
          totals(nn, mm, octave_scale(bin));
          scan(nn, mm, ab, abm, tc, tm);
          const int s = select(nn, ab, abm, above, above_m);
          const int sh = f.sh;
          const unsigned long long v = (unsigned long long)(NB - 1 - s);
          const unsigned long long l = lo + (v << sh), h = l + (1ull << sh);
          lo = l;
          hi = h < hi ? h : hi;
          __syncthreads();   // sh has been read
          tell_range(f.sel_n);
        } else {
          // the gathered tokens: sort, then walk to the cut
          const int cnt = min(f.n_list, CAP);
          int size = 2;
          while (size < cnt) size <<= 1;
          for (int i = cnt + tid; i < size; i += NT) f.list[i] = 0;
          __syncthreads();
          for (int k = 2; k <= size; k <<= 1)
            for (int j = k >> 1; j > 0; j >>= 1) {
              for (int i = tid; i < size / 2; i += NT) {
                const int a = 2 * i - (i & (j - 1)), b = a + j;   // pair (a, a + j)
                const unsigned long long x = f.list[a], y = f.list[b];
                const bool down = (a & k) == 0;
                if ((x < y) == down) {
                  f.list[a] = y;
                  f.list[b] = x;
                }
              }
              __syncthreads();
            }
          int nn[2], ab[2], tc;
          double mm[2], abm[2], tm;
          static_assert(CAP == 2 * NT && PB == 2, "two tokens and two bins a thread");
          for (int i = 0; i < 2; ++i) {
            const int at = 2 * tid + i;
            nn[i] = at < cnt ? 1 : 0;
            mm[i] = 0;
            if (at < cnt) {
              int b;
              uint32_t u;
              weigh(order_value((uint32_t)(f.list[at] >> 32)), tab, b, u);
              mm[i] = (double)u * octave_scale(bin);
            }
          }
          scan(nn, mm, ab, abm, tc, tm);
          const int s = select(nn, ab, abm, above, above_m);   // the cut's place in the list
          cut = f.list[s];
          if (s / 2 == tid) f.sel_through = above_m + mm[s % 2];   // weight through the cut
          __syncthreads();
          if (stage == 0 && top_p < 1.f) {
            stage = 1;
            target = fmax((double)top_p * f.sel_through, 1e-300);
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
      const unsigned long long r_lo = f.range_lo, r_hi = f.range_hi;
      if (guard > 24) {   // 64-bit keys end long before
        if (rank == 0 && tid == 0) raise_error(p.err, DFLASH_DERR_TIMEOUT);
        break;
      }
      clear();
      if (cmd == CMD_GATHER) cl.sync();   // the leader's list is empty before anyone adds to it
      each([&](float x, int id) {
        const unsigned long long k = key_of(x, id);
        if (k < r_lo || k >= r_hi || is_far(x)) return;
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
    cut = f.cut;
  }
  if (!greedy && min_p > 0.f) {
    const double x = (double)m + (double)temp * log((double)min_p);
    const unsigned long long k =
        (unsigned long long)order_image(__double2float_ru(fmax(x, -(double)FLT_MAX))) << 32;
    cut = k > cut ? k : cut;
  }

  // ---- the kept tokens' sum (and the race)
  const float xc = order_value((uint32_t)(cut >> 32));
  const uint32_t idc = ~(uint32_t)cut;
  auto kept = [&](float x, int id) { return x > xc || (x == xc && (uint32_t)id <= idc); };
  float s0 = 0.f, s1 = 0.f;
  unsigned long long best = 0;
  const float *noise = DRAW ? p.noise + (int64_t)row * V : nullptr;
  each([&](float x, int id) {
    if (!kept(x, id)) return;
    const float w = ex2((x - m) * weigh.c_hi);
    if (id & 1) s1 += w;
    else s0 += w;
    if (DRAW) {
      const unsigned long long k = argmax_key(w / noise[id], id);
      best = k > best ? k : best;
    }
  });
  const float sum = warp_sum(s0 + s1);
  if (DRAW) best = warp_max_key(best);
  __syncthreads();
  if (lane == 0) {
    f.fred[warp] = sum;
    if (DRAW) f.kred[warp] = best;
  }
  __syncthreads();
  if (tid < C) {
    double s = 0;
    for (int w = 0; w < NT / 32; ++w) s += (double)f.fred[w];
    Fixed &o = *cl.map_shared_rank(&f, tid);
    o.x_sum[rank] = s;
    if (DRAW) {
      for (int w = 0; w < NT / 32; ++w) best = f.kred[w] > best ? f.kred[w] : best;
      o.x_race[rank] = best;
    }
  }
  cl.sync();   // the last exchange: nothing remote after it
  double total = 0;
  for (int r = 0; r < C; ++r) total += f.x_sum[r];
  const float inv = (float)(1.0 / total);
  if (DRAW) {
    if (rank == 0 && tid == 0) {
      for (int r = 0; r < C; ++r) best = f.x_race[r] > best ? f.x_race[r] : best;
      const int id = argmax_key_index(best);
      p.ids[row] = id;
      if (p.prob) {
        float x = to_f32(((const T *)p.logits)[(int64_t)row * p.ld + id]);
        x = fminf(x, Elem<T>::largest());
        p.prob[row] = ex2((x - m) * weigh.c_hi) * inv;
      }
    }
    return;
  }
  // ---- probabilities: 16-byte stores from the row's first aligned element
  auto prob_at = [&](int i) {
    const float x = to_f32(slice[mis + i]);
    return kept(x, start + i) ? ex2((x - m) * weigh.c_hi) * inv : 0.f;
  };
  const int head = min(n, (int)((16 - ((uintptr_t)out & 15)) & 15) / 4);
  const int quads = (n - head) / 4;
  if (tid < head) out[tid] = prob_at(tid);
  for (int q = tid; q < quads; q += NT) {
    const int i = head + 4 * q;
    *reinterpret_cast<float4 *>(out + i) =
        make_float4(prob_at(i), prob_at(i + 1), prob_at(i + 2), prob_at(i + 3));
  }
  const int done = head + 4 * quads;
  if (tid < n - done) out[done + tid] = prob_at(done + tid);
}

size_t smem_bytes(int per, int es) {
  return (sizeof(Fixed) + 15) / 16 * 16 + (size_t)per * es + 32;
}
int slice_of(int vocab, int C) { return ((vocab + C - 1) / C + 15) / 16 * 16; }

template <typename T, bool DRAW> cudaError_t launch(const SampleParams &p, cudaStream_t s) {
  const int es = sizeof(T);
  int dev = 0, sms = 0;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  // the fewest CTAs whose slices leave room for two of them on an SM; more
  // while rows are too few to fill the GPU and a slice stays worth a CTA
  int C = 1;
  while (C < MAXC && smem_bytes(slice_of(p.vocab, C), es) > 108 * 1024) C *= 2;
  while (C < MAXC && (int64_t)p.rows * C * 2 <= sms && slice_of(p.vocab, C) > 4096) C *= 2;
  KernelParams kp;
  kp.p = p;
  kp.per = slice_of(p.vocab, C);
  for (int i = 0; i < 32; ++i) {
    const double w = std::exp2(28.0 - i / 32.0);
    kp.t.u[i] = (uint32_t)std::llround(w);
    kp.t.f[i] = (float)w;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.rows * C));
  cfg.blockDim = dim3(NT);
  cfg.dynamicSmemBytes = smem_bytes(kp.per, es);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = C;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, sampling_kernel<T, DRAW>, kp);
}

template <typename T, bool DRAW> cudaError_t prepare() {
  return cudaFuncSetAttribute(sampling_kernel<T, DRAW>, cudaFuncAttributeMaxDynamicSharedMemorySize,
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

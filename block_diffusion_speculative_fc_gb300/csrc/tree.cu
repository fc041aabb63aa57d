// Trees of drafted tokens: positions and ancestor masks from the parents, and the
// walk along the target's tokens.  A CTA a request; both are a few passes over at
// most 1024 rows in shared memory, so that launch and load latency bound them:
// one request of 64 rows 3 us either (GPU time; a call through the session 7 and 10
// us of host time), 128 requests of 17 to 250 rows 8 and 4 us.
#include "common.cuh"
#include "target_ops.h"

namespace dflash {
namespace {

// First row and number of rows of request b; false: no range of rows (flagged).
__device__ __forceinline__ bool tree_range(const int *row_start, int b, int total_rows, int most,
                                           unsigned int *err, int &start, int &n) {
  start = row_start[b];
  const int end = row_start[b + 1];
  n = end - start;
  if (start < 0 || start > end || end > total_rows) {
    if (threadIdx.x == 0) raise_error(err, DFLASH_DERR_ROW_RANGE);
    return false;
  }
  if (n > most) {
    if (threadIdx.x == 0) raise_error(err, DFLASH_DERR_TREE);
    return false;
  }
  return n > 0;
}

// ancestors(i) = {i} + ancestors(parent(i)), by pointer doubling: after k steps a
// row's mask holds its first 2^k ancestors and its pointer names the one 2^k
// above, so that a chain of 1024 rows takes 10 steps and a tree of depth 14
// four.  A mask is read while its own row may be adding to it: whatever is seen
// of it are ancestors, and those of the step before are all there.  The depth is
// the number of bits less one.
__global__ void __launch_bounds__(1024) tree_plan_kernel(const __grid_constant__ TreePlanParams p) {
  extern __shared__ uint32_t s_mask[];          // [n][W]
  __shared__ int s_up[2][1024];
  pdl_wait();
  const int b = blockIdx.x, tid = threadIdx.x, nt = blockDim.x, W = p.mask_words;
  int start, n;
  if (!tree_range(p.row_start, b, p.total_rows, 32 * W, p.err, start, n)) return;
  bool bad = false;
  for (int i = tid; i < n; i += nt) {
    const int up = p.parent[start + i];
    bad = bad || up < -1 || up >= i;
    s_up[0][i] = up;
  }
  for (int e = tid; e < n * W; e += nt) {
    const int i = e / W, w = e % W;
    s_mask[e] = i >> 5 == w ? 1u << (i & 31) : 0u;
  }
  const int root = p.root_pos[b];
  if (__syncthreads_or(bad)) {
    if (tid == 0) raise_error(p.err, DFLASH_DERR_TREE);
    return;
  }
  for (int cur = 0;; cur ^= 1) {
    bool more = false;
    for (int e = tid; e < n * W; e += nt) {
      const int i = e / W, w = e % W, up = s_up[cur][i];
      if (up >= 0) s_mask[e] |= *reinterpret_cast<volatile uint32_t *>(s_mask + up * W + w);
      if (w == 0) {
        const int next = up >= 0 ? s_up[cur][up] : -1;
        s_up[cur ^ 1][i] = next;
        more = more || next >= 0;
      }
    }
    if (!__syncthreads_or(more)) break;
  }
  for (int e = tid; e < n * W; e += nt) p.mask[(int64_t)start * W + e] = s_mask[e];
  if (p.positions)
    for (int i = tid; i < n; i += nt) {
      int bits = 0;
      for (int w = 0; w < W; ++w) bits += __popc(s_mask[i * W + w]);
      p.positions[start + i] = root + bits - 1;
    }
}

// A child stands behind its parent, so a step of the walk looks on from the row it
// stands on: all steps together pass over the rows once.  The first warp walks,
// 32 rows a look.
__global__ void __launch_bounds__(128) accept_tree_kernel(const __grid_constant__ AcceptTreeParams p) {
  __shared__ int s_parent[kMaxTreeRows], s_token[kMaxTreeRows], s_post[kMaxTreeRows];
  __shared__ int s_path[kMaxTreeRows], s_len, s_ok;
  pdl_wait();
  const int b = blockIdx.x, tid = threadIdx.x, nt = blockDim.x, lane = tid & 31;
  int start, n;
  if (!tree_range(p.row_start, b, p.total_rows, kMaxTreeRows, p.err, start, n)) return;
  bool bad = false;
  for (int i = tid; i < n; i += nt) {
    const int up = p.parent[start + i];
    bad = bad || up < -1 || up >= i;
    s_parent[i] = up;
    s_token[i] = p.tokens[start + i];
    s_post[i] = p.posterior[start + i];
  }
  const int at = p.seq_len[b];
  if (__syncthreads_or(bad)) {
    if (tid == 0) raise_error(p.err, DFLASH_DERR_TREE);
    return;
  }
  if (tid < 32) {
    int cur = 0, len = 1;
    if (lane == 0) s_path[0] = 0;
    while (len < p.max_path) {
      const int want = s_post[cur];
      int next = -1;
      for (int i0 = cur + 1; i0 < n && next < 0; i0 += 32) {
        const int i = i0 + lane;
        const unsigned hit = __ballot_sync(0xffffffffu, i < n && s_parent[i] == cur && s_token[i] == want);
        if (hit) next = i0 + __ffs(hit) - 1;
      }
      if (next < 0) break;
      cur = next;
      if (lane == 0) s_path[len] = cur;
      ++len;
    }
    __syncwarp();
    const int bonus = s_post[cur];
    bool bad_id = bonus < 0 || bonus >= p.vocab;
    for (int k = lane; k < len; k += 32) {
      const int id = s_token[s_path[k]];
      bad_id = bad_id || id < 0 || id >= p.vocab;
    }
    bad_id = __any_sync(0xffffffffu, bad_id) != 0;
    const bool over = p.output_ids && (at < 0 || (int64_t)at + len >= p.out_stride);
    if (lane == 0) {
      if (bad_id) raise_error(p.err, DFLASH_DERR_TOKEN_RANGE);
      else if (over) raise_error(p.err, DFLASH_DERR_OUTPUT_ROW);
      s_len = len;
      s_ok = !bad_id && !over;
      if (s_ok) {
        p.accept_len[b] = len - 1;
        p.commit_len[b] = len;
        p.bonus[b] = bonus;
        p.seq_len[b] = at + len;
      }
    }
  }
  __syncthreads();
  if (!s_ok) return;
  const int len = s_len, bonus = s_post[s_path[len - 1]];
  for (int k = tid; k < p.max_path; k += nt) {
    p.path[(int64_t)b * p.max_path + k] = k < len ? s_path[k] : -1;
    p.out_tokens[(int64_t)b * p.max_path + k] = k + 1 < len ? s_token[s_path[k + 1]] : k + 1 == len ? bonus : 0;
  }
  if (p.output_ids)
    for (int k = tid; k <= len; k += nt)
      p.output_ids[(int64_t)b * p.out_stride + at + k] = k < len ? s_token[s_path[k]] : bonus;
  if (p.row_weight) {
    // (a row is on the path where the path's first row at or behind it is the row itself)
    for (int i = tid; i < n; i += nt) {
      int lo = 0, hi = len;
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (s_path[mid] < i) lo = mid + 1;
        else hi = mid;
      }
      p.row_weight[start + i] = lo < len && s_path[lo] == i ? 1.f : 0.f;
    }
  }
}

size_t plan_smem(int words) { return (size_t)32 * words * words * 4; }

}  // namespace

cudaError_t launch_tree_plan(const TreePlanParams &p, cudaStream_t s) {
  // a thread a word of a mask, in the largest tree that the masks have room for
  const int nt = std::max(64, std::min(1024, 32 * p.mask_words * p.mask_words));
  return launch_pdl(tree_plan_kernel, dim3(p.B), dim3(nt), plan_smem(p.mask_words), s, p);
}

cudaError_t launch_accept_tree(const AcceptTreeParams &p, cudaStream_t s) {
  return launch_pdl(accept_tree_kernel, dim3(p.B), dim3(128), 0, s, p);
}

cudaError_t prepare_tree() {
  return cudaFuncSetAttribute(tree_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              (int)plan_smem(kMaxTreeRows / 32));
}

}  // namespace dflash

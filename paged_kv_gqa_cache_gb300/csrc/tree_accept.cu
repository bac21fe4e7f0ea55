// The drafted tokens that the model's own choices confirm, and the cache
// compacted to them, for sm_103a.
//
// Sequence s has n drafted tokens at cache positions L - n .. L - 1, a tree by
// parents.  Token i is accepted when its parent is accepted and draft[i] equals
// target[parent], what the model chose after the parent; one without parent when it
// equals the choice after the committed context, or always where that is not given.
// Of the accepted tokens the deepest (of these the lowest index) ends the path; the
// path's rows move, in every layer and in place, to positions L - n ..: row L - n +
// path[i] to row L - n + i, so that the cache is a line again.
//
// One launch: every CTA of a sequence finds the path itself (a few hundred bytes
// from L2; waiting for one that does would cost another launch) and moves it in
// its share of the layers.  The path by pointer doubling: after r rounds a token
// knows its depth and acceptance over 2^r ancestors, so log2(depth) rounds of two
// barriers do.  path[i] >= i and ascending, so a thread that moves one 16-byte
// column of all rows, in order, never reads a row that it has overwritten: no
// barrier, no second buffer.
// Bound by a chain of round trips (lengths, drafts, block ids, rows) where little
// moves, by bytes where much does (8 rows of 16 bytes in flight per thread).  36 layers
// of 8 heads, bf16: 32 sequences of 16 to 32 drafts 7.4 us (the bytes' own 4.5), 192 of
// 33 to 64 26.6 us (22.6, 0.85 of the copy rate); one of 5 drafts, 28 layers: 2.6 us.
#include "pa_device.cuh"

namespace pa {
namespace {

constexpr int kAcceptThreads = PA_MAX_TREE_LEN;  // a thread per token
constexpr int kMoveRows = 8;                     // rows in flight per thread
constexpr unsigned FULL = 0xffffffffu;
static_assert(kAcceptThreads == 256, "8 warps");

__device__ __forceinline__ int64_t block_sum(int64_t x, int64_t *part) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(FULL, x, off);
  if (lane == 0) part[warp] = x;
  __syncthreads();
  int64_t sum = 0;
#pragma unroll
  for (int i = 0; i < kAcceptThreads / 32; ++i) sum += part[i];
  return sum;
}

// GREEDY: the paths are found, else they are given.
template <bool GREEDY>
__global__ void __launch_bounds__(kAcceptThreads)
tree_accept_kernel(const __grid_constant__ TreeAcceptParams p, int layers_per_cta) {
  __shared__ int64_t s_tgt[kAcceptThreads], s_src[kAcceptThreads], s_dst[kAcceptThreads];
  __shared__ int32_t s_par[kAcceptThreads], s_hop[kAcceptThreads], s_dep[kAcceptThreads], s_path[kAcceptThreads];
  __shared__ int64_t s_part[kAcceptThreads / 32];
  __shared__ int32_t s_best[kAcceptThreads / 32];
  const int i = threadIdx.x, lane = i & 31, warp = i >> 5, s = blockIdx.x;
  const bool scribe = p.first && blockIdx.y == 0;  // writes the outputs and reports
  griddep_wait();  // (drafts, choices and lengths may be the previous kernels' outputs)
  const int n = __ldg(p.tree_lens + s), L = __ldg(p.context_lens + s);
  const int start = (int)((unsigned)L - (unsigned)n);  // (used where the lengths are good)
  bool ok = n >= 0 && n <= kAcceptThreads && (!GREEDY || n <= p.path_stride) &&
            (n == 0 || (L >= n && (!p.block_tables || L <= (int64_t)p.max_blocks_per_seq * kBlock)));
  int dep = 0;          // the path's length
  int64_t next = -1;
  if constexpr (GREEDY) {
    const bool judged = p.context_targets != nullptr;  // (the tokens without parent, that is)
    const int64_t choice = judged ? __ldg(p.context_targets + s) : -1;
    int64_t before = 0;  // rows of the sequences in front
    for (int j = i; j < s; j += kAcceptThreads) before += max(__ldg(p.tree_lens + j), 0);
    const int64_t row0 = block_sum(before, s_part);
    ok = ok && row0 + n <= p.num_tokens;
    int par = -1;
    int64_t draft = 0;
    if (ok && i < n) {
      par = __ldg(p.parents + row0 + i);
      draft = __ldg(p.draft + row0 + i);
      s_tgt[i] = __ldg(p.target + row0 + i);
      s_par[i] = par;
    }
    ok = !__syncthreads_or(!ok || (i < n && (par < -1 || par >= i)));
    // hop: the ancestor reached, -1 above a root, -2 not accepted; depth: tokens from here to it
    int hop = -2, depth = 1;
    if (ok && i < n && (par < 0 ? !judged || draft == choice : draft == s_tgt[par])) hop = par;
    while (true) {
      s_hop[i] = hop;
      s_dep[i] = depth;
      if (!__syncthreads_or(hop >= 0)) break;
      if (hop >= 0) {
        depth += s_dep[hop];
        hop = s_hop[hop];
      }
      __syncthreads();
    }
    const int mine = hop == -1 ? depth << 16 | (kAcceptThreads - 1 - i) : 0;
    const int top = __reduce_max_sync(FULL, mine);
    if (lane == 0) s_best[warp] = top;
    __syncthreads();
    int best = 0;
#pragma unroll
    for (int w = 0; w < kAcceptThreads / 32; ++w) best = max(best, s_best[w]);
    dep = best >> 16;
    const int node = kAcceptThreads - 1 - (best & 0xffff);
    if (ok) next = choice;  // (nothing accepted)
    if (dep > 0) {
      next = s_tgt[node];
      if (i == 0)
        for (int k = dep - 1, a = node; k >= 0; --k, a = s_par[a]) s_path[k] = a;
    }
    __syncthreads();
    if (scribe) {
      for (int k = i; k < p.path_stride; k += kAcceptThreads)
        p.path[(int64_t)s * p.path_stride + k] = k < dep ? s_path[k] : -1;
      if (i == 0) {
        p.path_lens[s] = dep;
        p.next_tokens[s] = next;
      }
    }
  } else {
    dep = __ldg(p.path_lens + s);
    ok = ok && dep >= 0 && dep <= n && dep <= p.path_stride;
    const int32_t *path = p.path + (int64_t)s * p.path_stride;
    int a = 0, front = -1;
    if (ok && i < dep) {
      a = __ldg(path + i);
      if (i > 0) front = __ldg(path + i - 1);
      s_path[i] = a;
    }
    ok = !__syncthreads_or(!ok || (i < dep && (a <= front || a >= n)));
    if (!ok) dep = 0;
  }
  if (scribe && i == 0) {
    // An attention call enqueued next reads the lengths before its dependency wait, so this
    // kernel never releases its dependents early and makes them visible before it ends.
    p.new_lens[s] = ok ? start + dep : -1;
    __threadfence();
    if (!ok) set_error(p.err, PA_ERR_RANGE, s);
  }
  if (p.num_layers == 0) return;
  // where the path's tokens lie and where they go (-1: they stay, or cannot be reached)
  bool stays = false;
  if (i < dep) {
    const int from = start + s_path[i], to = start + i;
    const int32_t *bt = p.block_tables + (int64_t)s * p.max_blocks_per_seq;
    stays = from == to;
    int64_t src = -1, dst = -1;
    if (!stays) {
      const int a = __ldg(bt + from / kBlock), b = __ldg(bt + to / kBlock);
      if ((unsigned)a < (unsigned)p.num_blocks && (unsigned)b < (unsigned)p.num_blocks) {
        src = (int64_t)a * kBlock + from % kBlock;
        dst = (int64_t)b * kBlock + to % kBlock;
      } else if (scribe) {
        set_error(p.err, PA_ERR_RANGE, s);
      }
    }
    s_src[i] = src;
    s_dst[i] = dst;
  }
  const int k0 = __syncthreads_count(stays);  // the tokens that stay come first
  if (k0 >= dep) return;
  const int l0 = blockIdx.y * layers_per_cta, l1 = min(l0 + layers_per_cta, p.num_layers);
  const int cols = 2 * p.row_vecs;
  for (int x = i; x < (l1 - l0) * cols; x += kAcceptThreads) {
    const int l = l0 + x / cols, c = x % cols;
    uint4 *base = static_cast<uint4 *>(c < p.row_vecs ? p.k[l] : p.v[l]) + (c < p.row_vecs ? c : c - p.row_vecs);
    for (int k = k0; k < dep; k += kMoveRows) {
      uint4 r[kMoveRows];
#pragma unroll
      for (int u = 0; u < kMoveRows; ++u)
        if (k + u < dep && s_src[k + u] >= 0) r[u] = base[s_src[k + u] * p.row_vecs];
#pragma unroll
      for (int u = 0; u < kMoveRows; ++u)
        if (k + u < dep && s_src[k + u] >= 0) st_v4(base + s_dst[k + u] * p.row_vecs, r[u]);
    }
  }
}

}  // namespace

cudaError_t launch_tree_accept(const TreeAcceptParams &p, int sms, cudaStream_t stream) {
  // CTAs for the whole GPU (8 on an SM), each with work for all of its threads
  const int per_seq = 8 * sms / p.num_seqs > 0 ? 8 * sms / p.num_seqs : 1;
  int layers = (p.num_layers + per_seq - 1) / per_seq;
  const int least = (kAcceptThreads + 2 * p.row_vecs - 1) / (2 * p.row_vecs);
  if (layers < least) layers = least;
  const dim3 grid(p.num_seqs, p.num_layers > 0 ? (p.num_layers + layers - 1) / layers : 1);
  return p.next_tokens ? launch_pdl(tree_accept_kernel<true>, grid, dim3(kAcceptThreads), 0, stream, p, layers)
                       : launch_pdl(tree_accept_kernel<false>, grid, dim3(kAcceptThreads), 0, stream, p, layers);
}

}  // namespace pa

// Eviction from the paged cache by accumulated attention weight, for sm_103a.
//
// For each sequence s and KV head h, of the ctx cached tokens
//   ctx <= budget:  all stay;
//   else:           the first `sinks`, the last `recent` and, of those between,
//                   the budget - sinks - recent of largest weight (ties: the
//                   lower index first) stay.
// The tokens that stay keep their order and move to positions 0 .. n - 1 of
// the destination block table, with their weights.  Each KV head keeps tokens
// of its own: a row of a page belongs to one head, and keys are rotated before
// they are stored, so a head's rows may move without the other heads'.
//
// One cluster of C CTAs per (sequence, KV head):
//   select   radix selection of the threshold weight over order-preserving
//            32-bit keys, 8 bits per pass: each CTA counts its slice of the
//            tokens into a histogram with one column per lane (column = bank:
//            no two lanes of a warp ever meet in a bank or on an address,
//            however few values the weights take), the CTAs add their counts
//            through the cluster, and every warp finds the digit by the same
//            scan.  A digit whose tokens all stay ends the selection.  The
//            slice's keys stay in shared memory where they fit.
//   rank     a kept token's new position = the kept tokens before it: each
//            warp counts its part of the slice, one scan over the warps and the
//            lower ranks' counts through the cluster, then ballots.
//   move     each half-warp takes every (32 C)-th new position, three rows at a
//            time through shared memory (cp.async), the next three on their way
//            meanwhile.  A token never moves up, so the sources of a group of
//            rows lie at or above its destinations: in place (a destination
//            table that repeats the source table, or weights_out = weights) a
//            cluster barrier between the reads and the writes of each group is
//            all the order it takes; apart, no barrier at all.
// HBM-bound: 4 bytes per token, then 512 read and 512 written per kept row.
#include "pa_device.cuh"

namespace pa {
namespace {

constexpr unsigned FULL = 0xffffffffu;
constexpr int kEvThreads = 512;
constexpr int kEvWarps = kEvThreads / 32;
constexpr int kEvHalfWarps = kEvThreads / 16;
constexpr int kEvKeys = 16384;       // keys of a CTA's slice held in shared memory (64 KB)
constexpr int kEvBins = 256;         // 8 bits per pass
constexpr int kEvRows = 3;           // rows per half-warp and group; two groups in shared memory

struct EvSmem {
  union {
    struct {
      uint32_t keys[kEvKeys];
      uint32_t hist[kEvBins * 32];     // [bin][lane]
    } sel;
    uint4 rows[2][kEvRows][kEvHalfWarps][2][16];  // the move: [group parity][row][half-warp][K, V][16 x 16 bytes]
  };
  uint32_t local[2][kEvBins];          // this CTA's counts, by pass parity
  uint32_t total[kEvBins];             // the cluster's
  uint32_t sure[kEvWarps], tie[kEvWarps];
  uint32_t counts[2];                  // sure, then tied tokens of the slice
};

// Order-preserving key of a weight (NaN below every number); -0 and +0 compare equal.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w == 0.f ? 0.f : w);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

__global__ void __launch_bounds__(kEvThreads, 2) kv_evict_kernel(const EvictParams p) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  EvSmem &sm = *reinterpret_cast<EvSmem *>(smem_raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int C = (int)cluster_nctarank(), rank = (int)cluster_ctarank();
  auto sync_all = [&] {  // every thread of the cluster
    if (C > 1) cluster_sync(); else __syncthreads();
  };
  const int item = blockIdx.x / C;
  const int hkv = p.num_kv_heads;
  const int s = item / hkv, h = item % hkv;
  griddep_wait();  // weights, lengths, tables and pool may come from the previous kernel
  const int ctx = __ldg(p.context_lens + s);
  const int n = min(ctx, p.budget);  // tokens that stay
  if (ctx < 1 || (int64_t)ctx > (int64_t)p.max_blocks_per_seq * kBlock || ctx > p.weights_stride ||
      (int64_t)n > (int64_t)p.dst_max_blocks * kBlock || n > p.out_stride) {  // uniform over the cluster
    if (h == 0 && rank == 0 && tid == 0) set_error(p.err, PA_ERR_RANGE, s);
    return;
  }
  const float *w = p.weights + ((int64_t)s * hkv + h) * p.weights_stride;
  float *w_out = p.weights_out + ((int64_t)s * hkv + h) * p.out_stride;
  int32_t *kept = p.kept + ((int64_t)s * hkv + h) * p.budget;
  const int32_t *bt = p.block_tables + (int64_t)s * p.max_blocks_per_seq;
  const int32_t *dt = p.dst_block_tables + (int64_t)s * p.dst_max_blocks;
  // In place if a destination page is the source page of the same index.
  bool same = p.weights_out == p.weights;
  for (int i = tid; i < (n + kBlock - 1) / kBlock; i += kEvThreads) same = same || __ldg(bt + i) == __ldg(dt + i);
  const bool ordered = __syncthreads_or(same) != 0;  // (the same in every CTA of the cluster)

  if (ctx > p.budget) {
    // ---- select ----
    const int lo_mid = p.sinks, hi_mid = ctx - p.recent;  // the tokens that compete (more than need of them)
    const uint32_t need = (uint32_t)(p.budget - p.sinks - p.recent);
    const int per = ((ctx + C - 1) / C + 31) & ~31;
    const int s0 = min(ctx, rank * per), s1 = min(ctx, s0 + per);  // this CTA's slice
    for (int i = tid; i < min(s1 - s0, kEvKeys); i += kEvThreads) sm.sel.keys[i] = weight_key(w[s0 + i]);
    auto key_at = [&](int i) { return i - s0 < kEvKeys ? sm.sel.keys[i - s0] : weight_key(w[i]); };
    uint32_t prefix = 0, left = need;  // digits found so far; tokens still wanted at them
    int shift = 32;                    // the digits' place: a key's are key >> shift
    for (int pass = 0; pass < 4 && need > 0; ++pass) {
      for (int i = tid; i < kEvBins * 32; i += kEvThreads) sm.sel.hist[i] = 0;
      __syncthreads();  // (the keys too are there)
      const int a = max(s0, lo_mid), b = min(s1, hi_mid);
      for (int i = a + tid; i < b; i += kEvThreads) {
        const uint32_t key = key_at(i);
        if (pass == 0 || (key >> shift) == prefix)
          atomicAdd(&sm.sel.hist[((key >> (shift - 8)) & (kEvBins - 1)) * 32 + lane], 1u);
      }
      __syncthreads();
      {  // two threads per digit
        uint32_t sum = 0;
        const int bin = tid >> 1, half = (tid & 1) * 16;
#pragma unroll
        for (int j = 0; j < 16; ++j) sum += sm.sel.hist[bin * 32 + half + ((j + (lane >> 1)) & 15)];
        sum += __shfl_xor_sync(FULL, sum, 1);
        if ((tid & 1) == 0) (C > 1 ? sm.local[pass & 1] : sm.total)[bin] = sum;
      }
      static_assert(kEvThreads == 2 * kEvBins, "two threads per digit");
      if (C > 1) {
        cluster_sync();
        if (tid < kEvBins) {
          uint32_t sum = 0;
          for (int r = 0; r < C; ++r) sum += ld_cluster_u32(map_to_rank(&sm.local[pass & 1][tid], r));
          sm.total[tid] = sum;
        }
      }
      __syncthreads();
      // every warp scans the digits from the heaviest down: lane l has digits 255 - 8 l .. 248 - 8 l
      uint32_t c[8], mine = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        c[j] = sm.total[kEvBins - 1 - 8 * lane - j];
        mine += c[j];
      }
      uint32_t incl = mine;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const uint32_t y = __shfl_up_sync(FULL, incl, off);
        if (lane >= off) incl += y;
      }
      uint32_t above = incl - mine;                      // tokens at digits before this lane's
      const int owner = __ffs(__ballot_sync(FULL, incl >= left)) - 1;  // exists: at least `left` tokens are counted
      uint32_t digit = 0, count = 0;
      bool found = false;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (!found) {
          if (above + c[j] >= left) {
            found = true;
            digit = kEvBins - 1 - 8 * lane - j;
            count = c[j];
          } else {
            above += c[j];
          }
        }
      digit = __shfl_sync(FULL, digit, owner);
      count = __shfl_sync(FULL, count, owner);
      left -= __shfl_sync(FULL, above, owner);
      prefix = (prefix << 8) | digit;
      shift -= 8;
      if (count == left) break;  // (uniform over the cluster) every token at these digits stays
      __syncthreads();           // the histogram and the totals are read before they are written again
    }
    // stay: the tokens outside the middle, those with larger digits, and the first `left` with equal ones
    const bool none = need == 0;
    auto kind = [&](int i, bool &is_sure, bool &is_tie) {
      const bool mid = i >= lo_mid && i < hi_mid;
      const uint32_t k = mid && !none ? key_at(i) >> shift : 0u;
      is_sure = i < s1 && (!mid || (!none && k > prefix));
      is_tie = i < s1 && mid && !none && k == prefix;
    };
    // ---- rank ----
    const int wper = (((s1 - s0) + kEvWarps - 1) / kEvWarps + 31) & ~31;
    const int w0 = s0 + warp * wper, w1 = min(s1, w0 + wper);  // this warp's part, 32 tokens per step
    uint32_t n_sure = 0, n_tie = 0;
    for (int i = w0; i < w1; i += 32) {
      bool a, b;
      kind(i + lane, a, b);
      n_sure += __popc(__ballot_sync(FULL, a));
      n_tie += __popc(__ballot_sync(FULL, b));
    }
    if (lane == 0) {
      sm.sure[warp] = n_sure;
      sm.tie[warp] = n_tie;
    }
    __syncthreads();
    uint32_t sure = 0, tie = 0, all_sure = 0, all_tie = 0;
#pragma unroll
    for (int i = 0; i < kEvWarps; ++i) {
      sure += i < warp ? sm.sure[i] : 0u;
      tie += i < warp ? sm.tie[i] : 0u;
      all_sure += sm.sure[i];
      all_tie += sm.tie[i];
    }
    if (C > 1) {
      if (tid == 0) {
        sm.counts[0] = all_sure;
        sm.counts[1] = all_tie;
      }
      cluster_sync();
      for (int r = 0; r < rank; ++r) {
        sure += ld_cluster_u32(map_to_rank(&sm.counts[0], r));
        tie += ld_cluster_u32(map_to_rank(&sm.counts[1], r));
      }
    }
    const uint32_t below = (1u << lane) - 1u;
    for (int i = w0; i < w1; i += 32) {
      bool a, b;
      kind(i + lane, a, b);
      const uint32_t ma = __ballot_sync(FULL, a), mb = __ballot_sync(FULL, b);
      const uint32_t ts = sure + __popc(ma & below), tt = tie + __popc(mb & below);
      if (a || (b && tt < left)) __stcg(kept + ts + min(tt, left), i + lane);
      sure += __popc(ma);
      tie += __popc(mb);
    }
  } else {
    for (int i = rank * kEvThreads + tid; i < n; i += C * kEvThreads) __stcg(kept + i, i);
  }
  for (int i = n + rank * kEvThreads + tid; i < p.budget; i += C * kEvThreads) kept[i] = -1;
  __threadfence();
  sync_all();  // every kept index is written; select has read its last weight and its shared memory is free

  // ---- move ----
  const int hw = tid >> 4, l16 = tid & 15;
  const int group = C * kEvHalfWarps * kEvRows;  // new positions per group
  const int64_t row_vecs = (int64_t)hkv * (kHeadDim * 2 / 16);  // 16-byte vectors per token of a pool
  const uint4 *kin = static_cast<const uint4 *>(p.k_cache), *vin = static_cast<const uint4 *>(p.v_cache);
  uint4 *kout = static_cast<uint4 *>(p.k_cache), *vout = static_cast<uint4 *>(p.v_cache);
  const int j_first = rank * kEvHalfWarps + hw, j_step = C * kEvHalfWarps;  // row i of group g: j_first + (g kEvRows + i) j_step
  int next[kEvRows];  // source indices of the group to be fetched next
  auto look = [&](int g0) {
#pragma unroll
    for (int i = 0; i < kEvRows; ++i) {
      const int j = g0 + j_first + i * j_step;
      next[i] = j < n ? __ldcg(kept + j) : -1;
    }
  };
  int64_t to[2][kEvRows];  // destinations of the two groups in flight (-1: no copy)
  float wv[2][kEvRows];
  auto fetch = [&](int g0, int b) {
#pragma unroll
    for (int i = 0; i < kEvRows; ++i) {
      const int j = g0 + j_first + i * j_step, src = next[i];
      to[b][i] = -1;
      if (src >= 0) {
        const int sb = __ldg(bt + (src >> 4)), db = __ldg(dt + (j >> 4));
        if (l16 == 0) wv[b][i] = w[src];
        if ((unsigned)sb >= (unsigned)p.num_blocks || (unsigned)db >= (unsigned)p.num_blocks) {
          if (l16 == 0) set_error(p.err, PA_ERR_RANGE, s);
        } else {
          const int64_t from = ((int64_t)sb * kBlock + (src & 15)) * row_vecs + h * 16 + l16;
          const int64_t dst = ((int64_t)db * kBlock + (j & 15)) * row_vecs + h * 16 + l16;
          if (from != dst) {  // (a row that stays where it is needs no copy)
            to[b][i] = dst;
            cp_async_16(&sm.rows[b][i][hw][0][l16], kin + from, 16);
            cp_async_16(&sm.rows[b][i][hw][1][l16], vin + from, 16);
          }
        }
      }
    }
    cp_async_commit();
  };
  auto store = [&](int g0, int b) {
#pragma unroll
    for (int i = 0; i < kEvRows; ++i) {
      const int j = g0 + j_first + i * j_step;
      if (j < n && l16 == 0) w_out[j] = wv[b][i];
      if (to[b][i] >= 0) {  // (a lane reads what it fetched itself)
        st_v4(kout + to[b][i], sm.rows[b][i][hw][0][l16]);
        st_v4(vout + to[b][i], sm.rows[b][i][hw][1][l16]);
      }
    }
  };
  look(0);
  fetch(0, 0);
  look(group);
  for (int g0 = 0; g0 < n; g0 += 2 * group) {  // (uniform over the cluster) two groups per turn: fixed register names
    fetch(g0 + group, 1);
    look(g0 + 2 * group);
    cp_async_wait<1>();
    if (ordered) sync_all();
    store(g0, 0);
    if (g0 + group >= n) break;
    fetch(g0 + 2 * group, 0);
    look(g0 + 3 * group);
    cp_async_wait<1>();
    if (ordered) sync_all();
    store(g0 + group, 1);
  }
  // (in place, each group's weights were read before its barrier, so the tail may be cleared)
  for (int i = n + rank * kEvThreads + tid; i < min(ctx, p.out_stride); i += C * kEvThreads) w_out[i] = 0.f;
  // An attention call enqueued next reads the lengths before its dependency
  // wait, so this kernel never releases its dependents early and makes the
  // length visible before it ends.
  if (h == 0 && rank == 0 && tid == 0) {
    p.new_lens[s] = n;
    __threadfence();
  }
}

}  // namespace

cudaError_t launch_evict(const EvictParams &p, int sms, cudaStream_t stream) {
  static KernelSetup setup;
  const int smem = (int)sizeof(EvSmem);
  cudaError_t e = kernel_setup(setup, kv_evict_kernel, smem, kEvThreads, nullptr);
  if (e != cudaSuccess) return e;
  const int items = p.num_seqs * p.num_kv_heads;
  int C = 8;
  while (C > 1 && items * C > 2 * sms) C >>= 1;
  return launch_pdl_cluster(kv_evict_kernel, dim3(items * C), dim3(kEvThreads), smem, C, stream, p);
}

}  // namespace pa

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
//            through the cluster, and every CTA finds the digit by the same
//            scan.  The slice's keys stay in shared memory where they fit.
//   rank     a kept token's new position = the kept tokens before it: an
//            index-ordered scan of the slice, with the counts of the lower
//            ranks' slices exchanged through the cluster.
//   move     chunks of new positions in ascending order, the rows of a chunk
//            dealt over the cluster's half-warps: read the rows, cluster
//            barrier, write them.  A token never moves up, so a chunk's
//            sources lie at or above its destinations: with the destination
//            table equal to the source table (in place) a write can only reach
//            rows of chunks already read.
// HBM-bound: 4 bytes per token, then 512 read and 512 written per kept row.
#include "pa_device.cuh"

namespace pa {
namespace {

constexpr unsigned FULL = 0xffffffffu;
constexpr int kEvThreads = 512;
constexpr int kEvWarps = kEvThreads / 32;
constexpr int kEvKeys = 16384;       // keys of a CTA's slice held in shared memory (64 KB)
constexpr int kEvBins = 256;         // 8 bits per pass
constexpr int kEvRows = 4;           // rows per half-warp and chunk
constexpr int kEvTile = 4 * kEvThreads;  // tokens per step of the rank scan

struct EvSmem {
  uint32_t hist[kEvBins * 32];       // [bin][lane]
  uint32_t local[2][kEvBins];        // this CTA's counts, by pass parity
  uint32_t scan[kEvWarps];
  uint32_t counts[2];                // sure or heavier tokens of the slice; tokens at the threshold
  uint32_t digit, above;             // the pass's outcome
  uint32_t keys[kEvKeys];
};

// Order-preserving key of a weight (NaN below every number), and a larger key
// for a larger weight; -0 and +0 compare equal.
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

// Inclusive sum over the CTA (every thread; two barriers).
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t *warp_sums, uint32_t &total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const uint32_t y = __shfl_up_sync(FULL, v, off);
    if (lane >= off) v += y;
  }
  if (lane == 31) warp_sums[warp] = v;
  __syncthreads();
  uint32_t base = 0, sum = 0;
#pragma unroll
  for (int i = 0; i < kEvWarps; ++i) {
    base += i < warp ? warp_sums[i] : 0u;
    sum += warp_sums[i];
  }
  total = sum;
  __syncthreads();
  return v + base;
}

__global__ void __launch_bounds__(kEvThreads, 2) kv_evict_kernel(const EvictParams p) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  EvSmem &sm = *reinterpret_cast<EvSmem *>(smem_raw);
  const int tid = threadIdx.x, lane = tid & 31;
  const int C = (int)cluster_nctarank(), rank = (int)cluster_ctarank();
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

  if (ctx > p.budget) {
    // ---- select ----
    const int lo_mid = p.sinks, hi_mid = ctx - p.recent;  // the tokens that compete (more than need of them)
    const uint32_t need = (uint32_t)(p.budget - p.sinks - p.recent);
    const int per = ((ctx + C - 1) / C + 3) & ~3;
    const int s0 = min(ctx, rank * per), s1 = min(ctx, s0 + per);  // this CTA's slice
    for (int i = tid; i < min(s1 - s0, kEvKeys); i += kEvThreads) sm.keys[i] = weight_key(w[s0 + i]);
    __syncthreads();
    auto key_at = [&](int i) { return i - s0 < kEvKeys ? sm.keys[i - s0] : weight_key(w[i]); };
    uint32_t prefix = 0, left = need;  // digits found so far; tokens still wanted at or below them
    for (int pass = 0; pass < 4 && need > 0; ++pass) {
      const int shift = 24 - 8 * pass;
      for (int i = tid; i < kEvBins * 32; i += kEvThreads) sm.hist[i] = 0;
      __syncthreads();
      const int a = max(s0, lo_mid), b = min(s1, hi_mid);
      for (int i = a + tid; i < b; i += kEvThreads) {
        const uint32_t key = key_at(i);
        if (pass == 0 || (key >> (shift + 8)) == prefix)
          atomicAdd(&sm.hist[((key >> shift) & (kEvBins - 1)) * 32 + lane], 1u);
      }
      __syncthreads();
      if (tid < kEvBins) {
        uint32_t sum = 0;
#pragma unroll 8
        for (int j = 0; j < 32; ++j) sum += sm.hist[tid * 32 + ((j + lane) & 31)];
        sm.local[pass & 1][tid] = sum;
      }
      if (C > 1) cluster_sync(); else __syncthreads();
      // thread t takes digit 255 - t: scan from the heaviest down
      uint32_t cnt = 0;
      if (tid < kEvBins)
        for (int r = 0; r < C; ++r)
          cnt += C > 1 ? ld_cluster_u32(map_to_rank(&sm.local[pass & 1][kEvBins - 1 - tid], r))
                       : sm.local[pass & 1][kEvBins - 1 - tid];
      uint32_t total;
      const uint32_t incl = block_scan(cnt, sm.scan, total);
      if (tid < kEvBins && incl >= left && incl - cnt < left) {
        sm.digit = kEvBins - 1 - tid;
        sm.above = incl - cnt;
      }
      __syncthreads();
      prefix = (prefix << 8) | sm.digit;
      left -= sm.above;
      // (the next pass's barriers order these reads before digit and above are written again)
    }
    // kept of the middle: key > prefix, and the first `left` tokens with key == prefix
    const bool none = need == 0;
    auto heavier = [&](int i) -> bool {  // stays whatever its rank among the ties
      return i < lo_mid || i >= hi_mid || (!none && key_at(i) > prefix);
    };
    auto tied = [&](int i) -> bool { return !none && i >= lo_mid && i < hi_mid && key_at(i) == prefix; };
    // ---- rank ----
    uint32_t c_sure = 0, c_tie = 0;
    for (int i = s0 + tid; i < s1; i += kEvThreads) {
      c_sure += heavier(i) ? 1u : 0u;
      c_tie += tied(i) ? 1u : 0u;
    }
    uint32_t t_sure, t_tie;
    block_scan(c_sure, sm.scan, t_sure);
    block_scan(c_tie, sm.scan, t_tie);
    if (tid == 0) {
      sm.counts[0] = t_sure;
      sm.counts[1] = t_tie;
    }
    if (C > 1) cluster_sync(); else __syncthreads();
    uint32_t sure = 0, tie = 0;  // in the slices before this one, then before the current tile
    for (int r = 0; r < rank; ++r) {
      sure += ld_cluster_u32(map_to_rank(&sm.counts[0], r));
      tie += ld_cluster_u32(map_to_rank(&sm.counts[1], r));
    }
    for (int i0 = s0; i0 < s1; i0 += kEvTile) {  // (block-uniform)
      uint32_t f = 0, v = 0;                     // per token: bit e sure, bit 4 + e tied; counts (ties << 16 | sure)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int i = i0 + 4 * tid + e;
        if (i < s1) {
          if (heavier(i)) f |= 1u << e, v += 1u;
          else if (tied(i)) f |= 16u << e, v += 65536u;
        }
      }
      uint32_t tile;
      const uint32_t before = block_scan(v, sm.scan, tile) - v;  // each count at most 2048: no carry
      uint32_t bs = sure + (before & 0xffffu), bt = tie + (before >> 16);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const bool is_sure = (f >> e) & 1u, is_tie = (f >> (4 + e)) & 1u;
        if (is_sure || (is_tie && bt < left)) __stcg(kept + bs + min(bt, left), i0 + 4 * tid + e);
        bs += is_sure;
        bt += is_tie;
      }
      sure += tile & 0xffffu;
      tie += tile >> 16;
    }
  } else {
    for (int i = rank * kEvThreads + tid; i < n; i += C * kEvThreads) __stcg(kept + i, i);
  }
  for (int i = n + rank * kEvThreads + tid; i < p.budget; i += C * kEvThreads) kept[i] = -1;
  __threadfence();
  if (C > 1) cluster_sync(); else __syncthreads();  // every kept index is written; every weight that select reads is read

  // ---- move ----
  const int32_t *bt = p.block_tables + (int64_t)s * p.max_blocks_per_seq;
  const int32_t *dt = p.dst_block_tables + (int64_t)s * p.dst_max_blocks;
  const int hw = tid >> 4, l16 = tid & 15;
  constexpr int kHalfWarps = kEvThreads / 16;
  const int chunk = C * kHalfWarps * kEvRows;
  const int64_t row_vecs = (int64_t)hkv * (kHeadDim * 2 / 16);  // 16-byte vectors per token of a pool
  const uint4 *kin = static_cast<const uint4 *>(p.k_cache), *vin = static_cast<const uint4 *>(p.v_cache);
  uint4 *kout = static_cast<uint4 *>(p.k_cache), *vout = static_cast<uint4 *>(p.v_cache);
  for (int c0 = 0; c0 < n; c0 += chunk) {  // (uniform over the cluster)
    uint4 kr[kEvRows], vr[kEvRows];
    int64_t to[kEvRows];
    float wr[kEvRows];
#pragma unroll
    for (int i = 0; i < kEvRows; ++i) {
      const int j = c0 + (i * C + rank) * kHalfWarps + hw;  // new position
      to[i] = -1;
      if (j < n) {
        const int src = __ldcg(kept + j);
        const int sb = __ldg(bt + (src >> 4)), db = __ldg(dt + (j >> 4));
        if (l16 == 0) wr[i] = w[src];
        if ((unsigned)sb >= (unsigned)p.num_blocks || (unsigned)db >= (unsigned)p.num_blocks) {
          if (l16 == 0) set_error(p.err, PA_ERR_RANGE, s);
        } else {
          const int64_t a = ((int64_t)sb * kBlock + (src & 15)) * row_vecs + h * 16 + l16;
          const int64_t b = ((int64_t)db * kBlock + (j & 15)) * row_vecs + h * 16 + l16;
          if (a != b) {  // (a row that stays where it is needs no copy)
            to[i] = b;
            kr[i] = kin[a];
            vr[i] = vin[a];
          }
        }
      }
    }
    if (C > 1) cluster_sync(); else __syncthreads();
#pragma unroll
    for (int i = 0; i < kEvRows; ++i) {
      const int j = c0 + (i * C + rank) * kHalfWarps + hw;
      if (j < n && l16 == 0) w_out[j] = wr[i];
      if (to[i] >= 0) {
        st_v4(kout + to[i], kr[i]);
        st_v4(vout + to[i], vr[i]);
      }
    }
  }
  // (each chunk's weights were read before its barrier, so the tail may be cleared in place)
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

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
//            however few values the weights take: with 11 bits and 4 columns
//            the zero weights of 131072 tokens made three passes cost 26 us,
//            where these four cost 12), the CTAs add their counts through the
//            cluster, and every warp finds the digit by the same scan from the
//            heaviest down.  A digit whose tokens all stay ends the
//            selection.  The slice's keys stay in shared memory where they fit.
//            A short sequence is selected by every CTA of its cluster alone: up
//            to kEvAlone tokens a pass is bound by its barriers, and those of a
//            cluster cost more than counting all tokens does (1000 tokens, 8
//            CTAs: 8.6 us together).
//   rank     a kept token's new position = the kept tokens before it: ballots
//            over 32 tokens at a time, lane i keeping the i-th, then one scan over
//            the lanes, the warps and the lower ranks.
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
constexpr int kEvAlone = 4096;       // tokens that a CTA selects from without its cluster
constexpr int kEvRows = 3;           // rows per half-warp and group; two groups in shared memory
constexpr uint32_t kStays = 0xffffffffu;  // the key of a token that stays whatever its weight (no weight's key)
static_assert(kEvThreads == 2 * kEvBins, "two threads sum a digit's columns");

struct EvSmem {
  union {
    struct {
      uint32_t keys[kEvKeys];
      uint4 hist[kEvBins][8];          // [digit][lane]
    } sel;
    uint4 rows[2][kEvRows][kEvHalfWarps][2][16];  // the move: [group parity][row][half-warp][K, V][16 x 16 bytes]
  };
  uint32_t local[2][kEvBins];          // this CTA's counts, by pass parity
  uint32_t total[kEvBins];             // the cluster's
  uint32_t warp_a[kEvWarps], warp_b[kEvWarps];
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
// Inclusive sum over the warp's lanes.
__device__ __forceinline__ uint32_t warp_scan(uint32_t v, int lane) {
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const uint32_t y = __shfl_up_sync(FULL, v, off);
    if (lane >= off) v += y;
  }
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
  // The CTAs that select together, and this one's place among them.
  const bool alone = C == 1 || ctx <= kEvAlone;
  const int SC = alone ? 1 : C, srank = alone ? 0 : rank;
  const int lo_mid = p.sinks, hi_mid = ctx - p.recent;  // the tokens that compete
  const int per = ((ctx + SC - 1) / SC + 31) & ~31;
  const int s0 = min(ctx, srank * per), s1 = min(ctx, s0 + per);  // this CTA's slice
  auto key_of = [&](int i) { return i < lo_mid || i >= hi_mid ? kStays : weight_key(w[i]); };
  if (ctx > p.budget) {
    constexpr int U = 8;  // loads in flight per thread
    const int m = min(s1 - s0, kEvKeys), m4 = (m + 3) & ~3;
    for (int i0 = tid; i0 < m4; i0 += U * kEvThreads) {
      float f[U];
#pragma unroll
      for (int u = 0; u < U; ++u) f[u] = i0 + u * kEvThreads < m ? w[s0 + i0 + u * kEvThreads] : 0.f;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = i0 + u * kEvThreads, j = s0 + i;
        if (i < m4) sm.sel.keys[i] = i >= m || j < lo_mid || j >= hi_mid ? kStays : weight_key(f[u]);
      }
    }
  }
  // In place if a destination page is the source page of the same index.
  bool same = p.weights_out == p.weights;
  for (int i = tid; i < (n + kBlock - 1) / kBlock; i += kEvThreads) same = same || __ldg(bt + i) == __ldg(dt + i);
  const bool ordered = __syncthreads_or(same) != 0;  // (the same in every CTA of the cluster)

  if (ctx > p.budget) {
    // ---- select ----
    const uint32_t need = (uint32_t)(p.budget - p.sinks - p.recent);
    auto key_at = [&](int i) { return i - s0 < kEvKeys ? sm.sel.keys[i - s0] : key_of(i); };
    uint32_t prefix = 0, left = need;  // digits found so far; tokens still wanted at them
    int shift = 32;                    // the digits' place: a key's are key >> shift
    if (need == 0) {                   // none of the middle stays
      prefix = kStays - 1;
      shift = 0;
    }
    for (int pass = 0; pass < 4 && need > 0; ++pass) {
#pragma unroll
      for (int j = 0; j < 4; ++j) sm.sel.hist[0][tid + j * kEvThreads] = make_uint4(0, 0, 0, 0);
      __syncthreads();
      const uint32_t hist = smem_u32(sm.sel.hist) + 4 * lane;
      auto tally = [&](uint32_t key) {  // (a token that stays anyway does not compete)
        if (key != kStays && (pass == 0 || (key >> shift) == prefix))
          asm volatile("red.shared.add.u32 [%0], 1;" ::"r"(hist + ((key >> (shift - 8)) & (kEvBins - 1)) * 128)
                       : "memory");
      };
      const int m4 = (min(s1 - s0, kEvKeys) + 3) >> 2;
#pragma unroll 4
      for (int i = tid; i < m4; i += kEvThreads) {
        const uint4 u = reinterpret_cast<const uint4 *>(sm.sel.keys)[i];
        tally(u.x), tally(u.y), tally(u.z), tally(u.w);
      }
      for (int i = s0 + kEvKeys + tid; i < s1; i += kEvThreads) tally(key_of(i));
      __syncthreads();
      {
        const int bin = tid >> 1;
        uint32_t sum = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {  // (eight lanes read eight banks' worth)
          const uint4 u = sm.sel.hist[bin][(tid & 1) * 4 + ((j + (lane >> 1)) & 3)];
          sum += (u.x + u.y) + (u.z + u.w);
        }
        sum += __shfl_xor_sync(FULL, sum, 1);
        if ((tid & 1) == 0) (SC > 1 ? sm.local[pass & 1] : sm.total)[bin] = sum;
      }
      if (SC > 1) {
        cluster_sync();
        if (tid < kEvBins) {
          uint32_t sum = 0;
          for (int r = 0; r < SC; ++r) sum += ld_cluster_u32(map_to_rank(&sm.local[pass & 1][tid], r));
          sm.total[tid] = sum;
        }
      }
      __syncthreads();
      // lane l scans the digits 255 - 8 l .. 248 - 8 l
      uint32_t c[8], mine = 0;
      {
        const uint4 u = *reinterpret_cast<const uint4 *>(&sm.total[kEvBins - 8 - 8 * lane]);
        const uint4 v = *reinterpret_cast<const uint4 *>(&sm.total[kEvBins - 4 - 8 * lane]);
        c[0] = v.w, c[1] = v.z, c[2] = v.y, c[3] = v.x, c[4] = u.w, c[5] = u.z, c[6] = u.y, c[7] = u.x;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) mine += c[j];
      const uint32_t incl = warp_scan(mine, lane);
      const int owner = __ffs(__ballot_sync(FULL, incl >= left)) - 1;  // exists: at least `left` tokens are counted
      uint32_t above = incl - mine, digit = 0, count = 0;
      bool open = true;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (open) {
          if (above + c[j] >= left) {
            open = false;
            digit = kEvBins - 1 - 8 * lane - j;
            count = c[j];
          } else {
            above += c[j];
          }
        }
      prefix = (prefix << 8) | __shfl_sync(FULL, digit, owner);
      left -= __shfl_sync(FULL, above, owner);
      shift -= 8;
      if (__shfl_sync(FULL, count, owner) == left) break;  // (uniform over the cluster) all tokens at these digits stay
      __syncthreads();  // (alone, the totals are read before the next pass writes them)
    }
    // ---- rank: the tokens with larger digits stay, and the first `left` with equal ones ----
    const int wper = (((s1 - s0) + kEvWarps - 1) / kEvWarps + 31) & ~31;
    const int w0 = s0 + warp * wper, w1 = min(s1, w0 + wper);  // this warp's part
    // 1024 tokens from i0 on: lane l gets the masks of the 32 from i0 + 32 l on
    auto masks = [&](int i0, uint32_t &ma, uint32_t &mb) {
      ma = mb = 0;
      const int steps = min(32, (w1 - i0 + 31) >> 5);
      const bool held = i0 - s0 + 1024 <= kEvKeys;  // (all in shared memory: no other test per step)
#pragma unroll 4
      for (int k = 0; k < steps; ++k) {  // (warp-uniform)
        const int i = i0 + 32 * k + lane;
        const uint32_t d = (held ? sm.sel.keys[i - s0] : i < w1 ? key_at(i) : 0u) >> shift;
        const uint32_t a = __ballot_sync(FULL, d > prefix), b = __ballot_sync(FULL, d == prefix);
        if (lane == k) ma = a, mb = b;
      }
      const int valid = w1 - i0 - 32 * lane;  // tokens of this lane's 32 that are the warp's
      if (valid < 32) {
        const uint32_t in = valid > 0 ? (1u << valid) - 1u : 0u;
        ma &= in;
        mb &= in;
      }
    };
    uint32_t n_sure = 0, n_tie = 0, ma = 0, mb = 0;
    for (int i0 = w0; i0 < w1; i0 += 1024) {
      masks(i0, ma, mb);
      n_sure += __popc(ma);
      n_tie += __popc(mb);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      n_sure += __shfl_xor_sync(FULL, n_sure, off);
      n_tie += __shfl_xor_sync(FULL, n_tie, off);
    }
    if (lane == 0) {
      sm.warp_a[warp] = n_sure;
      sm.warp_b[warp] = n_tie;
    }
    __syncthreads();
    uint32_t sure = 0, tie = 0, all_sure = 0, all_tie = 0;
#pragma unroll
    for (int i = 0; i < kEvWarps; ++i) {
      const uint32_t x = sm.warp_a[i], y = sm.warp_b[i];
      sure += i < warp ? x : 0u;
      tie += i < warp ? y : 0u;
      all_sure += x;
      all_tie += y;
    }
    if (SC > 1) {
      if (tid == 0) {
        sm.counts[0] = all_sure;
        sm.counts[1] = all_tie;
      }
      cluster_sync();
      for (int r = 0; r < srank; ++r) {
        sure += ld_cluster_u32(map_to_rank(&sm.counts[0], r));
        tie += ld_cluster_u32(map_to_rank(&sm.counts[1], r));
      }
    }
    for (int i0 = w0; i0 < w1; i0 += 1024) {
      if (wper > 1024) masks(i0, ma, mb);  // (else they are still there)
      const uint32_t is = warp_scan(__popc(ma), lane), it = warp_scan(__popc(mb), lane);
      const uint32_t ls = sure + is - __popc(ma), lt = tie + it - __popc(mb);  // before this lane's 32
      // of its ties the first left - lt stay
      uint32_t m = mb;
      for (int drop = (int)min((int64_t)__popc(mb), max((int64_t)0, (int64_t)lt + __popc(mb) - (int64_t)left)); drop > 0; --drop)
        m &= ~(0x80000000u >> __clz(m));
      m |= ma;
      int32_t *dst = kept + ls + min(lt, left);
      for (int i = i0 + 32 * lane; m; m &= m - 1) __stcg(dst++, i + __ffs(m) - 1);
      sure += __shfl_sync(FULL, is, 31);
      tie += __shfl_sync(FULL, it, 31);
    }
  } else {
    for (int i = srank * kEvThreads + tid; i < n; i += SC * kEvThreads) __stcg(kept + i, i);
  }
  for (int i = n + rank * kEvThreads + tid; i < p.budget; i += C * kEvThreads) kept[i] = -1;
  // Every kept index that this CTA will read is written, the shared memory of
  // the selection is free, and (the barrier of the first group in place, too)
  // the weights it read may be overwritten.
  if (SC > 1) {
    __threadfence();
    cluster_sync();
  } else {
    __syncthreads();
  }

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

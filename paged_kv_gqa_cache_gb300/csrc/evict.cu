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
//            cluster, and every warp finds the digit by the same two scans, of
//            16 groups and of the 16 digits in one, from the heaviest down.  A
//            digit whose tokens all stay ends the selection, and so do few
//            tokens at a digit, each of which is then compared with all others.
//            The slice's keys stay in shared memory where they fit.  A pass over
//            16384 keys is bound by its instructions (five a key) and by its
//            barriers.  A short sequence is selected by every CTA of its cluster
//            alone: up to kEvAlone tokens the barriers of a cluster cost more
//            than counting all tokens does (1000 tokens, 8 CTAs: 8.6 us
//            together, 3.8 alone).
//   rank     a kept token's new position = the kept tokens before it: ballots
//            over 32 tokens at a time, lane i keeping the i-th, then one scan over
//            the lanes, the warps and the lower ranks.  The indices are gathered
//            in shared memory and leave it in whole lines.
//   move     each half-warp takes every (32 C)-th new position through shared
//            memory (cp.async), the next row on its way meanwhile.  More rows in
//            flight are slower: the heads of a sequence then drift apart, and
//            with them the rows of one page (32 sequences of up to 8192 tokens:
//            97.7 us, 104.8 with two rows, 106.7 with three; 4 sequences of
//            131072, of which an eighth stays: 121.0, 118.7, 119.0).  A token
//            never moves up, so the sources of a group of rows lie at or above
//            its destinations: in place (a destination table that repeats the
//            source table, or weights_out = weights) a cluster barrier between
//            the reads and the writes of each group is all the order it takes,
//            and three rows per half-warp and barrier are faster (the same
//            sequences in place: 91.8 and 138 us, with one row 93.4 and 172);
//            apart, no barrier at all.
// HBM-bound: 4 bytes per token, then 512 read and 512 written per kept row.  The
// 32 sequences above, cut to 2048 with 8 KV heads: 97.7 us, 5.4 TB/s, of which
// the selection and ranking (13 us) leave HBM idle; the 4 long ones, cut to 16384:
// 121 us, 4.6 TB/s (22 us; then 256-byte rows apart from one another).  One
// sequence of 1000 cut to 512: 8.5 us, a chain of latencies (select 3.8, rank 1.7,
// move 2.1).  The cluster's size goes by the number of (sequence, KV head) items
// alone: 5 sequences of 131072 with 8 heads take 4 CTAs each, whose slices of 32768
// keys fit shared memory by half, and 239 us (floor 103; 4 sequences, 8 CTAs each:
// 123, floor 82; 8 sequences 293, floor 165).
#include <type_traits>

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
constexpr int kEvList = 4096;        // kept indices of a CTA that selects alone, held in shared memory
constexpr int kEvFew = 32;           // competing tokens that are ranked against one another
constexpr int kEvRows = 3;           // rows per half-warp and group in place (one apart); two groups in shared memory
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
  uint16_t list[kEvList];              // kept indices, of a CTA that selects alone
  uint32_t local[2][kEvBins];          // this CTA's counts, by pass parity
  uint32_t total[kEvBins];             // the cluster's
  uint32_t group[16];                  // the sums of 16 totals each
  uint32_t warp_a[kEvWarps], warp_b[kEvWarps];
  uint32_t few[kEvFew];                // keys of the last tokens that compete
  uint32_t num_few;
  uint32_t counts[2];                  // sure, then tied tokens of the slice
};

// Order-preserving key of a weight (NaN below every number); -0 and +0 compare
// equal.  No number's key has 16 leading ones (+inf: 0xff800000).
__device__ __forceinline__ uint32_t weight_key(float w) {
  const uint32_t u = __float_as_uint(w + 0.f);  // (-0 becomes +0)
  return w != w ? 0u : u ^ (uint32_t)((int32_t)u >> 31 | 0x80000000);
}
// Add 1 to a word of shared memory if key < bound, by predicate.
__device__ __forceinline__ void tally_below(uint32_t addr, uint32_t key, uint32_t bound) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.lt.u32 p, %1, %2;\n\t@p red.shared.add.u32 [%0], 1;\n\t}" ::"r"(addr), "r"(key),
      "r"(bound)
      : "memory");
}

__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void st_cluster_u32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ uint32_t add_cluster_u32(uint32_t addr, uint32_t v) {
  uint32_t old;
  asm volatile("atom.relaxed.cluster.shared::cluster.add.u32 %0, [%1], %2;" : "=r"(old) : "r"(addr), "r"(v) : "memory");
  return old;
}
__device__ __forceinline__ void cp_async_4(void *dst, const void *src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
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
  if (ctx < 1 || ctx > kLongMaxTokens || (int64_t)ctx > (int64_t)p.max_blocks_per_seq * kBlock ||
      ctx > p.weights_stride || (int64_t)n > (int64_t)p.dst_max_blocks * kBlock ||
      n > p.out_stride) {  // uniform over the cluster
    if (h == 0 && rank == 0 && tid == 0) {
      set_error(p.err, PA_ERR_RANGE, s);
      if (p.flags & PA_EVICT_MARK_LENGTHS) p.new_lens[s] = -1;
    }
    if (p.flags & PA_EVICT_MARK_KEPT) {
      int32_t *row = p.kept + ((int64_t)s * hkv + h) * p.budget;
      for (int i = rank * kEvThreads + tid; i < p.budget; i += C * kEvThreads) row[i] = -1;
    }
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
  const bool listed = alone && n <= kEvList && ctx <= 0x10000;  // the kept indices stay in shared memory
  const int lo_mid = p.sinks, hi_mid = ctx - p.recent;          // the tokens that compete
  const int per = ((ctx + SC - 1) / SC + 31) & ~31;
  const int s0 = min(ctx, srank * per), s1 = min(ctx, s0 + per);  // this CTA's slice
  const int m = min(s1 - s0, kEvKeys), m4 = (m + 3) >> 2;         // the part of it in shared memory
  if (ctx > p.budget) {  // the slice's weights, all on their way together
    if ((reinterpret_cast<uintptr_t>(w) & 15) == 0) {
      for (int i = tid; i < m4; i += kEvThreads)
        cp_async_16(&sm.sel.keys[4 * i], w + s0 + 4 * i, 4 * min(4, m - 4 * i));
    } else {
      for (int i = tid; i < m; i += kEvThreads) cp_async_4(&sm.sel.keys[i], w + s0 + i);
    }
    cp_async_commit();
#pragma unroll
    for (int j = 0; j < 4; ++j) sm.sel.hist[0][tid + j * kEvThreads] = make_uint4(0, 0, 0, 0);
    if (tid == 0) sm.num_few = 0;
  }
  // In place if a destination page is the source page of the same index.
  bool same = p.weights_out == p.weights;
  for (int i = tid; i < (n + kBlock - 1) / kBlock; i += kEvThreads) same |= __ldg(bt + i) == __ldg(dt + i);
  cp_async_wait<0>();
  const bool ordered = __syncthreads_or(same) != 0;  // (the same in every CTA of the cluster)

  if (ctx > p.budget) {
    // ---- select ----
    auto key_of = [&](int i, float x) { return i < lo_mid || i >= hi_mid ? kStays : weight_key(x); };
    auto key_at = [&](int i) { return i - s0 < kEvKeys ? sm.sel.keys[i - s0] : key_of(i, w[i]); };
    auto each_key = [&](auto &&f) {  // over the slice (the padding of the last four keys has the key kStays)
#pragma unroll 4
      for (int i = tid; i < m4; i += kEvThreads) {
        const uint4 u = reinterpret_cast<const uint4 *>(sm.sel.keys)[i];
        f(u.x), f(u.y), f(u.z), f(u.w);
      }
      for (int i = s0 + kEvKeys + tid; i < s1; i += kEvThreads) f(key_of(i, w[i]));
    };
    const uint32_t hist = smem_u32(sm.sel.hist) + 4 * lane;
    auto tally_first = [&](uint32_t key) { tally_below(hist + (key >> 24) * 128, key, kStays); };
    // weights to keys, in place, and the counts of the first pass
#pragma unroll 4
    for (int i = tid; i < m4; i += kEvThreads) {
      const float4 x = reinterpret_cast<const float4 *>(sm.sel.keys)[i];
      const int j = s0 + 4 * i;
      uint4 u = make_uint4(weight_key(x.x), weight_key(x.y), weight_key(x.z), weight_key(x.w));
      if (j < lo_mid || j + 4 > hi_mid || 4 * i + 4 > m) {  // the ends
        auto out = [&](int k) { return j + k < lo_mid || j + k >= hi_mid || 4 * i + k >= m; };
        if (out(0)) u.x = kStays;
        if (out(1)) u.y = kStays;
        if (out(2)) u.z = kStays;
        if (out(3)) u.w = kStays;
      }
      reinterpret_cast<uint4 *>(sm.sel.keys)[i] = u;
      tally_first(u.x), tally_first(u.y), tally_first(u.z), tally_first(u.w);
    }
    for (int i = s0 + kEvKeys + tid; i < s1; i += kEvThreads) tally_first(key_of(i, w[i]));
    const uint32_t need = (uint32_t)(p.budget - p.sinks - p.recent);
    uint32_t prefix = 0, left = need;  // digits found so far; tokens still wanted at them
    int shift = 32;                    // the digits' place: a key's are key >> shift
    if (need == 0) {                   // none of the middle stays
      prefix = kStays - 1;
      shift = 0;
      __syncthreads();  // the keys
    }
    for (int pass = 0; pass < 4 && need > 0; ++pass) {
      if (pass > 0) {
        const uint32_t base = prefix << shift, bound = 1u << shift;
        each_key([&](uint32_t key) {
          const uint32_t rest = key ^ base;  // (below the bound: the key has the digits found so far)
          tally_below(hist + (rest >> (shift - 8)) * 128, rest, bound);
        });
      }
      __syncthreads();
      {
        const int bin = tid >> 1;
        uint4 *row = sm.sel.hist[bin] + (tid & 1) * 4, u[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) u[j] = row[(j + (lane >> 1)) & 3];  // (eight lanes read eight banks' worth)
        uint32_t sum = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          sum += (u[j].x + u[j].y) + (u[j].z + u[j].w);
          row[(j + (lane >> 1)) & 3] = make_uint4(0, 0, 0, 0);  // for the next pass
        }
        sum += __shfl_xor_sync(FULL, sum, 1);
        // (below the digit 0xff of a first pass a second one is a token's that stays anyway)
        if (pass == 1 && prefix == 0xff && bin == 0xff) sum = 0;
        if ((tid & 1) == 0) (SC > 1 ? sm.local[pass & 1] : sm.total)[bin] = sum;
        if (SC == 1) {
          sum = __reduce_add_sync(FULL, tid & 1 ? 0u : sum);
          if (lane == 0) sm.group[warp] = sum;
        }
      }
      if (SC > 1) {
        cluster_sync();
        if (tid < kEvBins) {
          uint32_t sum = 0;
          for (int r = 0; r < SC; ++r) sum += ld_cluster_u32(map_to_rank(&sm.local[pass & 1][tid], r));
          sm.total[tid] = sum;
#pragma unroll
          for (int off = 8; off > 0; off >>= 1) sum += __shfl_xor_sync(FULL, sum, off);
          if ((lane & 15) == 0) sm.group[tid >> 4] = sum;
        }
      }
      __syncthreads();  // (the next totals are written behind the next pass's barrier)
      // Every warp finds the digit: the group of 16 from the heaviest down, then
      // the digit in it; lane l takes the l-th from the top (16 .. 31 nothing).
      uint32_t digit, count;
      {
        const int top = 15 - (lane & 15);
        uint32_t c = lane < 16 ? sm.group[top] : 0u, incl = warp_scan(c, lane);
        int owner = __ffs(__ballot_sync(FULL, incl >= left)) - 1;  // exists: at least `left` tokens are counted
        left -= __shfl_sync(FULL, incl - c, owner);
        digit = 16 * (15 - owner);
        c = lane < 16 ? sm.total[digit + top] : 0u;
        incl = warp_scan(c, lane);
        owner = __ffs(__ballot_sync(FULL, incl >= left)) - 1;
        left -= __shfl_sync(FULL, incl - c, owner);
        count = __shfl_sync(FULL, c, owner);
        digit += 15 - owner;
      }
      prefix = (prefix << 8) | digit;
      shift -= 8;
      if (count == left) break;  // (uniform over the cluster) all tokens at these digits stay
      if (count <= kEvFew && shift > 0) {  // few compete still: each against all
        const uint32_t base = prefix << shift, bound = 1u << shift;
        each_key([&](uint32_t key) {
          if ((key ^ base) < bound && key != kStays) {
            if (SC > 1) {
              for (int r = 0; r < SC; ++r) {
                const uint32_t at = add_cluster_u32(map_to_rank(&sm.num_few, r), 1);
                if (at < kEvFew) st_cluster_u32(map_to_rank(&sm.few[at], r), key);
              }
            } else {
              const uint32_t at = atomicAdd(&sm.num_few, 1u);
              if (at < kEvFew) sm.few[at] = key;
            }
          }
        });
        if (SC > 1) cluster_sync(); else __syncthreads();
        const uint32_t key = lane < count ? sm.few[lane] : 0;
        uint32_t larger = 0, equal = 0;
#pragma unroll
        for (uint32_t j = 0; j < kEvFew; ++j) {
          const uint32_t other = sm.few[j];
          larger += j < count && other > key;
          equal += j < count && other == key;
        }
        // the key that the wanted tokens end at
        const int at = __ffs(__ballot_sync(FULL, lane < count && larger < left && larger + equal >= left)) - 1;
        prefix = __shfl_sync(FULL, key, at);
        left -= __shfl_sync(FULL, larger, at);
        shift = 0;
        break;
      }
    }
    // ---- rank: the tokens with larger digits stay, and the first `left` with equal ones ----
    const uint32_t lo_key = prefix << shift;
    const uint32_t hi_key = min(lo_key | ((1u << shift) - 1u), kStays - 1u);  // (a token that stays anyway is above)
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
        const uint32_t key = held ? sm.sel.keys[i - s0] : i < w1 ? key_at(i) : 0u;
        const uint32_t a = __ballot_sync(FULL, key > hi_key), b = __ballot_sync(FULL, key >= lo_key) & ~a;
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
    uint32_t sure = 0, tie = 0, all_sure = 0, all_tie = 0;  // before this warp, of the slice
#pragma unroll
    for (int i = 0; i < kEvWarps; ++i) {
      const uint32_t x = sm.warp_a[i], y = sm.warp_b[i];
      sure += i < warp ? x : 0u;
      tie += i < warp ? y : 0u;
      all_sure += x;
      all_tie += y;
    }
    uint32_t sure0 = 0, tie0 = 0;  // before the slice
    if (SC > 1) {
      if (tid == 0) {
        sm.counts[0] = all_sure;
        sm.counts[1] = all_tie;
      }
      cluster_sync();
      for (int r = 0; r < srank; ++r) {
        sure0 += ld_cluster_u32(map_to_rank(&sm.counts[0], r));
        tie0 += ld_cluster_u32(map_to_rank(&sm.counts[1], r));
      }
      sure += sure0;
      tie += tie0;
    }
    // The indices are gathered in shared memory, where the keys were (all masks
    // are taken and held), and go out in whole lines.
    const uint32_t before0 = sure0 + min(tie0, left), behind0 = sure0 + all_sure + min(tie0 + all_tie, left);
    const bool staged = s1 - s0 <= kEvKeys;
    auto stays = [&](uint32_t at, int i) {
      if (listed) sm.list[at] = (uint16_t)i;
      else if (staged) sm.sel.keys[at - before0] = (uint32_t)i;
      else __stcg(kept + at, i);
    };
    for (int i0 = w0; i0 < w1; i0 += 1024) {
      if (wper > 1024) masks(i0, ma, mb);  // (else they are still there)
      const uint32_t is = warp_scan(__popc(ma), lane), it = warp_scan(__popc(mb), lane);
      const uint32_t ls = sure + is - __popc(ma), lt = tie + it - __popc(mb);  // before this lane's 32
      // of its ties the first left - lt stay
      uint32_t m = mb;  // (of this lane's 32 tokens)
      const int nb = __popc(mb);
      for (int drop = (int)min((int64_t)nb, max((int64_t)0, (int64_t)lt + nb - (int64_t)left)); drop > 0; --drop)
        m &= ~(0x80000000u >> __clz(m));
      m |= ma;
      // The masks are written out by all lanes: of steps <= 2^lg masks each lane
      // takes 2^lg bits.
      const int steps = min(32, (w1 - i0 + 31) >> 5), lg = 32 - __clz(steps - 1);
      const int from = lane >> (5 - lg), low = (lane << lg) & 31;
      const uint32_t whole = __shfl_sync(FULL, m, from), before = whole & ((1u << low) - 1u);
      uint32_t at = __shfl_sync(FULL, ls + min(lt, left), from) + __popc(before);
      uint32_t bits = whole ^ before;
      if (lg < 5 && low + (1 << lg) < 32) bits &= (1u << (low + (1 << lg))) - 1u;
      for (; bits; bits &= bits - 1) stays(at++, i0 + 32 * from + __ffs(bits) - 1);
      sure += __shfl_sync(FULL, is, 31);
      tie += __shfl_sync(FULL, it, 31);
    }
    __syncthreads();
    if (listed) {
      for (int j = rank * kEvThreads + tid; j < n; j += C * kEvThreads) kept[j] = sm.list[j];
    } else if (staged) {
      for (uint32_t j = before0 + tid; j < behind0; j += kEvThreads) __stcg(kept + j, (int)sm.sel.keys[j - before0]);
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
  const int64_t row_vecs = (int64_t)hkv * (kHeadDim * 2 / 16);  // 16-byte vectors per token of a pool
  const uint4 *kin = static_cast<const uint4 *>(p.k_cache), *vin = static_cast<const uint4 *>(p.v_cache);
  uint4 *kout = static_cast<uint4 *>(p.k_cache), *vout = static_cast<uint4 *>(p.v_cache);
  // row i of group g: j_first + (g R + i) j_step
  const int j_first = rank * kEvHalfWarps + hw, j_step = C * kEvHalfWarps;
  auto move = [&](auto rows_per_group) {
    constexpr int R = decltype(rows_per_group)::value;
    const int group = R * j_step;  // new positions per group
    int next[R];  // source indices of the group to be fetched next
    auto look = [&](int g0) {
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const int j = g0 + j_first + i * j_step;
        next[i] = j >= n ? -1 : ctx <= p.budget ? j : listed ? sm.list[j] : __ldcg(kept + j);
      }
    };
    int64_t to[2][R];  // destinations of the two groups in flight (-1: no copy)
    float wv[2][R];
    auto fetch = [&](int g0, int b) {
#pragma unroll
      for (int i = 0; i < R; ++i) {
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
      for (int i = 0; i < R; ++i) {
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
  };
  if (ordered) move(std::integral_constant<int, kEvRows>()); else move(std::integral_constant<int, 1>());
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

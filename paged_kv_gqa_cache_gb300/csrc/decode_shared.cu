// Paged GQA decode for sequences that share prefixes by groups, for sm_103a:
// each group's prefix is read and multiplied once for all of its sequences.
//
//   out[s][g] = softmax_j(scale q[s][g] . K_j) V_j over the whole context of s,
// the keys split in two: the shared prefix of the sequence's group and the rest.
// For online softmax states (m, l, o) over disjoint key sets the join is
//   m = max m_i,  l = sum l_i 2^(m_i - m),  o = sum o_i 2^(m_i - m),  out = o / l.
//
// Two kernels:
//   shared  One CTA per SM; each has an equal share of the prefix work and of
//           the rest.
//           Prefix: the query rows of a group's sequences for one KV head
//           (sequences x G rows) against the prefix are a matrix product: query
//           tiles of 128 rows, key tiles of 128 keys, on the tcgen05 tensor cores
//           with the tile machinery of prefill_kernel.cuh (no causal mask).  The
//           (query tile, key tile) pairs are dealt evenly; a piece of a query
//           tile's keys leaves its state in the workspace.  One query tile per KV
//           head is bound by HBM (64 KB of K and V per 0.78 us of tensor time,
//           against 1.47 us of an SM's share of HBM), more by the tensor cores;
//           then the key range is cut into blocks about as long as a CTA's share,
//           the query tiles of a block next to each other in the order, so that
//           the CTAs that need the same keys run at the same time and all but one
//           of them read L2 (mostly: of 126 MB of shared keys 172 come from HBM).
//           Suffix: the rest of each sequence, by the split workers of
//           decode_mma.cuh: the softmax warps consume, the loader and MMA warps
//           produce.  Their stages (8 x 3 x 8 KB) take the very 192 KB of the query
//           tile and the K and V rings, so the first pages are on their way when
//           the last P V has completed, while the query tile is still stored.
//           (As a kernel of its own behind the prefix the suffix paid a launch, a
//           schedule and a first trip to HBM: 57 us for 32 sequences and 32768
//           shared tokens, 122 for 192 in three groups.  Beside the prefix on SMs
//           of its own 54 and 139: its stream pushed the shared keys out of L2.
//           With half of the CTAs starting with the suffix 49.7 and 100.5.)
//   join    A warp per (sequence, KV head, part of the dims) adds up the pieces.
// Measured, 32 / 8 heads, bf16: 32 sequences, 32768 shared tokens and up to 1000
// each: 46.1 us (4.3 TB/s; HBM in both parts, 1.6 us a pair, and the ramps; the
// join takes 3 us); 192 in three groups of 4096 to 16384, up to 700 each: 100.5 us
// (4.3 TB/s; a pair of a large group 1.0 us: 192 KB through shared memory, 64 in
// by TMA, 64 to Q K^T and 64 to P V, are 0.8; the join takes 9; 98.5 us with P in
// one term).  4 sequences, 1024 shared, up to 200 each, 16 / 8 heads: 9.7 us, a
// chain of latencies.  A sequence more than fills whole query tiles costs one more
// (16384 shared, 32 / 8 heads, 32 and 33 sequences: 31.6 and 41.5 us).  Against the
// plain decode, which reads the prefix once per sequence, it is the faster from about
// (sequences - 1) x shared tokens = 10000 on at 8 KV heads (2 sequences, 4096 shared:
// 14.9 and 13.8 us, 16384: 24.4 and 29.2; 16, 256: 9.4 and 6.0, 1024: 11.2 and 12.5;
// 32, 1024: 14.7 and 25.3).
#include "decode_mma.cuh"
#include "prefill_kernel.cuh"

namespace pa {
namespace {

constexpr int kGroups = kMaxPrefixGroups;
constexpr int kJoinPieces = 8;  // pieces in flight in the join
// Two stages of K and three of V: a K tile is free again once S is computed, a V
// tile only after the softmax and P V (K 3 and V 2, both issued in one order by
// the same warps, left 1.9 us between key tiles where HBM's share is 1.5).
constexpr int kPKStages = 2, kPVStages = 3;
constexpr int kKLoad = 4, kVLoad = kLoadWarps - kKLoad;  // loader warps of each
constexpr int P_OFF_Q = 0;
constexpr int P_OFF_K = 2 * kHalf;
constexpr int P_OFF_V = P_OFF_K + kPKStages * 2 * kHalf;
constexpr int P_OFF_X = P_OFF_V + kPVStages * 2 * kHalf;  // (m, l) exchange [unit parity][half][128]
constexpr int P_OFF_PLAN = P_OFF_X + 2 * 2 * 128 * 8;
struct PBars {
  uint64_t q_full, q_free;
  uint64_t k_full[kPKStages], s_full[kPKStages];
  uint64_t v_full[kPVStages], p_full[kPVStages], pv_done[kPVStages];
  uint64_t x_full, o_free, drain;
  uint64_t idle;  // every MMA of the prefix has completed
  PageRing page[kSoftmaxWarps];  // the suffix workers' rings
  uint32_t tmem_base;
};
constexpr int kBarBytes = 1024;
static_assert(sizeof(PBars) <= kBarBytes, "barriers");
static_assert(kSoftmaxWarps * kStages * STAGE <= P_OFF_X, "the suffix workers' stages fit the rings");
static_assert(kKLoad * kStages * STAGE <= P_OFF_V, "the K loaders' lie in front of V");

// The groups and the order of the prefix work.  Group g: sequences end[g - 1]
// .. end[g] - 1, len[g] shared tokens; its pairs start at pairs[g], its units
// at units[g].  A unit is (KV head, key block, query tile); its key block has
// at most `share` key tiles when the group has several query tiles, else all.
struct SharedPlan {
  int32_t num_groups, share, ctas, total;  // total: pairs of all groups; ctas: the CTAs that share them
  int32_t end[kGroups], len[kGroups];
  int32_t pairs[kGroups + 1], units[kGroups + 1];
};
// What the join wants to know of a sequence.
struct SeqRecord {
  int32_t len, index, pairs, units;  // shared tokens; place in the group; the group's first pair and unit
  int32_t kt, mt, blocks, blen;      // the group's shape
};
// The tables that one CTA leaves in the workspace for the join.
struct SharedTables {
  int32_t *head;       // [0] total, [1] ctas of the plan
  SeqRecord *records;  // [num_seqs]
};
__host__ __device__ __forceinline__ SharedTables shared_tables(void *ws) {
  uint8_t *b = static_cast<uint8_t *>(ws);
  return {reinterpret_cast<int32_t *>(b), reinterpret_cast<SeqRecord *>(b + 16)};
}
constexpr int P_OFF_BAR = P_OFF_PLAN + ((int)sizeof(SharedPlan) + 127) / 128 * 128;
constexpr int P_OFF_PREFIX = P_OFF_BAR + kBarBytes;  // page prefix of the suffixes [num_seqs + 1]
constexpr int P_SMEM_MAX = 232448;
static_assert(P_OFF_PREFIX + (kSharedMaxSeqs + 1) * 4 + 1024 <= P_SMEM_MAX, "shared memory");

struct GroupShape {
  int kt, mt, blocks, blen;  // key tiles, query tiles, key blocks per KV head, key tiles per block (the last: fewer)
};
template <int G>
__device__ __forceinline__ GroupShape group_shape(int size, int len, int share) {
  constexpr int TQ = 128 / G;
  GroupShape s;
  s.kt = (len + 127) / 128;
  s.mt = (size + TQ - 1) / TQ;
  s.blocks = s.mt > 1 && s.kt > 0 ? (s.kt + share - 1) / share : 1;
  s.blen = (s.kt + s.blocks - 1) / s.blocks;  // <= share, and every block has a key tile
  return s;
}

// Every group's end and shared length (one warp).  A group of negative size
// counts as empty; one that runs past the sequences takes all that are left, so
// that no later group gets any of them; that one, one with a bad length and one
// with a single sequence share nothing.  Reported if asked (of the groups past
// the sequences the first).
__device__ __forceinline__ void load_groups(const SharedParams &p, SharedPlan &pl, bool report) {
  const int lane = threadIdx.x & 31;
  int carry = 0;
  for (int g0 = 0; g0 < p.num_groups; g0 += 32) {
    const int g = g0 + lane;
    int size = 0, n = 0;
    bool bad = false;
    if (g < p.num_groups) {
      size = __ldg(p.group_sizes + g);
      n = __ldg(p.prefix_lens + g);
      const bool bad_len = n < 0 || n % kBlock != 0 || n > (int64_t)p.max_blocks_per_seq * kBlock;
      bad = size < 0 || bad_len;
      size = max(0, min(size, p.num_seqs + 1));  // (the ends of all groups then fit 32 bits)
      if (bad_len || size < 2) n = 0;
    }
    int e = size;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int y = __shfl_up_sync(FULL, e, off);
      if (lane >= off) e += y;
    }
    e += carry;
    carry = __shfl_sync(FULL, e, 31);
    if (g < p.num_groups) {
      const bool over = e > p.num_seqs;
      if (report && (bad || (over && e - size <= p.num_seqs))) set_error(p.err, PA_ERR_RANGE, g);
      pl.end[g] = min(e, p.num_seqs);
      pl.len[g] = over ? 0 : n;
    }
  }
  __syncwarp();
}

// The rest of the plan from the groups' ends and lengths in it (one warp).
template <int G>
__device__ __forceinline__ void make_plan(SharedPlan &pl, int num_groups, int hkv, int grid) {
  const int lane = threadIdx.x & 31;
#pragma unroll 1
  for (int round = 0; round < 2; ++round) {  // the pairs, then (with the share known) the units
    int32_t *out = round ? pl.units : pl.pairs;
    int carry = 0;
    for (int g0 = 0; g0 < num_groups; g0 += 32) {
      const int g = g0 + lane;
      int mine = 0;
      if (g < num_groups && pl.len[g] > 0) {
        const GroupShape s = group_shape<G>(pl.end[g] - (g ? pl.end[g - 1] : 0), pl.len[g], round ? pl.share : 1);
        mine = hkv * s.mt * (round ? s.blocks : s.kt);
      }
      int incl = mine;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(FULL, incl, off);
        if (lane >= off) incl += y;
      }
      if (g < num_groups) out[g] = carry + incl - mine;
      carry += __shfl_sync(FULL, incl, 31);
    }
    if (lane == 0) {
      out[num_groups] = carry;
      if (!round) {
        pl.num_groups = num_groups;
        pl.total = carry;
        pl.ctas = carry < grid ? carry : grid;  // so that no share is empty
        pl.share = carry > 0 ? (carry + pl.ctas - 1) / pl.ctas : 1;
      }
    }
    __syncwarp();
  }
}

// CTA b's share of W pairs over n CTAs, [b W / n, (b + 1) W / n), and the CTA that owns pair y.
__device__ __forceinline__ int share_start(int b, int W, int n) { return b >= n ? W : (int)((int64_t)b * W / n); }
__device__ __forceinline__ int share_owner(int y, int W, int n) {
  return (int)((((int64_t)y + 1) * n + W - 1) / W - 1);
}

// A run of pairs of one unit: key tiles ka .. kb - 1 of query tile mt.
struct PUnit {
  int g, h, mt, ka, kb, kt_last, unit, seq0, size, len;
};
template <int G>
__device__ __forceinline__ PUnit punit_at(const SharedPlan &pl, int x, int x_end) {
  int lo = 0, hi = pl.num_groups - 1;  // the last group with pairs[g] <= x: the one that holds x
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (pl.pairs[mid] <= x) lo = mid; else hi = mid - 1;
  }
  PUnit u;
  u.g = lo;
  u.seq0 = lo ? pl.end[lo - 1] : 0;
  u.size = pl.end[lo] - u.seq0;
  u.len = pl.len[lo];
  const GroupShape s = group_shape<G>(u.size, u.len, pl.share);
  int r = x - pl.pairs[lo];
  u.h = r / (s.mt * s.kt);
  r -= u.h * s.mt * s.kt;
  const int j = r / (s.mt * s.blen);
  r -= j * s.mt * s.blen;
  const int bl = min(s.blen, s.kt - j * s.blen);
  u.mt = r / bl;
  r -= u.mt * bl;
  u.ka = j * s.blen + r;
  u.kb = u.ka + min(bl - r, x_end - x);
  u.kt_last = s.kt - 1;
  u.unit = pl.units[lo] + (u.h * s.blocks + j) * s.mt + u.mt;
  return u;
}

// The suffix's workers: consumer warp i and producer warp 8 + i.  Their numbers
// run from the last CTA down: with few pairs and pages the CTAs without pairs
// take the pages.
template <typename T, int G, bool CONSUME>
__device__ __forceinline__ bool suffix_worker(const CUtensorMap &kpage, const CUtensorMap &vmap, const SharedParams &sp,
                                              const DecodeParams &dp, const SharedPlan &pl, uint8_t *smem, PBars &bars,
                                              const int32_t *prefix) {
  const int64_t P = (int64_t)prefix[sp.num_seqs] * sp.num_kv_heads;
  const int64_t W0 = (int64_t)gridDim.x * kSoftmaxWarps, W = P < W0 ? P : W0;
  const int i = (threadIdx.x >> 5) % kSoftmaxWarps;
  const int64_t w = (int64_t)((int)gridDim.x - 1 - (int)blockIdx.x) * kSoftmaxWarps + i;
  if (w >= W) return true;
  FormArgs fa;
  fa.group_end = pl.end;
  fa.group_len = pl.len;
  fa.num_groups = sp.num_groups;
  uint8_t *stages = smem + i * (kStages * STAGE);
  if constexpr (CONSUME)
    return split_consumer16<T, G, kFormSuffix>(dp, fa, stages, bars.page[i], prefix, w, P, W);
  else
    return split_producer16<G, kFormSuffix>(kpage, vmap, dp, fa, stages, bars.page[i], prefix, w, P, W);
}

// ---- the shared kernel ----
// The roles of prefill_kernel.cuh, each looping over the CTA's runs of pairs
// with a key-tile counter c that runs on across them: warps 0..7 softmax and
// epilogue (the halves of a key tile never meet in the loop), warps 8..14
// load, warp 15 owns the tensor memory and issues the MMAs.  A run's Q is
// loaded once the previous run's last Q K^T has completed (q_free); its first
// P V product waits until the previous run's epilogue has read O (o_free).
// P goes into P V in two terms, P_hi = round(P) and P_lo = round(P - P_hi), like
// the suffix's, whatever the group's size: a sequence's output does not lose
// precision because others joined its group.  The 8 more MMAs per key tile are
// 0.26 us of tensor time.  A row's reference m_ref is kBelow under a maximum, and
// O is rescaled once a maximum is more than kTop above it.  bf16 has fp32's range:
// 0 and kRescale.  fp16 has 2^-25 to 65504, all of it used so that small weights
// are held nearly as in the suffix: P is 2^13 or more at the row's largest (a weight
// is off by 2^-38 of that one at most) and under 2^16.  The 2.9 between the two
// decide how often O is rescaled (192 sequences in three groups, fp16: 108.7 us; with
// 14 and 15 in their place 118, 13 and 15 115.5, 12 and 15 108; bf16 100.3).
// Then warp i < 8 consumes and warp 8 + i fetches the pages of a suffix worker.
template <typename T>
constexpr float kBelow = std::is_same<T, __half>::value ? 13.f : 0.f;
template <typename T>
constexpr float kTop = std::is_same<T, __half>::value ? 15.9f : kRescale;
template <typename T>
constexpr float kTopSum = std::is_same<T, __half>::value ? 61147.f : kRescaleSum;  // 2^kTop: a half-row sum bound
// The reference for a maximum mc, and what a maximum mc may reach above the
// reference: kBelow under it and kTop, while such sums are good to 2^-4; past that
// mc itself and nothing, since fp16 has no room for their roundings (weights under
// 2^-25 of the largest are then lost in fp16).
template <typename T>
__device__ __forceinline__ float reference_of(float mc) {
  return kBelow<T> == 0.f || fabsf(mc) >= 1048576.f ? mc : mc - kBelow<T>;
}
template <typename T>
__device__ __forceinline__ float top_of(float mc) {
  return kBelow<T> != 0.f && fabsf(mc) >= 1048576.f ? 0.f : kTop<T>;
}

template <typename T, int G>
__global__ void __launch_bounds__(kThreads, 1)
shared_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap kpage,
              const __grid_constant__ CUtensorMap vmap, const __grid_constant__ CUtensorMap qmap,
              const SharedParams sp, const PrefillParams p, const DecodeParams dp) {
  constexpr int TQ = 128 / G;
  constexpr bool kBF16 = std::is_same<T, __nv_bfloat16>::value;
  constexpr uint32_t IDESC_S = tc::idesc_f16(kBF16, 128, 128, false);
  constexpr uint32_t IDESC_O = tc::idesc_f16(kBF16, 128, 128, true);
  extern __shared__ uint8_t smem_raw[];
  __shared__ int warp_tot[kThreads / 32];
  uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  PBars &bars = *reinterpret_cast<PBars *>(smem + P_OFF_BAR);
  SharedPlan &pl = *reinterpret_cast<SharedPlan *>(smem + P_OFF_PLAN);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = (int)blockIdx.x;

  if (threadIdx.x == kThreads - 64) {
    tma_prefetch_desc(&kmap);
    tma_prefetch_desc(&kpage);
    tma_prefetch_desc(&vmap);
    tma_prefetch_desc(&qmap);
    mbar_init(&bars.q_full, 1);
    mbar_init(&bars.q_free, 1);
    for (int i = 0; i < kPKStages; ++i) {
      mbar_init(&bars.k_full[i], kKLoad);
      mbar_init(&bars.s_full[i], 1);
    }
    for (int i = 0; i < kPVStages; ++i) {
      mbar_init(&bars.v_full[i], kVLoad);
      mbar_init(&bars.p_full[i], kSoftmaxThreads);
      mbar_init(&bars.pv_done[i], 1);
    }
    mbar_init(&bars.x_full, kSoftmaxThreads);
    mbar_init(&bars.o_free, kSoftmaxThreads);
    mbar_init(&bars.drain, 1);
    mbar_init(&bars.idle, 1);
    for (int i = 0; i < kSoftmaxWarps; ++i) init_ring(bars.page[i]);
    fence_mbar_init();
  }
  if (warp == kWarpMma) {
    tc::tmem_alloc(&bars.tmem_base, kTmemCols);
    tc::tmem_relinquish();
  }
  // The plan and the page prefix of the suffixes, from the group metadata and the
  // lengths (like block tables they are read before the dependency wait), the same
  // in every CTA.  The last CTA reports what is wrong.
  const bool scribe = b == (int)gridDim.x - 1;
  int32_t *prefix = reinterpret_cast<int32_t *>(smem + P_OFF_PREFIX);
  if (warp == 0) load_groups(sp, pl, scribe);
  __syncthreads();
  if (warp == 0) make_plan<G>(pl, sp.num_groups, sp.num_kv_heads, (int)gridDim.x);
  scan_pages_of<kThreads>(sp.num_seqs, prefix, warp_tot, [&](int s) {
    const int ctx = __ldg(dp.context_lens + s);
    const int g = group_of(pl.end, sp.num_groups, s), len = g < sp.num_groups ? pl.len[g] : 0;
    if (ctx >= 1 && ctx <= (int64_t)sp.max_blocks_per_seq * kBlock && ctx >= len)
      return (ctx + kBlock - 1) / kBlock - len / kBlock;
    if (scribe) set_error(sp.err, PA_ERR_RANGE, s);
    return 0;
  });
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = bars.tmem_base;
  const int x0 = share_start(b, pl.total, pl.ctas), x1 = share_start(b + 1, pl.total, pl.ctas);
  bool timed_out = false;

  if (warp < kSoftmaxWarps) {
    regs_inc<kRegsSoftmax>();
    regs_taken();
    griddep_wait();
    // ---------------- softmax + epilogue (warps 0..7), run after run ----------------
    const int quad = warp & 3, ch = warp >> 2;
    const int r = quad * 32 + lane;
    const uint32_t lane_base = (uint32_t)(quad * 32) << 16;
    const uint32_t o_self = tmem + lane_base + kColO + ch * 128;
    const float sl2 = p.scale_log2;
    int c = 0, ui = 0;
    for (int x = x0; x < x1 && !timed_out; ++ui) {
      const PUnit U = punit_at<G>(pl, x, x1);
      x += U.kb - U.ka;
      const int span = U.len - 1;
      float m_ref = -INFINITY, l = 0.f;
      for (int kt = U.ka; kt < U.kb; ++kt, ++c) {
        const int sb = c & 1, ks = c % kPKStages, vs = c % kPVStages;
        if (!mbar_wait(&bars.s_full[ks], (c / kPKStages) & 1)) {
          timed_out = true;
          break;
        }
        tc::fence_after_sync();
        const uint32_t s_addr = tmem + lane_base + sb * 128 + ch * 64;
        const int kb = kt * 128 + ch * 64;  // first key of this half
        uint32_t v[2][32];
        tc::ld_32x32b_x32(s_addr, v[0]);
        tc::ld_32x32b_x32(s_addr + 32, v[1]);
        tc::wait_ld();
        const bool full = kb + 63 <= span;  // (the same in every thread of the half)
        const bool first = m_ref == -INFINITY;  // nothing accumulated for this row yet
        const bool common = __all_sync(FULL, full && !first);
        float mx = -INFINITY, ls = 0.f;
        if (common) ls = exp_pack_store<T, true>(v, s_addr, sl2, m_ref, true, kb, span);
        if (!common || ls > kTopSum<T>) {
          if (full) {
            float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int cc = 0; cc < 2; ++cc)
#pragma unroll
              for (int j = 0; j < 32; j += 4) {
                float &a = m4[cc * 2 + ((j >> 2) & 1)];
                a = fmax3(a, __uint_as_float(v[cc][j]), __uint_as_float(v[cc][j + 1]));
                a = fmax3(a, __uint_as_float(v[cc][j + 2]), __uint_as_float(v[cc][j + 3]));
              }
            mx = fmaxf(fmax3(m4[0], m4[1], m4[2]), m4[3]);
          } else {
#pragma unroll
            for (int cc = 0; cc < 2; ++cc)
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if (kb + cc * 32 + j <= span) mx = fmaxf(mx, __uint_as_float(v[cc][j]));
          }
        }
        const float mc = mx * sl2;
        const bool need = !first && mc > m_ref + top_of<T>(mc);
        const bool redo = __any_sync(FULL, need);
        if (redo) {  // warp-uniform; key tile c - 1 belongs to this run (first is false)
          if (common) tc::wait_st();
          const float m_new = reference_of<T>(mc), f = need ? ex2(m_ref - m_new) : 1.f;
          if (need) {
            l *= f;
            m_ref = m_new;
          }
          if (!mbar_wait(&bars.pv_done[(c - 1) % kPVStages], ((c - 1) / kPVStages) & 1)) {
            timed_out = true;
            break;
          }
          tc::fence_after_sync();
#pragma unroll
          for (int cc = 0; cc < 4; ++cc) {
            uint32_t ov[32];
            tc::ld_32x32b_x32(o_self + cc * 32, ov);
            tc::wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) ov[i] = __float_as_uint(__uint_as_float(ov[i]) * f);
            tc::st_32x32b_x32(o_self + cc * 32, ov);
          }
        }
        if (first) m_ref = reference_of<T>(mc);
        if (!common || redo) ls = exp_pack_store<T, true>(v, s_addr, sl2, m_ref, full, kb, span);
        l += ls;
        tc::wait_st();
        if (!mbar_wait(&bars.v_full[vs], (c / kPVStages) & 1)) {
          timed_out = true;
          break;
        }
        if (kt == U.kt_last) {  // value rows past the prefix, this half only
          const int z0 = max(U.len - kt * 128, ch * 64), z1 = ch * 64 + 64;
          uint8_t *vbase = smem + P_OFF_V + vs * 2 * kHalf;
          for (int idx = (warp & 3) * 32 + lane; idx < (z1 - z0) * 16; idx += kSoftmaxThreads / 2) {
            const int row = z0 + (idx >> 4), part = idx & 15;
            *reinterpret_cast<uint4 *>(vbase + (row >> 4) * kVPage + (part >> 3) * (kVPage / 2) + (row & 15) * 128 +
                                       (part & 7) * 16) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
        }
        tc::fence_before_sync();
        mbar_arrive(&bars.p_full[vs]);
      }
      if (timed_out) break;

      // ---- the run's state into the workspace ----
      const int cl = c - 1;
      bool ok = mbar_wait(&bars.pv_done[cl % kPVStages], (cl / kPVStages) & 1);
      tc::fence_after_sync();
      float2 *xm = reinterpret_cast<float2 *>(smem + P_OFF_X) + (ui & 1) * 256;
      if (ok) {
        xm[ch * 128 + r] = make_float2(m_ref, l);
        mbar_arrive(&bars.x_full);
        ok = mbar_wait(&bars.x_full, ui & 1);
      }
      if (!__all_sync(FULL, ok)) {  // warp-uniform before the warp-wide loads
        timed_out = true;
        break;
      }
      const float2 other = xm[(1 - ch) * 128 + r];
      const float m0 = ch == 0 ? m_ref : other.x, l0 = ch == 0 ? l : other.y;
      const float m1 = ch == 0 ? other.x : m_ref, l1 = ch == 0 ? other.y : l;
      const float M = fmaxf(m0, m1);
      const float f0 = (m0 == -INFINITY) ? 0.f : ex2(m0 - M);
      const float f1 = (m1 == -INFINITY) ? 0.f : ex2(m1 - M);
      // this thread's 64 dims of the row, both key halves, out of tensor memory; then O is free
      const uint32_t o0 = tmem + lane_base + kColO + ch * 64, o1 = o0 + 128;
      uint32_t a[64], bq[64];
      tc::ld_32x32b_x32(o0, *reinterpret_cast<uint32_t(*)[32]>(a));
      tc::ld_32x32b_x32(o0 + 32, *reinterpret_cast<uint32_t(*)[32]>(a + 32));
      tc::ld_32x32b_x32(o1, *reinterpret_cast<uint32_t(*)[32]>(bq));
      tc::ld_32x32b_x32(o1 + 32, *reinterpret_cast<uint32_t(*)[32]>(bq + 32));
      tc::wait_ld();
      tc::fence_before_sync();
      mbar_arrive(&bars.o_free);
      if (U.mt * TQ + r / G < U.size) {  // rows past the group's last sequence hold nothing
        const int64_t slot = U.unit + b;
        float4 *dst = reinterpret_cast<float4 *>(sp.ws_o) + (slot * 32 + ch * 16) * 128 + r;  // [dims / 4][row]
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          float y[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            y[e] = __uint_as_float(a[4 * i + e]) * f0 + __uint_as_float(bq[4 * i + e]) * f1;
          dst[i * 128] = make_float4(y[0], y[1], y[2], y[3]);
        }
        if (ch == 0) sp.ws_ml[slot * 128 + r] = make_float2(M, l0 * f0 + l1 * f1);
      }
    }
    // ---------------- the suffix: the worker whose producer is warp 8 + warp ----------------
    if (!timed_out && !suffix_worker<T, G, true>(kpage, vmap, sp, dp, pl, smem, bars, prefix)) timed_out = true;
    regs_dec<128>();
  } else {
    // every loader and MMA warp runs this one decrease (setmaxnreg acts on whole warpgroups)
    regs_dec<kRegsOther>();
    int key_tiles = 0;  // a loader warp's, over all runs
    if (warp != kWarpMma) {
      // ---------------- loader warps ----------------
      // Warps 0 .. 3 load K, each 4 of a key tile's 16 boxes (the 64-dim half b %
      // 2 of page b / 2), warps 4 .. 6 V, pages lw - 4, + 3, .., from parallel
      // lanes.  The block ids of 4 key tiles sit one per lane, the next 4 tiles'
      // already on their way: a table read per tile would hold up every copy by
      // an L2 trip.
      const int lw = warp - kWarpLoad0;
      const bool for_k = lw < kKLoad;
      const int box = for_k ? lw + kKLoad * lane : lw - kKLoad + kVLoad * lane;
      const int boxes = for_k ? 16 : 8, page = for_k ? box >> 1 : box;
      const int32_t *bt = nullptr;
      int npages = 0, wbase = 0;
      int32_t win = -1, win_next = -1;
      auto ids_from = [&](int base) { return base + lane < npages ? __ldg(bt + base + lane) : -1; };
      auto open_run = [&](const PUnit &U) {
        bt = p.block_tables + (int64_t)U.seq0 * p.max_blocks_per_seq;  // the group's first sequence
        npages = U.len / kBlock;
        wbase = U.ka * 8;
        win = ids_from(wbase);
        win_next = ids_from(wbase + 32);
      };
      // The id of a key tile's page (every lane; -1 past the prefix).
      auto id_of = [&](int t, int page) { return __shfl_sync(FULL, win, (t * 8 + page - wbase) & 31); };
      PUnit U;
      if (x0 < x1) {
        U = punit_at<G>(pl, x0, x1);
        open_run(U);
      }
      griddep_wait();  // Q, K and V may come from the kernels before
      if (scribe) {  // the join's tables (after the wait: the previous call's join may still read them)
        const SharedTables tb = shared_tables(sp.tables);
        const int i0 = lw * 32 + lane;
        if (i0 == 0) {
          tb.head[0] = pl.total;
          tb.head[1] = pl.ctas;
        }
        for (int i = i0; i <= sp.num_seqs; i += kLoadWarps * 32) {
          dp.meta[i] = prefix[i];
          if (i == sp.num_seqs) break;
          SeqRecord r = {};
          const int g = group_of(pl.end, sp.num_groups, i);
          if (g < sp.num_groups && pl.len[g] > 0) {
            const int seq0 = g ? pl.end[g - 1] : 0;
            const GroupShape sh = group_shape<G>(pl.end[g] - seq0, pl.len[g], pl.share);
            r = {pl.len[g], i - seq0, pl.pairs[g], pl.units[g], sh.kt, sh.mt, sh.blocks, sh.blen};
          }
          tb.records[i] = r;
        }
      }
      int c = 0, ui = 0, issued = 0;
      for (int x = x0; x < x1 && !timed_out; ++ui) {
        if (ui > 0) {
          U = punit_at<G>(pl, x, x1);
          open_run(U);
        }
        x += U.kb - U.ka;
        if (lw == 0 && lane == 0) {
          if (ui > 0 && !mbar_wait(&bars.q_free, (ui - 1) & 1)) timed_out = true;
          // (rows past the group belong to other sequences or read as zeros; nothing is stored for them)
          mbar_arrive_expect_tx(&bars.q_full, 2 * kHalf);
          tma_load_3d(smem + P_OFF_Q, &qmap, &bars.q_full, 0, U.h * G, U.seq0 + U.mt * TQ);
          tma_load_3d(smem + P_OFF_Q + kHalf, &qmap, &bars.q_full, 64, U.h * G, U.seq0 + U.mt * TQ);
        }
        timed_out = __any_sync(FULL, timed_out);
        for (int t = U.ka; t < U.kb && !timed_out; ++t, ++c) {
          if (t * 8 >= wbase + 32) {
            wbase += 32;
            win = win_next;
            win_next = ids_from(wbase + 32);
          }
          const int id = id_of(t, page);
          const bool in = box < boxes && t * 8 + page < npages;  // (the softmax warps zero V past the prefix)
          const bool ok = in && (unsigned)id < (unsigned)p.num_blocks;
          const unsigned okmask = __ballot_sync(FULL, ok);
          const int st = for_k ? c % kPKStages : c % kPVStages;
          // the stage is free: S of the key tile two before, P V of the one three before
          if (for_k ? c >= kPKStages && !mbar_wait(&bars.s_full[st], ((c - kPKStages) / kPKStages) & 1)
                    : c >= kPVStages && !mbar_wait(&bars.pv_done[st], ((c - kPVStages) / kPVStages) & 1))
            timed_out = true;
          if (__any_sync(FULL, timed_out)) {
            timed_out = true;
            break;
          }
          const uint32_t bytes = for_k ? 2048u : (uint32_t)kVPage;
          uint8_t *dst = for_k ? smem + P_OFF_K + st * 2 * kHalf + (box & 1) * kHalf + page * 2048
                               : smem + P_OFF_V + st * 2 * kHalf + page * kVPage;
          uint64_t *bar = for_k ? &bars.k_full[st] : &bars.v_full[st];
          if (in && !ok) {  // rare: keep the products finite
            set_error(p.err, PA_ERR_RANGE, U.seq0);
            for (uint32_t i = 0; i < bytes / 16; ++i) reinterpret_cast<uint4 *>(dst)[i] = make_uint4(0, 0, 0, 0);
            fence_proxy_async_smem();
          }
          __syncwarp();  // the zeroed boxes are written before the arrival below releases them
          if (lane == 0) mbar_arrive_expect_tx(bar, (uint32_t)__popc(okmask) * bytes);
          __syncwarp();
          if (ok) {
            if (for_k)
              tma_load_4d(dst, &kmap, bar, (box & 1) * 64, U.h, 0, id);
            else
              tma_load_5d(dst, &vmap, bar, 0, 0, 0, U.h, id);
          }
          issued = c + 1;
        }
      }
      key_tiles = c;
      if (timed_out) {  // a short, bounded chance for this warp's copies in flight to land
        if (lw == 0 && ui > 0) mbar_wait(&bars.q_full, (ui - 1) & 1, kWaitLimitNs / 8);
        const int n = for_k ? kPKStages : kPVStages;
        for (int t = issued - n > 0 ? issued - n : 0; t < issued; ++t)
          mbar_wait(for_k ? &bars.k_full[t % n] : &bars.v_full[t % n], (t / n) & 1, kWaitLimitNs / 8);
      }
    } else {
      // ---------------- MMA issuer (warp-uniform loop, one elected lane issues) ----------------
      griddep_wait();  // (for the suffix's pages)
      const bool leader = elect_one();
      auto wait_all = [&](uint64_t *bar, uint32_t parity) { return __all_sync(FULL, mbar_wait(bar, parity)) != 0; };
      const uint64_t qdesc = tc::desc_sw128(smem_u32(smem + P_OFF_Q), 16, 1024);
      const uint64_t kdesc0 = tc::desc_sw128(smem_u32(smem + P_OFF_K), 16, 1024);
      const uint64_t vdesc0 = tc::desc_sw128(smem_u32(smem + P_OFF_V), kVPage / 2, 1024);
      constexpr uint64_t kStageStep = (2 * kHalf) >> 4;
      constexpr uint64_t kHalfStep = kHalf >> 4;
      // the P V product of key tile pc (pending), issued once P is ready
      int pc = -1, p_run = 0;
      bool p_first = false;
      auto issue_pv = [&]() -> bool {
        const int jv = pc % kPVStages;
        if (!wait_all(&bars.p_full[jv], (pc / kPVStages) & 1)) return false;
        if (p_first && p_run > 0 && !wait_all(&bars.o_free, (p_run - 1) & 1)) return false;
        tc::fence_after_sync();
        const uint64_t vdesc = vdesc0 + (uint64_t)jv * kStageStep;
        const uint32_t p_col = tmem + (pc & 1) * 128;
        const uint32_t acc0 = p_first ? 0u : 1u;
        if (leader) {
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) {
            const uint32_t o_col = tmem + kColO + (kk >> 2) * 128;
            const uint32_t a_hi = p_col + 32 * (kk >> 1) + 8 * (kk & 1);
            const uint64_t bdesc = vdesc + (uint64_t)(kk * (kVPage >> 4));
            tc::mma_f16_ts(o_col, a_hi, bdesc, IDESC_O, (kk & 3) > 0 ? 1u : acc0);
            tc::mma_f16_ts(o_col, a_hi + 16, bdesc, IDESC_O, 1u);
          }
          tc::commit(&bars.pv_done[jv]);
        }
        __syncwarp();
        return true;
      };
      int c = 0, ui = 0;
      for (int x = x0; x < x1 && !timed_out; ++ui) {
        const PUnit U = punit_at<G>(pl, x, x1);
        x += U.kb - U.ka;
        // the previous run's last P V first: its epilogue need not wait for this run's Q and first K
        if (pc >= 0) {
          if (!issue_pv()) {
            timed_out = true;
            break;
          }
          pc = -1;
        }
        if (!wait_all(&bars.q_full, ui & 1)) {
          timed_out = true;
          break;
        }
        for (int kt = U.ka; kt < U.kb; ++kt, ++c) {
          const int ks = c % kPKStages;
          if (!wait_all(&bars.k_full[ks], (c / kPKStages) & 1)) {
            timed_out = true;
            break;
          }
          tc::fence_after_sync();
          const uint64_t kdesc = kdesc0 + (uint64_t)ks * kStageStep;
          const uint32_t s_col = tmem + (c & 1) * 128;
          if (leader) {
            tc::mma_f16(s_col, qdesc, kdesc, IDESC_S, 0u);
#pragma unroll
            for (int kk = 1; kk < 8; ++kk) {
              const uint64_t off = (uint64_t)((kk >> 2) * kHalfStep + (kk & 3) * 2);
              tc::mma_f16(s_col, qdesc + off, kdesc + off, IDESC_S, 1u);
            }
            tc::commit(&bars.s_full[ks]);
            if (kt == U.kb - 1) tc::commit(&bars.q_free);  // the run's Q is no longer read
          }
          __syncwarp();
          if (pc >= 0 && !issue_pv()) {
            timed_out = true;
            break;
          }
          pc = c;
          p_run = ui;
          p_first = kt == U.ka;
        }
      }
      if (!timed_out && pc >= 0 && !issue_pv()) timed_out = true;
      if (!timed_out && leader && x0 < x1) tc::commit(&bars.idle);
      __syncwarp();
      if (timed_out) {  // every MMA issued so far, bounded, before the tensor memory is freed
        if (leader) tc::commit(&bars.drain);
        __syncwarp();
        mbar_wait(&bars.drain, 0, kWaitLimitNs / 8);
      }
    }
    // ---------------- the suffix: this warp fetches consumer warp - 8's pages ----------------
    // The rings are idle once every MMA has completed: each copy was consumed by
    // one.  The K loaders' stages lie where Q and K were, idle when the last Q K^T
    // has completed (they have seen the one two before, on the same barrier).
    if (x0 < x1 && !timed_out) {
      const int last = key_tiles - 1;
      if (!(warp < kWarpLoad0 + kKLoad ? mbar_wait(&bars.s_full[last % kPKStages], (last / kPKStages) & 1)
                                       : mbar_wait(&bars.idle, 0)))
        timed_out = true;
    }
    timed_out = __any_sync(FULL, timed_out);
    if (!timed_out && !suffix_worker<T, G, false>(kpage, vmap, sp, dp, pl, smem, bars, prefix)) timed_out = true;
    regs_wait_taken();  // (the softmax warps hold their registers by now)
    regs_inc<128>();
  }
  if (timed_out) set_error(p.err, PA_ERR_TIMEOUT, b);
  tc::fence_before_sync();
  __syncthreads();
  if (warp == kWarpMma) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, kTmemCols);
  }
}

// ---- the join ----
// Warp (s, h, part): lane (gg, quad) adds up head gg's dims 4 quad .. 4 quad +
// 3 over the pieces of the prefix and of the suffix.
template <typename T, int G>
__global__ void __launch_bounds__(128)
shared_join_kernel(const SharedParams sp, const DecodeParams p) {
  constexpr int TQ = 128 / G, QW = 32 / G;  // dim quads per warp
  griddep_wait();
  griddep_launch_dependents();  // (it writes nothing that a kernel may read before its own wait)
  const int wid = blockIdx.x * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int hkv = p.num_kv_heads;
  if (wid >= p.num_seqs * hkv * G) return;
  const int part = wid % G, item = wid / G, s = item / hkv, h = item % hkv;
  const int gg = lane % G, quad = part * QW + lane / G;
  const SharedTables tb = shared_tables(sp.tables);
  const int4 ra = __ldcg(reinterpret_cast<const int4 *>(tb.records + s));
  const int4 rb = __ldcg(reinterpret_cast<const int4 *>(tb.records + s) + 1);
  const SeqRecord rec = {ra.x, ra.y, ra.z, ra.w, rb.x, rb.y, rb.z, rb.w};
  const int2 head = __ldcg(reinterpret_cast<const int2 *>(tb.head));
  const int ctx = __ldg(p.context_lens + s), len = rec.len;
  const int m0 = __ldcg(p.meta + s), m1 = __ldcg(p.meta + s + 1), mn = __ldcg(p.meta + p.num_seqs);
  if (ctx < 1 || ctx > (int64_t)p.max_blocks_per_seq * kBlock || ctx < len) return;  // reported; its rows are left
  // the suffix's pieces: slots item + wf ..
  const int pages = m1 - m0;
  const int64_t P = (int64_t)mn * hkv;
  const int64_t W = P < p.num_workers ? P : p.num_workers;
  const int64_t A = (int64_t)hkv * m0 + (int64_t)h * pages;
  const int wf = pages ? worker_of(A, P, W) : 0;
  const int nfs = pages ? worker_of(A + pages - 1, P, W) - wf + 1 : 0;
  if (len == 0 && nfs <= 1) return;  // the suffix worker wrote the output
  JoinState js;
  constexpr int U = kJoinPieces;
  for (int f0 = 0; f0 < nfs; f0 += U) {
    float2 ml[U];
    float4 o[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      ml[u] = make_float2(-INFINITY, 0.f);
      o[u] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (f0 + u < nfs) {
        const int64_t slot = ((int64_t)item + wf + f0 + u) * G + gg;
        ml[u] = __ldcg(reinterpret_cast<const float2 *>(p.ws_ml + slot * 2));
        o[u] = __ldcg(reinterpret_cast<const float4 *>(p.ws_o + slot * kHeadDim + 4 * quad));
      }
    }
    js.add(ml, o);
  }
  if (len > 0) {
    const int mt = rec.index / TQ, row = (rec.index % TQ) * G + gg;
    for (int j = 0; j < rec.blocks; ++j) {
      const int bl = min(rec.blen, rec.kt - j * rec.blen);
      const int xa = rec.pairs + (h * rec.kt + j * rec.blen) * rec.mt + mt * bl;  // the unit's first pair
      const int unit = rec.units + (h * rec.blocks + j) * rec.mt + mt;
      const int ff = share_owner(xa, head.x, head.y), fl = share_owner(xa + bl - 1, head.x, head.y);
      for (int f0 = ff; f0 <= fl; f0 += U) {
        float2 ml[U];
        float4 o[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          ml[u] = make_float2(-INFINITY, 0.f);
          o[u] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (f0 + u <= fl) {
            const int64_t slot = unit + f0 + u;
            ml[u] = __ldcg(sp.ws_ml + slot * 128 + row);
            o[u] = __ldcg(reinterpret_cast<const float4 *>(sp.ws_o) + (slot * 32 + quad) * 128 + row);
          }
        }
        js.add(ml, o);
      }
    }
  }
  js.store(reinterpret_cast<T *>(p.out) + ((int64_t)s * p.num_q_heads + h * G + gg) * kHeadDim + 4 * quad);
}

template <typename T, int G>
cudaError_t launch_shared_typed(const SharedParams &sp, const PrefillParams &pp, const DecodeParams &dp0,
                                const CUtensorMap *maps, int sms, cudaStream_t stream) {
  DecodeParams dp = dp0;
  static KernelSetup setup;
  const int smem = 1024 + P_OFF_PREFIX + (dp.num_seqs + 1) * 4;
  cudaError_t e = kernel_setup(setup, shared_kernel<T, G>, smem, kThreads, nullptr);
  if (e != cudaSuccess) return e;
  dp.num_workers = sms * kSoftmaxWarps;
  e = launch_pdl(shared_kernel<T, G>, dim3(sms), dim3(kThreads), smem, stream, maps[0], maps[1], maps[2], maps[3], sp,
                 pp, dp);
  if (e != cudaSuccess) return e;
  return launch_pdl(shared_join_kernel<T, G>, dim3((dp.num_seqs * dp.num_q_heads + 3) / 4), dim3(128), 0, stream, sp,
                    dp);
}

}  // namespace

namespace {
struct SharedLayout {
  size_t tables, decode, ml, o, total;
};
SharedLayout shared_layout(int num_seqs, int num_groups, int num_q_heads, int num_kv_heads, int sms) {
  const size_t group = num_q_heads / num_kv_heads;
  // pieces: at most one per unit and one more per CTA; units: at most one per CTA and one per query tile
  const size_t tiles = (size_t)num_kv_heads * (num_groups + (size_t)num_seqs * group / 128);
  const size_t slots = 2 * (size_t)sms + tiles;
  auto up = [](size_t n) { return (n + 255) & ~(size_t)255; };
  SharedLayout l;
  l.tables = 0;
  l.decode = up(16 + (size_t)num_seqs * sizeof(SeqRecord));
  l.ml = l.decode + up(decode_workspace_counters_offset(num_seqs, num_q_heads, num_kv_heads));
  l.o = l.ml + up(slots * 128 * sizeof(float2));
  l.total = l.o + slots * 128 * kHeadDim * sizeof(float);
  return l;
}
}  // namespace

size_t shared_workspace_bytes(int num_seqs, int num_groups, int num_q_heads, int num_kv_heads, int sms) {
  return shared_layout(num_seqs, num_groups, num_q_heads, num_kv_heads, sms).total;
}

cudaError_t launch_decode_shared(SharedParams sp, const PrefillParams &pp, DecodeParams dp, void *workspace,
                                 const CUtensorMap *maps, int dtype, int group, int sms, cudaStream_t stream) {
  const SharedLayout l = shared_layout(dp.num_seqs, sp.num_groups, dp.num_q_heads, dp.num_kv_heads, sms);
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  sp.tables = ws + l.tables;
  sp.ws_ml = reinterpret_cast<float2 *>(ws + l.ml);
  sp.ws_o = reinterpret_cast<float *>(ws + l.o);
  decode_workspace_carve(ws + l.decode, SIZE_MAX, dp.num_seqs, dp.num_q_heads, dp.num_kv_heads, dp);
#define PA_SHARED_CASE(T, G) \
  if (group == G) return launch_shared_typed<T, G>(sp, pp, dp, maps, sms, stream);
  if (dtype == PA_BF16) {
    PA_SHARED_CASE(__nv_bfloat16, 1)
    PA_SHARED_CASE(__nv_bfloat16, 2)
    PA_SHARED_CASE(__nv_bfloat16, 4)
    PA_SHARED_CASE(__nv_bfloat16, 8)
  } else {
    PA_SHARED_CASE(__half, 1)
    PA_SHARED_CASE(__half, 2)
    PA_SHARED_CASE(__half, 4)
    PA_SHARED_CASE(__half, 8)
  }
#undef PA_SHARED_CASE
  return cudaErrorInvalidValue;
}

}  // namespace pa

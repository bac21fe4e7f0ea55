// Paged GQA attention of drafted tokens that form a tree behind each sequence's
// cached context, for sm_103a (speculative decoding).
//
//   out[i][g] = softmax_j(scale q[i][g] . K_j) V_j over the L - n committed keys,
//               token i's ancestors in the tree, and i itself (the n drafted
//               tokens' K and V are the last n of the L cached ones)
//
// The n x G query rows of a sequence for one KV head against its keys are a
// matrix product: query tiles of 128 rows (128 / G tokens x the G heads), key
// tiles of 128 keys, on the tcgen05 tensor cores.  NT query tiles (1 or 2) form a
// group, taken by NT CTAs at the same time, a worker, so that one of them reads the
// keys from HBM and the other from L2 (each on its own: nothing passes between
// them).  All (group, key tile) pairs of the call are dealt evenly to the workers
// (one CTA per SM), so one long sequence or many short ones fill the GPU alike.  A
// worker's share is a row of runs: consecutive key tiles of one group.  A run that
// holds all keys of its group writes the outputs; a group cut between workers
// leaves a piece (m, l, o) per CTA, joined by a second kernel.  Only a worker's
// first and last run can be such pieces, so 2 slots per CTA hold them whatever the
// batch.  With several groups to a sequence the key range is cut into blocks at
// least as long as a share, the groups of a block next to each other in the order,
// so that the workers that need the same keys run at the same time.
//
// A pair is 64 KB of K and V, 1.47 us of an SM's share of HBM, beside 0.78 us of
// tensor time (P in two terms).  To keep the copies running across a change of
// runs the queries do not lie in shared memory but as the A operand in tensor
// memory, two tiles of them, fetched a run ahead: the rings of K and V have three
// key tiles each.  One warpgroup computes P, one prepares the next run's queries
// and masks, one looks at the drafted values and writes the outputs, while the next
// run is under way.  What a change of runs must not do: touch local memory (beside
// 227 KB of shared memory the L1 is small; spills of 250 bytes cost 5 us a change),
// read rows 16 bytes a lane (the queries: 124 against 101 us for 32 sequences of up
// to 8192), or signal behind stores (an arrival waits until they are in L2).
//
// The mask: per token a bit for each drafted token that it sees, found by a walk up
// the tree a run ahead; 128 bits of it per key tile that reaches the drafted keys.
// A row always sees itself.  A drafted value that is infinite or NaN must not reach
// the rows that do not see it (0 x inf): such values are zeroed in shared memory and
// the rows that see them made NaN.
//
// Measured (CUDA graphs): 192 sequences of up to 2900 tokens, chains of 1 to 8 drafts,
// 16 / 8 heads, bf16: 188 us, 0.94 of the copy rate; 32 of 100 to 8192, 16 to 32 drafts,
// 32 / 8: 96.3, 0.80; 5 of 40000 to 100001, 9 to 13 drafts, 32 / 4: 133, 0.86; 8 of 8000
// to 32768, 60 to 64 drafts (two query tiles), 32 / 8, fp16: 198, 0.54 (in bursts at 2
// GHz; 232 where thousands of calls in a row bring the SMs to 1.5 GHz under the power
// cap, which the calls that HBM bounds do not feel); one of 777, 5 drafts: 11.0, a chain of latencies (plan, one key tile, join).  With one query tile
// 152 equal contexts of 8192 run at 0.95; ragged batches lose what the SMs' unequal
// speeds leave at the end.  With two a pair takes 1.3 us, the tensor pipe 67 % busy: P
// waits for S, S for the P V that has left its columns, and tensor memory's loads and
// stores take turns with the products (of 202, without the low term's product 170,
// without its stores 185, without the maximum's pass 184, without exponentials 199).
// P V goes in halves of 64 keys, the first as soon as its P is ready (3 %, and 11.2 to
// 11.0).  More warps on the softmax gain nothing: the maxima found by the epilogue's
// warps cost 1 %, half of the keys each with the maxima exchanged 10; units of 64 keys,
// four of them in tensor memory, 28.
#include <limits.h>

#include "decode_mma.cuh"
#include "piece_softmax.cuh"

namespace pa {
namespace {

// Warps 0..3 softmax; 4..7 drafted values and epilogue; 8 and 9 load K, 10 V, 11 issues the
// MMAs; 12..15 queries and masks.
constexpr int kTThreads = 512, kTWarpEpi = 4, kTWarpLoad0 = 8, kTKLoad = 2, kTWarpMma = 11, kTWarpPrep = 12;
// Registers: 128 per thread at launch, given and taken by warpgroups (together what the
// launch holds, so an increase never waits forever).
constexpr int kTRegsSoftmax = 168, kTRegsEpi = 136, kTRegsLoad = 96, kTRegsPrep = 112;
static_assert(128 * (kTRegsSoftmax + kTRegsEpi + kTRegsLoad + kTRegsPrep) <= 65536, "register split fits the launch");
constexpr int kTStages = 3;  // of K, and of V (two CTAs per SM of one stage each: 1.7 to 1.95 us a pair, not 1.55)
constexpr int T_OFF_K = 0;
constexpr int T_OFF_V = T_OFF_K + kTStages * 2 * kHalf;
constexpr int kTMaskWords = PA_MAX_TREE_LEN / 32;
constexpr int T_OFF_MASK = T_OFF_V + kTStages * 2 * kHalf;     // [run parity][token][kTMaskWords]
constexpr int T_OFF_X = T_OFF_MASK + 2 * 128 * kTMaskWords * 4;  // (m, l) [run parity][128]
constexpr int T_OFF_STAGE = T_OFF_X + 2 * 128 * 8;  // 1 KB per warp of 4..7 and 12..15: rows on their way out and in
constexpr int T_OFF_BAR = T_OFF_STAGE + 8 * kStageBytes;
// Tensor memory: two of S / P, O, two of Q (64 columns of packed pairs).
constexpr uint32_t kTColO = 256, kTColQ = 384;
// What the other roles want to know of a run: published by the first loader warp a run
// ahead of its own (kb 0: no more).  8 would do: when run u + 1 is published, of runs of one
// key tile, tile u - 1 was loaded, so S of tile u - 4 is done, P V of tile u - 6 was issued
// and O of run u - 7 has been read.
constexpr int kTRuns = 10;
struct TRunInfo {
  int32_t ka, kb, start, len;  // its key tiles; the sequence's first drafted key, and keys
  int32_t row, live_rows;      // row of the query tile's first token in q and out; rows of queries
  int32_t h, s, tok0;          // KV head, sequence, the tile's first token in the tree
  int32_t whole, first;        // all keys of the group; the worker's first run
};
struct TBars {
  uint64_t k_full[kTStages], k_free[kTStages];
  uint64_t v_full[2][kTStages];  // [1]: a key tile that reaches the drafted keys (looked at before it is used)
  uint64_t v_free[kTStages];
  uint64_t s_full[2], p_full[2][2], o_done;  // p_full: per half of the keys; o_done: P V of a key tile added to O
  uint64_t q_full[2];          // per run: its queries and masks are in place
  uint64_t look[kTStages];     // per key tile that reaches the drafted keys: its values are fit for P V
  uint64_t x_full[2], run_done, o_free;  // per run: (m, l) written; every P V done; O read
  uint64_t side, drain;
  uint32_t bad[2][kTMaskWords];  // per run parity: drafted tokens whose values are not finite
  uint64_t run_full[kTRuns];
  TRunInfo info[kTRuns];
  uint32_t tmem_base;
  int32_t warp_tot[kTThreads / 32];
};
constexpr int T_BAR_BYTES = 960;
static_assert(sizeof(TBars) <= T_BAR_BYTES, "barriers");
constexpr int T_OFF_PLAN = T_OFF_BAR + T_BAR_BYTES;  // rows [num_seqs + 1], pairs [num_seqs + 1]
static_assert(T_OFF_PLAN + 2 * (kTreeMaxSeqs + 1) * 4 <= 232448, "shared memory");

// The order of the work: sequence s has rows[s + 1] - rows[s] drafted tokens and
// the pairs pairs[s] .. pairs[s + 1] - 1 (none for a sequence that is refused).
struct TreePlan {
  const int32_t *rows, *pairs, *context_lens;
  int32_t num_seqs, num_kv_heads, total, workers, share, cost;
};

// Part j of W things over n, [j W / n, (j + 1) W / n), and the part that holds thing y.
__device__ __forceinline__ int part_start(int j, int W, int n) { return j >= n ? W : (int)((int64_t)j * W / n); }
__device__ __forceinline__ int part_owner(int y, int W, int n) {
  return (int)((((int64_t)y + 1) * n + W - 1) / W - 1);
}

// A run of pairs: tiles va .. vb - 1 of group g of (sequence s, KV head h), within the unit
// of that group and key block j (tiles k0 .. k1 - 1).  A run costs more than its key
// tiles (queries, masks, epilogue): in the deal a group counts for `cost` tiles more,
// which come first and hold no keys; all of these numbers count them.
struct TRun {
  int s, h, g, j, va, vb, k0, k1;
  int kt, groups, blocks;  // the sequence's tiles, groups, key blocks
  int n, len, row0;        // its drafted tokens, keys, and first row
  // its key tiles
  __device__ __forceinline__ int ka(int cost) const { return max(va - cost, 0); }
  __device__ __forceinline__ int kb(int cost) const { return max(vb - cost, 0); }
  __device__ __forceinline__ bool whole(int cost) const { return blocks == 1 && va <= cost && vb == kt; }
  template <int TG>
  __device__ __forceinline__ void open_sequence(const TreePlan &pl) {
    row0 = pl.rows[s];
    n = pl.rows[s + 1] - row0;
    len = __ldg(pl.context_lens + s);
    kt = (len + 127) / 128 + pl.cost;
    groups = (n + TG - 1) / TG;
    blocks = groups > 1 ? max(kt / pl.share, 1) : 1;
  }
  __device__ __forceinline__ void open_block() {
    k0 = blocks == 1 ? 0 : part_start(j, kt, blocks);
    k1 = blocks == 1 ? kt : part_start(j + 1, kt, blocks);
  }
  // The run that holds pair x, of a share that ends at x_end.
  template <int TG>
  __device__ __forceinline__ void at(const TreePlan &pl, int x, int x_end) {
    int lo = 0, hi = pl.num_seqs - 1;  // the last sequence with pairs[s] <= x: the one that holds x
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (pl.pairs[mid] <= x) lo = mid; else hi = mid - 1;
    }
    s = lo;
    open_sequence<TG>(pl);
    int r = x - pl.pairs[s];
    h = r / (groups * kt);
    r -= h * groups * kt;
    j = part_owner(r / groups, kt, blocks);  // block j's pairs start at groups * (its first key tile)
    open_block();
    r -= groups * k0;
    g = r / (k1 - k0);
    va = k0 + r - g * (k1 - k0);
    vb = min(k1, va + (x_end - x));
  }
  // The next one, from pair x on (the last ended with its unit).
  template <int TG>
  __device__ __forceinline__ void next(const TreePlan &pl, int x, int x_end) {
    if (++g == groups) {
      g = 0;
      if (++j == blocks) {
        j = 0;
        if (++h == pl.num_kv_heads) {
          h = 0;
          do ++s;
          while (pl.pairs[s + 1] == pl.pairs[s]);
          open_sequence<TG>(pl);
        }
      }
      open_block();
    }
    va = k0;
    vb = min(k1, va + (x_end - x));
  }
};

// What the join wants to know of the group that starts in a worker's last run and
// ends in others (rows 0: none).
struct JoinRecord {
  int32_t rows, row0, h;      // query rows, first token's row in out, KV head
  int32_t pairs0, kt, groups, g, blocks, total, workers, pad[2];
};
static_assert(sizeof(JoinRecord) == 48, "three 16-byte loads");

// Whether one of the two 16-bit values of u is infinite or NaN.
template <typename T>
__device__ __forceinline__ bool not_finite2(uint32_t u) {
  constexpr uint32_t E = std::is_same<T, __half>::value ? 0x7c00u : 0x7f80u;
  return (u & E) == E || ((u >> 16) & E) == E;
}

// P = 2^(S * scale_log2 - m) of 32 keys as two terms of T over their S columns: 16
// columns of P_hi pairs, then 16 of P_lo.  Adds P to the sums.
template <typename T>
__device__ __forceinline__ void exp_pack_store32(const uint32_t (&v)[32], uint32_t s_addr, float sl2, float m,
                                                 float2 (&ls)[2]) {
  const float2 sl2v = make_float2(sl2, sl2), negm = make_float2(-m, -m), neg1 = make_float2(-1.f, -1.f);
  uint32_t hi[16], lo[16];
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const float2 e = __ffma2_rn(make_float2(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1])), sl2v, negm);
    const float2 pr = make_float2(ex2(e.x), ex2(e.y));
    ls[j & 1] = __fadd2_rn(ls[j & 1], pr);
    hi[j] = Pack<T>::from_f2(pr.x, pr.y);
    const float2 rest = __ffma2_rn(Pack<T>::to_f2(hi[j]), neg1, pr);  // P - P_hi, exact
    lo[j] = Pack<T>::from_f2(rest.x, rest.y);
  }
  tc::st_32x32b_x16(s_addr, hi);
  tc::st_32x32b_x16(s_addr + 16, lo);
}
// Scores that the row does not see become -inf.
__device__ __forceinline__ void hide32(uint32_t (&v)[32], uint32_t seen) {
#pragma unroll
  for (int j = 0; j < 32; ++j)
    if (!((seen >> j) & 1)) v[j] = 0xff800000u;
}
__device__ __forceinline__ float max64(const uint32_t (&a)[32], const uint32_t (&b)[32], float m) {
  float m4[4] = {m, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
  for (int j = 0; j < 32; j += 4) {
    m4[0] = fmax3(m4[0], __uint_as_float(a[j]), __uint_as_float(a[j + 1]));
    m4[1] = fmax3(m4[1], __uint_as_float(b[j]), __uint_as_float(b[j + 1]));
    m4[2] = fmax3(m4[2], __uint_as_float(a[j + 2]), __uint_as_float(a[j + 3]));
    m4[3] = fmax3(m4[3], __uint_as_float(b[j + 2]), __uint_as_float(b[j + 3]));
  }
  return fmaxf(fmax3(m4[0], m4[1], m4[2]), m4[3]);
}

// The roles loop over the CTA's runs, with a key-tile counter c that runs on across
// them: tile c has stage c % 3 of K and V and S / P columns c % 2.  Softmax warps whose
// 32 rows hold no query of the run (a small tree's tile is mostly empty) only keep pace
// on the barriers.
template <typename T, int G, int NT>
__global__ void __launch_bounds__(kTThreads, 1)
attn_tree_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                 const __grid_constant__ TreeParams p) {
  constexpr int TQ = 128 / G, TG = NT * TQ;  // tokens per query tile and group
  constexpr bool kBF16 = std::is_same<T, __nv_bfloat16>::value;
  constexpr uint32_t IDESC_S = tc::idesc_f16(kBF16, 128, 128, false);
  constexpr uint32_t IDESC_O = tc::idesc_f16(kBF16, 128, 128, true);
  extern __shared__ __align__(1024) uint8_t tree_smem[];
  uint8_t *smem = tree_smem;
  TBars &bars = *reinterpret_cast<TBars *>(smem + T_OFF_BAR);
  int32_t *rows = reinterpret_cast<int32_t *>(smem + T_OFF_PLAN), *pairs = rows + p.num_seqs + 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int worker = (int)blockIdx.x / NT, sub = (int)blockIdx.x % NT;

  if (threadIdx.x == kTThreads - 64) {
    tma_prefetch_desc(&kmap);
    tma_prefetch_desc(&vmap);
    for (int i = 0; i < kTStages; ++i) {
      mbar_init(&bars.k_full[i], kTKLoad);
      mbar_init(&bars.k_free[i], 1);
      mbar_init(&bars.v_full[0][i], 1);
      mbar_init(&bars.v_full[1][i], 1);
      mbar_init(&bars.v_free[i], 1);
      mbar_init(&bars.look[i], 128);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars.s_full[i], 1);
      mbar_init(&bars.p_full[i][0], 128);
      mbar_init(&bars.p_full[i][1], 128);
      mbar_init(&bars.q_full[i], 128);
      mbar_init(&bars.x_full[i], 128);
    }
    for (int i = 0; i < kTRuns; ++i) mbar_init(&bars.run_full[i], 1);
    mbar_init(&bars.run_done, 1);
    mbar_init(&bars.o_free, 128);
    mbar_init(&bars.side, 128);
    mbar_init(&bars.o_done, 1);
    mbar_init(&bars.drain, 1);
    for (int i = 0; i < kTMaskWords; ++i) bars.bad[0][i] = bars.bad[1][i] = 0;
    fence_mbar_init();
  }
  if (warp == kTWarpMma) {
    tc::tmem_alloc(&bars.tmem_base, kTmemCols);
    tc::tmem_relinquish();
  }
  // The plan, from the lengths (like block tables read before the dependency wait),
  // the same in every CTA.  The last CTA reports what is wrong.
  const bool scribe = blockIdx.x == gridDim.x - 1;
  scan_pages_of<kTThreads>(p.num_seqs, rows, bars.warp_tot,
                           [&](int s) { return min(max(__ldg(p.tree_lens + s), 0), p.num_tokens + 1); });
  scan_pages_of<kTThreads>(p.num_seqs, pairs, bars.warp_tot, [&](int s) {
    const int n = __ldg(p.tree_lens + s), len = __ldg(p.context_lens + s);
    if (n == 0) return 0;  // nothing drafted: no rows
    if (n > 0 && n <= PA_MAX_TREE_LEN && rows[s + 1] <= p.num_tokens && len >= n && len <= p.max_len)
      return p.num_kv_heads * ((n + TG - 1) / TG) * ((len + 127) / 128 + p.run_cost);
    if (scribe) set_error(p.err, PA_ERR_RANGE, s);
    return 0;
  });
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = bars.tmem_base;
  TreePlan pl;
  pl.rows = rows;
  pl.pairs = pairs;
  pl.context_lens = p.context_lens;
  pl.num_seqs = p.num_seqs;
  pl.num_kv_heads = p.num_kv_heads;
  pl.cost = p.run_cost;
  pl.total = pairs[p.num_seqs];
  pl.workers = min(pl.total, (int)gridDim.x / NT);  // so that no share is empty
  pl.share = pl.workers > 0 ? (pl.total + pl.workers - 1) / pl.workers : 1;
  const int x0 = part_start(worker, pl.total, pl.workers), x1 = part_start(worker + 1, pl.total, pl.workers);
  bool timed_out = false;
  // (the outcome of a wait is made warp-uniform: what follows is warp-wide)
  auto wait_all = [&](uint64_t *bar, uint32_t parity) { return __all_sync(FULL, mbar_wait(bar, parity)) != 0; };
  // the first token of this CTA's query tile (a group may be the last and not full: then the
  // second tile has fewer rows or none)
  auto first_token = [&](const TRun &U) { return U.g * TG + sub * TQ; };
  // This CTA's next run from pair x on (x0: the first), x behind it; false: no more.
  auto next_run = [&](TRun &U, int &x, bool &begun) {
    while (x < x1) {
      if (!begun) U.at<TG>(pl, x, x1); else U.next<TG>(pl, x, x1);
      begun = true;
      x += U.vb - U.va;
      // (else there are none of the group's keys in it, or no rows of this CTA)
      if (U.vb > pl.cost && first_token(U) < U.n) return true;
    }
    return false;
  };
  TRun U = {};
  int x = x0;
  bool begun = false;

  // (one instruction for the loader and MMA warps: setmaxnreg acts on whole warpgroups)
  if (warp >= kTWarpLoad0 && warp < kTWarpPrep) regs_dec<kTRegsLoad>();
  if (warp < kTWarpEpi) {
    regs_inc<kTRegsSoftmax>();
    griddep_wait();
    // ---------------- softmax (warps 0..3) ----------------
    const int r = threadIdx.x;  // tile row = TMEM lane
    const uint32_t lane_base = tmem + ((uint32_t)(warp * 32) << 16), o_addr = lane_base + kTColO;
    const uint32_t *masks = reinterpret_cast<const uint32_t *>(smem + T_OFF_MASK);
    float2 *xm = reinterpret_cast<float2 *>(smem + T_OFF_X);
    const float sl2 = p.scale_log2;
    int c = 0;
    for (int ui = 0; !timed_out; ++ui) {
      if (!wait_all(&bars.q_full[ui & 1], (ui >> 1) & 1)) {
        timed_out = true;
        break;
      }
      const TRunInfo &I = bars.info[ui % kTRuns];
      const int kt_end = I.kb, start = I.start;
      if (kt_end == 0) break;
      const bool live = r < I.live_rows, active = warp * 32 < I.live_rows;  // (active: warp-uniform)
      const uint32_t *mask = masks + ((ui & 1) * 128 + r / G) * kTMaskWords;
      float m_ref = -INFINITY, l = 0.f;
      for (int kt = I.ka; kt < kt_end; ++kt, ++c) {
        const int kb = kt * 128, st = c & 1;
        const bool full = kb + 128 <= start;  // (the same in every thread)
        if (!wait_all(&bars.s_full[st], (c >> 1) & 1)) {
          timed_out = true;
          break;
        }
        tc::fence_after_sync();
        if (active) {
          const uint32_t s_addr = lane_base + st * 128;
          // the maximum, then P: S is read twice, which costs less than the registers that would hold it
          uint32_t v[2][32];
          if (!full) {  // first the scores that the row does not see become -inf, in their place
            // bit i: key kb + i, drafted token kb + i - start (below 0: committed, seen by all)
            auto word = [&](int k) { return k < 0 ? 0xffffffffu : k < kTMaskWords ? mask[k] : 0u; };
#pragma unroll 1
            for (int q = 0; q < 4; ++q) {
              const int i = kb - start + 32 * q;
              const uint32_t seen = live ? __funnelshift_r(word(i >> 5), word((i >> 5) + 1), i & 31) : 0xffffffffu;
              __syncwarp();
              tc::ld_32x32b_x32(s_addr + q * 32, v[0]);
              tc::wait_ld();
              hide32(v[0], seen);
              tc::st_32x32b_x32(s_addr + q * 32, v[0]);
            }
            tc::wait_st();
          }
          float mx = -INFINITY;
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            tc::ld_32x32b_x32(s_addr + hf * 64, v[0]);
            tc::ld_32x32b_x32(s_addr + hf * 64 + 32, v[1]);
            tc::wait_ld();
            mx = max64(v[0], v[1], mx);
          }
          const float mc = mx == -INFINITY ? mx : mx * sl2;  // -inf: the row has seen nothing of the tile
          const bool first = m_ref == -INFINITY;             // nothing accumulated for this row yet
          const bool need = !first && mc > m_ref + top_of<T>(mc);
          if (__any_sync(FULL, need)) {  // warp-uniform; key tile c - 1 belongs to this run (first is false)
            const float m_new = reference_of<T>(mc), f = need ? ex2(m_ref - m_new) : 1.f;
            if (need) {
              l *= f;
              m_ref = m_new;
            }
            if (!wait_all(&bars.o_done, (c - 1) & 1)) {
              timed_out = true;
              break;
            }
            tc::fence_after_sync();
#pragma unroll
            for (int cc = 0; cc < 4; ++cc) {
              tc::ld_32x32b_x32(o_addr + cc * 32, v[0]);
              tc::wait_ld();
#pragma unroll
              for (int k = 0; k < 32; ++k) v[0][k] = __float_as_uint(__uint_as_float(v[0][k]) * f);
              tc::st_32x32b_x32(o_addr + cc * 32, v[0]);
            }
          }
          if (first) m_ref = reference_of<T>(mc);
          const float m = m_ref == -INFINITY ? 0.f : m_ref;
          float2 ls[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
          tc::ld_32x32b_x32(s_addr, v[0]);
#pragma unroll
          for (int cc = 0; cc < 4; ++cc) {
            tc::wait_ld();
            if (cc < 3) tc::ld_32x32b_x32(s_addr + cc * 32 + 32, v[(cc + 1) & 1]);
            exp_pack_store32<T>(v[cc & 1], s_addr + cc * 32, sl2, m, ls);
            if (cc == 1) {  // the first half's P V goes ahead
              tc::wait_st();
              tc::fence_before_sync();
              mbar_arrive(&bars.p_full[st][0]);
            }
          }
          l += (ls[0].x + ls[0].y) + (ls[1].x + ls[1].y);
          tc::wait_st();
        } else {
          mbar_arrive(&bars.p_full[st][0]);
        }
        if (kt == kt_end - 1) {
          xm[(ui & 1) * 128 + r] = make_float2(m_ref, l);
          mbar_arrive(&bars.x_full[ui & 1]);
        }
        tc::fence_before_sync();
        mbar_arrive(&bars.p_full[st][1]);
      }
    }
  } else if (warp < kTWarpLoad0) {
    regs_inc<kTRegsEpi>();
    griddep_wait();
    // ---------------- drafted values and outputs (warps 4..7) ----------------
    const int r = threadIdx.x & 127;
    const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16), o_addr = lane_base + kTColO;
    const uint32_t *masks = reinterpret_cast<const uint32_t *>(smem + T_OFF_MASK);
    const float2 *xm = reinterpret_cast<const float2 *>(smem + T_OFF_X);
    uint4 *stage = reinterpret_cast<uint4 *>(smem + T_OFF_STAGE + (warp & 3) * kStageBytes);
    int c0 = 0, sides = 0;
    uint32_t landed = 0;  // per stage the parity of its next drafted key tile
    for (int ui = 0;; ++ui) {
      if (!wait_all(&bars.q_full[ui & 1], (ui >> 1) & 1)) {
        timed_out = true;
        break;
      }
      const TRunInfo &I = bars.info[ui % kTRuns];
      if (I.kb == 0) break;

      // Value rows from the first drafted one on, key tile by key tile: past the last key
      // they may hold anything and are zeroed; before it, what is not finite is (see above).
      const int start = I.start;
      for (int kt = max(I.ka, start >> 7); kt < I.kb && !timed_out; ++kt) {
        const int st = (c0 + kt - I.ka) % kTStages, kb = kt * 128;
        if (!wait_all(&bars.v_full[1][st], (landed >> st) & 1)) {
          timed_out = true;
          break;
        }
        landed ^= 1u << st;
        const int z0 = max(start - kb, 0), zl = I.len - kb;
        uint8_t *vbase = smem + T_OFF_V + st * 2 * kHalf;
        for (int idx = r; idx < (128 - z0) * 16; idx += 128) {
          const int row = z0 + (idx >> 4), part = idx & 15;
          uint4 *w = reinterpret_cast<uint4 *>(vbase + (row >> 4) * kVPage + (part >> 3) * (kVPage / 2) +
                                               (row & 15) * 128 + (part & 7) * 16);
          if (row < zl) {
            const uint4 y = *w;
            if (!not_finite2<T>(y.x) && !not_finite2<T>(y.y) && !not_finite2<T>(y.z) && !not_finite2<T>(y.w)) continue;
            const int a = kb + row - start;
            atomicOr(&bars.bad[ui & 1][a >> 5], 1u << (a & 31));
          }
          *w = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
        mbar_arrive(&bars.look[st]);
      }
      c0 += I.kb - I.ka;

      // the run's outputs, or its state into the workspace
      if (timed_out || !wait_all(&bars.x_full[ui & 1], (ui >> 1) & 1) || !wait_all(&bars.run_done, ui & 1)) {
        timed_out = true;
        break;
      }
      tc::fence_after_sync();
      const bool live = r < I.live_rows, active = (warp & 3) * 32 < I.live_rows;  // (active: warp-uniform)
      float2 ml = xm[(ui & 1) * 128 + r];
      uint32_t any = 0, hit = 0;
#pragma unroll
      for (int k = 0; k < kTMaskWords; ++k) {
        const uint32_t w = *reinterpret_cast<volatile uint32_t *>(&bars.bad[ui & 1][k]);
        any |= w;
        if (w && live) hit |= w & masks[((ui & 1) * 128 + r / G) * kTMaskWords + k];
      }
      if (any) {  // (rare; the same in every thread)
        if (hit) ml.y = __int_as_float(0x7fffffff);
        mbar_arrive(&bars.side);  // every thread has read them
        if (!wait_all(&bars.side, sides++ & 1)) {
          timed_out = true;
          break;
        }
        if (r < kTMaskWords) bars.bad[ui & 1][r] = 0;  // (looked for again in the run after the next, behind o_free)
      }
      // (what follows the arrival on o_free does not look at the run's record)
      const int64_t out0 = ((int64_t)I.row * p.num_q_heads + I.h * G) * kHeadDim;
      const int live_rows = I.live_rows;
      if (I.whole) {
        // O into registers, and the next run may have it: an arrival behind the stores
        // would wait until they have reached L2
        uint32_t y[64];
        if (active) {
          const float inv = 1.f / ml.y;
#pragma unroll
          for (int cc = 0; cc < 4; ++cc) {
            uint32_t a[32];
            tc::ld_32x32b_x32(o_addr + cc * 32, a);
            tc::wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i)
              y[cc * 16 + i] =
                  Pack<T>::from_f2(__uint_as_float(a[2 * i]) * inv, __uint_as_float(a[2 * i + 1]) * inv);
          }
          tc::fence_before_sync();
        }
        mbar_arrive(&bars.o_free);
        if (active) {  // 64 bytes of 8 rows per store
#pragma unroll
          for (int cc = 0; cc < 4; ++cc)
#pragma unroll
            for (int pass = 0; pass < 2; ++pass) {
              if ((lane >> 4) == pass) {
                const int row = lane & 15;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  stage[row * 4 + (i ^ (row & 3))] = make_uint4(y[16 * cc + 4 * i], y[16 * cc + 4 * i + 1],
                                                                y[16 * cc + 4 * i + 2], y[16 * cc + 4 * i + 3]);
              }
              __syncwarp();
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const int at = 8 * i + (lane >> 2), row = (warp & 3) * 32 + pass * 16 + at;
                T *op = static_cast<T *>(p.out) + out0 + ((int64_t)(row / G) * p.num_q_heads + row % G) * kHeadDim;
                if (row < live_rows)
                  reinterpret_cast<uint4 *>(op)[4 * cc + (lane & 3)] = stage[at * 4 + ((lane & 3) ^ (at & 3))];
              }
              __syncwarp();
            }
        }
      } else {
        if (active) {
          const int64_t slot = 2 * (int)blockIdx.x + (I.first ? 0 : 1);  // (the share's first run, or its last)
          float4 *piece = reinterpret_cast<float4 *>(p.ws_o) + slot * 32 * 128 + r;  // [dims / 4][row]
#pragma unroll 1
          for (int cc = 0; cc < 4; ++cc) {
            uint32_t a[32];
            tc::ld_32x32b_x32(o_addr + cc * 32, a);
            tc::wait_ld();
            if (live) {
#pragma unroll
              for (int i = 0; i < 8; ++i)
                piece[(cc * 8 + i) * 128] =
                    make_float4(__uint_as_float(a[4 * i]), __uint_as_float(a[4 * i + 1]),
                                __uint_as_float(a[4 * i + 2]), __uint_as_float(a[4 * i + 3]));
            }
            __syncwarp();  // (the next chunk's load is warp-wide)
          }
          if (live) p.ws_ml[slot * 128 + r] = ml;
          tc::fence_before_sync();
        }
        mbar_arrive(&bars.o_free);
      }
      __syncwarp();
    }
  } else if (warp >= kTWarpPrep) {
    regs_dec<kTRegsPrep>();
    griddep_wait();
    // ---------------- queries and masks, a run ahead (warps 12..15) ----------------
    const int r = threadIdx.x & 127;
    const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    uint32_t *masks = reinterpret_cast<uint32_t *>(smem + T_OFF_MASK);
    uint4 *stage = reinterpret_cast<uint4 *>(smem + T_OFF_STAGE + (4 + (warp & 3)) * kStageBytes);
    for (int un = 0;; ++un) {
      // into the buffers of the run's parity, which the run two before has left
      if (!wait_all(&bars.run_full[un % kTRuns], (un / kTRuns) & 1) ||
          (un >= 2 && !wait_all(&bars.o_free, (un - 2) & 1))) {
        timed_out = true;
        break;
      }
      const TRunInfo &I = bars.info[un % kTRuns];
      if (I.kb != 0) {
        const int par = un & 1;
        // The queries: 64 bytes of 8 rows per load, all 32 rows of the warp (rows past the
        // tree are zeros), turned so that a lane holds its row's on the way to tensor memory.
        const T *q0 = static_cast<const T *>(p.q) + ((int64_t)I.row * p.num_q_heads + I.h * G) * kHeadDim;
        const int live_rows = I.live_rows;
        uint4 w[16];
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // row 8 i + lane / 4 of the warp
          const int row = (warp & 3) * 32 + 8 * i + (lane >> 2);
          const uint4 *src = reinterpret_cast<const uint4 *>(
                                 q0 + ((int64_t)(row / G) * p.num_q_heads + row % G) * kHeadDim) + (lane & 3);
#pragma unroll
          for (int cc = 0; cc < 4; ++cc) w[4 * cc + i] = row < live_rows ? __ldg(src + 4 * cc) : make_uint4(0, 0, 0, 0);
        }
        if (r < live_rows / G && I.kb * 128 > I.start) {  // (a run that ends in front of the tree needs no mask)
          uint32_t *mask = masks + (par * 128 + r) * kTMaskWords;
#pragma unroll
          for (int k = 0; k < kTMaskWords; ++k) mask[k] = 0;
          const int32_t *parents = p.parents + (I.row - I.tok0);
          int a = I.tok0 + r;
          while (true) {
            mask[a >> 5] |= 1u << (a & 31);
            const int up = __ldg(parents + a);
            if (up < 0 || up >= a) {
              if (up != -1) set_error(p.err, PA_ERR_RANGE, I.s);  // (the walk ends: as one without parent)
              break;
            }
            a = up;
          }
        }
        __syncwarp();
#pragma unroll
        for (int cc = 0; cc < 4; ++cc) {
          uint32_t v[16];
#pragma unroll
          for (int pass = 0; pass < 2; ++pass) {  // 16 rows at a time, the pieces swizzled against bank conflicts
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int row = 8 * i + (lane >> 2);
              stage[row * 4 + ((lane & 3) ^ (row & 3))] = w[4 * cc + 2 * pass + i];
            }
            __syncwarp();
            if ((lane >> 4) == pass) {
              const int row = lane & 15;
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const uint4 y = stage[row * 4 + (i ^ (row & 3))];
                v[4 * i] = y.x;
                v[4 * i + 1] = y.y;
                v[4 * i + 2] = y.z;
                v[4 * i + 3] = y.w;
              }
            }
            __syncwarp();
          }
          tc::st_32x32b_x16(lane_base + kTColQ + par * 64 + cc * 16, v);
        }
        tc::wait_st();
        tc::fence_before_sync();
      }
      const bool more = I.kb != 0;  // (read before the arrival)
      mbar_arrive(&bars.q_full[un & 1]);
      if (!more) break;
    }
  } else if (warp != kTWarpMma) {
    // ---------------- loader warps: 8 boxes of a key tile each, from parallel lanes ----------------
    // The first two: K, the 64-dim half (box & 1) of page box / 2; the third: V, a page per
    // box.  The block ids of 4 key tiles sit one per lane, the next 4 tiles' already on
    // their way: a table read per tile would hold up every copy by an L2 trip.
    const int lw = warp - kTWarpLoad0;
    const bool for_k = lw < kTKLoad;
    const int box = for_k ? lw + kTKLoad * lane : lane, boxes = for_k ? 16 : 8;
    const int page = for_k ? box >> 1 : box;
    uint64_t *free = for_k ? bars.k_free : bars.v_free;
    uint8_t *dst0 = smem + (for_k ? T_OFF_K + (box & 1) * kHalf + page * 2048 : T_OFF_V + page * kVPage);
    const uint32_t bytes = for_k ? 2048u : (uint32_t)kVPage;
    int c = 0;
    // Keys that one worker alone reads leave L2 to what is read again (pieces, queries).
    const uint64_t once = policy_evict_first(), often = policy_evict_last();
    uint32_t issued = 0;  // per barrier (8 bits per kind, 2 per stage) bit 1: any copy, bit 0: the last one's parity
    bool waited = false;
    TRun N = {};
    bool more = true;
    for (int ui = -1; !timed_out; ++ui) {  // (the first time round only the first run is published)
      if (!more) break;
      U = N;
      more = next_run(N, x, begun);
      if (lw == 0 && lane == 0) {  // run ui + 1
        TRunInfo &I = bars.info[(ui + 1) % kTRuns];
        const int tok0 = first_token(N);
        I.ka = N.ka(pl.cost);
        I.kb = more ? N.kb(pl.cost) : 0;
        I.start = N.len - N.n;
        I.len = N.len;
        I.row = N.row0 + tok0;
        I.live_rows = min(TQ, N.n - tok0) * G;
        I.h = N.h;
        I.s = N.s;
        I.tok0 = tok0;
        I.whole = N.whole(pl.cost);
        I.first = x - (N.vb - N.va) == x0;
        mbar_arrive(&bars.run_full[(ui + 1) % kTRuns]);
      }
      __syncwarp();
      if (ui < 0) continue;
      const int32_t *bt = p.block_tables + (int64_t)U.s * p.max_blocks_per_seq;
      const int npages = (U.len + kBlock - 1) / kBlock;
      const int tail = for_k ? INT_MAX : (U.len - U.n) >> 7;  // the first key tile that reaches the drafted keys
      const int ka = U.ka(pl.cost), kb = U.kb(pl.cost);
      const uint64_t policy = U.groups > 1 ? often : once;
      int wbase = ka * 8;
      auto ids_from = [&](int base) { return base + lane < npages ? __ldg(bt + base + lane) : -1; };
      int32_t win = ids_from(wbase), win_next = ids_from(wbase + 32);
      if (!waited) griddep_wait();  // K and V may come from the kernels before
      waited = true;
      for (int t = ka; t < kb; ++t, ++c) {
        if (t * 8 >= wbase + 32) {
          wbase += 32;
          win = win_next;
          win_next = ids_from(wbase + 32);
        }
        const int id = __shfl_sync(FULL, win, (t * 8 + page - wbase) & 31);
        const bool in = box < boxes && t * 8 + page < npages;  // (V past the last key is zeroed, see above)
        const bool ok = in && (unsigned)id < (unsigned)p.num_blocks;
        const unsigned okmask = __ballot_sync(FULL, ok);
        const int st = c % kTStages;
        if (c >= kTStages && !wait_all(free + st, (c / kTStages - 1) & 1)) {  // the stage is free
          timed_out = true;
          break;
        }
        uint8_t *dst = dst0 + st * 2 * kHalf;
        uint64_t *full = (for_k ? bars.k_full : bars.v_full[t >= tail]) + st;
        if (in && !ok) {  // rare: keep the products finite
          set_error(p.err, PA_ERR_RANGE, U.s);
          for (uint32_t i = 0; i < bytes / 16; ++i) reinterpret_cast<uint4 *>(dst)[i] = make_uint4(0, 0, 0, 0);
          fence_proxy_async_smem();
        }
        __syncwarp();  // the zeroed boxes are written before the arrival below releases them
        if (lane == 0) mbar_arrive_expect_tx(full, (uint32_t)__popc(okmask) * bytes);
        __syncwarp();
        const int bit = 2 * st + (t >= tail ? 8 : 0);
        issued = issued >> bit & 2 ? issued ^ 1u << bit : issued | 2u << bit;
        if (ok) {
          if (for_k)
            tma_load_4d_hint(dst, &kmap, full, (box & 1) * 64, U.h, 0, id, policy);
          else
            tma_load_5d_hint(dst, &vmap, full, 0, 0, 0, U.h, id, policy);
        }
      }
    }
    if (timed_out)  // a short, bounded chance for this warp's copies in flight to land
      for (int i = 0; i < kTStages; ++i)
        for (int k = 0; k < (for_k ? 1 : 2); ++k) {
          const uint32_t used = issued >> (2 * i + 8 * k) & 3;
          if (used & 2) mbar_wait((for_k ? bars.k_full : bars.v_full[k]) + i, used & 1, kWaitLimitNs / 8);
        }
  } else {
    // ---------------- MMA issuer (warp-uniform loop, one elected lane issues) ----------------
    griddep_wait();
    griddep_launch_dependents();  // (the join waits for this grid; its blocks start as CTAs leave)
    if (lane == 0 && sub == 0) {  // the join's record (after the wait: the previous call's join may still read)
      JoinRecord rec = {};
      if (x0 < x1) {
        // The group of the last pair: joined here if its first unit began in this share and others go on with it.
        TRun Z = {};
        Z.at<TG>(pl, x1 - 1, x1);
        const int unit = x1 - 1 - (Z.va - Z.k0), end = unit + Z.k1 - Z.k0;  // its unit's pairs
        const bool cut = part_owner(unit + pl.cost, pl.total, pl.workers) != part_owner(end - 1, pl.total, pl.workers);
        if (unit >= x0 && Z.k0 == 0 && (Z.blocks > 1 || cut)) {  // (its keys, that is)
          rec.rows = min(TG, Z.n - Z.g * TG) * G;
          rec.row0 = Z.row0 + Z.g * TG;
          rec.h = Z.h;
          rec.pairs0 = pairs[Z.s] + Z.h * Z.groups * Z.kt;
          rec.kt = Z.kt;
          rec.groups = Z.groups;
          rec.g = Z.g;
          rec.blocks = Z.blocks;
          rec.total = pl.total;
          rec.workers = pl.workers;
        }
      }
      reinterpret_cast<JoinRecord *>(p.records)[worker] = rec;
    }
    __syncwarp();
    const bool leader = elect_one();
    const uint64_t kdesc0 = tc::desc_sw128(smem_u32(smem + T_OFF_K), 16, 1024);
    const uint64_t vdesc0 = tc::desc_sw128(smem_u32(smem + T_OFF_V), kVPage / 2, 1024);
    constexpr uint64_t kStageStep = (2 * kHalf) >> 4;
    constexpr uint64_t kHalfStep = kHalf >> 4;
    // the P V product of key tile pc (pending), issued once P is ready
    int pc = -1, p_run = 0;
    uint32_t looked = 0, landed = 0;  // per stage the parity of its next look, and of its next other key tile
    bool p_first = false, p_last = false, p_tail = false;
    auto issue_pv = [&]() -> bool {
      const int st = pc % kTStages;
      if (p_tail) {
        if (!wait_all(&bars.look[st], (looked >> st) & 1)) return false;
        looked ^= 1u << st;
      } else {
        if (!wait_all(&bars.v_full[0][st], (landed >> st) & 1)) return false;
        landed ^= 1u << st;
      }
      if (p_first && p_run > 0 && !wait_all(&bars.o_free, (p_run - 1) & 1)) return false;
      const uint64_t vdesc = vdesc0 + (uint64_t)st * kStageStep;
#pragma unroll
      for (int half = 0; half < 2; ++half) {  // (as soon as P of its 64 keys is ready)
        if (!wait_all(&bars.p_full[pc & 1][half], (pc >> 1) & 1)) return false;
        tc::fence_after_sync();
        if (leader) {
#pragma unroll
          for (int kk = 4 * half; kk < 4 * half + 4; ++kk) {
            const uint32_t a_hi = tmem + (pc & 1) * 128 + 32 * (kk >> 1) + 8 * (kk & 1);
            const uint64_t bdesc = vdesc + (uint64_t)(kk * (kVPage >> 4));
            tc::mma_f16_ts(tmem + kTColO, a_hi, bdesc, IDESC_O, kk > 0 || !p_first ? 1u : 0u);
            tc::mma_f16_ts(tmem + kTColO, a_hi + 16, bdesc, IDESC_O, 1u);
          }
        }
        __syncwarp();
      }
      if (leader) {
        tc::commit(&bars.o_done);
        tc::commit(&bars.v_free[st]);
        if (p_last) tc::commit(&bars.run_done);
      }
      __syncwarp();
      return true;
    };
    int c = 0;
    for (int ui = 0; !timed_out; ++ui) {
      if (!wait_all(&bars.q_full[ui & 1], (ui >> 1) & 1)) {
        timed_out = true;
        break;
      }
      const int ka = bars.info[ui % kTRuns].ka, kb = bars.info[ui % kTRuns].kb, start = bars.info[ui % kTRuns].start;
      if (kb == 0) break;
      for (int kt = ka; kt < kb; ++kt, ++c) {
        const int st = c % kTStages;
        if (!wait_all(&bars.k_full[st], (c / kTStages) & 1)) {
          timed_out = true;
          break;
        }
        tc::fence_after_sync();
        if (leader) {
          // S = Q K^T over the P of key tile c - 2, whose P V was issued: they run in order
          const uint64_t kdesc = kdesc0 + (uint64_t)st * kStageStep;
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)  // 16-element k-steps
            tc::mma_f16_ts(tmem + (c & 1) * 128, tmem + kTColQ + (ui & 1) * 64 + 8 * kk,
                           kdesc + (uint64_t)((kk >> 2) * kHalfStep + (kk & 3) * 2), IDESC_S, kk > 0 ? 1u : 0u);
          tc::commit(&bars.s_full[c & 1]);
          tc::commit(&bars.k_free[st]);
        }
        __syncwarp();
        if (pc >= 0 && !issue_pv()) {
          timed_out = true;
          break;
        }
        pc = c;
        p_run = ui;
        p_first = kt == ka;
        p_last = kt == kb - 1;
        p_tail = kt * 128 + 128 > start;
      }
    }
    if (!timed_out && pc >= 0 && !issue_pv()) timed_out = true;
    if (timed_out) {  // every MMA issued so far, bounded, before the tensor memory is freed
      if (leader) tc::commit(&bars.drain);
      __syncwarp();
      mbar_wait(&bars.drain, 0, kWaitLimitNs / 8);
    }
  }
  if (timed_out) set_error(p.err, PA_ERR_TIMEOUT, (int)blockIdx.x);
  tc::fence_before_sync();
  __syncthreads();
  if (warp == kTWarpMma) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, kTmemCols);
  }
}

// ---- the join ----
// Block (worker, part): the group of the worker's record, per thread and round 4
// items of a row's 4 dims each, so that their pieces are in flight together.
constexpr int kTJoinThreads = 256, kTJoinParts = 4, kTJoinItems = 4, kTJoinPieces = 2;
template <typename T, int G, int NT>
__global__ void __launch_bounds__(kTJoinThreads) attn_tree_join_kernel(const __grid_constant__ TreeParams p) {
  griddep_wait();
  griddep_launch_dependents();  // (it writes nothing that a kernel may read before its own wait)
  JoinRecord rec;
  {
    const int4 *src = reinterpret_cast<const int4 *>(p.records) + blockIdx.x * 3;
    int4 *dst = reinterpret_cast<int4 *>(&rec);
    dst[0] = __ldcg(src);
    dst[1] = __ldcg(src + 1);
    dst[2] = __ldcg(src + 2);
  }
  const int items = rec.rows * 32, stride = gridDim.y * kTJoinThreads;
  for (int i0 = (int)blockIdx.y * kTJoinThreads + (int)threadIdx.x; i0 < items; i0 += kTJoinItems * stride) {
    JoinState js[kTJoinItems];
    // lanes: G neighbouring rows x 32 / G dim quads, so that pieces are read in runs and outputs are written so
    auto row_of = [&](int i) { return (i / 32) / G * G + i % G; };
    auto quad_of = [&](int i) { return (i / G) % 32; };
    for (int j = 0; j < rec.blocks; ++j) {
      const int k0 = part_start(j, rec.kt, rec.blocks), bl = part_start(j + 1, rec.kt, rec.blocks) - k0;
      const int xa = rec.pairs0 + rec.groups * k0 + rec.g * bl;  // the unit's first pair
      const int ff = part_owner(xa, rec.total, rec.workers), fl = part_owner(xa + bl - 1, rec.total, rec.workers);
      const int second = part_start(ff, rec.total, rec.workers) < xa ? 1 : 0;  // worker ff's piece is not its first run
      for (int f0 = ff; f0 <= fl; f0 += kTJoinPieces) {
        float2 ml[kTJoinItems][kTJoinPieces];
        float4 o[kTJoinItems][kTJoinPieces];
#pragma unroll
        for (int n = 0; n < kTJoinItems; ++n) {
          const int i = i0 + n * stride, row = row_of(i), tr = row & 127;
          const int cta = row >> 7;
#pragma unroll
          for (int u = 0; u < kTJoinPieces; ++u) {
            ml[n][u] = make_float2(-INFINITY, 0.f);
            o[n][u] = make_float4(0.f, 0.f, 0.f, 0.f);
            // (a worker with no more than the group's cost has no piece)
            // (a piece without keys does not exist)
            auto until = [&]() { return min(part_start(f0 + u + 1, rec.total, rec.workers), xa + bl); };
            if (i < items && f0 + u <= fl && k0 + until() - xa > p.run_cost) {
              const int64_t slot = 2 * ((f0 + u) * NT + cta) + (f0 + u == ff ? second : 0);
              ml[n][u] = __ldcg(p.ws_ml + slot * 128 + tr);
              o[n][u] = __ldcg(reinterpret_cast<const float4 *>(p.ws_o) + (slot * 32 + quad_of(i)) * 128 + tr);
            }
          }
        }
#pragma unroll
        for (int n = 0; n < kTJoinItems; ++n) js[n].add(ml[n], o[n]);
      }
    }
#pragma unroll
    for (int n = 0; n < kTJoinItems; ++n) {
      const int i = i0 + n * stride, row = row_of(i);
      if (i < items)
        js[n].store(static_cast<T *>(p.out) +
                    ((int64_t)(rec.row0 + row / G) * p.num_q_heads + rec.h * G + row % G) * kHeadDim + 4 * quad_of(i));
    }
  }
}

template <typename T, int G, int NT>
cudaError_t launch_tree_typed(TreeParams p, const CUtensorMap *maps, int sms, cudaStream_t stream) {
  static KernelSetup setup;
  const int smem = T_OFF_PLAN + 2 * (p.num_seqs + 1) * 4;
  cudaError_t e = kernel_setup(setup, attn_tree_kernel<T, G, NT>, smem, kTThreads, nullptr);
  if (e != cudaSuccess) return e;
  const int workers = sms / NT > 0 ? sms / NT : 1;
  // A call of a few key tiles per worker, by the bound on its lengths, is spread as evenly as its
  // key tiles go, without the runs' cost, which would leave workers without keys: 4 sequences of
  // 300 with 8 drafts, 32 / 8 heads, 12.7 us against 14.6, one of 777, 16 / 8, 11.2 against 12.4;
  // 16 of 500, 16 / 8, 18.3 against 17.6, and 4 of 600 with 60 drafts, 32 / 8, 20.3 against 18.7.
  // The lengths themselves are not known here: a bound far above them has the second figures.
  const int64_t groups = (int64_t)p.num_kv_heads * (p.num_seqs + (int64_t)p.num_tokens * G / (128 * NT));
  p.run_cost = groups * ((p.max_len + 127) / 128) > 4 * workers ? kTreeRunCost : 0;
  const dim3 grid(workers * NT), block(kTThreads);
  e = launch_pdl(attn_tree_kernel<T, G, NT>, grid, block, smem, stream, maps[0], maps[1], p);
  if (e != cudaSuccess) return e;
  const dim3 parts(workers, kTJoinParts * NT);
  return launch_pdl(attn_tree_join_kernel<T, G, NT>, parts, dim3(kTJoinThreads), 0, stream, p);
}

struct TreeLayout {
  size_t ml, o, total;
};
TreeLayout tree_layout(int sms) {
  auto up = [](size_t n) { return (n + 255) & ~(size_t)255; };
  const size_t ctas = sms > 1 ? sms : 2, rows = 2 * ctas * 128;  // a CTA's first and last run
  TreeLayout l;
  l.ml = up(ctas * sizeof(JoinRecord));
  l.o = l.ml + up(rows * sizeof(float2));
  l.total = l.o + rows * kHeadDim * sizeof(float);
  return l;
}

}  // namespace

size_t tree_workspace_bytes(int sms) { return tree_layout(sms).total; }

cudaError_t launch_attn_tree(TreeParams p, void *workspace, const CUtensorMap *maps, int dtype, int group, int sms,
                             cudaStream_t stream) {
  const TreeLayout l = tree_layout(sms);
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  p.records = reinterpret_cast<int32_t *>(ws);
  p.ws_ml = reinterpret_cast<float2 *>(ws + l.ml);
  p.ws_o = reinterpret_cast<float *>(ws + l.o);
  // Two query tiles per group where the average tree fills more than one.  Two against one,
  // 32 / 8 heads, bf16: 19 sequences of 8192 with 33 drafts 171 us against 188, with 64 165
  // against 195; 64 of 1024 with 33 87 against 96; one of 20000 with 33 40 against 64.  With
  // 96 drafts, three tiles, a CTA in four has none: 325 against 283.
  const bool two = (int64_t)p.num_tokens * group > (int64_t)p.num_seqs * 128;
#define PA_TREE_CASE(T, G) \
  if (group == G) \
    return two ? launch_tree_typed<T, G, 2>(p, maps, sms, stream) : launch_tree_typed<T, G, 1>(p, maps, sms, stream);
  if (dtype == PA_BF16) {
    PA_TREE_CASE(__nv_bfloat16, 1)
    PA_TREE_CASE(__nv_bfloat16, 2)
    PA_TREE_CASE(__nv_bfloat16, 4)
    PA_TREE_CASE(__nv_bfloat16, 8)
  } else {
    PA_TREE_CASE(__half, 1)
    PA_TREE_CASE(__half, 2)
    PA_TREE_CASE(__half, 4)
    PA_TREE_CASE(__half, 8)
  }
#undef PA_TREE_CASE
  return cudaErrorInvalidValue;
}

}  // namespace pa

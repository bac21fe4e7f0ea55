// Paged GQA attention of drafted tokens that form a tree behind each sequence's
// cached context, for sm_103a (speculative decoding).
//
//   out[i][g] = softmax_j(scale q[i][g] . K_j) V_j over the L - n committed keys,
//               token i's ancestors in the tree, and i itself (the n drafted
//               tokens' K and V are the last n of the L cached ones)
//
// The n x G query rows of a sequence for one KV head against its keys are a
// matrix product: query tiles of 128 rows (128 / G tokens x the G heads), key
// tiles of 128 keys, on the tcgen05 tensor cores with the tile machinery of
// prefill_kernel.cuh.  All (query tile, key tile) pairs of the call are dealt
// evenly to one CTA per SM, so one long sequence or many short ones fill the GPU
// alike.  A CTA's share is a row of runs: consecutive key tiles of one query tile.
// A run that holds all keys of its query tile writes the outputs; a query tile cut
// between CTAs leaves a piece (m, l, o) per CTA, joined by a second kernel.  Only a
// CTA's first and last run can be such pieces, so 2 slots per CTA hold them whatever
// the batch.  One query tile (n G <= 128) is bound by HBM: 64 KB of K and V per
// pair, 1.47 us of an SM's share, beside 0.78 us of tensor time (P in two terms).
// With several, the key range is cut into blocks at least as long as a CTA's share,
// the query tiles of a block next to each other in the order, so that the CTAs that
// need the same keys run at the same time and all but one of them read L2.
//
// The mask: 64 bits per row and half key tile, found from the parents where the
// tile reaches the drafted keys (a walk up the tree, its length the token's depth
// within 64 keys, while the keys are on their way).  A row always sees itself.  A
// drafted value that is infinite or NaN must not reach the rows that do not see it
// (0 x inf): such values are zeroed in shared memory and the rows that see them
// made NaN.
#include "decode_mma.cuh"
#include "piece_softmax.cuh"

namespace pa {
namespace {

constexpr int kTJoinPieces = 8;  // pieces in flight in the join
constexpr int kTKStages = 2, kTVStages = 3;  // (as the shared prefixes: a V tile is held longer than a K tile)
constexpr int kTKLoad = 4, kTVLoad = kLoadWarps - kTKLoad;
constexpr int T_OFF_Q = 0;
constexpr int T_OFF_K = 2 * kHalf;
constexpr int T_OFF_V = T_OFF_K + kTKStages * 2 * kHalf;
constexpr int T_OFF_X = T_OFF_V + kTVStages * 2 * kHalf;  // (m, l) exchange [run parity][half][128]
constexpr int T_OFF_STAGE = T_OFF_X + 2 * 2 * 128 * 8;    // 1 KB of output staging per softmax warp
constexpr int T_OFF_BAR = T_OFF_STAGE + kSoftmaxWarps * kStageBytes;
struct TBars {
  uint64_t q_full, q_free;
  uint64_t k_full[kTKStages], s_full[kTKStages];
  uint64_t v_full[kTVStages], p_full[kTVStages], pv_done[kTVStages];
  uint64_t x_full, o_free, drain;
  uint64_t tail[2];    // per half: its threads have looked at the drafted values of a key tile
  uint64_t bad[2][2];  // [key-tile parity][half]: keys whose drafted values are not finite
  uint32_t tmem_base;
};
constexpr int T_BAR_BYTES = 512;
static_assert(sizeof(TBars) <= T_BAR_BYTES, "barriers");
constexpr int T_OFF_PLAN = T_OFF_BAR + T_BAR_BYTES;  // rows [num_seqs + 1], pairs [num_seqs + 1]
static_assert(T_OFF_PLAN + 2 * (kTreeMaxSeqs + 1) * 4 + 1024 <= 232448, "shared memory");

// The order of the work: sequence s has rows[s + 1] - rows[s] drafted tokens and
// the pairs pairs[s] .. pairs[s + 1] - 1 (none for a sequence that is refused).
struct TreePlan {
  const int32_t *rows, *pairs;
  int32_t num_seqs, total, ctas, share;
};

// Part j of W things over n, [j W / n, (j + 1) W / n), and the part that holds thing y.
__device__ __forceinline__ int part_start(int j, int W, int n) { return j >= n ? W : (int)((int64_t)j * W / n); }
__device__ __forceinline__ int part_owner(int y, int W, int n) {
  return (int)((((int64_t)y + 1) * n + W - 1) / W - 1);
}

// A run of pairs: key tiles ka .. kb - 1 of query tile mt of (sequence s, KV head h).
struct TRun {
  int s, h, mt, ka, kb, kt, nmt, blocks;  // kt, nmt, blocks: the sequence's key tiles, query tiles, key blocks
  int n, len, row0;                       // its drafted tokens, keys, and first row
  int first_pair;                         // of the unit (query tile and key block) that the run is part of
  bool whole;                             // the run holds all keys of its query tile
};
template <int G>
__device__ __forceinline__ TRun trun_at(const TreePlan &pl, const int32_t *context_lens, int x, int x_end) {
  constexpr int TQ = 128 / G;
  int lo = 0, hi = pl.num_seqs - 1;  // the last sequence with pairs[s] <= x: the one that holds x
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (pl.pairs[mid] <= x) lo = mid; else hi = mid - 1;
  }
  TRun u;
  u.s = lo;
  u.row0 = pl.rows[lo];
  u.n = pl.rows[lo + 1] - u.row0;
  u.len = __ldg(context_lens + lo);
  u.kt = (u.len + 127) / 128;
  u.nmt = (u.n + TQ - 1) / TQ;
  u.blocks = u.nmt > 1 ? max(u.kt / pl.share, 1) : 1;
  int r = x - pl.pairs[lo];
  u.h = r / (u.nmt * u.kt);
  r -= u.h * u.nmt * u.kt;
  const int j = part_owner(r / u.nmt, u.kt, u.blocks);  // block j's pairs start at nmt * (its first key tile)
  const int k0 = part_start(j, u.kt, u.blocks), bl = part_start(j + 1, u.kt, u.blocks) - k0;
  r -= u.nmt * k0;
  u.mt = r / bl;
  r -= u.mt * bl;
  u.ka = k0 + r;
  u.kb = min(k0 + bl, u.ka + (x_end - x));
  u.first_pair = x - r;
  u.whole = u.blocks == 1 && r == 0 && u.kb == u.kt;
  return u;
}

// What the join wants to know of the query tile that starts in a CTA's last run
// and ends in others (rows 0: none).
struct JoinRecord {
  int32_t rows, row0, head0;      // query rows, first token's row in out, first query head
  int32_t pairs0, kt, nmt, mt, blocks, total, ctas, pad[2];
};
static_assert(sizeof(JoinRecord) == 48, "three 16-byte loads");

// P = 2^(S * scale_log2 - m) of this thread's 64 keys, those visible per `seen`
// (bit i: key i of the half), in two terms over the S columns as exp_pack_store.
template <typename T>
__device__ __forceinline__ float exp_pack_store_seen(const uint32_t (&v)[2][32], uint32_t s_addr, float sl2,
                                                     float m_ref, const uint32_t (&seen)[2]) {
  const float2 sl2v = make_float2(sl2, sl2), negm = make_float2(-m_ref, -m_ref), neg1 = make_float2(-1.f, -1.f);
  float2 ls[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
  for (int cc = 0; cc < 2; ++cc) {
    uint32_t pk[32];
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const float2 e =
          __ffma2_rn(make_float2(__uint_as_float(v[cc][2 * j]), __uint_as_float(v[cc][2 * j + 1])), sl2v, negm);
      float2 pr = make_float2(ex2(e.x), ex2(e.y));
      pr.x = (seen[cc] >> (2 * j)) & 1 ? pr.x : 0.f;
      pr.y = (seen[cc] >> (2 * j + 1)) & 1 ? pr.y : 0.f;
      ls[cc] = __fadd2_rn(ls[cc], pr);
      pk[j] = Pack<T>::from_f2(pr.x, pr.y);
      const float2 lo = __ffma2_rn(Pack<T>::to_f2(pk[j]), neg1, pr);
      pk[16 + j] = Pack<T>::from_f2(lo.x, lo.y);
    }
    tc::st_32x32b_x32(s_addr + cc * 32, pk);
  }
  const float2 t = __fadd2_rn(ls[0], ls[1]);
  return t.x + t.y;
}

// Whether one of the two 16-bit values of u is infinite or NaN.
template <typename T>
__device__ __forceinline__ bool not_finite2(uint32_t u) {
  constexpr uint32_t E = std::is_same<T, __half>::value ? 0x7c00u : 0x7f80u;
  return (u & E) == E || ((u >> 16) & E) == E;
}

// The roles of prefill_kernel.cuh, each looping over the CTA's runs with a
// key-tile counter c that runs on across them (as in decode_shared.cu): warps 0..7
// softmax and epilogue, warps 8..14 load (4 K, 3 V), warp 15 owns the tensor
// memory and issues the MMAs.  Softmax warps whose 32 rows hold no query of the
// run (a small tree's tile is mostly empty) only keep pace on the barriers.
template <typename T, int G>
__global__ void __launch_bounds__(kThreads, 1)
attn_tree_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                 const __grid_constant__ CUtensorMap qmap, const __grid_constant__ TreeParams p) {
  constexpr int TQ = 128 / G;
  constexpr bool kBF16 = std::is_same<T, __nv_bfloat16>::value;
  constexpr uint32_t IDESC_S = tc::idesc_f16(kBF16, 128, 128, false);
  constexpr uint32_t IDESC_O = tc::idesc_f16(kBF16, 128, 128, true);
  extern __shared__ uint8_t smem_raw[];
  __shared__ int warp_tot[kThreads / 32];
  uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  TBars &bars = *reinterpret_cast<TBars *>(smem + T_OFF_BAR);
  int32_t *rows = reinterpret_cast<int32_t *>(smem + T_OFF_PLAN), *pairs = rows + p.num_seqs + 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = (int)blockIdx.x;

  if (threadIdx.x == kThreads - 64) {
    tma_prefetch_desc(&kmap);
    tma_prefetch_desc(&vmap);
    tma_prefetch_desc(&qmap);
    mbar_init(&bars.q_full, 1);
    mbar_init(&bars.q_free, 1);
    for (int i = 0; i < kTKStages; ++i) {
      mbar_init(&bars.k_full[i], kTKLoad);
      mbar_init(&bars.s_full[i], 1);
    }
    for (int i = 0; i < kTVStages; ++i) {
      mbar_init(&bars.v_full[i], kTVLoad);
      mbar_init(&bars.p_full[i], kSoftmaxThreads);
      mbar_init(&bars.pv_done[i], 1);
    }
    mbar_init(&bars.x_full, kSoftmaxThreads);
    mbar_init(&bars.o_free, kSoftmaxThreads);
    mbar_init(&bars.drain, 1);
    for (int i = 0; i < 2; ++i) mbar_init(&bars.tail[i], kSoftmaxThreads / 2);
    for (int i = 0; i < 4; ++i) bars.bad[i >> 1][i & 1] = 0;
    fence_mbar_init();
  }
  if (warp == kWarpMma) {
    tc::tmem_alloc(&bars.tmem_base, kTmemCols);
    tc::tmem_relinquish();
  }
  // The plan, from the lengths (like block tables read before the dependency wait),
  // the same in every CTA.  The last CTA reports what is wrong.
  const bool scribe = b == (int)gridDim.x - 1;
  scan_pages_of<kThreads>(p.num_seqs, rows, warp_tot,
                          [&](int s) { return min(max(__ldg(p.tree_lens + s), 0), p.num_tokens + 1); });
  scan_pages_of<kThreads>(p.num_seqs, pairs, warp_tot, [&](int s) {
    const int n = __ldg(p.tree_lens + s), len = __ldg(p.context_lens + s);
    if (n == 0) return 0;  // nothing drafted: no rows
    if (n > 0 && n <= PA_MAX_TREE_LEN && rows[s + 1] <= p.num_tokens && len >= n && len <= p.max_len)
      return p.num_kv_heads * ((n + TQ - 1) / TQ) * ((len + 127) / 128);
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
  pl.num_seqs = p.num_seqs;
  pl.total = pairs[p.num_seqs];
  pl.ctas = min(pl.total, (int)gridDim.x);  // so that no share is empty
  pl.share = pl.ctas > 0 ? (pl.total + pl.ctas - 1) / pl.ctas : 1;
  const int x0 = part_start(b, pl.total, pl.ctas), x1 = part_start(b + 1, pl.total, pl.ctas);
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
    // (the outcome of a wait is made warp-uniform: what follows is warp-wide)
    auto wait_all = [&](uint64_t *bar, uint32_t parity) { return __all_sync(FULL, mbar_wait(bar, parity)) != 0; };
    int c = 0, ui = 0, tails = 0;
    for (int x = x0; x < x1 && !timed_out; ++ui) {
      const TRun U = trun_at<G>(pl, p.context_lens, x, x1);
      x += U.kb - U.ka;
      const int start = U.len - U.n;                    // the first drafted key
      const int tok = U.mt * TQ + r / G;                // this row's token in the tree
      const int live_rows = min(TQ, U.n - U.mt * TQ) * G;
      const bool live = r < live_rows, active = quad * 32 < live_rows;  // (active: warp-uniform)
      const int32_t *parents = p.parents + U.row0;
      const float sl2 = live ? p.scale_log2 : 0.f;  // (rows past the tree: no rescaling on their account)
      float m_ref = -INFINITY, l = 0.f;
      for (int kt = U.ka; kt < U.kb; ++kt, ++c) {
        const int sb = c & 1, ks = c % kTKStages, vs = c % kTVStages;
        const int kb = kt * 128 + ch * 64;  // first key of this half
        const bool full = kb + 63 < start;  // (the same in every thread of the half)
        uint32_t seen[2] = {0xffffffffu, 0xffffffffu};
        if (!full && active && live) {
          const int committed = start - kb;  // keys of this half in front of the tree
          seen[0] = committed <= 0 ? 0u : committed >= 32 ? 0xffffffffu : (1u << committed) - 1u;
          seen[1] = committed <= 32 ? 0u : (1u << (committed - 32)) - 1u;  // (committed < 64)
          int a = tok;
          while (start + a >= kb) {
            const int i = start + a - kb;
            if (i < 32) seen[0] |= 1u << i;
            else if (i < 64) seen[1] |= 1u << (i - 32);
            const int up = __ldg(parents + a);
            if (up < 0 || up >= a) {
              if (up != -1) set_error(p.err, PA_ERR_RANGE, U.s);  // (the walk ends: as one without parent)
              break;
            }
            a = up;
          }
        }
        if (!wait_all(&bars.s_full[ks], (c / kTKStages) & 1)) {
          timed_out = true;
          break;
        }
        tc::fence_after_sync();
        const uint32_t s_addr = tmem + lane_base + sb * 128 + ch * 64;
        uint32_t v[2][32];
        if (active) {
          tc::ld_32x32b_x32(s_addr, v[0]);
          tc::ld_32x32b_x32(s_addr + 32, v[1]);
          tc::wait_ld();
          const bool first = m_ref == -INFINITY;  // nothing accumulated for this row yet
          const bool common = __all_sync(FULL, full && !first);
          float mx = -INFINITY, ls = 0.f;
          if (common) ls = exp_pack_store<T, true>(v, s_addr, sl2, m_ref, true, 0, 0);
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
                  if ((seen[cc] >> j) & 1) mx = fmaxf(mx, __uint_as_float(v[cc][j]));
            }
          }
          const float mc = mx == -INFINITY ? mx : mx * sl2;
          const bool need = !first && mc > m_ref + top_of<T>(mc);
          const bool redo = __any_sync(FULL, need);
          if (redo) {  // warp-uniform; key tile c - 1 belongs to this run (first is false)
            if (common) tc::wait_st();
            const float m_new = reference_of<T>(mc), f = need ? ex2(m_ref - m_new) : 1.f;
            if (need) {
              l *= f;
              m_ref = m_new;
            }
            if (!wait_all(&bars.pv_done[(c - 1) % kTVStages], ((c - 1) / kTVStages) & 1)) {
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
          if (!common || redo)
            ls = full ? exp_pack_store<T, true>(v, s_addr, sl2, m_ref, true, 0, 0)
                      : exp_pack_store_seen<T>(v, s_addr, sl2, m_ref, seen);
          l += ls;
          tc::wait_st();
        }
        if (!wait_all(&bars.v_full[vs], (c / kTVStages) & 1)) {
          timed_out = true;
          break;
        }
        if (!full) {
          // value rows of this half from the first drafted one on: past the last key they
          // may hold anything and are zeroed; before it, what is not finite is (see above)
          const int z0 = max(start - kb, 0), zl = U.len - kb;
          uint8_t *vbase = smem + T_OFF_V + vs * 2 * kHalf;
          uint64_t bad = 0;
          for (int idx = quad * 32 + lane; idx < (64 - z0) * 16; idx += kSoftmaxThreads / 2) {
            const int i = z0 + (idx >> 4), part = idx & 15, row = ch * 64 + i;
            uint4 *w = reinterpret_cast<uint4 *>(vbase + (row >> 4) * kVPage + (part >> 3) * (kVPage / 2) +
                                                 (row & 15) * 128 + (part & 7) * 16);
            const bool past = i >= zl;
            if (!past) {
              const uint4 y = *w;
              if (!not_finite2<T>(y.x) && !not_finite2<T>(y.y) && !not_finite2<T>(y.z) && !not_finite2<T>(y.w))
                continue;
              bad |= 1ull << i;
            }
            *w = make_uint4(0, 0, 0, 0);
          }
          unsigned long long *flag = reinterpret_cast<unsigned long long *>(&bars.bad[c & 1][ch]);
          if (bad) atomicOr(flag, (unsigned long long)bad);
          fence_proxy_async_smem();
          mbar_arrive(&bars.tail[ch]);
          if (!wait_all(&bars.tail[ch], tails++ & 1)) {
            timed_out = true;
            break;
          }
          const uint64_t all = *reinterpret_cast<volatile unsigned long long *>(flag);
          if (all) {  // (rare; the same in every thread of the half)
            if (((uint32_t)all & seen[0]) | ((uint32_t)(all >> 32) & seen[1])) l = __int_as_float(0x7fffffff);
            mbar_arrive(&bars.tail[ch]);  // every thread has read it
            if (!wait_all(&bars.tail[ch], tails++ & 1)) {
              timed_out = true;
              break;
            }
            if (quad == 0 && lane == 0) *flag = 0;
          }
        }
        tc::fence_before_sync();
        mbar_arrive(&bars.p_full[vs]);
      }
      if (timed_out) break;

      // ---- the run's outputs, or its state into the workspace ----
      const int cl = c - 1;
      bool ok = wait_all(&bars.pv_done[cl % kTVStages], (cl / kTVStages) & 1);
      tc::fence_after_sync();
      float2 *xm = reinterpret_cast<float2 *>(smem + T_OFF_X) + (ui & 1) * 256;
      if (ok) {
        xm[ch * 128 + r] = make_float2(m_ref, l);
        mbar_arrive(&bars.x_full);
        ok = wait_all(&bars.x_full, ui & 1);
      }
      if (!ok) {
        timed_out = true;
        break;
      }
      if (!active) {
        mbar_arrive(&bars.o_free);
        continue;
      }
      const float2 other = xm[(1 - ch) * 128 + r];
      const float m0 = ch == 0 ? m_ref : other.x, l0 = ch == 0 ? l : other.y;
      const float m1 = ch == 0 ? other.x : m_ref, l1 = ch == 0 ? other.y : l;
      const float M = fmaxf(m0, m1);
      float f0 = (m0 == -INFINITY) ? 0.f : ex2(m0 - M);
      float f1 = (m1 == -INFINITY) ? 0.f : ex2(m1 - M);
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
      const float lsum = l0 * f0 + l1 * f1;
      if (U.whole) {
        const float inv = 1.f / lsum;
        f0 *= inv;
        f1 *= inv;
        T *op = reinterpret_cast<T *>(p.out) +
                ((int64_t)(U.row0 + tok) * p.num_q_heads + U.h * G + r % G) * kHeadDim + ch * 64;
#pragma unroll
        for (int cc = 0; cc < 2; ++cc) {
          uint4 w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t *ww = reinterpret_cast<uint32_t *>(&w[i]);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int d = 32 * cc + 8 * i + 2 * e;
              ww[e] = Pack<T>::from_f2(__uint_as_float(a[d]) * f0 + __uint_as_float(bq[d]) * f1,
                                       __uint_as_float(a[d + 1]) * f0 + __uint_as_float(bq[d + 1]) * f1);
            }
          }
          store_rows_coalesced(reinterpret_cast<uint4 *>(smem + T_OFF_STAGE + warp * kStageBytes), op + cc * 32, live,
                               w, lane);
        }
      } else if (live) {
        const int64_t slot = 2 * b + (ui > 0 ? 1 : 0);
        float4 *dst = reinterpret_cast<float4 *>(p.ws_o) + (slot * 32 + ch * 16) * 128 + r;  // [dims / 4][row]
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          float y[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            y[e] = __uint_as_float(a[4 * i + e]) * f0 + __uint_as_float(bq[4 * i + e]) * f1;
          dst[i * 128] = make_float4(y[0], y[1], y[2], y[3]);
        }
        if (ch == 0) p.ws_ml[slot * 128 + r] = make_float2(M, lsum);
      }
    }
    regs_dec<128>();
  } else {
    // every loader and MMA warp runs this one decrease (setmaxnreg acts on whole warpgroups)
    regs_dec<kRegsOther>();
    if (warp != kWarpMma) {
      // ---------------- loader warps (as the prefix loaders of decode_shared.cu) ----------------
      const int lw = warp - kWarpLoad0;
      const bool for_k = lw < kTKLoad;
      const int box = for_k ? lw + kTKLoad * lane : lw - kTKLoad + kTVLoad * lane;
      const int boxes = for_k ? 16 : 8, page = for_k ? box >> 1 : box;
      const int32_t *bt = nullptr;
      int npages = 0, wbase = 0;
      int32_t win = -1, win_next = -1;  // block ids of 4 key tiles, one per lane, and of the next 4
      auto ids_from = [&](int base) { return base + lane < npages ? __ldg(bt + base + lane) : -1; };
      auto open_run = [&](const TRun &U) {
        bt = p.block_tables + (int64_t)U.s * p.max_blocks_per_seq;
        npages = (U.len + kBlock - 1) / kBlock;
        wbase = U.ka * 8;
        win = ids_from(wbase);
        win_next = ids_from(wbase + 32);
      };
      auto id_of = [&](int t, int page) { return __shfl_sync(FULL, win, (t * 8 + page - wbase) & 31); };
      TRun U;
      if (x0 < x1) {
        U = trun_at<G>(pl, p.context_lens, x0, x1);
        open_run(U);
      }
      griddep_wait();  // Q, K and V may come from the kernels before
      int c = 0, ui = 0, issued = 0;
      for (int x = x0; x < x1 && !timed_out; ++ui) {
        if (ui > 0) {
          U = trun_at<G>(pl, p.context_lens, x, x1);
          open_run(U);
        }
        x += U.kb - U.ka;
        if (lw == 0 && lane == 0) {
          if (ui > 0 && !mbar_wait(&bars.q_free, (ui - 1) & 1)) {
            timed_out = true;
          } else {
            // (rows past the tree belong to other sequences or read as zeros; nothing is stored for them)
            mbar_arrive_expect_tx(&bars.q_full, 2 * kHalf);
            tma_load_3d(smem + T_OFF_Q, &qmap, &bars.q_full, 0, U.h * G, U.row0 + U.mt * TQ);
            tma_load_3d(smem + T_OFF_Q + kHalf, &qmap, &bars.q_full, 64, U.h * G, U.row0 + U.mt * TQ);
          }
        }
        timed_out = __any_sync(FULL, timed_out);
        for (int t = U.ka; t < U.kb && !timed_out; ++t, ++c) {
          if (t * 8 >= wbase + 32) {
            wbase += 32;
            win = win_next;
            win_next = ids_from(wbase + 32);
          }
          const int id = id_of(t, page);
          const bool in = box < boxes && t * 8 + page < npages;  // (the softmax warps zero V past the last key)
          const bool ok = in && (unsigned)id < (unsigned)p.num_blocks;
          const unsigned okmask = __ballot_sync(FULL, ok);
          const int st = for_k ? c % kTKStages : c % kTVStages;
          // the stage is free: S of the key tile two before, P V of the one three before
          if (for_k ? c >= kTKStages && !mbar_wait(&bars.s_full[st], ((c - kTKStages) / kTKStages) & 1)
                    : c >= kTVStages && !mbar_wait(&bars.pv_done[st], ((c - kTVStages) / kTVStages) & 1))
            timed_out = true;
          if (__any_sync(FULL, timed_out)) {
            timed_out = true;
            break;
          }
          const uint32_t bytes = for_k ? 2048u : (uint32_t)kVPage;
          uint8_t *dst = for_k ? smem + T_OFF_K + st * 2 * kHalf + (box & 1) * kHalf + page * 2048
                               : smem + T_OFF_V + st * 2 * kHalf + page * kVPage;
          uint64_t *bar = for_k ? &bars.k_full[st] : &bars.v_full[st];
          if (in && !ok) {  // rare: keep the products finite
            set_error(p.err, PA_ERR_RANGE, U.s);
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
      if (timed_out) {  // a short, bounded chance for this warp's copies in flight to land
        if (lw == 0 && ui > 0) mbar_wait(&bars.q_full, (ui - 1) & 1, kWaitLimitNs / 8);
        const int n = for_k ? kTKStages : kTVStages;
        for (int t = issued - n > 0 ? issued - n : 0; t < issued; ++t)
          mbar_wait(for_k ? &bars.k_full[t % n] : &bars.v_full[t % n], (t / n) & 1, kWaitLimitNs / 8);
      }
    } else {
      // ---------------- MMA issuer (warp-uniform loop, one elected lane issues) ----------------
      griddep_wait();
      if (lane == 0) {  // the join's record of this CTA (after the wait: the previous call's join may still read)
        JoinRecord rec = {};
        if (x0 < x1) {
          // The last run: found from the last pair, then from the start of its unit
          // (or of the CTA's share, whichever comes later) to see whether it began here.
          const TRun U = trun_at<G>(pl, p.context_lens, x1 - 1, x1);
          const int k0 = part_start(part_owner(U.ka, U.kt, U.blocks), U.kt, U.blocks);
          const int end = U.first_pair + part_start(part_owner(U.ka, U.kt, U.blocks) + 1, U.kt, U.blocks) - k0;
          if (U.first_pair >= x0 && k0 == 0 && (U.blocks > 1 || end > x1)) {
            rec.rows = min(TQ, U.n - U.mt * TQ) * G;
            rec.row0 = U.row0 + U.mt * TQ;
            rec.head0 = U.h * G;
            rec.pairs0 = pairs[U.s] + U.h * U.nmt * U.kt;
            rec.kt = U.kt;
            rec.nmt = U.nmt;
            rec.mt = U.mt;
            rec.blocks = U.blocks;
            rec.total = pl.total;
            rec.ctas = pl.ctas;
          }
        }
        reinterpret_cast<JoinRecord *>(p.records)[b] = rec;
      }
      __syncwarp();
      const bool leader = elect_one();
      auto wait_all = [&](uint64_t *bar, uint32_t parity) { return __all_sync(FULL, mbar_wait(bar, parity)) != 0; };
      const uint64_t qdesc = tc::desc_sw128(smem_u32(smem + T_OFF_Q), 16, 1024);
      const uint64_t kdesc0 = tc::desc_sw128(smem_u32(smem + T_OFF_K), 16, 1024);
      const uint64_t vdesc0 = tc::desc_sw128(smem_u32(smem + T_OFF_V), kVPage / 2, 1024);
      constexpr uint64_t kStageStep = (2 * kHalf) >> 4;
      constexpr uint64_t kHalfStep = kHalf >> 4;
      // the P V product of key tile pc (pending), issued once P is ready
      int pc = -1, p_run = 0;
      bool p_first = false;
      auto issue_pv = [&]() -> bool {
        const int jv = pc % kTVStages;
        if (!wait_all(&bars.p_full[jv], (pc / kTVStages) & 1)) return false;
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
        const TRun U = trun_at<G>(pl, p.context_lens, x, x1);
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
          const int ks = c % kTKStages;
          if (!wait_all(&bars.k_full[ks], (c / kTKStages) & 1)) {
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
      if (timed_out) {  // every MMA issued so far, bounded, before the tensor memory is freed
        if (leader) tc::commit(&bars.drain);
        __syncwarp();
        mbar_wait(&bars.drain, 0, kWaitLimitNs / 8);
      }
    }
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
// Block (b, part): the query tile of CTA b's record, a thread per row and 4 dims.
constexpr int kTJoinThreads = 128;
template <typename T, int G>
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
  // lanes: G neighbouring rows x 32 / G dim quads, so that pieces are read in runs and outputs are written so
  for (int i = (int)blockIdx.y * kTJoinThreads + (int)threadIdx.x; i < rec.rows * 32; i += gridDim.y * kTJoinThreads) {
    const int row = (i / 32) / G * G + i % G, quad = (i / G) % 32;
    JoinState js;
    constexpr int U = kTJoinPieces;
    for (int j = 0; j < rec.blocks; ++j) {
      const int k0 = part_start(j, rec.kt, rec.blocks), bl = part_start(j + 1, rec.kt, rec.blocks) - k0;
      const int xa = rec.pairs0 + rec.nmt * k0 + rec.mt * bl;  // the unit's first pair
      const int ff = part_owner(xa, rec.total, rec.ctas), fl = part_owner(xa + bl - 1, rec.total, rec.ctas);
      const int second = part_start(ff, rec.total, rec.ctas) < xa ? 1 : 0;  // the piece of CTA ff is not its first run
      for (int f0 = ff; f0 <= fl; f0 += U) {
        float2 ml[U];
        float4 o[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          ml[u] = make_float2(-INFINITY, 0.f);
          o[u] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (f0 + u <= fl) {
            const int64_t slot = 2 * (f0 + u) + (f0 + u == ff ? second : 0);
            ml[u] = __ldcg(p.ws_ml + slot * 128 + row);
            o[u] = __ldcg(reinterpret_cast<const float4 *>(p.ws_o) + (slot * 32 + quad) * 128 + row);
          }
        }
        js.add(ml, o);
      }
    }
    js.store(reinterpret_cast<T *>(p.out) +
             ((int64_t)(rec.row0 + row / G) * p.num_q_heads + rec.head0 + row % G) * kHeadDim + 4 * quad);
  }
}

template <typename T, int G>
cudaError_t launch_tree_typed(const TreeParams &p, const CUtensorMap *maps, int sms, cudaStream_t stream) {
  static KernelSetup setup;
  const int smem = 1024 + T_OFF_PLAN + 2 * (p.num_seqs + 1) * 4;
  cudaError_t e = kernel_setup(setup, attn_tree_kernel<T, G>, smem, kThreads, nullptr);
  if (e != cudaSuccess) return e;
  e = launch_pdl(attn_tree_kernel<T, G>, dim3(sms), dim3(kThreads), smem, stream, maps[0], maps[1], maps[2], p);
  if (e != cudaSuccess) return e;
  return launch_pdl(attn_tree_join_kernel<T, G>, dim3(sms, 8), dim3(kTJoinThreads), 0, stream, p);
}

struct TreeLayout {
  size_t ml, o, total;
};
TreeLayout tree_layout(int sms) {
  auto up = [](size_t n) { return (n + 255) & ~(size_t)255; };
  const size_t slots = 2 * (size_t)sms;  // a CTA's first and last run
  TreeLayout l;
  l.ml = up((size_t)sms * sizeof(JoinRecord));
  l.o = l.ml + up(slots * 128 * sizeof(float2));
  l.total = l.o + slots * 128 * kHeadDim * sizeof(float);
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
#define PA_TREE_CASE(T, G) \
  if (group == G) return launch_tree_typed<T, G>(p, maps, sms, stream);
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

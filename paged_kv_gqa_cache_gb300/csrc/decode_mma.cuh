#pragma once
// Split worker of the long-context decodes over a 16-bit pool, for sm_103a:
// the page ranges, fragments and log-sum-exp joins of decode_kernel.cuh, with
// the page step on mma.sync m16n8k16 (a decode has at most 8 query rows per KV
// head: too few for a 128-row tcgen05 tile, while on the CUDA cores 8 heads
// cost eight multiply-adds per K/V element and bound the call).
//
//   S = Q K^T      rows = the G query heads (rows G .. 15 zero), columns = the
//                  page's 16 keys (two n-tiles), k = the 128 dims; Q and K as
//                  they are (exact products, fp32 sums), the scale on the fp32
//                  scores.
//   O^T += V^T P^T rows = dims (m-tile mt: dims 16 mt ..), columns = heads, k
//                  = the 16 keys.  The C fragment of S is exactly the B
//                  fragment of this product, so P stays in registers.
//   P is fed as two terms, P_hi = round(P) and P_lo = round(P - P_hi), to the
//   16-bit type: one rounding of P would double the output's rounding variance
//   (each weight off by up to half a step), two keep P to 2^-16 or better for 8
//   more products per page, which the tensor cores have to spare.  fp16 ends at
//   2^-25 below and 65504 above, and the weights of a row may lie further apart
//   (tens of thousands of keys 18 nats below one, which carry the row where that
//   one's value is small): P is 2^15 at its largest there (kUnit), so that a weight
//   is off by 2^-40 of the row's largest at most beside the 2^-22 of its own.  The
//   factor stands in l and O alike and leaves both before they leave the warp.
//
// K and V pages land in the 128-byte swizzle (one 4 KB box each, the two
// 64-dim halves 2 KB apart), which ldmatrix reads without bank conflicts: K
// rows as the B operand, V rows transposed as the A operand, at one address
// formula.
#include "decode_kernel.cuh"

namespace pa {
namespace {

// The forms of the worker.
enum DecodeForm {
  kFormScores = 1,  // every key's scores go to the workspace, every item becomes fragments
  kFormSuffix = 2   // the keys past a shared prefix; an item of a sequence with a prefix becomes fragments
};
// The first of n ascending group ends behind sequence s (n: none).
__device__ __forceinline__ int group_of(const int32_t *end, int n, int s) {
  int lo = 0, hi = n;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (end[mid] <= s) lo = mid + 1; else hi = mid;
  }
  return lo;
}
struct FormArgs {
  float *scores = nullptr;             // kFormScores: [page of the global numbering][G][16 keys], log2 domain
  const int32_t *group_end = nullptr;  // kFormSuffix: sequences before the end of group g, ascending [num_groups]
  const int32_t *group_len = nullptr;  //   the tokens that its sequences share, a multiple of 16 (0: none)
  int32_t num_groups = 0;              //   sequences behind the last group share nothing
  __device__ __forceinline__ int shared_len(int s) const {
    const int g = group_of(group_end, num_groups, s);
    return g < num_groups ? group_len[g] : 0;
  }
};

// Exclusive prefix of pages(s) over sequences into prefix[0 .. n], by NT threads
// (warp_tot: NT / 32 ints of shared memory).
template <int NT, typename Pages>
__device__ void scan_pages_of(int n, int32_t *prefix, int *warp_tot, Pages pages) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int carry = 0;
  for (int s0 = 0; s0 < n; s0 += NT) {
    const int s = s0 + tid;
    const int mine = s < n ? pages(s) : 0;
    int incl = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int y = __shfl_up_sync(FULL, incl, off);
      if (lane >= off) incl += y;
    }
    if (lane == 31) warp_tot[warp] = incl;
    __syncthreads();
    int base = carry, total = 0;
#pragma unroll
    for (int i = 0; i < NT / 32; ++i) {
      base += (i < warp) ? warp_tot[i] : 0;
      total += warp_tot[i];
    }
    if (s < n) prefix[s] = base + incl - mine;
    carry += total;
    __syncthreads();
  }
  if (tid == 0) prefix[n] = carry;
  __syncthreads();
}

// The largest P of a row, a power of two.
template <typename T>
constexpr float kUnit = std::is_same<T, __half>::value ? 32768.f : 1.f;

template <typename T>
__device__ __forceinline__ void mma16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                      uint32_t b1) {
  if constexpr (std::is_same<T, __nv_bfloat16>::value)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Four 8 x 8 matrices of 16-bit elements from shared memory (lane l gives the
// row l % 8 of matrix l / 8), plain or transposed.  Volatile: the stage they
// read is refilled by a copy.
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// An item's running state: O^T fragments (lane (g, t) = (lane / 4, lane % 4):
// heads 2t and 2t + 1 at dims 16 mt + g and 16 mt + g + 8), and for head g the
// maximum (log2 domain, the same in its quad) and this lane's part of the sum;
// the sum and O are of kUnit 2^(s - m).
struct Mma16 {
  float acc[8][4];
  float m, l;
};

// The A operand of the G query rows (rows G .. 15 zero): head g at dims 16 ks +
// 2t, + 1 and + 8, + 9.
template <typename T, int G>
__device__ __forceinline__ void load_q16(const T *qp, int lane, uint32_t (&qa)[8][2]) {
  const int g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int ks = 0; ks < 8; ++ks) {
    qa[ks][0] = g < G ? *reinterpret_cast<const uint32_t *>(qp + g * kHeadDim + 16 * ks + 2 * t) : 0u;
    qa[ks][1] = g < G ? *reinterpret_cast<const uint32_t *>(qp + g * kHeadDim + 16 * ks + 2 * t + 8) : 0u;
  }
}

// One 16-key page at stage (K rows, then V rows 4 KB on), its first nv >= 1
// keys visible: scores, online softmax, O^T += V^T P^T.  scores: null, or where
// the page's [G][16] scores go.
template <typename T, int G>
__device__ __forceinline__ void decode_page16(uint32_t stage, int nv, const uint32_t (&qa)[8][2], float scale_log2,
                                              Mma16 &st, int lane, float *scores) {
  const int g = lane >> 2, t = lane & 3;
  // lane l addresses row l % 8 of matrix l / 8: keys 8 (matrix / 2) .., chunk 2 step + matrix % 2
  const int mrow = lane & 7, mkey = ((lane >> 4) << 3) + mrow, mchunk = (lane >> 3) & 1;
  const uint32_t row = stage + mkey * 128;
  float c[2][4] = {};
#pragma unroll
  for (int ks = 0; ks < 8; ++ks) {
    uint32_t b[4];
    ldsm4(b, row + (ks >> 2) * 2048 + (((2 * (ks & 3) + mchunk) ^ mrow) << 4));
    mma16<T>(c[0], qa[ks][0], 0u, qa[ks][1], 0u, b[0], b[1]);
    mma16<T>(c[1], qa[ks][0], 0u, qa[ks][1], 0u, b[2], b[3]);
  }
  float s[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) s[i] = c[i >> 1][i & 1] * scale_log2;
  const bool full = nv == kBlock;  // (warp-uniform)
  if (!full) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (8 * (i >> 1) + 2 * t + (i & 1) >= nv) s[i] = -INFINITY;
  }
  if (scores && g < G) {  // 32 contiguous bytes per head and store
    *reinterpret_cast<float2 *>(scores + g * kBlock + 2 * t) = make_float2(s[0], s[1]);
    *reinterpret_cast<float2 *>(scores + g * kBlock + 8 + 2 * t) = make_float2(s[2], s[3]);
  }
  float mx = fmaxf(fmaxf(s[0], s[1]), fmaxf(s[2], s[3]));
  mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, 1));
  mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, 2));
  const float mn = fmaxf(st.m, mx);
  const float base = mn == -INFINITY ? 0.f : mn;
  const float alpha = ex2(st.m - base);  // 0 while nothing was accumulated
  float p[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) p[i] = ex2(s[i] - base) * kUnit<T>;
  st.l = st.l * alpha + ((p[0] + p[1]) + (p[2] + p[3]));
  st.m = mn;
  // the accumulators hold heads 2t and 2t + 1: their factors come from those heads' quads
  const float f0 = __shfl_sync(FULL, alpha, 8 * t), f1 = __shfl_sync(FULL, alpha, 8 * t + 4);
  if (__any_sync(FULL, f0 != 1.f || f1 != 1.f)) {
#pragma unroll
    for (int mt = 0; mt < 8; ++mt) {
      st.acc[mt][0] *= f0;
      st.acc[mt][1] *= f1;
      st.acc[mt][2] *= f0;
      st.acc[mt][3] *= f1;
    }
  }
  uint32_t hi[2], lo[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    hi[i] = Pack<T>::from_f2(p[2 * i], p[2 * i + 1]);
    const float2 h = Pack<T>::to_f2(hi[i]);
    lo[i] = Pack<T>::from_f2(p[2 * i] - h.x, p[2 * i + 1] - h.y);
  }
  // value rows of keys that are not visible may hold any bytes (a NaN): zeroed in the fragments
  uint32_t keep0 = ~0u, keep1 = ~0u;
  if (!full) {
    keep0 = (2 * t < nv ? 0xffffu : 0u) | (2 * t + 1 < nv ? 0xffff0000u : 0u);
    keep1 = (2 * t + 8 < nv ? 0xffffu : 0u) | (2 * t + 9 < nv ? 0xffff0000u : 0u);
  }
#pragma unroll
  for (int mt = 0; mt < 8; ++mt) {
    uint32_t a[4];
    ldsm4_t(a, row + 4096 + (mt >> 2) * 2048 + (((2 * (mt & 3) + mchunk) ^ mrow) << 4));
    if (!full) {
      a[0] &= keep0;
      a[1] &= keep0;
      a[2] &= keep1;
      a[3] &= keep1;
    }
    mma16<T>(st.acc[mt], a[0], a[1], a[2], a[3], hi[0], hi[1]);
    mma16<T>(st.acc[mt], a[0], a[1], a[2], a[3], lo[0], lo[1]);
  }
}

// 5-D tiled load with an L2 eviction-priority hint.
__device__ __forceinline__ void tma_load_5d_hint(void *dst, const CUtensorMap *map, uint64_t *bar, int c0, int c1,
                                                 int c2, int c3, int c4, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3, %4, %5, %6}], [%7], %8;" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4), "r"(smem_u32(bar)), "l"(policy)
      : "memory");
}

// The join of online-softmax pieces for one head's 4 dims: pieces (m, l) with o
// come U at a time (m = -inf: none).
struct JoinState {
  float M = -INFINITY, L = 0.f;
  float4 O = {0.f, 0.f, 0.f, 0.f};
  template <int U>
  __device__ __forceinline__ void add(const float2 (&ml)[U], const float4 (&o)[U]) {
    float mx = M;
#pragma unroll
    for (int u = 0; u < U; ++u) mx = fmaxf(mx, ml[u].x);
    if (mx == -INFINITY) {  // no scores, or NaN alone (a maximum skips them): such a sum stays
#pragma unroll
      for (int u = 0; u < U; ++u) L += ml[u].y;
      return;
    }
    const float f = ex2(M - mx);
    L *= f;
    O.x *= f, O.y *= f, O.z *= f, O.w *= f;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const float w = ex2(ml[u].x - mx);
      L = fmaf(ml[u].y, w, L);
      O.x = fmaf(o[u].x, w, O.x);
      O.y = fmaf(o[u].y, w, O.y);
      O.z = fmaf(o[u].z, w, O.z);
      O.w = fmaf(o[u].w, w, O.w);
    }
    M = mx;
  }
  template <typename T>
  __device__ __forceinline__ void store(T *dst) const {
    const float inv = 1.f / L;
    uint2 pk;
    pk.x = Pack<T>::from_f2(O.x * inv, O.y * inv);
    pk.y = Pack<T>::from_f2(O.z * inv, O.w * inv);
    *reinterpret_cast<uint2 *>(dst) = pk;
  }
};

// ---- a split worker: a producer warp that fetches its pages, a consumer warp ----
// Worker w of W (as decode_split_worker): the pages [w P / W, (w + 1) P / W) of
// the global numbering, through a ring of kStages stages.  Two warps, because
// one that did both spent 480 of its 2450 cycles a page on the cursor, the block
// id and the two tensor copies.
struct PageRing {
  uint64_t full[kStages];  // the page landed (or cannot be read: bad)
  uint64_t free[kStages];  // the consumer has read it
  int32_t bad[kStages];
};
__device__ __forceinline__ void init_ring(PageRing &r) {  // one thread, before a barrier of both warps
#pragma unroll
  for (int st = 0; st < kStages; ++st) {
    mbar_init(&r.full[st], 1);
    mbar_init(&r.free[st], 1);
  }
}

// kmap, vmap: the pool's K and V in whole-page boxes, 128-byte swizzled; stages:
// kStages stages, 1024-byte aligned; prefix: the page prefix over sequences.
// Returns false if a wait gave up (reported by the caller).
template <int G, int FORM>
__device__ __forceinline__ bool split_producer16(const CUtensorMap &kmap, const CUtensorMap &vmap,
                                                 const DecodeParams &p, const FormArgs fa, uint8_t *stages,
                                                 PageRing &ring, const int32_t *prefix, int64_t w, int64_t P,
                                                 int64_t W) {
  const int lane = threadIdx.x & 31;
  const int n = p.num_seqs, hkv = p.num_kv_heads;
  const int64_t x0 = w * P / W;
  const int npages = (int)((w + 1) * P / W - x0);
  Cursor ic = locate(prefix, n, hkv, x0);
  int win_s = -1, win_base = -1, win_first = 0;
  int32_t win = -1;  // one of 32 block ids per lane
  // A page is read once: it leaves L2 to what is read again (scores, fragments,
  // shared keys).  With weights 97.4 -> 96.3 us and 157.7 -> 155.4 (32 and 5
  // sequences), shared prefixes 48.5 -> 47.7 and 101.5 -> 99.2 (32 and 192).
  const uint64_t once = policy_evict_first();
  int st = 0, phase = 1;  // a fresh ring is free: the first waits pass
  bool ok_all = true;
  for (int x = 0; x < npages; ++x) {
    const int base = ic.page & ~31;
    if (ic.s != win_s || base != win_base) {
      if constexpr (FORM == kFormSuffix)
        if (ic.s != win_s) win_first = fa.shared_len(ic.s) / kBlock;
      win_s = ic.s;
      win_base = base;
      win = base + lane < ic.pages
                ? __ldg(p.block_tables + (int64_t)ic.s * p.max_blocks_per_seq + win_first + base + lane)
                : -1;
    }
    if (ic.page == 0 && x > 0 && lane < 2 * G) {  // a new item: its query rows towards L2, pages ahead of their use
      const char *q = static_cast<const char *>(p.q) +
                      ((int64_t)ic.s * p.num_q_heads + (int64_t)ic.h * G) * (kHeadDim * 2) + lane * 128;
      asm volatile("prefetch.global.L2 [%0];" ::"l"(q));
    }
    const int blk = __shfl_sync(FULL, win, ic.page & 31);
    const bool ok = (unsigned)blk < (unsigned)p.num_blocks;
    if (!mbar_wait(&ring.free[st], phase)) ok_all = false;
    if (!__all_sync(FULL, ok_all)) {  // give the copies still in flight a short, bounded chance to land
      for (int y = x - kStages > 0 ? x - kStages : 0; y < x; ++y)
        mbar_wait(&ring.full[y % kStages], (y / kStages) & 1, kWaitLimitNs / 8);
      return false;
    }
    if (lane == 0) {
      ring.bad[st] = ok ? 0 : 1;
      if (ok) {
        mbar_arrive_expect_tx(&ring.full[st], STAGE);
        tma_load_5d_hint(stages + st * STAGE, &kmap, &ring.full[st], 0, 0, 0, ic.h, blk, once);
        tma_load_5d_hint(stages + st * STAGE + STAGE / 2, &vmap, &ring.full[st], 0, 0, 0, ic.h, blk, once);
      } else {
        set_error(p.err, PA_ERR_RANGE, ic.s);
        mbar_arrive(&ring.full[st]);
      }
    }
    __syncwarp();
    advance(ic, prefix, n, hkv);
    if (++st == kStages) st = 0, phase ^= 1;
  }
  return true;
}

template <typename T, int G, int FORM>
__device__ __forceinline__ bool split_consumer16(const DecodeParams &p, const FormArgs fa, const uint8_t *stages,
                                                 PageRing &ring, const int32_t *prefix, int64_t w, int64_t P,
                                                 int64_t W) {
  const int lane = threadIdx.x & 31;
  const int n = p.num_seqs, hkv = p.num_kv_heads;
  const int64_t x0 = w * P / W;
  const int npages = (int)((w + 1) * P / W - x0);
  Cursor cc = locate(prefix, n, hkv, x0);
  uint32_t qa[8][2];
  Mma16 st16;
  int ctx = 0, first = 0, st = 0, phase = 0;
  bool open = false, whole = false;
  const uint32_t stage0 = smem_u32(stages);
  float *scores = nullptr;
  if constexpr (FORM == kFormScores) scores = fa.scores + x0 * (kBlock * G);
  for (int x = 0; x < npages; ++x) {
    if (!open) {
      load_q16<T, G>(reinterpret_cast<const T *>(p.q) +
                         ((int64_t)cc.s * p.num_q_heads + (int64_t)cc.h * G) * kHeadDim,
                     lane, qa);  // (from L2: the producer asked for them pages ago)
#pragma unroll
      for (int mt = 0; mt < 8; ++mt) st16.acc[mt][0] = st16.acc[mt][1] = st16.acc[mt][2] = st16.acc[mt][3] = 0.f;
      st16.m = -INFINITY;
      st16.l = 0.f;
      ctx = __ldg(p.context_lens + cc.s);
      if constexpr (FORM == kFormSuffix) first = fa.shared_len(cc.s) / kBlock;
      whole = cc.page == 0;
      open = true;
    }
    if (!mbar_wait(&ring.full[st], phase)) return false;
    if (!ring.bad[st]) {
      decode_page16<T, G>(stage0 + st * STAGE, min(kBlock, ctx - (first + cc.page) * kBlock), qa, p.scale_log2, st16,
                          lane, scores);
    } else if constexpr (FORM == kFormScores) {  // a page that could not be read has no weight
      for (int i = lane; i < kBlock * G; i += 32) scores[i] = -INFINITY;
    }
    if constexpr (FORM == kFormScores) scores += kBlock * G;
    __syncwarp();  // every lane has read the stage
    if (lane == 0) mbar_arrive(&ring.free[st]);
    if (++st == kStages) st = 0, phase ^= 1;

    const bool last_of_item = cc.page == cc.pages - 1;
    if (last_of_item || x == npages - 1) {
      // lane (g, t): heads 2t, 2t + 1 at dims 16 mt + g, 16 mt + g + 8; head hh's (m, l) in lanes 4 hh .. 4 hh + 3
      const int g = lane >> 2, t = lane & 3;
      const bool final_out = FORM == kFormSuffix && whole && last_of_item && first == 0;
      float l = st16.l;
      l += __shfl_xor_sync(FULL, l, 1);
      l += __shfl_xor_sync(FULL, l, 2);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int hh = 2 * t + c;
        const float mh = __shfl_sync(FULL, st16.m, 4 * hh), lh = __shfl_sync(FULL, l, 4 * hh);
        if (hh < G) {
          if (final_out) {
            const float inv = 1.f / lh;
            T *op = reinterpret_cast<T *>(p.out) +
                    ((int64_t)cc.s * p.num_q_heads + cc.h * G + hh) * kHeadDim + g;
#pragma unroll
            for (int mt = 0; mt < 8; ++mt) {
              op[16 * mt] = (T)(st16.acc[mt][c] * inv);
              op[16 * mt + 8] = (T)(st16.acc[mt][2 + c] * inv);
            }
          } else {
            const int64_t fslot = ((int64_t)cc.s * hkv + cc.h + w) * G + hh;
            float *dst = p.ws_o + fslot * kHeadDim + g;
#pragma unroll
            for (int mt = 0; mt < 8; ++mt) {
              dst[16 * mt] = st16.acc[mt][c] * (1.f / kUnit<T>);
              dst[16 * mt + 8] = st16.acc[mt][2 + c] * (1.f / kUnit<T>);
            }
            if (g == 0) *reinterpret_cast<float2 *>(p.ws_ml + fslot * 2) = make_float2(mh, lh * (1.f / kUnit<T>));
          }
        }
      }
      open = false;
    }
    advance(cc, prefix, n, hkv);
  }
  return true;
}

}  // namespace
}  // namespace pa

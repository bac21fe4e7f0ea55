// Paged GQA decode that also accumulates the attention weight every cached
// token received, for sm_103a (the split worker: decode_mma.cuh).
//
//   out[s][g]           = softmax_j(scale q[s][g] . K_j) V_j
//   weights_out[s][h][j] = weights_in[s][h][j] + sum over the G query heads g of
//                          KV head h of their softmax weight of token j
//
// A weight needs its row's final maximum and sum, which exist only after the
// last page.  Reading K again would cost half of the decode; instead the split
// pass leaves each key's G scores (log2 domain, fp32: 4 G bytes next to the 512
// of its K and V rows) in the workspace, and the pass that joins the fragments
// turns them into weights: CTA (item, 0) joins the outputs, CTA (item, c > 0)
// takes kChunkKeys keys, first joining the (m, l) of the item's fragments
// itself (a few hundred bytes), so that no CTA waits for another.
// HBM-bound: K and V once; the scores and weights stream at 8 G + 8 bytes a key.
// 32 sequences of 100 to 8192 tokens, 32 / 8 heads, bf16: 95.5 .. 96.3 us (5.4
// TB/s; the split pass 86, at 6.0), 5 of 40000 to 100001, 32 / 4 heads: 153.8 ..
// 155.4 (5.4 TB/s; the split pass 137).  One sequence of 777: 7.6 us, of which the
// split pass takes 4.7.
#include "decode_mma.cuh"

namespace pa {
namespace {

constexpr int kChunkKeys = 2048;  // (1024: 97.5 and 157.4 us for the two batches below, 4096: 96.6 and 153.5)
constexpr int kJoinPieces = 8;    // fragments in flight (4: 97.3 and 161.4; 16: 98.3 and 154.7)
constexpr int kWeightThreads = 256;
constexpr int kKeysPerThread = kChunkKeys / kWeightThreads;
static_assert(kWeightThreads / 32 >= 8, "a warp per query head of a KV head");

// Per CTA kWorkers consumer warps, then their producer warps; per worker its
// stages and ring, then the page prefix.
constexpr int kWorkers = 4;
constexpr int kScoreThreads = 2 * kWorkers * 32;
constexpr int kRingOff = kWorkers * kStages * STAGE;
constexpr int kPrefixOff = (kRingOff + kWorkers * (int)sizeof(PageRing) + 15) / 16 * 16;

template <typename T, int G>
__global__ void __launch_bounds__(kScoreThreads, 2)
decode_scores_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                     const DecodeParams p, float *scores, int max_len) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  __shared__ int warp_tot[kScoreThreads / 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, slot = warp % kWorkers;
  PageRing *rings = reinterpret_cast<PageRing *>(smem + kRingOff);
  int32_t *prefix = reinterpret_cast<int32_t *>(smem + kPrefixOff);
  if (threadIdx.x == 0) {
    tma_prefetch_desc(&kmap);
    tma_prefetch_desc(&vmap);
    for (int i = 0; i < kWorkers; ++i) init_ring(rings[i]);
    fence_mbar_init();
  }
  FormArgs fa;
  fa.scores = scores;
  griddep_wait();
  scan_pages_of<kScoreThreads>(p.num_seqs, prefix, warp_tot, [&](int s) {
    const int ctx = __ldg(p.context_lens + s);
    if (ctx >= 1 && ctx <= (int64_t)p.max_blocks_per_seq * kBlock && ctx <= max_len) return (ctx + kBlock - 1) / kBlock;
    if (blockIdx.x == 0) set_error(p.err, PA_ERR_RANGE, s);
    return 0;
  });
  const int64_t P = (int64_t)prefix[p.num_seqs] * p.num_kv_heads;
  const int64_t W = P < p.num_workers ? P : p.num_workers;
  const int w = blockIdx.x * kWorkers + slot;
  if (blockIdx.x == 0 && warp == 0)  // for the pass that joins the fragments
    for (int i = lane; i <= p.num_seqs; i += 32) p.meta[i] = prefix[i];
  if (w < W) {
    uint8_t *stages = smem + slot * kStages * STAGE;
    const bool ok = warp < kWorkers
                        ? split_consumer16<T, G, kFormScores>(p, fa, stages, rings[slot], prefix, w, P, W)
                        : split_producer16<G, kFormScores>(kmap, vmap, p, fa, stages, rings[slot], prefix, w, P, W);
    if (!ok) set_error(p.err, PA_ERR_TIMEOUT, w);
  }
  griddep_launch_dependents();
}

template <typename T, int G>
__global__ void __launch_bounds__(kWeightThreads)
decode_weights_kernel(const DecodeParams p, const float *scores, const float *weights_in, float *weights_out,
                      int64_t weights_stride) {
  __shared__ float s_m[G], s_inv[G];
  griddep_wait();
  griddep_launch_dependents();  // (it writes nothing that a kernel may read before its own wait)
  const int item = blockIdx.y, hkv = p.num_kv_heads;
  const int s = item / hkv, h = item % hkv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int32_t first = __ldg(p.meta + s), pages = __ldg(p.meta + s + 1) - first;
  const int ctx = __ldg(p.context_lens + s);
  const int64_t P = (int64_t)__ldg(p.meta + p.num_seqs) * hkv;
  if (pages == 0) return;  // a bad length: reported, nothing written
  const int64_t W = P < p.num_workers ? P : p.num_workers;
  const int64_t A = (int64_t)hkv * first + (int64_t)h * pages;
  const int wf = worker_of(A, P, W), nf = worker_of(A + pages - 1, P, W) - wf + 1;
  const int64_t slot0 = (int64_t)item + wf;
  if (blockIdx.x == 0) {  // the outputs: warp -> head, lane -> its dims 4 lane ..
    for (int g = warp; g < G; g += kWeightThreads / 32) {
      JoinState js;
      for (int f0 = 0; f0 < nf; f0 += kJoinPieces) {
        float2 ml[kJoinPieces];
        float4 o[kJoinPieces];
#pragma unroll
        for (int u = 0; u < kJoinPieces; ++u) {
          ml[u] = make_float2(-INFINITY, 0.f);
          o[u] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (f0 + u < nf) {
            const int64_t slot = (slot0 + f0 + u) * G + g;
            ml[u] = __ldcg(reinterpret_cast<const float2 *>(p.ws_ml + slot * 2));
            o[u] = __ldcg(reinterpret_cast<const float4 *>(p.ws_o + slot * kHeadDim + 4 * lane));
          }
        }
        js.add(ml, o);
      }
      js.store(reinterpret_cast<T *>(p.out) + ((int64_t)s * p.num_q_heads + h * G + g) * kHeadDim + 4 * lane);
    }
    return;
  }
  const int j0 = ((int)blockIdx.x - 1) * kChunkKeys;
  if (j0 >= ctx) return;
  // this thread's keys j0 + thread + 256 u: their scores and weights on the way first
  const float *sc = scores + A * (kBlock * G);
  const int64_t row = (int64_t)item * weights_stride;
  constexpr int U = 4;  // keys in flight
  static_assert(kKeysPerThread % U == 0, "whole batches");
  float v[U][G], w[U];
  auto fetch = [&](int b) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = j0 + (int)threadIdx.x + (b + u) * kWeightThreads;
      w[u] = 0.f;
#pragma unroll
      for (int g = 0; g < G; ++g) v[u][g] = -INFINITY;
      if (k < ctx) {
        const float *page = sc + (int64_t)(k >> 4) * (kBlock * G) + (k & 15);
#pragma unroll
        for (int g = 0; g < G; ++g) v[u][g] = page[g * kBlock];
        if (weights_in) w[u] = weights_in[row + k];
      }
    }
  };
  fetch(0);
  if (warp < G) {  // head `warp`: the row's maximum and sum over its fragments
    float m = -INFINITY, l = 0.f;
    for (int f = lane; f < nf; f += 32) {
      const float2 ml = *reinterpret_cast<const float2 *>(p.ws_ml + ((slot0 + f) * G + warp) * 2);
      const float mn = fmaxf(m, ml.x);
      if (mn > -INFINITY) l = l * exp2f(m - mn) + ml.y * exp2f(ml.x - mn);
      m = mn;
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      const float m2 = __shfl_xor_sync(FULL, m, off), l2 = __shfl_xor_sync(FULL, l, off);
      const float mn = fmaxf(m, m2);
      if (mn > -INFINITY) l = l * exp2f(m - mn) + l2 * exp2f(m2 - mn);
      m = mn;
    }
    if (lane == 0) {
      s_m[warp] = m > -INFINITY ? m : 0.f;
      s_inv[warp] = l == 0.f ? 0.f : 1.f / l;  // (no page could be read: no weight; a NaN stays one)
    }
  }
  __syncthreads();
  float m[G], inv[G];
#pragma unroll
  for (int g = 0; g < G; ++g) {
    m[g] = s_m[g];
    inv[g] = s_inv[g];
  }
#pragma unroll
  for (int b = 0; b < kKeysPerThread; b += U) {
    if (b) fetch(b);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = j0 + (int)threadIdx.x + (b + u) * kWeightThreads;
      float sum = 0.f;
#pragma unroll
      for (int g = 0; g < G; ++g) sum = fmaf(exp2f(v[u][g] - m[g]), inv[g], sum);
      if (k < ctx) weights_out[row + k] = w[u] + sum;
    }
  }
}

template <typename T, int G>
cudaError_t launch_weights_typed(const DecodeParams &p0, const CUtensorMap &kmap, const CUtensorMap &vmap,
                                 const DecodeWeightsParams &wp, int sms, cudaStream_t stream) {
  DecodeParams p = p0;
  const int smem = 1024 + kPrefixOff + (p.num_seqs + 1) * 4;
  static KernelSetup setup;
  int per_sm = 0;
  cudaError_t e = kernel_setup(setup, decode_scores_kernel<T, G>, smem, kScoreThreads, &per_sm);
  if (e != cudaSuccess) return e;
  int grid = sms * per_sm;
  const int64_t pages = (int64_t)p.num_seqs * p.num_kv_heads * ((wp.max_len + kBlock - 1) / kBlock);
  const int64_t want = ((pages + 3) / 4 + kWorkers - 1) / kWorkers;  // at least 4 pages per worker
  if (want < grid) grid = (int)want;
  if (grid < 1) grid = 1;
  if (grid * kWorkers > kDecodeMaxWorkers) grid = kDecodeMaxWorkers / kWorkers;
  p.num_workers = grid * kWorkers;
  e = launch_pdl(decode_scores_kernel<T, G>, dim3(grid), dim3(kScoreThreads), smem, stream, kmap, vmap, p, wp.scores,
                 wp.max_len);
  if (e != cudaSuccess) return e;
  const dim3 wgrid(1 + (wp.max_len + kChunkKeys - 1) / kChunkKeys, p.num_seqs * p.num_kv_heads);
  return launch_pdl(decode_weights_kernel<T, G>, wgrid, dim3(kWeightThreads), 0, stream, p,
                    (const float *)wp.scores, wp.weights_in, wp.weights_out, wp.weights_stride);
}

}  // namespace

cudaError_t launch_decode_weights(const DecodeParams &p, const CUtensorMap &kmap, const CUtensorMap &vmap, int dtype,
                                  int group, const DecodeWeightsParams &wp, int sms, cudaStream_t stream) {
#define PA_WEIGHTS_CASE(T, G) \
  if (group == G) return launch_weights_typed<T, G>(p, kmap, vmap, wp, sms, stream);
  if (dtype == PA_BF16) {
    PA_WEIGHTS_CASE(__nv_bfloat16, 1)
    PA_WEIGHTS_CASE(__nv_bfloat16, 2)
    PA_WEIGHTS_CASE(__nv_bfloat16, 4)
    PA_WEIGHTS_CASE(__nv_bfloat16, 8)
  } else {
    PA_WEIGHTS_CASE(__half, 1)
    PA_WEIGHTS_CASE(__half, 2)
    PA_WEIGHTS_CASE(__half, 4)
    PA_WEIGHTS_CASE(__half, 8)
  }
#undef PA_WEIGHTS_CASE
  return cudaErrorInvalidValue;
}

}  // namespace pa

// Rotary embedding of new queries and keys, with the K/V rows written into
// their slots, for sm_103a: half or interleaved layout, the whole head or its
// first rotary_dim dims, any frequencies (scaled for long contexts by the
// caller), optional RMSNorm in front (page "Модуль 12: Финальный проект:
// мини-движок инференса", qwen_serve/model.py, apply_rope; page "Модуль 04:
// KV-кэш и арифметика памяти", section 4: the key is rotated to its absolute
// position before it is stored).
//
// For each new token at position p, with angle_i = p * inv_freq[i] and (c, s)
// = attention_factor * (cos, sin)(angle_i), a pair (a, b) of a query or key
// row becomes (a c - b s, b c + a s): dims i and i + d / 2 in the half layout,
// 2 i and 2 i + 1 in the interleaved one; dims past d = rotary_dim and value
// rows pass through.  fp32 throughout, rounded once to the 16-bit type.
//
// Angles.  At a far position the product p * inv_freq loses its fraction in
// fp32 (2^20 rad leave 2^-4 rad), and fp64 trigonometry is slow on this part.
// The frequency in turns (inv_freq / 2 pi, a double, once per thread and
// launch) is held as a 64-bit fixed-point fraction; p times it modulo 2^64 is
// then the exact fraction of a turn of that frequency, whatever p, in one
// integer multiplication, and its top 32 bits go through sincospif.  The
// phase error is p * 2^-53 of the frequency (what fp64 itself would leave)
// plus pi * 2^-25 from the conversion to fp32.
//
// HBM-bound: one pass over q, k and v (24.6 KB in and out per token at 32 / 8
// heads).  16 lanes hold one head row, 8 values each, chosen so that a lane
// holds both values of its 4 pairs: dims 4 l .. and d / 2 + 4 l .. of the
// rotated part in the half layout (two 8-byte accesses), 8 l .. in the
// interleaved one, so that no value crosses a lane and a lane's 4 (cos, sin)
// stay in registers for all rows of the token.  A CTA takes 4 tokens at a time
// (2 warps each), or, when there are too few tokens to fill the GPU so, one
// (8 warps): its threads compute the tokens' angles once for all heads, through
// shared memory (two buffers, one barrier per step), while the first rows'
// loads are on their way.
#include "pa_device.cuh"

namespace pa {
namespace {

constexpr unsigned FULL = 0xffffffffu;
constexpr int kRopeKvThreads = 256;
constexpr int kBatch = 4;  // rows per half-warp whose loads are in flight together

// kPairs: a lane holds both values of its pairs (interleaved, or half with
// rotary_dim a multiple of 8); kExchange: any even rotary_dim in the half
// layout, values exchanged through shared memory.
enum RopeMode { kInterleaved = 0, kHalfPairs = 1, kHalfExchange = 2 };

// The fraction of a turn per position as a 64-bit fixed-point number.
__device__ __forceinline__ long long turns_fixed(double inv_freq) {
  const double t = inv_freq * 0.15915494309189533577;  // 1 / (2 pi)
  return __double2ll_rn((t - rint(t)) * 18446744073709551616.0);
}

// TOK tokens per CTA and step, 8 / TOK warps each.
template <typename T, int MODE, bool NORM, int TOK>
__global__ void __launch_bounds__(kRopeKvThreads, 4) rope_kv_kernel(const RopeKvParams p) {
  constexpr int kWarps = kRopeKvThreads / 32 / TOK;  // warps per token
  constexpr int kStep = 2 * kWarps;                  // rows per pass of them
  __shared__ __align__(16) float2 cs_buf[2][TOK][kHeadDim / 2];
  __shared__ float stage_buf[MODE == kHalfExchange ? kRopeKvThreads / 16 * kHeadDim : 1];
  const int tid = threadIdx.x, lane = tid & 31, l16 = lane & 15;
  const int hq = p.num_q_heads, hkv = p.num_kv_heads;
  const int rows = hq + 2 * hkv, d = p.rotary_dim;
  // this lane's values: dims d0 .. d0 + 3 and d1 .. d1 + 3; its pairs' angles: pair 4 l16 + i
  const bool split = MODE == kHalfPairs && 8 * l16 < d;
  const int d0 = split ? 4 * l16 : 8 * l16, d1 = split ? d / 2 + 4 * l16 : 8 * l16 + 4;
  float *stage = stage_buf + (MODE == kHalfExchange ? (tid >> 4) * kHeadDim : 0);
  const int tok = tid / (32 * kWarps);                          // this warp's token of the step
  const int r_first = ((tid >> 5) % kWarps) * 2 + (lane >> 4);  // this half-warp's first row
  griddep_wait();  // q, k, v may be the previous kernel's output; the pool may be read by it
  long long turns = 0;
  if (tid < TOK * 64 && (tid & 63) < d / 2) turns = turns_fixed(__ldg(p.inv_freq + (tid & 63)));
  uint2 wq[2], wk[2];
  if constexpr (NORM) {
    wq[0] = *reinterpret_cast<const uint2 *>(static_cast<const T *>(p.q_weight) + d0);
    wq[1] = *reinterpret_cast<const uint2 *>(static_cast<const T *>(p.q_weight) + d1);
    wk[0] = *reinterpret_cast<const uint2 *>(static_cast<const T *>(p.k_weight) + d0);
    wk[1] = *reinterpret_cast<const uint2 *>(static_cast<const T *>(p.k_weight) + d1);
  }
  int buf = 0;
  for (int t0 = blockIdx.x * TOK; t0 < p.num_tokens; t0 += gridDim.x * TOK) {  // (block-uniform)
    const int t = t0 + tok;
    const int pos = t < p.num_tokens ? __ldg(p.positions + t) : -1;
    const int64_t slot = t < p.num_tokens ? __ldg(p.slots + t) : -1;
    const bool ok = pos >= 0 && slot >= 0 && slot < p.num_slots;  // else nothing of the token is written
    if (!ok && t < p.num_tokens && tid % (32 * kWarps) == 0) set_error(p.err, PA_ERR_RANGE, t);
    auto load = [&](int r, uint2 (&x)[2]) {
      const T *src = r < hq         ? static_cast<const T *>(p.q) + ((int64_t)t * hq + r) * kHeadDim
                     : r < hq + hkv ? static_cast<const T *>(p.k) + ((int64_t)t * hkv + (r - hq)) * kHeadDim
                                    : static_cast<const T *>(p.v) + ((int64_t)t * hkv + (r - hq - hkv)) * kHeadDim;
      if constexpr (MODE == kHalfPairs) {
        x[0] = *reinterpret_cast<const uint2 *>(src + d0);
        x[1] = *reinterpret_cast<const uint2 *>(src + d1);
      } else {
        const uint4 u = *reinterpret_cast<const uint4 *>(src + d0);
        x[0] = make_uint2(u.x, u.y);
        x[1] = make_uint2(u.z, u.w);
      }
    };
    uint2 raw[kBatch][2];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int r = r_first + i * kStep;
      raw[i][0] = raw[i][1] = make_uint2(0, 0);
      if (ok && r < rows) load(r, raw[i]);
    }
    // the step's angles, while the rows are on their way
    if (tid < TOK * 64 && (tid & 63) < d / 2) {
      const int at = t0 + (tid >> 6);
      const int pa = at < p.num_tokens ? __ldg(p.positions + at) : 0;
      const long long turn = (long long)((unsigned long long)turns * (unsigned long long)(unsigned)pa);
      float s, c;
      sincospif((float)(int)(turn >> 32) * 4.656612873077393e-10f, &s, &c);  // 2^-31: half turns
      cs_buf[buf][tid >> 6][tid & 63] = make_float2(c * p.attention_factor, s * p.attention_factor);
    }
    __syncthreads();
    if (ok) {  // (warp-uniform)
      float2 cs[4];
      if constexpr (MODE != kHalfExchange) {
        const float4 *src = reinterpret_cast<const float4 *>(cs_buf[buf][tok] + 4 * l16);
        const float4 u = src[0], v = src[1];  // (pairs past rotary_dim / 2 are not used)
        cs[0] = make_float2(u.x, u.y), cs[1] = make_float2(u.z, u.w);
        cs[2] = make_float2(v.x, v.y), cs[3] = make_float2(v.z, v.w);
      }
      for (int r0 = 0; r0 < rows; r0 += kStep * kBatch) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const int r = r0 + r_first + i * kStep;
          if (r0 + i * kStep + ((tid >> 5) % kWarps) * 2 >= rows) break;  // (warp-uniform)
          uint2 out[2] = {raw[i][0], raw[i][1]};
          if (r0 + i * kStep + ((tid >> 5) % kWarps) * 2 < hq + hkv) {  // the warp holds a query or key row
            float x[8];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const float2 f = Pack<T>::to_f2(raw[i][k].x), g = Pack<T>::to_f2(raw[i][k].y);
              x[4 * k] = f.x, x[4 * k + 1] = f.y, x[4 * k + 2] = g.x, x[4 * k + 3] = g.y;
            }
            float inv = 1.f;
            if constexpr (NORM) {
              float ss = 0.f;
#pragma unroll
              for (int k = 0; k < 8; ++k) ss = fmaf(x[k], x[k], ss);
#pragma unroll
              for (int off = 8; off > 0; off >>= 1) ss += __shfl_xor_sync(FULL, ss, off);
              inv = rsqrtf(ss * (1.f / kHeadDim) + p.eps);
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const uint2 w = r < hq ? wq[k] : wk[k];
                const float2 f = Pack<T>::to_f2(w.x), g = Pack<T>::to_f2(w.y);
                x[4 * k] *= f.x * inv, x[4 * k + 1] *= f.y * inv;
                x[4 * k + 2] *= g.x * inv, x[4 * k + 3] *= g.y * inv;
              }
            }
            if constexpr (MODE == kInterleaved) {
#pragma unroll
              for (int k = 0; k < 4; ++k)
                if (8 * l16 + 2 * k < d) {
                  const float a = x[2 * k], b = x[2 * k + 1];
                  x[2 * k] = a * cs[k].x - b * cs[k].y;
                  x[2 * k + 1] = b * cs[k].x + a * cs[k].y;
                }
            } else if constexpr (MODE == kHalfPairs) {
              if (split) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  const float a = x[k], b = x[4 + k];
                  x[k] = a * cs[k].x - b * cs[k].y;
                  x[4 + k] = b * cs[k].x + a * cs[k].y;
                }
              }
            } else {
#pragma unroll
              for (int k = 0; k < 8; ++k) stage[8 * l16 + k] = x[k];
              __syncwarp();
              const int half = d >> 1;
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                const int j = 8 * l16 + k;
                if (j < d) {
                  const bool low = j < half;
                  const float2 c = cs_buf[buf][tok][low ? j : j - half];
                  const float y = stage[low ? j + half : j - half];
                  x[k] = x[k] * c.x + (low ? -y : y) * c.y;
                }
              }
              __syncwarp();
            }
            if (r < hq + hkv) {
#pragma unroll
              for (int k = 0; k < 2; ++k)
                out[k] = make_uint2(Pack<T>::from_f2(x[4 * k], x[4 * k + 1]),
                                    Pack<T>::from_f2(x[4 * k + 2], x[4 * k + 3]));
            }
          }
          if (r < rows) {
            T *dst = r < hq         ? static_cast<T *>(p.q_out) + ((int64_t)t * hq + r) * kHeadDim
                     : r < hq + hkv ? static_cast<T *>(p.k_cache) + (slot * hkv + (r - hq)) * kHeadDim
                                    : static_cast<T *>(p.v_cache) + (slot * hkv + (r - hq - hkv)) * kHeadDim;
            if constexpr (MODE == kHalfPairs) {
              *reinterpret_cast<uint2 *>(dst + d0) = out[0];
              *reinterpret_cast<uint2 *>(dst + d1) = out[1];
            } else {
              *reinterpret_cast<uint4 *>(dst + d0) = make_uint4(out[0].x, out[0].y, out[1].x, out[1].y);
            }
          }
          const int rn = r + kStep * kBatch;  // this buffer's next row
          if (rn < rows) load(rn, raw[i]);
        }
      }
    }
    buf ^= 1;  // a thread is at most one step ahead of the slowest (the barrier), so two buffers do
  }
  griddep_launch_dependents();
}

template <typename T, int TOK>
cudaError_t launch_rope_kv_typed(const RopeKvParams &p, int grid, cudaStream_t stream) {
  const int mode = p.interleaved ? kInterleaved : p.rotary_dim % 8 == 0 ? kHalfPairs : kHalfExchange;
#define PA_ROPE_CASE(M, N) \
  if (mode == M && (p.q_weight != nullptr) == N) \
    return launch_pdl(rope_kv_kernel<T, M, N, TOK>, dim3(grid), dim3(kRopeKvThreads), 0, stream, p);
  PA_ROPE_CASE(kInterleaved, false)
  PA_ROPE_CASE(kInterleaved, true)
  PA_ROPE_CASE(kHalfPairs, false)
  PA_ROPE_CASE(kHalfPairs, true)
  PA_ROPE_CASE(kHalfExchange, false)
  PA_ROPE_CASE(kHalfExchange, true)
#undef PA_ROPE_CASE
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_rope_kv(const RopeKvParams &p, int dtype, int sms, cudaStream_t stream) {
  const int cap = sms * 4;  // one wave: 4 CTAs fit on an SM
  if (p.num_tokens <= cap) {  // a token per CTA
    return dtype == PA_BF16 ? launch_rope_kv_typed<__nv_bfloat16, 1>(p, p.num_tokens, stream)
                            : launch_rope_kv_typed<__half, 1>(p, p.num_tokens, stream);
  }
  const int want = (p.num_tokens + 3) / 4, grid = want < cap ? want : cap;
  return dtype == PA_BF16 ? launch_rope_kv_typed<__nv_bfloat16, 4>(p, grid, stream)
                          : launch_rope_kv_typed<__half, 4>(p, grid, stream);
}

}  // namespace pa

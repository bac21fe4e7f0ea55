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
// heads), if the issue slots allow it.  16 lanes hold one head row, 8 values
// each, chosen so that a lane holds both values of its 4 pairs: dims 4 l .. and
// d / 2 + 4 l .. of the rotated part in the half layout (two 8-byte accesses),
// 8 l .. in the interleaved one, so that no value crosses a lane and a lane's 4
// (cos, sin) stay in registers for all rows of the token.  Queries, keys and
// values are swept one kind after the other, so that a row costs no address
// beyond a constant offset and the norm's weights are widened once per kind,
// and two fp32 values go through one instruction.  A CTA takes 4 tokens at a
// time (2 warps each), or, when there are too few tokens to fill the GPU so,
// one (8 warps): its threads compute the tokens' angles once for all heads,
// through shared memory (two buffers, one barrier per step), while the first
// rows' loads are on their way.
// 16383 tokens of 32 / 8 heads with the norm, bf16: 64.6 us, 6.24 TB/s; with
// all rows in one loop, addresses and weights per row, it was issue-bound at
// 76.8, and with 4 CTAs on an SM, 64 registers and spills, 72.  512 tokens,
// without: 3.4 us; 8 tokens of 16 / 8 heads: 1.7.
//
// AXES: pair i turns by the position on axis pair_axis[i] (of up to four: time, height
// and width of images and video); a thread then multiplies each of its pairs by its own
// axis's position, the rest is the same.  A variant of its own, because the choice in
// the loop slowed the call with one axis (75 against 69.5 us of graph time, the 16383
// tokens).  16383 tokens of 32 / 8 heads with the norm, three axes, bf16: 71.5 us, 0.83 of
// the copy rate; 911 tokens without: 4.6; 8 of 16 / 8 heads: 2.0.  A step's positions
// loaded a step ahead: 76 (registers).
#include "pa_device.cuh"

namespace pa {
namespace {

constexpr unsigned FULL = 0xffffffffu;
constexpr int kRopeKvThreads = 256;
constexpr int kBatchQ = 4, kBatchKv = 2;  // rows of a kind per half-warp whose loads are in flight together

// kPairs: a lane holds both values of its pairs (interleaved, or half with
// rotary_dim a multiple of 8); kExchange: any even rotary_dim in the half
// layout, values exchanged through shared memory.
enum RopeMode { kInterleaved = 0, kHalfPairs = 1, kHalfExchange = 2 };

// The fraction of a turn per position as a 64-bit fixed-point number.
__device__ __forceinline__ long long turns_fixed(double inv_freq) {
  const double t = inv_freq * 0.15915494309189533577;  // 1 / (2 pi)
  return __double2ll_rn((t - rint(t)) * 18446744073709551616.0);
}

__device__ __forceinline__ float2 twice(float a) { return make_float2(a, a); }

// TOK tokens per CTA and step, 8 / TOK warps each.
template <typename T, int MODE, bool NORM, int TOK, bool AXES>
__global__ void __launch_bounds__(kRopeKvThreads, 3) rope_kv_kernel(const RopeKvParams p) {
  constexpr int kWarps = kRopeKvThreads / 32 / TOK;  // warps per token
  constexpr int kStep = 2 * kWarps;                  // rows per pass of them
  __shared__ __align__(16) float2 cs_buf[2][TOK][kHeadDim / 2];
  __shared__ __align__(16) float stage_buf[MODE == kHalfExchange ? kRopeKvThreads / 16 * kHeadDim : 1];
  const int tid = threadIdx.x, lane = tid & 31, l16 = lane & 15;
  const int hq = p.num_q_heads, hkv = p.num_kv_heads, d = p.rotary_dim;
  // this lane's values: dims d0 .. d0 + 3 and d1 .. d1 + 3; its pairs' angles: pair 4 l16 + i
  const bool split = MODE == kHalfPairs && 8 * l16 < d;
  const int d0 = split ? 4 * l16 : 8 * l16, d1 = split ? d / 2 + 4 * l16 : 8 * l16 + 4;
  float *stage = stage_buf + (MODE == kHalfExchange ? (tid >> 4) * kHeadDim : 0);
  const int tok = tid / (32 * kWarps);  // this warp's token of the step
  // The first rows of this warp's pair of half-warps: of the queries and keys,
  // and of the values, which start with the other half of the warps.
  const int w_qk = ((tid >> 5) % kWarps) * 2, w_v = (w_qk + kStep / 2) % kStep;
  const int r_qk = w_qk + (lane >> 4), r_v = w_v + (lane >> 4);
  griddep_wait();  // q, k, v may be the previous kernel's output; the pool may be read by it
  long long turns = 0;
  int64_t axis = 0;  // where the positions of this thread's pair begin
  if (tid < TOK * 64 && (tid & 63) < d / 2) {
    turns = turns_fixed(__ldg(p.inv_freq + (tid & 63)));
    if (AXES) axis = (int64_t)p.pair_axis[tid & 63] * p.num_tokens;
  }
  auto read = [&](const T *src, uint2 (&x)[2]) {
    if constexpr (MODE == kHalfPairs) {
      x[0] = *reinterpret_cast<const uint2 *>(src + d0);
      x[1] = *reinterpret_cast<const uint2 *>(src + d1);
    } else {
      const uint4 u = *reinterpret_cast<const uint4 *>(src + d0);
      x[0] = make_uint2(u.x, u.y);
      x[1] = make_uint2(u.z, u.w);
    }
  };
  auto write = [&](T *dst, const uint2 (&x)[2]) {
    if constexpr (MODE == kHalfPairs) {
      *reinterpret_cast<uint2 *>(dst + d0) = x[0];
      *reinterpret_cast<uint2 *>(dst + d1) = x[1];
    } else {
      *reinterpret_cast<uint4 *>(dst + d0) = make_uint4(x[0].x, x[0].y, x[1].x, x[1].y);
    }
  };
  auto widen = [](const uint2 (&u)[2], float2 (&x)[4]) {
    x[0] = Pack<T>::to_f2(u[0].x), x[1] = Pack<T>::to_f2(u[0].y);
    x[2] = Pack<T>::to_f2(u[1].x), x[3] = Pack<T>::to_f2(u[1].y);
  };
  int buf = 0;
  for (int t0 = blockIdx.x * TOK; t0 < p.num_tokens; t0 += gridDim.x * TOK) {  // (block-uniform)
    const int t = t0 + tok;
    int pos = t < p.num_tokens ? __ldg(p.positions + t) : -1;
    if (AXES && t < p.num_tokens) {
#pragma unroll
      for (int a = 1; a < PA_ROPE_MAX_AXES; ++a)  // (their signs; all loads on their way together)
        pos |= a < p.num_axes ? __ldg(p.positions + (int64_t)a * p.num_tokens + t) : 0;
    }
    const int64_t slot = t < p.num_tokens ? __ldg(p.slots + t) : -1;
    const bool ok = pos >= 0 && slot >= 0 && slot < p.num_slots;  // else nothing of the token is written
    if (!ok && t < p.num_tokens && tid % (32 * kWarps) == 0) set_error(p.err, PA_ERR_RANGE, t);
    const T *q = static_cast<const T *>(p.q) + ((int64_t)t * hq + r_qk) * kHeadDim;
    const T *k = static_cast<const T *>(p.k) + ((int64_t)t * hkv + r_qk) * kHeadDim;
    const T *v = static_cast<const T *>(p.v) + ((int64_t)t * hkv + r_v) * kHeadDim;
    // the first rows of each kind, all on their way together
    uint2 raw_q[kBatchQ][2] = {}, raw_k[kBatchKv][2] = {}, raw_v[kBatchKv][2] = {};
    if (ok) {
#pragma unroll
      for (int i = 0; i < kBatchQ; ++i)
        if (r_qk + i * kStep < hq) read(q + i * kStep * kHeadDim, raw_q[i]);
#pragma unroll
      for (int i = 0; i < kBatchKv; ++i) {
        if (r_qk + i * kStep < hkv) read(k + i * kStep * kHeadDim, raw_k[i]);
        if (r_v + i * kStep < hkv) read(v + i * kStep * kHeadDim, raw_v[i]);
      }
    }
    // the step's angles, meanwhile
    if (tid < TOK * 64 && (tid & 63) < d / 2) {
      const int at = t0 + (tid >> 6);
      const int pa = at < p.num_tokens ? __ldg(p.positions + axis + at) : 0;
      const long long turn = (long long)((unsigned long long)turns * (unsigned long long)(unsigned)pa);
      float s, c;
      sincospif((float)(int)(turn >> 32) * 4.656612873077393e-10f, &s, &c);  // 2^-31: half turns
      cs_buf[buf][tid >> 6][tid & 63] = make_float2(c * p.attention_factor, s * p.attention_factor);
    }
    __syncthreads();
    if (ok) {  // (warp-uniform)
      float2 c[2], s[2], ns[2];  // of this lane's 4 pairs: cos, sin, -sin
      if constexpr (MODE != kHalfExchange) {
        const float4 *src = reinterpret_cast<const float4 *>(cs_buf[buf][tok] + 4 * l16);
        const float4 a = src[0], b = src[1];  // (pairs past rotary_dim / 2 are not used)
        c[0] = make_float2(a.x, a.z), s[0] = make_float2(a.y, a.w), ns[0] = make_float2(-a.y, -a.w);
        c[1] = make_float2(b.x, b.z), s[1] = make_float2(b.y, b.w), ns[1] = make_float2(-b.y, -b.w);
      }
      float2 weight[4];  // of the norm, for the kind of row at hand
      auto rotate = [&](uint2 (&u)[2]) {
        float2 x[4];
        widen(u, x);
        if constexpr (NORM) {
          float2 sq = __fmul2_rn(x[0], x[0]);
#pragma unroll
          for (int i = 1; i < 4; ++i) sq = __ffma2_rn(x[i], x[i], sq);
          float ss = sq.x + sq.y;
#pragma unroll
          for (int off = 8; off > 0; off >>= 1) ss += __shfl_xor_sync(FULL, ss, off);
          const float2 inv = twice(rsqrtf(ss * (1.f / kHeadDim) + p.eps));
#pragma unroll
          for (int i = 0; i < 4; ++i) x[i] = __fmul2_rn(__fmul2_rn(x[i], inv), weight[i]);
        }
        if constexpr (MODE == kInterleaved) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (8 * l16 + 2 * i < d) {
              const float cc = i & 1 ? c[i >> 1].y : c[i >> 1].x, sc = i & 1 ? s[i >> 1].y : s[i >> 1].x;
              x[i] = make_float2(x[i].x * cc - x[i].y * sc, x[i].y * cc + x[i].x * sc);
            }
        } else if constexpr (MODE == kHalfPairs) {
          if (split) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float2 a = x[i], b = x[2 + i];
              x[i] = __ffma2_rn(b, ns[i], __fmul2_rn(a, c[i]));
              x[2 + i] = __ffma2_rn(a, s[i], __fmul2_rn(b, c[i]));
            }
          }
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) reinterpret_cast<float2 *>(stage)[4 * l16 + i] = x[i];
          __syncwarp();
          const int half = d >> 1;
          auto turned = [&](int j, float y) {
            if (j >= d) return y;
            const bool low = j < half;
            const float2 w = cs_buf[buf][tok][low ? j : j - half];
            const float z = stage[low ? j + half : j - half];
            return y * w.x + (low ? -z : z) * w.y;
          };
#pragma unroll
          for (int i = 0; i < 4; ++i)
            x[i] = make_float2(turned(8 * l16 + 2 * i, x[i].x), turned(8 * l16 + 2 * i + 1, x[i].y));
          __syncwarp();
        }
        u[0] = make_uint2(Pack<T>::from_f2(x[0].x, x[0].y), Pack<T>::from_f2(x[1].x, x[1].y));
        u[1] = make_uint2(Pack<T>::from_f2(x[2].x, x[2].y), Pack<T>::from_f2(x[3].x, x[3].y));
      };
      // All rows of a kind: n of them, this warp's from w on, this half-warp's
      // first at src and dst; a buffer's next row is fetched once it is free.
      auto sweep = [&](auto &raw, const T *src, T *dst, int n, int w, auto &&compute) {
        constexpr int B = sizeof(raw) / sizeof(raw[0]);
        for (; w < n; w += B * kStep, src += B * kStep * kHeadDim, dst += B * kStep * kHeadDim) {
#pragma unroll
          for (int i = 0; i < B; ++i) {
            if (w + i * kStep >= n) break;  // (warp-uniform)
            const int r = w + i * kStep + (lane >> 4);
            compute(raw[i]);
            if (r < n) write(dst + i * kStep * kHeadDim, raw[i]);
            if (r + B * kStep < n) read(src + (B + i) * kStep * kHeadDim, raw[i]);
          }
        }
      };
      auto weigh = [&](const void *of) {
        if constexpr (NORM) {
          uint2 u[2];
          read(static_cast<const T *>(of), u);
          widen(u, weight);
        }
      };
      weigh(p.q_weight);
      sweep(raw_q, q, static_cast<T *>(p.q_out) + ((int64_t)t * hq + r_qk) * kHeadDim, hq, w_qk, rotate);
      weigh(p.k_weight);
      sweep(raw_k, k, static_cast<T *>(p.k_cache) + (slot * hkv + r_qk) * kHeadDim, hkv, w_qk, rotate);
      sweep(raw_v, v, static_cast<T *>(p.v_cache) + (slot * hkv + r_v) * kHeadDim, hkv, w_v, [](uint2 (&)[2]) {});
    }
    buf ^= 1;  // a thread is at most one step ahead of the slowest (the barrier), so two buffers do
  }
  griddep_launch_dependents();
}

template <typename T, int TOK, bool AXES>
cudaError_t launch_rope_kv_typed(const RopeKvParams &p, int grid, cudaStream_t stream) {
  const int mode = p.interleaved ? kInterleaved : p.rotary_dim % 8 == 0 ? kHalfPairs : kHalfExchange;
#define PA_ROPE_CASE(M, N) \
  if (mode == M && (p.q_weight != nullptr) == N) \
    return launch_pdl(rope_kv_kernel<T, M, N, TOK, AXES>, dim3(grid), dim3(kRopeKvThreads), 0, stream, p);
  PA_ROPE_CASE(kInterleaved, false)
  PA_ROPE_CASE(kInterleaved, true)
  PA_ROPE_CASE(kHalfPairs, false)
  PA_ROPE_CASE(kHalfPairs, true)
  PA_ROPE_CASE(kHalfExchange, false)
  PA_ROPE_CASE(kHalfExchange, true)
#undef PA_ROPE_CASE
  return cudaErrorInvalidValue;
}

template <bool AXES>
cudaError_t launch_rope_kv_axes(const RopeKvParams &p, int dtype, int sms, cudaStream_t stream) {
  const int cap = sms * 3;  // one wave: 3 CTAs fit on an SM
  if (p.num_tokens <= cap) {  // a token per CTA
    return dtype == PA_BF16 ? launch_rope_kv_typed<__nv_bfloat16, 1, AXES>(p, p.num_tokens, stream)
                            : launch_rope_kv_typed<__half, 1, AXES>(p, p.num_tokens, stream);
  }
  const int want = (p.num_tokens + 3) / 4, grid = want < cap ? want : cap;
  return dtype == PA_BF16 ? launch_rope_kv_typed<__nv_bfloat16, 4, AXES>(p, grid, stream)
                          : launch_rope_kv_typed<__half, 4, AXES>(p, grid, stream);
}

}  // namespace

cudaError_t launch_rope_kv(const RopeKvParams &p, int dtype, int sms, cudaStream_t stream) {
  return p.num_axes > 1 ? launch_rope_kv_axes<true>(p, dtype, sms, stream)
                        : launch_rope_kv_axes<false>(p, dtype, sms, stream);
}

}  // namespace pa

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
// heads).  A CTA takes one token at a time: its first d / 2 threads compute
// the token's angles once for all of its heads, through shared memory (two
// buffers, one barrier per token); 16 lanes hold one head row (8 values each,
// 16-byte loads and stores), and a thread issues the loads of all its rows of
// the token before the angles and the first use.
#include "pa_device.cuh"

namespace pa {
namespace {

constexpr unsigned FULL = 0xffffffffu;
constexpr int kRopeKvThreads = 256;
constexpr int kRowsAtOnce = kRopeKvThreads / 16;  // head rows one pass of the CTA covers
constexpr int kPasses = 3;                        // passes whose loads are in flight together

enum RopeMode { kInterleaved = 0, kHalfLanes = 1, kHalfAny = 2 };

// The fraction of a turn per position as a 64-bit fixed-point number.
__device__ __forceinline__ long long turns_fixed(double inv_freq) {
  const double t = inv_freq * 0.15915494309189533577;  // 1 / (2 pi)
  return __double2ll_rn((t - rint(t)) * 18446744073709551616.0);
}

// 8 values of one row (16 lanes per row, this lane's dims d0 .. d0 + 7) after
// the optional norm, rotated.  cs: the token's (cos, sin) pairs.  Every lane
// of the warp takes part (kHalfLanes shuffles, kHalfAny exchanges through the
// warp's staging rows).
template <int MODE>
__device__ __forceinline__ void rotate_row(float (&x)[8], const float2 *cs, int d, int lane, float *stage) {
  const int l16 = lane & 15, d0 = l16 * 8;
  if constexpr (MODE == kInterleaved) {
#pragma unroll
    for (int e = 0; e < 8; e += 2)
      if (d0 + e < d) {
        const float2 c = cs[(d0 + e) >> 1];
        const float a = x[e], b = x[e + 1];
        x[e] = a * c.x - b * c.y;
        x[e + 1] = b * c.x + a * c.y;
      }
  } else if constexpr (MODE == kHalfLanes) {  // d a multiple of 16: the partner's 8 dims are one lane's
    const int hl = d >> 4;                    // lanes per half
    const bool lo = l16 < hl;
    const int src = (lane & 16) | (lo ? l16 + hl : (l16 < 2 * hl ? l16 - hl : l16));
    float y[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = __shfl_sync(FULL, x[e], src);
    if (l16 < 2 * hl) {
      const float4 *c4 = reinterpret_cast<const float4 *>(cs + (lo ? d0 : d0 - (d >> 1)));
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        const float4 c = c4[e >> 1];  // (cos, sin) of two consecutive pairs
        const float s0 = lo ? -c.y : c.y, s1 = lo ? -c.w : c.w;
        x[e] = x[e] * c.x + y[e] * s0;
        x[e + 1] = x[e + 1] * c.z + y[e + 1] * s1;
      }
    }
  } else {
    float *row = stage + (lane >> 4) * kHeadDim;
#pragma unroll
    for (int e = 0; e < 8; ++e) row[d0 + e] = x[e];
    __syncwarp();
    const int half = d >> 1;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int j = d0 + e;
      if (j < d) {
        const bool lo = j < half;
        const float2 c = cs[lo ? j : j - half];
        const float y = row[lo ? j + half : j - half];
        x[e] = x[e] * c.x + (lo ? -y : y) * c.y;
      }
    }
    __syncwarp();
  }
}

template <typename T, int MODE, bool NORM>
__global__ void __launch_bounds__(kRopeKvThreads) rope_kv_kernel(const RopeKvParams p) {
  __shared__ __align__(16) float2 cs_buf[2][kHeadDim / 2];
  __shared__ float stage_buf[MODE == kHalfAny ? kRopeKvThreads / 32 * 2 * kHeadDim : 1];
  const int tid = threadIdx.x, lane = tid & 31, l16 = lane & 15;
  const int hq = p.num_q_heads, hkv = p.num_kv_heads;
  const int rows = hq + 2 * hkv, d = p.rotary_dim;
  float *stage = stage_buf + (MODE == kHalfAny ? (tid >> 5) * 2 * kHeadDim : 0);
  griddep_wait();  // q, k, v may be the previous kernel's output; the pool may be read by it
  long long turns = 0;
  if (tid < d / 2) turns = turns_fixed(__ldg(p.inv_freq + tid));
  float wq[8], wk[8];
  if constexpr (NORM) {
    const uint4 a = *reinterpret_cast<const uint4 *>(static_cast<const T *>(p.q_weight) + 8 * l16);
    const uint4 b = *reinterpret_cast<const uint4 *>(static_cast<const T *>(p.k_weight) + 8 * l16);
    const uint32_t ua[4] = {a.x, a.y, a.z, a.w}, ub[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 fa = Pack<T>::to_f2(ua[i]), fb = Pack<T>::to_f2(ub[i]);
      wq[2 * i] = fa.x, wq[2 * i + 1] = fa.y;
      wk[2 * i] = fb.x, wk[2 * i + 1] = fb.y;
    }
  }
  int buf = 0;
  for (int t = blockIdx.x; t < p.num_tokens; t += gridDim.x) {
    const int pos = __ldg(p.positions + t);
    const int64_t slot = __ldg(p.slots + t);
    if (pos < 0 || slot < 0 || slot >= p.num_slots) {  // (the same in every thread) nothing of it is written
      if (tid == 0) set_error(p.err, PA_ERR_RANGE, t);
      continue;
    }
    auto source = [&](int r) {
      return r < hq         ? static_cast<const T *>(p.q) + ((int64_t)t * hq + r) * kHeadDim
             : r < hq + hkv ? static_cast<const T *>(p.k) + ((int64_t)t * hkv + (r - hq)) * kHeadDim
                            : static_cast<const T *>(p.v) + ((int64_t)t * hkv + (r - hq - hkv)) * kHeadDim;
    };
    bool first = true;
    for (int r0 = 0; r0 < rows; r0 += kRowsAtOnce * kPasses) {
      uint4 raw[kPasses];
#pragma unroll
      for (int i = 0; i < kPasses; ++i) {
        const int r = r0 + i * kRowsAtOnce + (tid >> 4);
        raw[i] = r < rows ? *reinterpret_cast<const uint4 *>(source(r) + 8 * l16) : make_uint4(0, 0, 0, 0);
      }
      if (first) {  // the token's angles, while the rows are on their way
        if (tid < d / 2) {
          const long long turn = (long long)((unsigned long long)turns * (unsigned long long)(unsigned)pos);
          float s, c;
          sincospif((float)(int)(turn >> 32) * 4.656612873077393e-10f, &s, &c);  // 2^-31: half turns
          cs_buf[buf][tid] = make_float2(c * p.attention_factor, s * p.attention_factor);
        }
        __syncthreads();
        first = false;
      }
#pragma unroll
      for (int i = 0; i < kPasses; ++i) {
        const int r = r0 + i * kRowsAtOnce + (tid >> 4);
        const int rw = r0 + i * kRowsAtOnce + (tid >> 5) * 2;  // the warp's first row
        if (rw >= rows) break;                                 // (warp-uniform)
        uint4 out = raw[i];
        if (rw < hq + hkv) {  // (warp-uniform) the warp holds a query or key row
          const uint32_t u[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
          float x[8];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 f = Pack<T>::to_f2(u[k]);
            x[2 * k] = f.x, x[2 * k + 1] = f.y;
          }
          if constexpr (NORM) {
            float ss = 0.f;
#pragma unroll
            for (int k = 0; k < 8; ++k) ss = fmaf(x[k], x[k], ss);
#pragma unroll
            for (int off = 8; off > 0; off >>= 1) ss += __shfl_xor_sync(FULL, ss, off);
            const float inv = rsqrtf(ss * (1.f / kHeadDim) + p.eps);
#pragma unroll
            for (int k = 0; k < 8; ++k) x[k] *= inv * (r < hq ? wq[k] : wk[k]);
          }
          rotate_row<MODE>(x, cs_buf[buf], d, lane, stage);
          if (r < hq + hkv)
            out = make_uint4(Pack<T>::from_f2(x[0], x[1]), Pack<T>::from_f2(x[2], x[3]), Pack<T>::from_f2(x[4], x[5]),
                             Pack<T>::from_f2(x[6], x[7]));
        }
        if (r < rows) {
          T *dst = r < hq         ? static_cast<T *>(p.q_out) + ((int64_t)t * hq + r) * kHeadDim
                   : r < hq + hkv ? static_cast<T *>(p.k_cache) + (slot * hkv + (r - hq)) * kHeadDim
                                  : static_cast<T *>(p.v_cache) + (slot * hkv + (r - hq - hkv)) * kHeadDim;
          st_v4(dst + 8 * l16, out);
        }
      }
    }
    buf ^= 1;  // a thread is at most one token ahead of the slowest (the barrier), so two buffers do
  }
  griddep_launch_dependents();
}

template <typename T>
cudaError_t launch_rope_kv_typed(const RopeKvParams &p, int grid, cudaStream_t stream) {
  const int mode = p.interleaved ? kInterleaved : p.rotary_dim % 16 == 0 ? kHalfLanes : kHalfAny;
#define PA_ROPE_CASE(M, N) \
  if (mode == M && (p.q_weight != nullptr) == N) \
    return launch_pdl(rope_kv_kernel<T, M, N>, dim3(grid), dim3(kRopeKvThreads), 0, stream, p);
  PA_ROPE_CASE(kInterleaved, false)
  PA_ROPE_CASE(kInterleaved, true)
  PA_ROPE_CASE(kHalfLanes, false)
  PA_ROPE_CASE(kHalfLanes, true)
  PA_ROPE_CASE(kHalfAny, false)
  PA_ROPE_CASE(kHalfAny, true)
#undef PA_ROPE_CASE
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_rope_kv(const RopeKvParams &p, int dtype, cudaStream_t stream) {
  const int cap = sm_count() * 4;
  const int grid = p.num_tokens < cap ? p.num_tokens : cap;
  return dtype == PA_BF16 ? launch_rope_kv_typed<__nv_bfloat16>(p, grid, stream)
                          : launch_rope_kv_typed<__half>(p, grid, stream);
}

}  // namespace pa
